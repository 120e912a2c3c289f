"""PagedCache as a user holds it: its calls on a stream of the caller's, blocks of any number of
rows, what a refused reservation leaves behind."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _filled(b, lens, Hkv=2, D=64, page_size=16, layers=1, seed=0, **kw):
    """A cache whose slots hold `lens` tokens of random keys and values."""
    c = b.PagedCache(len(lens), 64, page_size, 16, layers, Hkv, D, **kw)
    c.reserve(_i32(lens))
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn((sum(lens), Hkv, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    for n in range(layers):
        c.write(n, k, v, _i32(np.concatenate([[0], np.cumsum(lens)])))
    return c


def _busy():
    """Work for some milliseconds on the current stream."""
    x = torch.randn((4096, 4096), device="cuda")
    for _ in range(30):
        x = x @ x * 1e-3
    return x


@pytest.mark.parametrize("Hq", [4, 32])  # both kernels
def test_attend_on_a_stream_while_another_is_busy(b, Hq):
    lens, new = [100, 200, 37], [5, 8, 2]
    c = _filled(b, lens)
    q = torch.randn((sum(new), Hq, 64), device="cuda").bfloat16()
    q_start = _i32(np.concatenate([[0], np.cumsum(new)]))
    ws = b.workspace(b.paged_attention_workspace_size(sum(new), 3, Hq, 2, 64, 8), "cuda")
    want = b.paged_attention(q, c.k[0], c.v[0], c.page_table, c.seq_len, q_start, 8, 0.125, ws=ws)
    torch.cuda.synchronize()
    # freed memory that holds other values than zero, for the scratch to be made of
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            torch.full((64 << 20,), 0x5A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        side.wait_stream(torch.cuda.current_stream())
        busy = _busy()
        out = c.attend(0, q, q_start, 8, 0.125, stream=side)
        side.synchronize()
        assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])
        torch.cuda.synchronize()
        del busy
    assert c.status() == 0


def test_attend_over_blocks_of_many_sizes_keeps_its_memory(b):
    c = _filled(b, [90, 150])
    held = None
    for T in range(2, 40, 3):
        new = [T // 2, T - T // 2]
        q = torch.randn((T, 8, 64), device="cuda").bfloat16()
        q_start = _i32([0, new[0], T])
        got = c.attend(0, q, q_start, 20, 0.125)
        ws = b.workspace(b.paged_attention_workspace_size(T, 2, 8, 2, 64, 20), "cuda")
        want = b.paged_attention(q, c.k[0], c.v[0], c.page_table, c.seq_len, q_start, 20, 0.125, ws=ws)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
        size = sum(w.numel() for w in c._attention_ws.values())
        held = held or size
        assert size == held
    assert c.status() == 0
