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


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("Hq", [4, 32])
def test_queries_of_slots_without_room_see_nothing(b, Hq, cache):
    scales = dict(k_scale=torch.full((2,), 0.05, device="cuda"), v_scale=torch.full((2,), 0.05, device="cuda"))
    c = _filled(b, [40, 33, 0, 70], dtype=cache, **(scales if cache.itemsize == 1 else {}))
    new = [3, 5, 4, 2]
    q = torch.randn((sum(new), Hq, 64), device="cuda").bfloat16()
    q_start = _i32(np.concatenate([[0], np.cumsum(new)]))
    args = (q, c.k[0], c.v[0], c.page_table, c.seq_len, q_start, 5, 0.125)
    kw = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    want = b.paged_attention(*args, **kw)
    for granted in ([3, 5, 4, 2], [1, 0, 4, 0], [0, 0, 0, 0]):
        for window in (0, 16):
            want = b.paged_attention(*args, **kw, window=window)
            got = b.paged_attention(*args, **kw, window=window, granted=_i32(granted))
            for r, g in enumerate(granted):
                rows = slice(int(q_start[r]), int(q_start[r + 1]))
                if g:
                    assert torch.equal(got["out"][rows], want["out"][rows]), (granted, r)
                    assert torch.equal(got["lse"][rows], want["lse"][rows]), (granted, r)
                else:
                    assert (got["out"][rows] == 0).all() and (got["lse"][rows] == -float("inf")).all(), (granted, r)
    with pytest.raises(b.DSparkError):
        b.paged_attention(*args, **kw, granted=_i32([1, 1, 1]))
    with pytest.raises(b.DSparkError):
        b.paged_attention(*args, **kw, granted=torch.ones(4, device="cuda"))


def test_refused_reservation(b):
    """A pool that runs out: the slot that got no room keeps its context, stores nothing and its queries
    see nothing; one that asked for nothing attends as ever; room given back serves it."""
    c = b.PagedCache(3, 6, 16, 6, 1, 2, 64)
    c.reserve(_i32([30, 16, 33]))  # 2 + 1 + 3 pages: the pool is full
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn((79, 2, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    c.write(0, k, v, _i32([0, 30, 46, 79]))
    plan = c.reserve(_i32([2, 4, 0]))
    assert plan["granted"].tolist() == [2, 0, 0] and c.seq_len.tolist() == [32, 16, 33]
    before = c.k.clone()
    q_start, q = _i32([0, 2, 6, 7]), torch.randn((7, 4, 64), generator=g, device="cuda").bfloat16()
    nk, nv = (torch.randn((7, 2, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    c.write(0, nk, nv, _i32([0, 2, 6, 6]))
    page = int(c.page_table[0, 1])
    assert torch.equal(c.k[:, [p for p in range(6) if p != page]], before[:, [p for p in range(6) if p != page]])
    o = c.attend(0, q, q_start, 4, 0.125)
    want = b.paged_attention(q, c.k[0], c.v[0], c.page_table, c.seq_len, q_start, 4, 0.125)
    assert (o["out"][2:6] == 0).all() and (o["lse"][2:6] == -float("inf")).all()
    for rows in (slice(0, 2), slice(6, 7)):
        assert torch.equal(o["out"][rows], want["out"][rows]) and torch.equal(o["lse"][rows], want["lse"][rows])
    c.truncate(_i32([99, 99, 16]))
    assert c.reserve(_i32([0, 4, 0]))["granted"].tolist() == [0, 4, 0]
    c.write(0, nk, nv, _i32([0, 0, 4, 4]))
    o = c.attend(0, q, _i32([0, 0, 4, 4]), 4, 0.125)
    assert torch.isfinite(o["lse"][:4]).all() and c.seq_len.tolist() == [32, 20, 16]
    assert c.status() == 0


def test_loop_on_a_pool_that_runs_out(b):
    """Requests without room emit nothing that round; what they answer in the end is what the dense
    model says (tolerance: tests/test_gpu_serving_loop.py)."""
    from tests.test_gpu_serving_loop import _loop, _prompts
    prompts = _prompts([30, 9, 20])
    loop = _loop(torch.bfloat16, prompts, page_size=8, num_pages=24)  # 8 pages a slot, of 24
    hold = loop.cache.ref_count  # all but three of the free pages are taken by someone else
    free = (hold == 0).nonzero()[:, 0]
    hold[free[3:]] = 1
    seqs, lps, refused, after = [list(p) for p in prompts], [[] for _ in prompts], 0, 0
    for k in range(14):
        if k == 7:
            hold[free[3:]] = 0  # they come back
        before, anchors = loop.cache.seq_len.tolist(), loop.x0.tolist()
        o = loop.step()
        for r, n in enumerate(o["n_out"].tolist()):
            if n == 0:
                refused += 1
                assert loop.cache.seq_len[r] == before[r] and loop.x0[r] == anchors[r]
                assert (o["tokens"][r] == -1).all() and torch.isnan(o["logprob"][r]).all()
            after += n * (k >= 7)
            seqs[r] += o["tokens"][r, :n].tolist()
            lps[r] += o["logprob"][r, :n].tolist()
    assert refused >= 3 and after > 7
    assert loop.cache.seq_len.tolist() == [len(s) - 1 for s in seqs] and loop.cache.status() == 0
    for r, seq in enumerate(seqs):
        dense = torch.log_softmax(loop.target.dense(torch.tensor(seq, device="cuda")), 1)
        at = len(prompts[r]) - 1
        want = dense[torch.arange(at, len(seq) - 1), torch.tensor(seq[at + 1:], device="cuda")]
        assert (torch.tensor(lps[r], device="cuda") - want).abs().max() < 0.15
    with pytest.raises(RuntimeError):
        _loop(torch.bfloat16, _prompts([30, 9, 20]), page_size=8, num_pages=9)


def test_write_before_any_reservation_reports_its_places(b):
    """Nothing has been refused yet: rows that have no place are reported, not passed over."""
    c = b.PagedCache(2, 4, 8, 2, 1, 1, 16)
    x = torch.ones((2, 1, 16), device="cuda").bfloat16()
    c.write(0, x, x, _i32([0, 1, 2]))
    assert c.status() == 1 and (c.k == 0).all()


def test_loop_with_long_prompts(b):
    """Prompts of more tokens than an attention call takes queries go in block by block."""
    from tests.test_gpu_serving_loop import _loop, _prompts
    prompts = _prompts([300, 9, 129, 130, 257])
    loop = _loop(torch.bfloat16, prompts, page_size=16, num_pages=125)
    assert loop.cache.seq_len.tolist() == [299, 8, 128, 129, 256]
    seqs, lps = [list(p) for p in prompts], [[] for _ in prompts]
    for _ in range(4):
        o = loop.step()
        for r, n in enumerate(o["n_out"].tolist()):
            seqs[r] += o["tokens"][r, :n].tolist()
            lps[r] += o["logprob"][r, :n].tolist()
    assert loop.cache.status() == 0
    for r, seq in enumerate(seqs):
        dense = torch.log_softmax(loop.target.dense(torch.tensor(seq, device="cuda")), 1)
        at = len(prompts[r]) - 1
        want = dense[torch.arange(at, len(seq) - 1), torch.tensor(seq[at + 1:], device="cuda")]
        assert (torch.tensor(lps[r], device="cuda") - want).abs().max() < 0.15


def test_status_of_a_captured_block(b):
    """Before the graph's first replay its scratch holds what was there; after a replay, its reports."""
    c = _filled(b, [40, 33])
    q, q_start = torch.randn((4, 8, 64), device="cuda").bfloat16(), _i32([0, 2, 4])
    torch.full((96 << 20,), 0x5A, dtype=torch.uint8, device="cuda")  # what freed memory may hold
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.attend(0, q, q_start, 2, 0.125)
    for ws in c._attention_ws.values():
        ws[:256] = 0x5A
    assert c.status() == 0
    graph.replay()
    assert c.status() == 0
    want = b.paged_attention(q, c.k[0], c.v[0], c.page_table, c.seq_len, q_start, 2, 0.125)
    assert torch.equal(out["out"], want["out"])
    c.page_table[1, 0] = 99
    graph.replay()
    assert c.status() == 1
