"""dspark_adjust_logits against a 64-bit form: types, odd vocabularies, strides, histories from empty to
long, ids out of range, repeated ids, masks, in place, rows of no slot, streams and graphs.

Tolerance.  Four operations in fp32 (the division or product, frequency * n, and the subtractions and
biases): each is off by 2^-24 of the largest magnitude on the way, so 2^-21 of it covers eight; each
further bias adds one.  Then half a step of the stored type (subnormal fp16 numbers: half of 2^-24)."""
import math

import numpy as np
import pytest
import torch

from tests import position_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _case(new, hist, V, dtype, seed=0, width=None, biases=0, masks=None, prompt=True, penalties=True):
    """Numpy arrays by argument name; the logits as a tensor."""
    rng = np.random.default_rng(seed)
    R, N = len(new), sum(new)
    L = width or max(1, max(hist))
    ids = lambda *s: np.minimum((V * rng.random(s) ** 3).astype(np.int32), V - 1)
    c = dict(tokens=ids(N), q_start=np.concatenate([[0], np.cumsum(new)]).astype(np.int32), history=ids(R, L),
             history_len=np.array(hist, np.int32))
    if prompt:
        c["prompt_len"] = np.array([n // 2 for n in hist], np.int32)
    if penalties:
        c.update(repetition=(1 + 0.5 * rng.random(R)).astype(np.float32), frequency=(rng.random(R) - 0.3).astype(np.float32),
                 presence=(rng.random(R) - 0.3).astype(np.float32))
    if biases:
        c.update(bias_ids=rng.integers(-1, V, (R, biases)).astype(np.int32),
                 bias=(4 * rng.random((R, biases)) - 2).astype(np.float32))
    if masks is not None:
        c["mask"] = rng.integers(-2 ** 31, 2 ** 31, (masks, -(-V // 32))).astype(np.int32)
        c["mask_row"] = rng.integers(-1, masks, N).astype(np.int32) if masks else np.full(N, -1, np.int32)
    return torch.randn((N, V), generator=torch.Generator().manual_seed(seed)).mul(4).to(dtype).cuda(), c


def _gpu(c):
    return {k: torch.as_tensor(v).cuda() for k, v in c.items()}


def _compare(got, x, c):
    want, most = ref.adjusted(x.double().cpu().numpy(), c.get("tokens"), c["q_start"],
                              **{k: v for k, v in c.items() if k not in ("tokens", "q_start")})
    got = got.double().cpu().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    extra = 0 if "bias_ids" not in c else c["bias_ids"].shape[1]
    tol = (2.0 ** -21 + extra * 2.0 ** -24) * most + torch.finfo(x.dtype).eps / 2 * np.abs(np.where(fine, want, 0))
    tol = tol + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
    off = np.abs(np.where(fine, got - np.where(fine, want, 0), 0))
    assert (off <= tol).all(), (np.argwhere(off > tol)[0], off.max())


def _check(b, x, c, **kw):
    got = b.adjust_logits(x, **{"tokens": None, **_gpu(c)}, **kw)
    _compare(got, x, c)
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 7, 31, 32, 33, 1000, 8191, 8192, 8193, 20001])
def test_vocabularies(b, dtype, V):
    """Slices and pieces that end anywhere, every kind of adjustment at once."""
    x, c = _case([3, 0, 1, 5], [40, 3, 0, 600], V, dtype, seed=V, biases=min(V, 20), masks=4)
    _check(b, x, c)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("what", ["repetition", "frequency", "presence", "bias", "mask", "nothing", "mask without rows"])
def test_one_at_a_time(b, dtype, what):
    x, c = _case([4, 2], [100, 7], 3001, dtype, seed=5, biases=9, masks=6)
    keep = {"bias": ("bias_ids", "bias"), "mask": ("mask", "mask_row"), "nothing": (), "mask without rows": ("mask",)}
    for k in ("repetition", "frequency", "presence", "bias_ids", "bias", "mask", "mask_row"):
        if k not in keep.get(what, (what,)):
            del c[k]
    got = _check(b, x, c)
    if what == "nothing":
        assert torch.equal(got, x)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_count_the_tokens_before_them(b, dtype):
    """A block that repeats one id: each row sees it once more; the prompt's end may lie inside the block."""
    x, c = _case([12, 20], [3, 0], 500, dtype, seed=7)
    c["tokens"][:] = 17
    c["prompt_len"][:] = [6, 0]
    got = _check(b, x, c)
    n = torch.arange(1, 21, device="cuda").float()
    f, a, rho = (float(c[k][1]) for k in ("frequency", "presence", "repetition"))
    z = x[12:, 17].float()
    want = torch.where(z > 0, z / rho, z * rho) - f * n - a
    assert torch.allclose(got[12:, 17].float(), want, rtol=torch.finfo(dtype).eps, atol=1e-5)
    c["tokens"][:] = -1  # nothing is fed in that counts
    _check(b, x, c)


def test_ids_and_lengths_out_of_range(b):
    x, c = _case([3, 3, 3], [50, 60, 0], 777, torch.float32, seed=8, biases=12, masks=3)
    c["history"][0, ::3] = -1
    c["history"][1, ::4] = [777, 2 ** 31 - 1, -2 ** 31, 800, 10 ** 9] * 3
    c["tokens"][1::2] = 777
    c["bias_ids"][0] = [5, 5, -1, 777, 5, 2 ** 31 - 1, -5, 5, 6, 6, 5, 0]
    c["mask_row"][:] = [0, 3, -7, 2 ** 31 - 1, 1, 2, 0, 100, -1]
    c["history_len"][:] = [1000, 60, -3]  # past the width, whole, below 0
    c["prompt_len"][:] = [-4, 1 << 30, 0]
    got = _check(b, x, c)
    again = b.adjust_logits(x, **_gpu(c))
    assert torch.equal(got, again)


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_in_place(b, dtype):
    x, c = _case([2, 3, 1], [30, 0, 500], 1003, dtype, seed=9, biases=5, masks=3)
    want = _check(b, x, c)
    wide = torch.full((6, 1100), 5.0, dtype=dtype, device="cuda")
    for shift_in, shift_out in ((0, 0), (1, 1), (1, 2), (8, 3)):  # rows whose alignments agree, and not
        src = wide.clone()[:, shift_in:shift_in + 1003]
        src.copy_(x)
        dst = wide.clone()
        b.adjust_logits(src, **_gpu(c), out=dst[:, shift_out:shift_out + 1003])
        assert torch.equal(dst[:, shift_out:shift_out + 1003], want)
        assert (dst[:, :shift_out] == 5).all() and (dst[:, shift_out + 1003:] == 5).all()
        got = b.adjust_logits(src, **_gpu(c), out=src)
        assert got is src and torch.equal(src, want)
    h = torch.as_tensor(np.pad(c["history"], ((0, 0), (0, 9)), constant_values=1)).cuda()[:, :c["history"].shape[1]]
    m = torch.as_tensor(np.pad(c["mask"], ((0, 0), (0, 4)))).cuda()[:, :c["mask"].shape[1]]
    assert torch.equal(b.adjust_logits(x, **{**_gpu(c), "history": h, "mask": m}), want)


def test_special_values(b):
    """NaN, infinities and masks of the type's lowest value, adjusted and masked; biases of -inf ban ids."""
    x, c = _case([3], [50], 300, torch.float32, seed=10, biases=3, masks=1)
    x[:, 0], x[:, 1], x[:, 2], x[:, 3] = math.nan, math.inf, -math.inf, torch.finfo(torch.float32).min
    c["history"][0, :8] = [0, 1, 2, 3, 4, 4, 4, 5]
    c["repetition"][:] = 0.5
    c["bias_ids"][0], c["bias"][0] = [4, 1, 5], [-math.inf, 1.0, 2.0]
    c["mask"][:] = -1
    c["mask"][0, 0] &= ~0b1001
    c["mask_row"][:] = [0, -1, 0]
    got = b.adjust_logits(x, **_gpu(c))
    assert (got[:, 4] == -math.inf).all() and (got[[0, 2], 0] == -math.inf).all() and torch.isnan(got[1, 0])
    assert (got[:, 1] == math.inf).all() and (got[:, 2] == -math.inf).all()
    # (an id of the prompt's: x < 0 is multiplied by 0.5, exactly)
    assert (got[[0, 2], 3] == -math.inf).all() and got[1, 3] == torch.finfo(torch.float32).min * 0.5
    c["mask"][:] = 0  # nothing is left
    assert (b.adjust_logits(x, **_gpu(c))[[0, 2]] == -math.inf).all()


def test_rows_of_no_slot_are_left(b):
    x, c = _case([3, 2], [50, 9], 2000, torch.bfloat16, seed=11)
    big = torch.cat([x[:2], x, x[:4]])
    c["q_start"] = c["q_start"] + 2
    c["tokens"] = np.concatenate([c["tokens"][:2], c["tokens"], c["tokens"][:4]])
    out = torch.full_like(big, 5.0)
    b.adjust_logits(big, **_gpu(c), out=out)
    assert (out[:2] == 5).all() and (out[7:] == 5).all()
    got = out.clone()
    got[:2], got[7:] = big[:2], big[7:]
    _compare(got, big, c)


@pytest.mark.parametrize("V,N,dtype", [(50257, 3, torch.float32), (151936, 9, torch.bfloat16)])
def test_long_histories_and_blocks(b, V, N, dtype):
    x, c = _case([N, 200], [60000, 131072], V, dtype, seed=12, biases=300, masks=5)
    rows = np.unique(np.concatenate([[0, N - 1, N, N + 7, N + 8, N + 100, N + 199]]))
    got = b.adjust_logits(x, **_gpu(c))
    # a few rows, each as a slot of one row whose history holds the block before it
    for n in rows:
        r, i = (0, n) if n < N else (1, n - N)
        seq = np.concatenate([c["history"][r, :c["history_len"][r]], c["tokens"][c["q_start"][r]:n + 1]])
        one = {k: v[r:r + 1] for k, v in c.items() if k in ("prompt_len", "repetition", "frequency", "presence", "bias_ids", "bias")}
        one.update(q_start=np.array([0, 1], np.int32), history=seq[None].astype(np.int32), history_len=np.array([len(seq)], np.int32),
                   mask=c["mask"], mask_row=c["mask_row"][n:n + 1])
        _compare(got[n:n + 1], x[n:n + 1], one)


def test_streams_and_graphs(b):
    x, c = _case([3, 2], [50, 9], 5000, torch.bfloat16, seed=13, biases=4, masks=2)
    d = _gpu(c)
    want = b.adjust_logits(x, **d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = b.adjust_logits(x, **d, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.adjust_logits(x, **d, out=out)
    d["history_len"] -= 5
    g.replay()
    assert torch.equal(out, b.adjust_logits(x, **d))
    assert b.adjust_logits(x[:0], d["tokens"][:0], torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 5000)
