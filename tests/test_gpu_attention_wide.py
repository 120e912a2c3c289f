"""dspark_paged_attention for blocks of more query rows than one small tile holds, which another
kernel takes (D <= 128, pages of a multiple of 8 tokens): the same contract, against the same 64-bit
form with the same tolerances as for few rows (tests/test_gpu_attention.py)."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_attention import _case, _check, _compare, _i32, _run

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
TYPES = [(torch.bfloat16, None), (torch.float16, None), (torch.bfloat16, E4M3), (torch.float16, E4M3)]


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq", [4, 32])
def test_pools_expanded_over_their_heads(b, dtype, cache, Hq):
    """One head's keys and values seen as several by a stride of 0, by few rows and by many; the
    pool is the end of its allocation."""
    c = _case([60, 90, 17], [2, 3, 1], Hq, 4, 64, 16, dtype, cache, seed=12, extra=0)
    dev = {}
    for n in ("k", "v"):
        one = c[n][:, :1].contiguous()
        c[n] = one.expand(-1, 4, -1, -1)
        dev[n] = one.cuda().expand(-1, 4, -1, -1)
    o, ws = _run(b, c, 0.125, dev=dev)
    assert b.device_status(ws) == 0
    _compare(c, o, 0.125)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,nq,tail", [(1, 1, 17.0), (1, 1, 25.5), (8, 1, 21.3), (4, 8, 17.0), (4, 8, 25.5), (16, 8, 23.0)])
def test_a_long_tail_of_small_weights(b, dtype, cache, Hq, nq, tail):
    """One likely token, and 70,000 whose weights are 2^-tail of its own: they are small numbers for
    16 bits, and together a share of the sum that the output has to show.  The likely token's value is
    0, so the output is the tail's alone."""
    n = 70000
    c = _case([n], [nq], Hq, 1, 64, 64, dtype, cache, seed=21, garbage=False)
    k, v = torch.zeros(c["k"].shape), torch.ones(c["v"].shape)
    page, slot = c["table"][0, 3], 5
    k[page, 0, slot, 0] = 8.0
    v[page, 0, slot] = 0.0
    c["k"], c["v"] = k.to(c["k"].dtype), v.to(c["v"].dtype)
    c["q"] = torch.zeros(c["q"].shape)
    c["q"][..., 0] = 4.0
    c["q"] = c["q"].to(dtype)
    if cache:
        c["scales"] = (torch.ones(1), torch.ones(1))
    scale = tail * math.log(2.0) / 32.0
    o, ws = _run(b, c, scale)
    assert b.device_status(ws) == 0
    _compare(c, o, scale)


# (Hq, H, D, page, queries): 20 to 128 query rows a cache head, whole and partly filled panels
LAYOUTS = [(20, 1, 96, 128, 1), (64, 1, 16, 8, 1), (16, 1, 48, 8, 2), (34, 2, 32, 56, 2), (32, 2, 128, 16, 2),
           (32, 2, 128, 32, 4), (48, 2, 80, 24, 3), (24, 1, 112, 40, 5), (32, 2, 128, 64, 8), (64, 2, 64, 16, 4)]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D,ps,nq", LAYOUTS)
def test_blocks(b, dtype, cache, Hq, H, D, ps, nq):
    lens = [nq, 1, 127, 128, 129, 0, 255, 256, 300, 1000, 40]
    new = [min(n, max(1, nq - i % 3)) for i, n in enumerate(lens)]
    _check(b, _case(lens, new, Hq, H, D, ps, dtype, cache, seed=D + nq), max_q=nq)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,nq", [(32, 2), (32, 4), (32, 8), (4, 1)])
@pytest.mark.parametrize("per_tile", [-12.0, 3.0, 20.0])
def test_scores_that_grow_along_the_context(b, dtype, cache, Hq, nq, per_tile):
    """Scores of 2^per_tile more (or less) every 128 tokens: what was summed is rescaled again and again,
    for half of the query rows; for the others they shrink.  Many tiles for every worker."""
    lens = [3001, 2900, 3100, 2807] * 8
    c = _case(lens, [nq] * 32, Hq, 2, 128, 64, dtype, cache, seed=17, garbage=False)
    step = per_tile * math.log(2.0) / 128.0 * 8.0  # in products, at a scale of 1/8
    k = c["k"].float()
    for r, n in enumerate(lens):
        at = torch.as_tensor(c["table"][r, : -(-n // 64)])
        pos = (torch.arange(len(at))[:, None] * 64 + torch.arange(64)).float()
        k[at, :, :, 0] = (step * (pos - n / 2) / 4.0)[:, None, :]
    c["k"] = k.to(c["k"].dtype)
    q = c["q"].float()
    q[:, ::2, 0], q[:, 1::2, 0] = 4.0, -4.0
    c["q"] = (q * torch.where(torch.arange(128) == 0, 1.0, 0.25)).to(dtype)
    if cache:
        c["scales"] = (torch.ones(2), torch.ones(2))
    _check(b, c, scale=0.125)


@pytest.mark.parametrize("Hq,H,nq", [(32, 2, 2), (32, 2, 8)])
def test_large_and_small_scores(b, Hq, H, nq):
    for scale, mult in ((1.0, 30.0), (-0.5, 1.0), (0.0, 1.0), (1e-3, 1e-3)):
        c = _case([77, 200, 900], [1, nq, nq], Hq, H, 128, 16, torch.bfloat16, seed=4)
        c["q"] = (c["q"].float() * mult).to(torch.bfloat16)
        _check(b, c, scale=scale)
    # queries past fp16's range over an e4m3 cache
    c = _case([77, 200], [1, nq], Hq, H, 128, 16, torch.bfloat16, E4M3, seed=4)
    c["q"] = (c["q"].float() * 1e6).to(torch.bfloat16)
    _check(b, c, scale=1e-7)
    c["q"] = (c["q"].float() * 1e-12).to(torch.bfloat16)
    c["q"][0] = 0
    _check(b, c, scale=1e5)


@pytest.mark.parametrize("window", [1, 7, 100, 128, 400])
@pytest.mark.parametrize("dtype,cache", TYPES[:3])
@pytest.mark.parametrize("Hq,nq", [(32, 2), (32, 8)])
def test_window(b, window, dtype, cache, Hq, nq):
    _check(b, _case([1, 50, 333, 700, 65], [1, nq, nq, 1, 2], Hq, 2, 128, 16, dtype, cache, seed=window), window=window)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,nq", [(32, 2), (32, 8)])
def test_unseen_values_have_no_influence(b, dtype, cache, Hq, nq):
    """NaN and infinities in the block's last token, which only its last query sees."""
    c = _case([140, 70], [nq, nq], Hq, 2, 128, 8, dtype, cache, seed=9)
    clean = _check(b, c)
    bad = math.nan if cache else math.inf
    for r, n in enumerate(c["lens"]):
        page = c["table"][r, (n - 1) // 8]
        for pool in (c["k"], c["v"]):
            x = pool.float()
            x[page, :, (n - 1) % 8] = bad
            x[page, :, (n - 1) % 8, 5] = math.nan
            pool.copy_(x.to(pool.dtype))
    o, ws = _run(b, c, 128 ** -0.5)
    last = [c["q_start"][r + 1] - 1 for r in range(2)]
    rest = [t for t in range(2 * nq) if t not in last]
    assert torch.equal(o["out"][rest], clean["out"][rest]) and torch.equal(o["lse"][rest], clean["lse"][rest])
    assert torch.isnan(o["out"][last].float()).any() and b.device_status(ws) == 0


@pytest.mark.parametrize("dtype,cache", TYPES[:3])
@pytest.mark.parametrize("D", [64, 128])
def test_strides(b, dtype, cache, D):
    """Pools [P, ps, H, D] seen as [P, H, ps, D], inside a larger allocation; queries that are a slice
    of a wider projection."""
    c = _case([33, 170, 9], [2, 4, 3], 32, 2, D, 16, dtype, cache, seed=6)
    P, H, ps, _ = c["k"].shape
    dev = {}
    for n in ("k", "v"):
        big = torch.zeros((P, ps + 1, H, D + 32), dtype=torch.uint8, device="cuda")
        big = big.view(cache) if cache else big.to(c[n].dtype)
        dev[n] = big[:, :ps, :, 16:16 + D].permute(0, 2, 1, 3)
        dev[n].copy_(c[n].cuda())
    wide = torch.zeros((9, 3, 32, D + 16), dtype=dtype, device="cuda")
    dev["q"] = wide[:, 1, :, 8:8 + D]
    dev["q"].copy_(c["q"].cuda())
    o, ws = _run(b, c, 0.125, dev=dev)
    assert b.device_status(ws) == 0
    _compare(c, o, 0.125)


def test_offsets_past_32_bits(b):
    """Pages 1.5 GB apart: element and byte offsets pass 32 bits."""
    for dtype, cache, stride in ((torch.bfloat16, None, 1_500_000_000), (torch.float16, E4M3, 2_400_000_000)):
        c = _case([60, 20], [2, 3], 32, 2, 64, 16, dtype, cache, seed=7, extra=0)
        P, H, ps, D = c["k"].shape
        size = c["k"].element_size()
        dev = {}
        for n in ("k", "v"):
            raw = torch.empty((P - 1) * stride * size + H * ps * D * size, dtype=torch.uint8, device="cuda")
            pool = raw.view(c[n].dtype).as_strided((P, H, ps, D), (stride, ps * D, D, 1))
            pool.copy_(c[n].cuda())
            dev[n] = pool
        o, ws = _run(b, c, 0.125, dev=dev)
        assert b.device_status(ws) == 0
        _compare(c, o, 0.125)
        del dev, pool, raw, o
        torch.cuda.empty_cache()


@pytest.mark.parametrize("cache", [None, E4M3])
def test_pages_out_of_range_are_reported_and_read_as_zeros(b, cache):
    for bad in (1 << 20, -1, -(1 << 31), 2 ** 31 - 1):
        c = _case([40, 140, 40], [2, 2, 2], 32, 2, 128, 8, torch.bfloat16, cache, seed=8, garbage=False)
        zero = next(p for p in range(c["k"].shape[0]) if p not in set(c["table"].ravel().tolist()))
        for pool in (c["k"], c["v"]):
            pool[zero] = torch.zeros(pool[zero].shape).to(pool.dtype)
        table = c["table"].copy()
        c["table"][1, 2] = bad
        o, ws = _run(b, c, 0.125)
        assert b.device_status(ws) == 1
        table[1, 2] = zero
        _compare(dict(c, table=table), o, 0.125)


def test_bad_requests_are_reported_and_harmless(b):
    for what in ("len", "negative", "queries", "order"):
        c = _case([40, 40, 40], [2, 2, 2], 32, 2, 128, 8, torch.bfloat16, seed=8, garbage=False)
        kw = {}
        if what == "len":
            c["lens"][1] = 41
        elif what == "negative":
            c["lens"][1] = -5
        elif what == "queries":
            c["q_start"] = np.array([0, 1, 5, 6])
            kw["max_q"] = 3
        else:
            c["q_start"] = np.array([0, 2, 9, 6])
        o, ws = _run(b, c, 0.125, **kw)
        assert b.device_status(ws) == 1, what
        good = _case([40, 40, 40], [2, 2, 2], 32, 2, 128, 8, torch.bfloat16, seed=8, garbage=False)
        if what == "queries":
            good["q_start"], good["new"] = np.array([0, 1, 5, 6]), [1, 4, 1]
        want, _ = _run(b, good, 0.125)
        n0 = c["q_start"][1]
        assert torch.equal(o["out"][:n0], want["out"][:n0]), what


def test_queries_of_no_request_are_not_written(b):
    c = _case([40, 20], [2, 1], 32, 2, 128, 8, torch.bfloat16, seed=3)
    c["q"] = torch.cat([c["q"], c["q"], c["q"]])
    c["q_start"] = c["q_start"] + 3
    o, ws = _run(b, c, 0.125)
    assert b.device_status(ws) == 0
    assert (o["out"][:3] == 77).all() and (o["out"][6:] == 77).all() and (o["lse"][:3] == 77).all()
    inner = dict(c, q=c["q"][3:6], q_start=c["q_start"] - 3)
    _compare(inner, dict(out=o["out"][3:6], lse=o["lse"][3:6]), 0.125)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_many_short_contexts(b, dtype, cache):
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 500, 220).tolist()
    new = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 9, 220))]
    _check(b, _case(lens, new, 32, 2, 128, 16, dtype, cache, seed=2, garbage=False))


@pytest.mark.parametrize("gone", [-1, 1 << 20])
@pytest.mark.parametrize("dtype,cache", TYPES[:3])
@pytest.mark.parametrize("Hq,D,ps", [(4, 64, 8), (4, 64, 5), (4, 256, 16), (32, 128, 8), (32, 64, 16)])
def test_pages_before_every_window_may_be_gone(b, dtype, cache, Hq, D, ps, gone):
    """Pages that no query sees any more need not be in the table, and are not reported; one that the
    first query still sees is."""
    lens, new, window = [37, 300, 513, 90], [1, 3, 5, 2], 21
    c = _case(lens, new, Hq, 2, D, ps, dtype, cache, seed=23, garbage=False)
    want = _check(b, c, window=window)
    for r, (n, m) in enumerate(zip(lens, new)):
        c["table"][r, : max(0, n - m - window + 1) // ps] = gone
    o, ws = _run(b, c, D ** -0.5, window)
    assert b.device_status(ws) == 0
    assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])
    c["table"][1, (300 - 3 - window + 1) // ps] = gone
    o, ws = _run(b, c, D ** -0.5, window)
    assert b.device_status(ws) == 1
