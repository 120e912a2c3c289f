"""dspark_paged_attention against a 64-bit form: types, head layouts, lengths from zero to
long, odd sizes, pages that end anywhere, windows, strides, what a query must not see (NaN and
infinities included), offsets past 32 bits, bad tables, streams and graphs.

Tolerances.  Scores are fp32 sums of D products: each is off by at most
d = 2^-24 (D + 8) max_j sum |q k_j| scale, and so is the normaliser, which adds
2^-24 (L/8 + 64 + |lse|) for its own sum.  The output adds, relative to sum_j w_j |v_j|, one
rounding of each weight to 16 bits (half a step h: 2^-8 bf16, 2^-11 fp16), the sum's
2^-24 (L/8 + 64) and 2 d, and one rounding to the output's type (h relative to the output).
With an e4m3 cache the weights, and the queries scaled by a power of two, are fp16."""
import math

import numpy as np
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _case(lens, new, Hq, H, D, ps, dtype, cache=None, seed=0, extra=2, garbage=True, scale_v=1.0):
    """Pools whose free pages and page tails hold NaN where `garbage`."""
    cache = cache or dtype
    R = len(lens)
    g = torch.Generator().manual_seed(seed)
    W = max(1, max(-(-n // ps) for n in lens))
    per = [-(-n // ps) for n in lens]
    P = sum(per) + extra
    order = np.random.default_rng(seed).permutation(P)
    table = np.full((R, W), -1)
    at = 0
    for r in range(R):
        table[r, :per[r]] = order[at:at + per[r]]
        at += per[r]
    pools = []
    for _ in range(2):
        x = torch.randn((P, H, ps, D), generator=g)
        if garbage:
            live = torch.zeros((P, ps), dtype=torch.bool)
            for r in range(R):
                for j in range(lens[r]):
                    live[table[r, j // ps], j % ps] = True
            x[~live[:, None, :].expand(P, H, ps)] = math.nan
        pools.append(x.to(cache))
    T = sum(new)
    q = (torch.randn((T, Hq, D), generator=g) * 1.5).to(dtype)
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(int)
    scales = (None, None)
    if cache == torch.float8_e4m3fn:
        scales = tuple(torch.rand(H, generator=g) + 0.5 for _ in range(2))
    return dict(q=q, k=pools[0], v=pools[1], table=table, lens=list(lens), new=list(new), q_start=q_start,
                scales=scales, ps=ps)


def _run(b, c, scale, window=0, dev=None, max_q=None, ws=None, **kw):
    d = dict(q=c["q"].cuda(), k=c["k"].cuda(), v=c["v"].cuda())
    d.update(dev or {})
    ks, vs = (None if s is None else s.cuda() for s in c["scales"])
    T, Hq, D = c["q"].shape
    max_q = max_q or max(1, max(c["new"]))
    ws = b.workspace(b.paged_attention_workspace_size(T, len(c["lens"]), Hq, c["k"].shape[1], D, max_q),
                     "cuda") if ws is None else ws
    out = dict(out=torch.full((T, Hq, D), 77.0, dtype=c["q"].dtype, device="cuda"),
               lse=torch.full((T, Hq), 77.0, device="cuda"))
    o = b.paged_attention(d["q"], d["k"], d["v"], _i32(c["table"]), _i32(c["lens"]), _i32(c["q_start"]), max_q, scale,
                          k_scale=ks, v_scale=vs, window=window, out=out, ws=ws, **kw)
    return o, ws


def _compare(c, o, scale, window=0):
    q64, k64, v64 = (c[n].cuda().to(torch.float64) if c[n].dtype != torch.float8_e4m3fn
                     else c[n].cuda().float().double() for n in ("q", "k", "v"))
    want, lse, mag, dot = ref.attention(q64, k64, v64, c["table"], c["lens"], c["q_start"], scale, *c["scales"],
                                        window=window)
    got, got_lse = o["out"].double(), o["lse"].double()
    D = c["q"].shape[2]
    L = max(c["lens"])
    e = 2.0 ** -24
    delta = e * (D + 8) * dot
    h = HALF_STEP[c["q"].dtype]
    hw = 2.0 ** -11 if c["k"].dtype == torch.float8_e4m3fn else h
    sums = e * (L / 8 + 64)
    empty = lse == -math.inf
    assert torch.equal(got_lse == -math.inf, empty)
    assert (got[empty] == 0).all()
    tol = delta + sums + e * lse.abs()
    bad = ((got_lse - lse).abs() > tol) & ~empty
    assert not bad.any(), (bad.nonzero()[0].tolist(), got_lse[bad][0].item(), lse[bad][0].item(), tol[bad][0].item())
    tol = (hw + sums + 2 * delta[..., None]) * mag + h * want.abs() + 1e-7
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item(), tol[bad][0].item(),
                           int(bad.sum()))


def _check(b, c, scale=None, window=0, **kw):
    scale = c["q"].shape[2] ** -0.5 if scale is None else scale
    o, ws = _run(b, c, scale, window, **kw)
    assert b.device_status(ws) == 0
    _compare(c, o, scale, window)
    return o


TYPES = [(torch.bfloat16, None), (torch.float16, None), (torch.bfloat16, torch.float8_e4m3fn),
         (torch.float16, torch.float8_e4m3fn)]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D,ps", [(1, 1, 16, 1), (4, 4, 64, 16), (8, 2, 128, 16), (6, 2, 80, 5), (8, 1, 256, 64),
                                       (40, 8, 48, 24), (16, 1, 112, 128), (5, 1, 64, 8), (64, 1, 128, 32)])
def test_one_new_token(b, dtype, cache, Hq, H, D, ps):
    lens = [1, 2, 15, 16, 17, 31, 64, 65, 127, 128, 129, 300]
    _check(b, _case(lens, [1] * len(lens), Hq, H, D, ps, dtype, cache, seed=D + ps))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D,ps", [(2, 2, 64, 16), (8, 2, 128, 16), (6, 2, 80, 7), (8, 1, 256, 64), (32, 8, 128, 32),
                                       (16, 2, 128, 1)])
def test_verified_block(b, dtype, cache, Hq, H, D, ps):
    new = [0, 1, 2, 5, 8, 16, 3, 1]
    lens = [40, 1, 2, 64, 100, 16, 259, 0]
    lens[-1], new[-1] = 0, 0
    _check(b, _case(lens, new, Hq, H, D, ps, dtype, cache, seed=D))


@pytest.mark.parametrize("Hq,H", [(1, 1), (8, 1), (64, 1), (6, 3)])
def test_long_blocks(b, Hq, H):
    """Up to 128 queries a request: more rows than one tile holds."""
    _check(b, _case([128, 150, 400], [128, 33, 100], Hq, H, 64, 16, torch.bfloat16, seed=3))


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_queries_that_see_nothing(b, dtype, cache):
    """More queries than context (their positions are negative), and empty contexts."""
    _check(b, _case([0, 3, 1, 20], [2, 5, 4, 20], 4, 2, 64, 4, dtype, cache, seed=5))


@pytest.mark.parametrize("window", [1, 2, 7, 64, 100, 1000])
@pytest.mark.parametrize("dtype,cache", TYPES[:3])
def test_window(b, window, dtype, cache):
    _check(b, _case([1, 50, 333, 700, 65], [1, 6, 4, 1, 3], 8, 2, 64, 16, dtype, cache, seed=window), window=window)


@pytest.mark.parametrize("Hq,window", [(4, 2 ** 31 - 1), (4, 2 ** 31 - 9), (32, 2 ** 31 - 1)])
def test_window_beyond_any_context(b, Hq, window):
    """Windows near 32 bits with more queries than context (negative positions), narrow and wide blocks."""
    _check(b, _case([2, 30, 0, 70], [8, 8, 3, 5], Hq, 2, 64, 16, torch.bfloat16, seed=9), window=window)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_long_context(b, dtype, cache):
    _check(b, _case([20011, 3, 9000], [1, 1, 2], 8, 2, 128, 16, dtype, cache, seed=1, garbage=False))


def test_many_requests(b):
    rng = np.random.default_rng(0)
    lens = rng.integers(1, 400, 700).tolist()
    _check(b, _case(lens, [1] * 700, 4, 1, 64, 16, torch.bfloat16, seed=2, garbage=False))
    new = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 6, 700))]
    _check(b, _case(lens, new, 8, 2, 64, 32, torch.float16, seed=2, garbage=False))


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_unseen_values_have_no_influence(b, dtype, cache):
    """NaN and infinities in what a query does not see: later tokens of its own block, and
    tokens before its window."""
    for Hq, H, nq in ((4, 2, 3), (16, 2, 8)):
        c = _case([40, 70], [nq, nq], Hq, H, 64, 8, dtype, cache, seed=9)
        clean = _check(b, c)
        bad = float("nan") if cache else float("inf")
        for r, n in enumerate(c["lens"]):
            page = c["table"][r, (n - 1) // 8]
            for pool in (c["k"], c["v"]):
                x = pool.float()
                x[page, :, (n - 1) % 8] = bad
                x[page, :, (n - 1) % 8, 5] = math.nan
                pool.copy_(x.to(pool.dtype))
        o, _ = _run(b, c, 64 ** -0.5)
        last = [c["q_start"][r + 1] - 1 for r in range(2)]
        rest = [t for t in range(2 * nq) if t not in last]
        assert torch.equal(o["out"][rest], clean["out"][rest]) and torch.equal(o["lse"][rest], clean["lse"][rest])
        assert torch.isnan(o["out"][last].float()).any()
        c = _case([40, 70], [nq, nq], Hq, H, 64, 8, dtype, cache, seed=9)
        clean = _check(b, c, window=20)
        for r, n in enumerate(c["lens"]):  # the last query sees n-20..n-1, the first n-nq-19..n-nq
            for j in range(n - nq - 19 + 1):
                for pool in (c["k"], c["v"]):
                    x = pool[c["table"][r, j // 8], :, j % 8].float()
                    pool[c["table"][r, j // 8], :, j % 8] = torch.full_like(x, math.nan).to(pool.dtype)
        o, _ = _run(b, c, 64 ** -0.5, 20)
        first = [c["q_start"][r] for r in range(2)]
        rest = [t for t in range(2 * nq) if t not in first]
        assert torch.equal(o["out"][rest], clean["out"][rest]) and torch.equal(o["lse"][rest], clean["lse"][rest])


def test_large_and_small_scores(b):
    for scale, mult in ((1.0, 30.0), (-0.5, 1.0), (0.0, 1.0), (1e-3, 1e-3)):
        c = _case([77, 200], [1, 4], 8, 2, 64, 16, torch.bfloat16, seed=4)
        c["q"] = (c["q"].float() * mult).to(torch.bfloat16)
        _check(b, c, scale=scale)
    # queries past fp16's range over an e4m3 cache
    c = _case([77, 200], [1, 4], 8, 2, 64, 16, torch.bfloat16, torch.float8_e4m3fn, seed=4)
    c["q"] = (c["q"].float() * 1e6).to(torch.bfloat16)
    _check(b, c, scale=1e-7)
    c["q"] = (c["q"].float() * 1e-12).to(torch.bfloat16)
    c["q"][0] = 0
    _check(b, c, scale=1e5)


@pytest.mark.parametrize("dtype,cache", TYPES[:3])
def test_strides(b, dtype, cache):
    """Pools [P, ps, H, D] seen as [P, H, ps, D], inside a larger allocation; queries that are a
    slice of a wider projection; a page table that is a slice."""
    c = _case([33, 70, 9], [2, 1, 3], 8, 2, 64, 16, dtype, cache, seed=6)
    P, H, ps, D = c["k"].shape
    pools = []
    for n in ("k", "v"):
        big = torch.zeros((P, ps + 1, H, D + 32), dtype=torch.uint8, device="cuda").to(c[n].dtype) \
            if not cache else torch.zeros((P, ps + 1, H, D + 32), dtype=torch.uint8, device="cuda").view(cache)
        view = big[:, :ps, :, 16:16 + D].permute(0, 2, 1, 3)
        view.copy_(c[n].cuda())
        pools.append(view)
    wide = torch.zeros((6, 3, 8, D + 16), dtype=dtype, device="cuda")
    q = wide[:, 1, :, 8:8 + D]
    q.copy_(c["q"].cuda())
    o, ws = _run(b, c, 0.125, dev=dict(q=q, k=pools[0], v=pools[1]))
    assert b.device_status(ws) == 0
    _compare(c, o, 0.125)


def test_offsets_past_32_bits(b):
    """Pages 1.5 GB apart: element and byte offsets pass 32 bits."""
    for dtype, cache, stride in ((torch.bfloat16, None, 1_500_000_000), (torch.float16, torch.float8_e4m3fn, 2_400_000_000)):
        c = _case([60, 20], [1, 3], 4, 2, 64, 16, dtype, cache, seed=7, extra=0)
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


def test_bad_tables_are_reported_and_harmless(b):
    base = dict(seed=8, garbage=False)
    for what in ("page", "len", "negative", "queries", "order"):
        c = _case([40, 40, 40], [2, 2, 2], 4, 2, 64, 8, torch.bfloat16, **base)
        kw = {}
        if what == "page":
            c["table"][1, 2] = 1 << 20
        elif what == "len":
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
        good = _case([40, 40, 40], [2, 2, 2], 4, 2, 64, 8, torch.bfloat16, **base)
        if what == "queries":
            good["q_start"], good["new"] = np.array([0, 1, 5, 6]), [1, 4, 1]
        want, _ = _run(b, good, 0.125)
        n0 = c["q_start"][1]
        assert torch.equal(o["out"][:n0], want["out"][:n0]), what


def test_queries_of_no_request_are_not_written(b):
    c = _case([40, 20], [2, 1], 4, 2, 64, 8, torch.bfloat16, seed=3)
    c["q"] = torch.cat([c["q"], c["q"], c["q"]])
    c["q_start"] = c["q_start"] + 3
    o, ws = _run(b, c, 0.125)
    assert b.device_status(ws) == 0
    assert (o["out"][:3] == 77).all() and (o["out"][6:] == 77).all() and (o["lse"][:3] == 77).all()
    inner = dict(c, q=c["q"][3:6], q_start=c["q_start"] - 3)
    _compare(inner, dict(out=o["out"][3:6], lse=o["lse"][3:6]), 0.125)


@pytest.mark.parametrize("new", [[1, 1, 1], [4, 7, 2]])
@pytest.mark.parametrize("cache", [None, torch.float8_e4m3fn])
def test_deterministic_on_any_stream_and_in_a_graph(b, new, cache):
    c = _case([3000, 70, 900], new, 8, 2, 128, 16, torch.bfloat16, cache, seed=11)
    ks, vs = (None if s is None else s.cuda() for s in c["scales"])
    T, R, mq = sum(new), 3, max(new)
    args = (c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), _i32(c["table"]), _i32(c["lens"]), _i32(c["q_start"]), mq, 0.09)
    ws = b.workspace(b.paged_attention_workspace_size(T, R, 8, 2, 128, mq), "cuda")
    ws[256:].random_(0, 256)  # another call's leavings
    first = {k: v.clone() for k, v in b.paged_attention(*args, k_scale=ks, v_scale=vs, ws=ws).items()}
    out = {k: torch.zeros_like(v) for k, v in first.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.paged_attention(*args, k_scale=ks, v_scale=vs, ws=ws, out=out, stream=side)
    side.synchronize()
    assert all(torch.equal(out[k], first[k]) for k in first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.paged_attention(*args, k_scale=ks, v_scale=vs, ws=ws, out=out)
    for _ in range(3):
        out["out"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], first[k]) for k in first)
    # buffers made by the call itself, on the stream that it runs on
    for _ in range(3):
        mine = b.paged_attention(*args, k_scale=ks, v_scale=vs, stream=side)
        side.synchronize()
        assert torch.equal(mine["out"], first["out"]) and torch.equal(mine["lse"], first["lse"])
    # without the normalisers
    only = b.paged_attention(*args, k_scale=ks, v_scale=vs, ws=ws, out=dict(out=torch.zeros_like(first["out"])))
    assert torch.equal(only["out"], first["out"])


def test_no_queries(b):
    c = _case([5], [0], 2, 1, 64, 8, torch.bfloat16)
    o, _ = _run(b, c, 0.1)
    assert o["out"].shape == (0, 2, 64)
