"""dspark_chunk_attention against a 64-bit form: blocks of any length, mixed with single queries, of every
type and head layout, over pages that end anywhere, windows, strides, what a query must not see, bad
tables, streams and graphs.  The tolerances are those of tests/test_gpu_attention.py."""
import math

import numpy as np
import pytest
import torch

from tests import position_ref as ref
from tests.test_gpu_attention import HALF_STEP, _case, _i32

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
TYPES = [(torch.bfloat16, None), (torch.float16, None), (torch.bfloat16, E4M3), (torch.float16, E4M3)]


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _run(b, c, scale, window=0, dev=None, ws=None, **kw):
    d = dict(q=c["q"].cuda(), k=c["k"].cuda(), v=c["v"].cuda())
    d.update(dev or {})
    ks, vs = (None if s is None else s.cuda() for s in c["scales"])
    T, Hq, D = c["q"].shape
    ws = b.workspace(b.chunk_attention_workspace_size(T, len(c["lens"]), Hq, c["k"].shape[1], D), "cuda") if ws is None else ws
    out = dict(out=torch.full((T, Hq, D), 77.0, dtype=c["q"].dtype, device="cuda"),
               lse=torch.full((T, Hq), 77.0, device="cuda"))
    o = b.chunk_attention(d["q"], d["k"], d["v"], _i32(c["table"]), _i32(c["lens"]), _i32(c["q_start"]), scale, k_scale=ks,
                          v_scale=vs, window=window, out=out, ws=ws, **kw)
    return o, ws


def _compare(c, o, scale, window=0, lens=None):
    q64, k64, v64 = (c[n].cuda().to(torch.float64) if c[n].dtype != E4M3 else c[n].cuda().float().double()
                     for n in ("q", "k", "v"))
    lens = c["lens"] if lens is None else lens
    want, lse, mag, dot = ref.attention(q64, k64, v64, c["table"], lens, c["q_start"], scale, *c["scales"], window=window)
    got, got_lse = o["out"].double(), o["lse"].double()
    D, L, e = c["q"].shape[2], max(c["lens"]), 2.0 ** -24
    delta = e * (D + 8) * dot
    h = HALF_STEP[c["q"].dtype]
    hw = 2.0 ** -11 if c["k"].dtype == E4M3 else h
    sums = e * (L / 8 + 64)
    empty = lse == -math.inf
    assert torch.equal(got_lse == -math.inf, empty)
    assert (got[empty] == 0).all()
    tol = delta + sums + e * lse.abs()
    bad = ~((got_lse - lse).abs() <= tol) & ~empty & ~torch.isnan(lse)
    assert not bad.any(), (bad.nonzero()[0].tolist(), got_lse[bad][0].item(), lse[bad][0].item(), tol[bad][0].item())
    tol = (hw + sums + 2 * delta[..., None]) * mag + h * want.abs() + 1e-7
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), ~odd)
    bad = ~((got - want).abs() <= tol) & ~odd
    assert not bad.any(), (bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item(), tol[bad][0].item(),
                           int(bad.sum()))


def _check(b, c, scale=None, window=0, lens=None, **kw):
    scale = c["q"].shape[2] ** -0.5 if scale is None else scale
    o, ws = _run(b, c, scale, window, **kw)
    assert b.device_status(ws) == 0
    _compare(c, o, scale, window, lens)
    return o


# (Hq, H, D, page): pages of 5 and D = 256 go by rows
LAYOUTS = [(1, 1, 16, 8), (4, 4, 64, 16), (8, 2, 128, 16), (8, 2, 80, 5), (4, 1, 256, 64), (40, 8, 48, 24), (7, 1, 112, 128),
           (64, 1, 128, 32), (5, 1, 64, 8), (3, 3, 128, 64), (12, 2, 96, 40)]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D,ps", LAYOUTS)
def test_blocks_of_any_length(b, dtype, cache, Hq, H, D, ps):
    lens = [1, 129, 300, 0, 520, 700, 128, 257, 40, 1000]
    new = [1, 129, 140, 0, 520, 3, 128, 256, 17, 131]
    _check(b, _case(lens, new, Hq, H, D, ps, dtype, cache, seed=D))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("G,n", [(1, 127), (1, 128), (1, 129), (1, 255), (1, 256), (1, 257), (1, 513), (4, 31), (4, 32), (4, 33),
                                 (4, 63), (4, 64), (4, 65), (4, 191), (6, 43), (6, 85), (6, 86)])
def test_blocks_around_a_tile(b, dtype, cache, G, n):
    """Query rows around one and two tiles of 128, over contexts that end around a tile of keys."""
    lens = [n, n + 1, n + 127, n + 128, n + 129, 384 + n % 3]
    _check(b, _case(lens, [min(n, x) for x in lens], G, 1, 128, 16, dtype, cache, seed=n))


@pytest.mark.parametrize("dtype,cache", [TYPES[0], TYPES[3]])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 128, 129, 200, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (2, 2, 64)])
def test_windows(b, dtype, cache, window, Hq, H, D):
    lens, new = [700, 129, 1500, 300, 5], [300, 129, 150, 1, 5]
    c = _case(lens, new, Hq, H, D, 16, dtype, cache, seed=window % 97)
    _check(b, c, window=window)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_pages_before_every_window_may_be_gone(b, dtype, cache):
    c = _case([900, 700], [130, 200], 8, 2, 128, 16, dtype, cache)
    for r, (n, m) in enumerate(zip(c["lens"], c["new"])):
        c["table"][r, :(n - m - 100 + 1) // 16] = -1
    _check(b, c, window=100)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_long_contexts_split_over_the_card(b, dtype, cache):
    """One request whose few items are shared by many SMs; a whole prompt; many short ones."""
    _check(b, _case([20000], [140], 8, 2, 128, 64, dtype, cache, seed=1))
    _check(b, _case([2500], [2500], 8, 2, 128, 16, dtype, cache, seed=2))
    n = [1 + 37 * i % 200 for i in range(150)]
    _check(b, _case([x + 11 * i % 90 for i, x in enumerate(n)], n, 4, 1, 64, 16, dtype, cache, seed=3))


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_same_answers_as_the_call_for_short_blocks(b, dtype, cache):
    """Within both calls' tolerances, a block of 128 queries is what paged_attention gives."""
    c = _case([1000, 700], [128, 100], 8, 2, 128, 16, dtype, cache, seed=5)
    o, _ = _run(b, c, 0.1)
    ks, vs = (None if s is None else s.cuda() for s in c["scales"])
    p = b.paged_attention(c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), _i32(c["table"]), _i32(c["lens"]), _i32(c["q_start"]), 128,
                          0.1, k_scale=ks, v_scale=vs)
    _compare(c, o, 0.1)
    _compare(c, p, 0.1)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("nq,tail", [(1, 17.0), (150, 17.0), (150, 25.5)])
def test_a_long_tail_of_small_weights(b, dtype, cache, nq, tail):
    """One likely token, and 70,000 whose weights are 2^-tail of its own; its value is 0, so the output is
    the tail's alone."""
    n = 70000
    c = _case([n], [nq], 2, 1, 64, 64, dtype, cache, seed=21, garbage=False)
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
    _check(b, c, scale=tail * math.log(2.0) / 32.0)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("per_tile", [-12.0, 3.0, 20.0])
def test_scores_that_grow_along_the_context(b, dtype, cache, per_tile):
    """Scores of 2^per_tile more (or less) every 128 tokens, for half of the heads; the others' shrink."""
    lens, nq = [3001, 1500], 150
    c = _case(lens, [nq] * 2, 8, 2, 128, 64, dtype, cache, seed=17, garbage=False)
    step = per_tile * math.log(2.0) / 128.0 * 8.0
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


def test_large_small_and_negative_scales(b):
    for scale, mult in ((1.0, 30.0), (-0.5, 1.0), (0.0, 1.0), (1e-3, 1e-3)):
        c = _case([177, 200, 900], [150, 1, 130], 8, 2, 128, 16, torch.bfloat16, seed=4)
        c["q"] = (c["q"].float() * mult).to(torch.bfloat16)
        _check(b, c, scale=scale)
    for mult, scale in ((1e6, 1e-7), (1e-12, 1e11), (1.0, -0.1)):  # queries past fp16's range over an e4m3 cache
        c = _case([177, 200], [150, 1], 8, 2, 128, 16, torch.bfloat16, E4M3, seed=4)
        c["q"] = (c["q"].float() * mult).to(torch.bfloat16)
        _check(b, c, scale=scale)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_what_some_queries_do_not_see(b, dtype, cache, window, what):
    """Keys and values that are not finite, at positions that only the later (or, with a window, the
    earlier) queries of a block see, and that none sees."""
    if cache and what == math.inf:
        pytest.skip("e4m3 has no infinities")
    c = _case([300, 700], [200, 300], 4, 1, 128, 16, dtype, cache, seed=6)
    k, v = c["k"].float(), c["v"].float()
    for r, j, pool in ((0, 150, v), (0, 222, v), (0, 223, v), (1, 500, v), (1, 640, k), (1, 401, v)):
        pool[c["table"][r, j // 16], 0, j % 16, 3 * r:3 * r + 2] = what
    c["k"], c["v"] = k.to(c["k"].dtype), v.to(c["v"].dtype)
    o, ws = _run(b, c, 0.1, window)
    assert b.device_status(ws) == 0
    q, kk, vv = c["q"].double().cuda(), c["k"].float().double().cuda(), c["v"].float().double().cuda()
    want, lse, mag, _ = ref.attention(q, kk, vv, c["table"], c["lens"], c["q_start"], 0.1, *c["scales"], window=window)
    got = o["out"].double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine)
    assert fine.any(2).any() and (~fine).any()
    # (the rows that see nothing odd, to the usual tolerance)
    hw = 2.0 ** -11 if cache == E4M3 else HALF_STEP[dtype]
    tol = (hw + 2.0 ** -12) * torch.where(fine, mag, 0) + HALF_STEP[dtype] * torch.where(fine, want, 0).abs() + 1e-7
    assert ((torch.where(fine, got - want, 0)).abs() <= tol).all()


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_strides_of_queries_and_pools(b, dtype, cache):
    c = _case([300, 131, 20], [200, 131, 3], 6, 2, 64, 16, dtype, cache, seed=7)
    T = c["q"].shape[0]
    packed = torch.full((T, 11, 64), math.nan, dtype=dtype, device="cuda")
    packed[:, 2:8] = c["q"].cuda()
    tokens_first = {n: c[n].cuda().transpose(1, 2).contiguous().transpose(1, 2) for n in ("k", "v")}
    want, _ = _run(b, c, 0.125)
    _compare(c, want, 0.125)
    got, _ = _run(b, c, 0.125, dev=dict(q=packed[:, 2:8], **tokens_first))
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    # one query's row read by every head; one head's pool seen as two
    d = dict(c, q=c["q"][:, :1].expand(-1, 6, -1))
    got, _ = _run(b, d, 0.125, dev=dict(q=c["q"][:, :1].cuda().expand(-1, 6, -1)))
    _compare(d, got, 0.125)
    d = dict(c, **{n: c[n][:, :1].expand(-1, 2, -1, -1) for n in ("k", "v")})
    got, _ = _run(b, d, 0.125, dev={n: c[n][:, :1].contiguous().cuda().expand(-1, 2, -1, -1) for n in ("k", "v")})
    _compare(d, got, 0.125)


@pytest.mark.parametrize("dtype,cache", [TYPES[0], TYPES[2]])
def test_offsets_past_32_bits(b, dtype, cache):
    size = 1 if cache else 2
    pages = (1 << 32) // (64 * 128 * size) + 40
    c = _case([400], [200], 4, 1, 128, 64, dtype, cache, seed=8, extra=0)
    place = torch.tensor([pages - 1, 5, pages - 30, 7, pages - 2, 0, pages - 9][:c["k"].shape[0]])
    dev = {}
    for n in ("k", "v"):
        big = torch.empty((pages, 1, 64, 128), dtype=c[n].dtype, device="cuda")
        for i, p in enumerate(place.tolist()):
            big[p] = c[n][i].cuda()
        dev[n] = big
    small = {n: c[n] for n in ("k", "v")}
    table = c["table"]
    c["table"] = place.numpy()[table]
    o, ws = _run(b, c, 0.09, dev=dev)
    assert b.device_status(ws) == 0
    _compare(dict(c, table=table, **small), o, 0.09)


def test_refused_slots_and_rows_of_no_slot(b):
    c = _case([300, 200, 150], [200, 100, 150], 4, 2, 128, 16, torch.bfloat16, seed=9)
    o, ws = _run(b, c, 0.1, granted=_i32([200, 0, 150]))
    assert b.device_status(ws) == 0
    assert (o["out"][200:300] == 0).all() and (o["lse"][200:300] == -math.inf).all()
    _compare(c, o, 0.1, lens=[300, 0, 150])
    # queries past and before the slots'
    big = dict(c, q=torch.cat([c["q"][:7], c["q"], c["q"][:200]]), q_start=c["q_start"] + 7)
    o, ws = _run(b, big, 0.1)
    assert b.device_status(ws) == 0
    assert (o["out"][:7] == 77).all() and (o["out"][457:] == 77).all() and (o["lse"][457:] == 77).all()
    _compare(c, dict(out=o["out"][7:457], lse=o["lse"][7:457]), 0.1)
    # more queries than the context has positions: the first ones see nothing
    c = _case([100, 300], [150, 300], 4, 2, 128, 16, torch.bfloat16, seed=10)
    _check(b, c)
    # no queries at all
    c = _case([100, 300], [0, 0], 4, 2, 128, 16, torch.bfloat16, seed=10)
    o, ws = _run(b, c, 0.1)
    assert b.device_status(ws) == 0 and o["out"].numel() == 0
    big = dict(c, q=torch.zeros((9, 4, 128), dtype=torch.bfloat16))
    o, ws = _run(b, big, 0.1)
    assert (o["out"] == 77).all() and b.device_status(ws) == 0


@pytest.mark.parametrize("cache", [None, E4M3])
def test_bad_tables_are_reported(b, cache):
    c = _case([300, 200, 150], [200, 100, 150], 4, 2, 128, 16, torch.bfloat16, cache, seed=11, garbage=False)
    want, _ = _run(b, c, 0.1)
    for bad in (-1, 1 << 30, c["k"].shape[0]):
        d = dict(c, table=c["table"].copy())
        d["table"][1, 2] = bad
        o, ws = _run(b, d, 0.1)
        assert b.device_status(ws) == 1
        for t in (slice(0, 200), slice(300, 450)):
            assert torch.equal(o["out"][t], want["out"][t])
        zeroed = {n: c[n].clone() for n in ("k", "v")}  # the page reads as zeros
        for n in zeroed:
            zeroed[n].view(torch.uint8 if cache else torch.int16)[c["table"][1, 2]] = 0
        _compare(dict(c, **zeroed), o, 0.1)
    for lens, q_start in (([300, -1, 150], None), ([300, 1 << 30, 150], None), (None, [0, 200, 100, 450]), (None, [0, 200, 300, 451]),
                          (None, [-5, 200, 300, 450])):
        d = dict(c, lens=lens or c["lens"], q_start=np.array(q_start) if q_start else c["q_start"])
        o, ws = _run(b, d, 0.1)
        assert b.device_status(ws) == 1
        if lens:
            assert (o["out"][200:300] == 77).all() and torch.equal(o["out"][:200], want["out"][:200])


@pytest.mark.parametrize("cache", [None, E4M3])
def test_repeated_streams_and_graphs(b, cache):
    """The same bits every time, on another stream, from a graph replayed over other lengths, and from two
    graphs with a workspace each that replay at once."""
    c = _case([3000, 200, 150], [300, 100, 150], 8, 2, 128, 16, torch.bfloat16, cache, seed=12)
    want, ws = _run(b, c, 0.1)
    for _ in range(3):
        o, _ = _run(b, c, 0.1, ws=ws)
        assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, _ = _run(b, c, 0.1, stream=side)
    side.synchronize()
    assert torch.equal(o["out"], want["out"])
    ks, vs = (None if s is None else s.cuda() for s in c["scales"])
    lens, args = _i32(c["lens"]), [c[n].cuda() for n in ("q", "k", "v")]
    table, q_start = _i32(c["table"]), _i32(c["q_start"])
    graphs, outs = [], []
    for _ in range(2):
        outs.append(dict(out=torch.zeros_like(args[0]), lse=torch.zeros(args[0].shape[:2], device="cuda")))
        w = torch.zeros_like(ws)
        w = w[(-w.data_ptr()) % 256:]
        w = b.workspace(ws.numel(), "cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.chunk_attention(*args, table, lens, q_start, 0.1, k_scale=ks, v_scale=vs, out=outs[-1], ws=w)
        graphs.append((g, w))
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(other):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for x in outs:
        assert torch.equal(x["out"], want["out"]) and torch.equal(x["lse"], want["lse"])
    lens -= torch.tensor([100, 50, 0], dtype=torch.int32, device="cuda")
    graphs[0][0].replay()
    torch.cuda.synchronize()
    _compare(dict(c, lens=lens.tolist()), outs[0], 0.1)


def test_cache_attends_over_long_blocks(b):
    """PagedCache.attend hands blocks of more than 128 queries to this call, refused slots included."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    cache = b.PagedCache(3, 40, 16, 30, 1, 2, 64)
    rates = b.rotary_rates(64)
    new = [200, 150, 400]
    plan = cache.reserve(_i32(new))
    assert plan["granted"].tolist() == [200, 150, 0]  # 13 and 10 of 40 pages; 25 do not fit
    q, k, v = rnd(750, 8, 64), rnd(750, 2, 64), rnd(750, 2, 64)
    q_start = _i32([0, 200, 350, 750])
    turned = cache.append(0, q, k, v, q_start, rates)
    o = cache.attend(0, turned, q_start, 400, 0.125)
    assert cache.status() == 0
    assert (o["out"][350:] == 0).all() and (o["lse"][350:] == -math.inf).all()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in new]).cuda()
    rq, rk = b.rotary(q, pos, rates), b.rotary(k, pos, rates)
    assert torch.equal(turned[:350], rq[:350])
    for t in (slice(0, 200), slice(200, 350)):
        kk, vv = rk[t].double().repeat_interleave(4, 1), v[t].double().repeat_interleave(4, 1)
        s = torch.einsum("qhd,khd->hqk", rq[t].double(), kk) * 0.125
        n = s.shape[1]
        s = s.masked_fill(~torch.ones((n, n), dtype=torch.bool, device="cuda").tril(), -math.inf)
        w = torch.softmax(s, 2)
        want = torch.einsum("hqk,khd->qhd", w, vv)
        mag = torch.einsum("hqk,khd->qhd", w, vv.abs())
        assert ((o["out"][t].double() - want).abs() <= 2.0 ** -8 * (mag + want.abs()) * 1.01 + 1e-6).all()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("window", [0, 150])
def test_many_items_with_values_that_some_do_not_see(b, dtype, cache, window):
    """Values that are NaN in every request, near the diagonal and along the blocks, with several items of two
    row tiles a CTA: each row has them in its sums, or not, by what it sees alone."""
    g = torch.Generator().manual_seed(21)
    new = torch.randint(250, 400, (24,), generator=g).tolist()
    before = torch.randint(0, 300, (24,), generator=g).tolist()
    c = _case([x + y for x, y in zip(new, before)], new, 16, 8, 64, 16, dtype, cache, seed=22)
    v = c["v"].float()
    for r in range(24):
        for j in torch.randint(0, new[r], (3,), generator=g).tolist():
            at, h = before[r] + j, int(torch.randint(0, 8, (1,), generator=g))
            v[c["table"][r, at // 16], h, at % 16, h:h + 2] = math.nan
    c["v"] = v.to(c["v"].dtype)
    out = _check(b, c, 0.125, window)["out"].float()
    assert torch.isnan(out).any() and torch.isfinite(out).any()
