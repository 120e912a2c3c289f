"""The ends of what the rotary, append, long-block attention and logit-adjustment calls take: the largest
sizes, scales and windows, and shapes at the borders of the kernels' fast paths."""
import decimal
import math

import numpy as np
import pytest
import torch

from tests import test_gpu_adjust as adjust
from tests import test_gpu_append as append
from tests import test_gpu_chunk_attention as chunk
from tests.test_gpu_attention import _case, _i32

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def test_query_rows_up_to_the_limit(b):
    """One request of 2^31 - 64 query rows: their count plus an item's does not fit 32 bits.  All but the last
    128 tokens lie before the context and see nothing."""
    T, G, D, n = (1 << 25) - 1, 64, 16, 128
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("the result takes 64 GB")
    g = torch.Generator().manual_seed(0)
    q = torch.randn((1, G, D), generator=g).bfloat16().cuda()
    k, v = (torch.randn((8, 1, 16, D), generator=g).bfloat16().cuda() for _ in range(2))
    out = torch.empty((T, G, D), dtype=torch.bfloat16, device="cuda")
    step = 1 << 21
    for t in range(0, T, step):
        out[t:t + step] = 77.0
    ws = b.workspace(b.chunk_attention_workspace_size(T, 1, G, 1, D), "cuda")
    b.chunk_attention(q.expand(T, G, D), k, v, _i32([np.arange(8)]), _i32([n]), _i32([0, T]), 0.25, out=dict(out=out), ws=ws)
    assert b.device_status(ws) == 0
    for t in range(0, T - n, step):
        assert not out[t:min(t + step, T - n)].any(), t
    kk, vv = (x.transpose(1, 2).reshape(n, D).double() for x in (k, v))
    s = torch.einsum("gd,sd->gs", q[0].double(), kk) * 0.25
    j = torch.arange(n, device="cuda")
    w = torch.softmax(s.expand(n, G, n).masked_fill(j > j[:, None, None], -math.inf), 2)
    want, mag = w @ vv, w @ vv.abs()
    # a half step of each weight and of the result, and fp32's sums
    assert ((out[T - n:].double() - want).abs() <= 2.0 ** -8 * (mag + want.abs()) + 2.0 ** -16 * mag).all()
    del out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,cache", [chunk.TYPES[0], chunk.TYPES[2]])
@pytest.mark.parametrize("D", [128, 256])
def test_the_longest_windows(b, dtype, cache, D):
    """Windows up to the limit with the call's rows, over slots with far more queries than positions: where the
    window of a query that sees nothing would begin lies at the end of 32 bits."""
    lens, new = [60, 100, 700], [700, 900, 300]
    c = _case(lens, new, 2, 1, D, 256, dtype, cache, seed=31)
    width = (1 << 23) - 2
    c["table"] = np.pad(c["table"], ((0, 0), (0, width - c["table"].shape[1])), constant_values=-1)
    window = (1 << 31) - 1024 - sum(new)
    with pytest.raises(b.DSparkError, match="must be below 2\\^31 - 1024"):
        chunk._run(b, c, 0.1, window)
    o, ws = chunk._run(b, c, 0.1, window - 1, granted=_i32([0, 900, 300]))
    assert b.device_status(ws) == 0
    small = dict(c, table=c["table"][:, :8])
    chunk._compare(small, o, 0.1, window - 1, lens=[0, 100, 700])


@pytest.mark.parametrize("words", [32, 40])
def test_a_mask_without_rows(b, words):
    """A step in which no row is under a grammar: masks of shape [0, words], every row's choice out of range."""
    x, c = adjust._case([3, 1], [40, 3], 1000, torch.bfloat16, seed=2, biases=3)
    d = adjust._gpu(c)
    want = b.adjust_logits(x, **d)
    mask = torch.zeros((0, words), dtype=torch.int32, device="cuda")
    for row in ([-1] * 4, [0, 7, -1, 2]):
        for out in (None, x.clone()):
            got = b.adjust_logits(x if out is None else out, **d, mask=mask, mask_row=_i32(row), out=out)
            assert torch.equal(got, want)
    # (a tensor of no rows may say any strides)
    odd = torch.as_strided(torch.zeros(1, dtype=torch.int32, device="cuda"), (0, words), (0, 0))
    assert torch.equal(b.adjust_logits(x, **d, mask=odd, mask_row=_i32([-1] * 4)), want)
    with pytest.raises(b.DSparkError, match="a mask row for each of the 4 rows, got 0"):
        b.adjust_logits(x, **d, mask=mask)
    with pytest.raises(b.DSparkError, match="at least 32 words"):
        b.adjust_logits(x, **d, mask=mask[:, :31], mask_row=_i32([-1] * 4))


@pytest.mark.parametrize("in_place", [False, True])
def test_inputs_written_just_before(b, in_place):
    """Everything that adjust_logits reads beside the logits, written by the kernels right before it on the stream,
    eagerly and in a graph: what it gives is what the same inputs give after a wait."""
    x, c = adjust._case([3, 8, 1, 5], [900, 3000, 0, 2000], 20001, torch.bfloat16, seed=3, biases=20, masks=6)
    names = [n for n in c if n != "q_start"]
    sets = []
    for seed in range(4):
        d = adjust._gpu(adjust._case([3, 8, 1, 5], [900, 3000, 0, 2000], 20001, torch.bfloat16, seed=seed, biases=20, masks=6)[1])
        sets.append(d)
    want = [b.adjust_logits(x, **d) for d in sets]
    torch.cuda.synchronize()
    live = {n: t.clone() for n, t in sets[0].items()}
    logits = x.clone()

    def step(i):
        logits.copy_(x)
        for n in names:
            live[n].copy_(sets[i][n])
        return b.adjust_logits(logits, **live, out=logits if in_place else None)

    graphs = []
    for i in range(4):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step(i)))
    for k in range(100):
        i = k * 7 % 4
        got = step(i)
        assert torch.equal(got, want[i]), k
        graphs[i][0].replay()
        assert torch.equal(graphs[i][1], want[i]), k


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_scales_of_keys_with_signs_and_without_a_value(b, dtype, scale):
    """An e4m3 cache whose heads' scales are positive, negative, NaN and 0, in long blocks as in short ones: signs
    count, a NaN reaches every query that sees something and no other head."""
    lens, new = [100, 300, 700], [150, 128, 300]  # (the first 50 queries see nothing)
    c = _case(lens, new, 8, 4, 128, 16, dtype, E4M3, seed=14)
    c["scales"] = (torch.tensor([0.7, -0.7, math.nan, 0.0]), c["scales"][1])
    o, ws = chunk._run(b, c, scale)
    assert b.device_status(ws) == 0
    chunk._compare(c, o, scale)
    out, lse = o["out"], o["lse"]
    assert torch.isnan(out[50:, 4:6]).all() and torch.isnan(lse[50:, 4:6]).all()
    assert (out[:50] == 0).all() and (lse[:50] == -math.inf).all() and torch.isfinite(out[50:, :4]).all()
    short = _case([100, 300], [128, 100], 8, 4, 128, 16, dtype, E4M3, seed=15)
    short["scales"] = c["scales"]
    o, _ = chunk._run(b, short, scale)
    ks, vs = (s.cuda() for s in short["scales"])
    p = b.paged_attention(short["q"].cuda(), short["k"].cuda(), short["v"].cuda(), _i32(short["table"]), _i32(short["lens"]),
                          _i32(short["q_start"]), 128, scale, k_scale=ks, v_scale=vs)
    for a in (o, p):
        chunk._compare(short, a, scale)
    assert torch.equal(torch.isnan(o["out"]), torch.isnan(p["out"])) and torch.equal(torch.isnan(o["lse"]), torch.isnan(p["lse"]))


def test_scores_of_a_scale_below_normal_products(b):
    """Products near fp32's end, brought back by a scale below 1e-37: the scores are ordinary ones."""
    c = _case([200, 300], [150, 129], 4, 1, 64, 16, torch.bfloat16, seed=16)
    c["q"], c["k"] = (c["q"].float() * 1.5e18).bfloat16(), (c["k"].float() * 1.5e18).bfloat16()
    chunk._check(b, c, scale=2e-38)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [math.inf, -math.inf, -3e38, -1e31, -1e19, -0.7, -1e-31, -1e-44, 0.0, -0.0, math.nan])
def test_divisions_by_any_scale(b, dtype, scale):
    """Values stored in an e4m3 cache by cache_append as by cache_write, whatever their scales: infinite, negative, 0 and
    NaN; bit for bit, but for the sign of a 0 that a negative scale divides."""
    make = lambda: append.Case([300], [300], 1, 2, 64, 16, dtype, E4M3, seed=2)
    c, d = make(), make()
    c.scales = [torch.tensor([scale, 1.0], device="cuda") for _ in range(2)]
    size = torch.tensor([1.0, 1e-3, 30.0], device="cuda").repeat(100)[:, None, None]
    c.v = (c.v.float() * size).to(dtype)
    c.v[7, :, 3], c.v[9, :, 60], c.v[11, :, 0], c.v[12, :, 1], c.v[13, :, 2] = math.inf, -math.inf, math.nan, 0.0, -0.0
    if dtype == torch.bfloat16:
        c.v[14:20] *= 1e36
    c.call(b, b.rotary_rates(64), q=None)
    b.cache_write(c.k, c.v, *d.pools, _i32(d.table), _i32(d.lens), _i32(d.q_start), k_scale=c.scales[0], v_scale=c.scales[1])
    got, want = (append._bits(x.pools[1]).int() for x in (c, d))
    if math.copysign(1.0, scale) < 0:  # (0 / s is -0: the quotient's -0 and the residual's +0 add up to +0, the same value)
        got, want = (torch.where(x == 128, 0, x) for x in (got, want))
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,cache", append.TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,H,D,rot,ps", [(1, 1, 16, 2, 1), (8, 2, 80, 40, 20), (6, 2, 80, 20, 5), (5, 1, 96, 24, 16), (64, 1, 48, 46, 8),
                                           (12, 4, 256, 250, 64), (3, 3, 64, 8, 16)])
def test_appends_that_turn_any_part(b, dtype, cache, interleaved, Hq, H, D, rot, ps):
    """Parts of a row that are no whole pieces: against the 64-bit form, the two calls one after the other, and in
    place inside a packed projection."""
    lens, new = [1, 5, 64, 130, 7, 300], [1, 5, 3, 30, 0, 2]
    rates = b.rotary_rates(rot)
    how = dict(interleaved=interleaved, magnitude=1.1)
    make = lambda: append.Case(lens, new, Hq, H, D, ps, dtype, cache, seed=D + rot)
    c, d, e = make(), make(), make()
    q_out = c.call(b, rates, **how)
    c.check(b, q_out, rates, **how)
    assert b.device_status(c.ws) == 0
    pos = _i32(c.positions())
    assert torch.equal(q_out, b.rotary(d.q, pos, rates, **how))
    b.cache_write(b.rotary(d.k, pos, rates, **how), d.v, *d.pools, _i32(d.table), _i32(d.lens), _i32(d.q_start),
                  k_scale=d.scales[0], v_scale=d.scales[1])
    assert torch.equal(append._bits(c.pools[1]), append._bits(d.pools[1]))
    if cache != E4M3:  # (an e4m3 cache takes the turned keys without a rounding between)
        assert torch.equal(append._bits(c.pools[0]), append._bits(d.pools[0]))
    packed = torch.cat([e.q, e.k, e.v], 1)
    e.q, e.k, e.v = packed[:, :Hq], packed[:, Hq:Hq + H], packed[:, Hq + H:]
    assert torch.equal(e.call(b, rates, q_out=e.q, **how), q_out)
    for x, y in zip(c.pools, e.pools):
        assert torch.equal(append._bits(x), append._bits(y))


def test_appends_of_any_part_leave_what_is_not_theirs(b):
    """Refused slots, rows of no slot, bad pages, elements that are not finite, a graph."""
    rates = b.rotary_rates(20)
    c = append.Case([40, 9, 100], [3, 2, 50], 4, 2, 80, 16, torch.bfloat16, torch.bfloat16, beyond=6)
    q_out = torch.full_like(c.q, 9.0)
    c.call(b, rates, q_out=q_out, granted=_i32([3, 0, 50]))
    c.check(b, q_out, rates, skip=[1])
    assert (q_out[3:5] == 9).all() and (q_out[55:] == 9).all() and b.device_status(c.ws) == 0
    c = append.Case([40, 9, 100], [3, 2, 50], 4, 2, 80, 16, torch.bfloat16, torch.bfloat16)
    c.table[1, 0] = 1 << 20
    q_out = torch.full_like(c.q, 9.0)
    c.call(b, rates, q_out=q_out)
    assert b.device_status(c.ws) == 1
    assert (q_out[3:5] == 9).all() and (q_out[:3] != 9).any() and (q_out[5:] != 9).any()
    c = append.Case([40], [3], 1, 1, 80, 16, torch.bfloat16, torch.bfloat16)
    c.k[1, 0, 3], c.k[1, 0, 40] = math.nan, math.inf  # of a pair, and past the part that turns
    c.call(b, rates, q=None)
    row = c.pools[0][c.table[0, 38 // 16], 0, 38 % 16]
    assert torch.isnan(row).nonzero()[:, 0].tolist() == [3, 13] and torch.equal(row[20:], c.k[1, 0, 20:])
    d = append.Case([40, 300], [30, 100], 6, 2, 80, 16, torch.float16, torch.float16)
    want, pools = d.call(b, rates), [p.clone() for p in d.pools]
    args, out = (_i32(d.table), _i32(d.lens), _i32(d.q_start)), torch.zeros_like(d.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.cache_append(d.q, d.k, d.v, *d.pools, *args, rates, ws=d.ws, q_out=out)
    for p in d.pools:
        p.fill_(3.0)
    g.replay()
    assert torch.equal(out, want) and all(torch.equal(x, y) for x, y in zip(d.pools, pools))


def test_paged_cache_appends_any_part(b):
    cache = b.PagedCache(2, 8, 16, 4, 1, 2, 80)
    cache.reserve(_i32([20, 7]))
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((27, h, 80), generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    rates = b.rotary_rates(40)
    pos = _i32(list(range(20)) + list(range(7)))
    assert torch.equal(cache.append(0, q, k, v, _i32([0, 20, 27]), rates), b.rotary(q, pos, rates))
    page = cache.page_table[1, 0].item()
    assert torch.equal(cache.k[0, page, :, :7], b.rotary(k, pos, rates)[20:].transpose(0, 1)) and cache.status() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_at_far_positions(b, interleaved):
    """The rotation of unit vectors at the ends of the positions' range, from the frequencies themselves in 90 digits:
    off by the angle's 1e-7 radians, a step of the sine and cosine and their rounding."""
    pi = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 1999999999, 1 << 30, 100003, 1, 0]
    x = torch.zeros((len(pos), 1, 64), device="cuda")
    u, w = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    x[..., u] = 1.0
    for how in (dict(), dict(scaling="linear", factor=3.0)):
        y = b.rotary(x, _i32(pos), b.rotary_rates(64, 500000.0, **how), interleaved=interleaved).double().cpu()
        for i, p in enumerate(pos):
            with decimal.localcontext(decimal.Context(prec=90)):
                f = [decimal.Decimal(500000) ** (decimal.Decimal(-k) / 32) / decimal.Decimal(how.get("factor", 1.0)) for k in range(32)]
                a = torch.tensor([float((p * z) % (2 * pi)) for z in f], dtype=torch.float64)
            off = torch.maximum((y[i, 0, u] - a.cos()).abs(), (y[i, 0, w] - a.sin()).abs())
            assert (off <= 1e-7 + 2.0 ** -23 + 2.0 ** -24).all(), (p, off.max())


@pytest.mark.parametrize("dtype,cache", chunk.TYPES)
@pytest.mark.parametrize("window", [0, 100, 700])
@pytest.mark.parametrize("Hq,H,D,ps", [(4, 1, 256, 64), (4, 2, 128, 20), (2, 1, 64, 5), (8, 8, 144, 12)])
def test_long_blocks_that_go_by_rows(b, dtype, cache, window, Hq, H, D, ps):
    """Shapes that the tensor-memory kernel does not take, over prompts of thousands of tokens, with windows, beside
    single queries and slots with more queries than positions; values that some rows do not see among them."""
    lens, new = [2600, 700, 1, 90, 3000, 0], [2600, 300, 1, 130, 1, 0]
    c = _case(lens, new, Hq, H, D, ps, dtype, cache, seed=D + ps)
    v = c["v"].float()
    for r, j in ((0, 1000), (0, 2599), (1, 650), (4, 2990)):
        v[c["table"][r, j // ps], 0, j % ps, 3:5] = math.nan
    c["v"] = v.to(c["v"].dtype)
    for r, (n, m) in enumerate(zip(lens, new)):  # (pages before every window are gone)
        if window:
            c["table"][r, :max(0, n - m - window + 1) // ps] = -1
    out = chunk._check(b, c, window=window)["out"].float()
    assert torch.isnan(out).any() and torch.isfinite(out).any()
