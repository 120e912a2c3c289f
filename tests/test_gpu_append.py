"""dspark_cache_append against a 64-bit form and against dspark_rotary and dspark_cache_write: layouts,
types, strides, refused slots, rows of no slot, bad tables, streams and graphs.

Tolerance: dspark_rotary's (tests/test_gpu_rotary.py); an e4m3 cache adds the division's 2^-24 and half
a step, 2^-4 of the value (2^-10 below the smallest normal number)."""
import numpy as np
import pytest
import torch

from tests import position_ref as ref

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, E4M3), (torch.float16, E4M3)]


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _bits(x):
    return x.contiguous().view(torch.uint8 if x.element_size() == 1 else torch.int16)


class Case:
    def __init__(self, lens, new, Hq, H, D, ps, dtype, cache, seed=0, beyond=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.dtype, self.cache = lens, new, dtype, cache
        per = [-(-n // ps) for n in lens]
        P = sum(per) + 2
        order = np.random.default_rng(seed).permutation(P)
        self.table = np.full((len(lens), max(1, max(per))), -1)
        at = 0
        for r, n in enumerate(per):
            self.table[r, :n] = order[at:at + n]
            at += n
        self.q_start = np.concatenate([[0], np.cumsum(new)])
        T = sum(new) + beyond
        rnd = lambda *s: (torch.randn(s, generator=g) * 2).to(dtype).cuda()
        self.q, self.k, self.v = rnd(T, Hq, D), rnd(T, H, D), rnd(T, H, D)
        self.pools = [torch.full((P, H, ps, D), 3.0).to(cache).cuda() for _ in range(2)]
        self.scales = [torch.rand(H, generator=g).cuda() * 0.1 + 0.01 for _ in range(2)] if cache == E4M3 else [None, None]
        self.ps = ps

    def call(self, b, rates, q="q", **kw):
        self.ws = b.workspace(256, "cuda")
        return b.cache_append(self.q if q == "q" else None, self.k, self.v, *self.pools, _i32(self.table), _i32(self.lens),
                              _i32(self.q_start), rates, k_scale=self.scales[0], v_scale=self.scales[1], ws=self.ws, **kw)

    def positions(self):
        return np.concatenate([np.arange(n - m, n) for n, m in zip(self.lens, self.new)] + [np.zeros(0, int)])

    def check(self, b, q_out, rates, skip=(), **how):
        T = sum(self.new)
        pos = self.positions()
        half = torch.finfo(self.dtype).eps / 2
        tiny = 2.0 ** -25 if self.dtype == torch.float16 else 0.0
        rows = np.concatenate([np.full(m, r) for r, m in enumerate(self.new)] + [np.zeros(0, int)]).astype(int)
        there = ~np.isin(rows, skip)
        num = rates.cpu().numpy()
        if q_out is not None:
            want, mag = ref.turned(self.q[:T].double().cpu().numpy(), pos, num, **how)
            off = np.abs(q_out[:T].double().cpu().numpy() - want)
            tol = 2.0 ** -21 * mag + (half * np.abs(want) + tiny) * (mag > 0)
            assert (off <= tol)[there].all()
        want_k, mag = ref.turned(self.k[:T].double().cpu().numpy(), pos, num, **how)
        wants = [(want_k, mag), (self.v[:T].double().cpu().numpy(), np.zeros_like(mag))]
        for pool, (want, mag), scale in zip(self.pools, wants, self.scales):
            x = pool.float().double().cpu().numpy()
            left = np.ones(x.shape[0::2][:2], bool)  # [page, token]: untouched
            for i, (r, p) in enumerate(zip(rows, pos)):
                if not there[i]:
                    continue
                page, slot = self.table[r, p // self.ps], p % self.ps
                left[page, slot] = False
                w, m = want[i], mag[i]
                if scale is None:
                    tol = 2.0 ** -21 * m + (half * np.abs(w) + tiny) * (m > 0)
                else:
                    s = scale.double().cpu().numpy()[:, None]
                    w, m = w / s, m / s
                    clip = np.clip(w, -448, 448)
                    tol = 2.0 ** -21 * m + 2.0 ** -23 * np.abs(w)
                    tol = tol + 2.0 ** -4 * (np.abs(clip) + tol) + 2.0 ** -10
                    w = clip
                assert (np.abs(x[page, :, slot] - w) <= tol).all(), (i, r, p)
            assert (pool.float().cpu().numpy().transpose(0, 2, 1, 3)[left] == 3.0).all()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,H,D,rot,ps", [(1, 1, 16, 16, 1), (8, 2, 64, 64, 16), (32, 8, 128, 128, 16), (6, 2, 80, 32, 5),
                                           (5, 1, 256, 128, 64), (64, 1, 48, 48, 8)])
def test_layouts(b, dtype, cache, interleaved, Hq, H, D, rot, ps):
    lens, new = [1, 5, 64, 130, 7, 300], [1, 5, 3, 30, 0, 2]
    rates = b.rotary_rates(rot)
    how = dict(interleaved=interleaved, magnitude=1.1)
    c = Case(lens, new, Hq, H, D, ps, dtype, cache, seed=D)
    c.check(b, c.call(b, rates, **how), rates, **how)
    assert b.device_status(c.ws) == 0
    d = Case(lens, new, Hq, H, D, ps, dtype, cache, seed=D)
    assert d.call(b, rates, q=None, **how) is None  # keys and values alone
    for x, y in zip(c.pools, d.pools):
        assert torch.equal(_bits(x), _bits(y))


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_as_rotary_then_write(b, dtype, cache):
    """The same bits as the two calls one after the other give, where the cache holds the type of the keys
    (an e4m3 cache takes them without the rounding between)."""
    lens, new = [4000, 77, 9000], [700, 77, 1]
    rates = b.rotary_rates(96, scaling="bands", factor=4.0, original_len=2048)
    c = Case(lens, new, 12, 4, 128, 32, dtype, cache, seed=1)
    q_out = c.call(b, rates)
    d = Case(lens, new, 12, 4, 128, 32, dtype, cache, seed=1)
    pos = _i32(c.positions())
    assert torch.equal(q_out, b.rotary(d.q, pos, rates))
    b.cache_write(b.rotary(d.k, pos, rates), d.v, *d.pools, _i32(d.table), _i32(d.lens), _i32(d.q_start), k_scale=d.scales[0],
                  v_scale=d.scales[1])
    assert torch.equal(_bits(c.pools[1]), _bits(d.pools[1]))
    if cache != E4M3:
        assert torch.equal(_bits(c.pools[0]), _bits(d.pools[0]))


def test_refused_slots_and_rows_of_no_slot(b):
    rates = b.rotary_rates(64)
    c = Case([40, 9, 100], [3, 2, 50], 4, 2, 64, 16, torch.bfloat16, torch.bfloat16, beyond=6)
    q_out = torch.full_like(c.q, 9.0)
    c.call(b, rates, q_out=q_out, granted=_i32([3, 0, 50]))
    c.check(b, q_out, rates, skip=[1])
    assert (q_out[3:5] == 9).all() and (q_out[55:] == 9).all()
    assert b.device_status(c.ws) == 0
    # rows before the first slot's
    c = Case([40, 9], [3, 2], 4, 2, 64, 16, torch.bfloat16, torch.bfloat16, beyond=6)
    c.q_start = c.q_start + 4
    q_out = torch.full_like(c.q, 9.0)
    c.call(b, rates, q_out=q_out)
    assert (q_out[:4] == 9).all() and (q_out[9:] == 9).all() and (q_out[4:9] != 9).any()


def test_strides_and_in_place(b):
    """One packed projection [T, Hq + 2 H, D], turned where it lies; a pool whose pages hold tokens first."""
    rates = b.rotary_rates(64)
    c = Case([40, 300], [30, 100], 6, 2, 64, 16, torch.float16, torch.float16)
    packed = torch.cat([c.q, c.k, c.v], 1)
    d = Case([40, 300], [30, 100], 6, 2, 64, 16, torch.float16, torch.float16)
    want = d.call(b, rates)
    c.q, c.k, c.v = packed[:, :6], packed[:, 6:8], packed[:, 8:]
    c.pools = [p.transpose(1, 2).contiguous().transpose(1, 2) for p in c.pools]
    got = c.call(b, rates, q_out=c.q)
    assert got.data_ptr() == packed.data_ptr() and torch.equal(got, want)
    for x, y in zip(c.pools, d.pools):
        assert torch.equal(x, y)
    assert torch.equal(packed[:, 6:], torch.cat([d.k, d.v], 1))


def test_bad_tables_are_reported(b):
    rates = b.rotary_rates(64)
    for change in ("page", "length"):
        c = Case([40, 9, 100], [3, 2, 50], 4, 2, 64, 16, torch.bfloat16, torch.bfloat16)
        if change == "page":
            c.table[1, 0] = 1 << 20
        else:
            c.lens = [40, 1, 100]  # two new tokens in a context of one
        q_out = torch.full_like(c.q, 9.0)
        c.call(b, rates, q_out=q_out)
        assert b.device_status(c.ws) == 1
        assert (q_out[3] == 9).all() and (q_out[:3] != 9).any() and (q_out[5:] != 9).any()


def test_offsets_past_32_bits(b):
    """A slot whose pages lie past 2^32 bytes and 2^31 elements of the pool."""
    pages = (1 << 31) // (16 * 128) + 40
    pools = [torch.zeros((pages, 1, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rates = b.rotary_rates(128)
    k, v = (torch.randn((20, 1, 128), device="cuda").bfloat16() for _ in range(2))
    table = _i32([[pages - 1, 3, pages - 30]])
    b.cache_append(None, k, v, *pools, table, _i32([40]), _i32([0, 20]), rates)
    want = b.rotary(k, torch.arange(20, 40, dtype=torch.int32, device="cuda"), rates)
    got = [torch.cat([p[3, 0, 4:], p[pages - 30, 0, :8]]) for p in pools]
    assert torch.equal(got[0], want[:, 0]) and torch.equal(got[1], v[:, 0])


def test_streams_and_graphs(b):
    rates = b.rotary_rates(64)
    c = Case([40, 300], [30, 100], 6, 2, 64, 16, torch.bfloat16, torch.bfloat16)
    want = c.call(b, rates)
    pools = [p.clone() for p in c.pools]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for p in c.pools:
        p.fill_(0)
    side.wait_stream(torch.cuda.current_stream())
    ws, args = b.workspace(256, "cuda"), (_i32(c.table), _i32(c.lens), _i32(c.q_start))
    torch.cuda.synchronize()
    got = b.cache_append(c.q, c.k, c.v, *c.pools, *args, rates, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    q_out = torch.zeros_like(c.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.cache_append(c.q, c.k, c.v, *c.pools, *args, rates, ws=ws, q_out=q_out)
    for p in c.pools:
        p.fill_(3.0)
    g.replay()
    assert torch.equal(q_out, want)
    for x, y in zip(c.pools, pools):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-31, 1e-29, 3.3e-3, 0.7, 1.0, 1e29, 1e31, 3e38])
def test_scales_of_any_size(b, dtype, scale):
    """Values divided by scales to the ends of fp32's range, as cache_write stores them: bit for bit."""
    c = Case([400], [400], 1, 2, 64, 16, dtype, E4M3, seed=2)
    c.scales = [torch.tensor([scale, scale * 1.0001 if scale < 1e38 else scale], device="cuda") for _ in range(2)]
    size = torch.tensor([1.0, 1e-3, 30.0, 448.0 * scale if 1e-3 < scale < 1e3 else 1.0], device="cuda").repeat(100)[:, None, None]
    c.v = (c.v.float() * size).to(dtype)
    c.v[7, 0, 3], c.v[9, 1, 60], c.v[11, 0, 0], c.v[12, 0, 1] = float("inf"), float("-inf"), float("nan"), 0.0
    c.call(b, b.rotary_rates(64), q=None)
    d = Case([400], [400], 1, 2, 64, 16, dtype, E4M3, seed=2)
    b.cache_write(c.k, c.v, *d.pools, _i32(d.table), _i32(d.lens), _i32(d.q_start), k_scale=c.scales[0], v_scale=c.scales[1])
    assert torch.equal(_bits(c.pools[1]), _bits(d.pools[1]))
