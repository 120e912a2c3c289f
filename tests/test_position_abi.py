"""Refusals of the rotary, append, chunk-attention and logit-adjustment calls: arguments are checked on
the host before anything is launched, so these calls never reach the GPU.  Also the rates."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import position_ref as ref
from tests.test_serving_abi import INVALID, OK, P, SMALL, UNSUPPORTED, _with


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import build
    build.build()
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _message(b):
    return b.lib.dspark_last_error_message().decode()


def test_rotary(b):
    def call(T=4, H=2, D=64, rot=64, dt=1, il=0, inv=0, mag=1.0, xs=(128, 64), os=(128, 64), null=(), shift=None, out=None):
        p = _with(P[:4], null, shift)
        return b.lib.dspark_rotary(T, H, D, rot, dt, il, inv, p[0], *xs, p[1], p[2], mag, out or p[3], *os, None)

    assert call(T=-1) == INVALID and call(H=0) == INVALID and call(D=0, rot=0) == INVALID
    for rot in (0, 1, 3, 63, 66, -2):
        assert call(rot=rot) == INVALID, rot
    assert call(dt=3) == INVALID and call(il=2) == INVALID and call(inv=-1) == INVALID
    assert call(D=1026, rot=64, xs=(4096, 2048), os=(4096, 2048)) == UNSUPPORTED
    assert call(H=1 << 21, D=64, os=(1 << 27, 64)) == UNSUPPORTED
    for m in (math.nan, math.inf):
        assert call(mag=m) == INVALID
    for i in range(4):
        assert call(null=[i]) == INVALID, i
    assert call(shift={0: 1}) == INVALID and call(shift={3: 1}) == INVALID and call(dt=0, shift={3: 2}) == INVALID
    assert call(xs=(-128, 64)) == INVALID
    for os in ((0, 64), (128, 0), (63, 64), (128, 63)):
        assert call(os=os) == INVALID, os
        assert "lie on one another" in _message(b)
    assert call(out=P[0], os=(192, 64)) == INVALID and "strides of x" in _message(b)
    assert call(T=0, null=[0, 1, 3]) == OK


def _geometry(call):
    for k in ("R", "num_pages", "page_size", "max_pages"):
        assert call(**{k: 0}) == INVALID, k
    assert call(R=8193) == UNSUPPORTED and call(num_pages=(1 << 22) + 1) == UNSUPPORTED
    assert call(page_size=1 << 30) == UNSUPPORTED and call(table_stride=7) == INVALID
    assert call(ws=16) == SMALL


def test_cache_append(b):
    def call(T=5, R=4, Hq=4, Hkv=2, D=64, rot=64, il=0, num_pages=64, page_size=16, max_pages=8, dt=1, kv=1, qs=(256, 64),
             ins=(128, 64), os=(256, 64), strides=(2048, 1024, 64), table_stride=8, mag=1.0, ws=256, null=(), shift=None, q_out=None):
        p = _with(P[:14], set(null) | ({10, 11} if kv != 3 else set()), shift)
        return b.lib.dspark_cache_append(T, R, Hq, Hkv, D, rot, il, num_pages, page_size, max_pages, dt, kv, p[0], *qs, p[1], p[2],
                                         *ins, q_out or p[3], *os, p[4], p[5], *strides, p[6], table_stride, p[7], p[8], p[9], p[10],
                                         p[11], p[12], mag, p[13], ws, None)

    _geometry(call)
    assert call(T=-1) == INVALID and call(Hq=-1) == INVALID and call(Hkv=0) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 12, 13):
        assert call(null=[i]) == INVALID, i
    assert call(kv=3, null=[10]) == INVALID and call(kv=3, null=[11]) == INVALID
    assert call(kv=2) == INVALID and call(dt=0, kv=0) == INVALID
    assert call(D=72, rot=16) == UNSUPPORTED and call(D=272, rot=16) == UNSUPPORTED
    assert call(rot=24) == UNSUPPORTED and call(rot=80) == INVALID and call(rot=0) == INVALID
    assert call(il=2) == INVALID and call(mag=math.nan) == INVALID
    assert call(Hq=1 << 21, os=(1 << 27, 64)) == UNSUPPORTED
    for strides in ((0, 1024, 64), (2048, 0, 64), (2048, 1024, 0), (2047, 1024, 64)):
        assert call(strides=strides) == INVALID, strides
    for kw in (dict(qs=(250, 64)), dict(ins=(128, 60)), dict(os=(256, 4)), dict(os=(56, 64)), dict(os=(256, 0))):
        assert call(**kw) == INVALID, kw
    for i in (0, 1, 2, 3, 4, 5, 13):
        assert call(shift={i: 8}) == INVALID, i
    assert call(q_out=P[0], os=(512, 64)) == INVALID and "strides of q" in _message(b)
    assert call(T=0, null=[0, 1, 2, 3]) == OK


def test_chunk_attention(b):
    need = b.chunk_attention_workspace_size(300, 4, 8, 2, 64)
    assert need > 256

    def call(T=300, R=4, Hq=8, Hkv=2, D=64, num_pages=64, page_size=16, max_pages=8, dt=1, kv=1, qs=(512, 64),
             strides=(2048, 1024, 64), table_stride=8, scale=0.1, window=0, ws=1 << 40, null=(), shift=None):
        p = _with(P[:12], set(null) | ({7, 8} if kv != 3 else set()), shift)
        return b.lib.dspark_chunk_attention(T, R, Hq, Hkv, D, num_pages, page_size, max_pages, dt, kv, p[0], *qs, p[1], p[2],
                                            *strides, p[3], table_stride, p[4], p[5], p[6], scale, p[7], p[8], window, p[9], p[10],
                                            p[11], ws, None)

    _geometry(call)
    assert call(T=-1) == INVALID and call(Hq=7) == INVALID and call(Hkv=0) == INVALID and call(window=-1) == INVALID
    assert call(Hq=130) == UNSUPPORTED and call(T=1 << 29) == UNSUPPORTED
    assert call(D=72) == UNSUPPORTED and call(D=272) == UNSUPPORTED and call(kv=2) == INVALID
    for s in (math.nan, math.inf):
        assert call(scale=s) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 9, 11):
        assert call(null=[i]) == INVALID, i
    assert call(kv=3, null=[7]) == INVALID and call(kv=3, null=[8]) == INVALID
    for i in (0, 1, 2, 9, 11):
        assert call(shift={i: 8}) == INVALID, i
    assert call(qs=(512, 60)) == INVALID and call(strides=(2048, 1024, 60)) == INVALID
    assert call(ws=need - 1) == SMALL
    assert call(T=0, null=[0, 6, 9, 10]) == OK
    for bad in (dict(T=-1), dict(R=0), dict(R=8193), dict(Hq=7), dict(Hq=130), dict(D=8), dict(D=264)):
        assert b.chunk_attention_workspace_size(**{**dict(T=300, R=4, Hq=8, Hkv=2, D=64), **bad}) == 0, bad


def test_adjust_logits(b):
    def call(N=4, V=100, R=2, dt=0, rs=100, os=100, hs=50, hw=50, nb=3, ms=4, mr=4, null=(), shift=None, out=None):
        p = _with(P[:14], null, shift)
        return b.lib.dspark_adjust_logits(N, V, R, dt, p[0], rs, p[1], p[2], p[3], hs, hw, p[4], p[5], p[6], p[7], p[8], nb, p[9], p[10],
                                          p[11], ms, mr, p[12], out or p[13], os, None)

    assert call(N=-1) == INVALID and call(V=0, rs=0) == INVALID and call(R=0) == INVALID
    assert call(V=(1 << 20) + 1, rs=1 << 21, os=1 << 21) == UNSUPPORTED and call(R=8193) == UNSUPPORTED
    assert call(dt=3) == INVALID and call(rs=99) == INVALID and call(os=99) == INVALID
    assert call(hs=49) == INVALID and call(hw=-1) == INVALID and call(nb=-1) == INVALID
    assert call(ms=3) == INVALID and call(mr=-1) == INVALID and call(mr=3, null=[12]) == INVALID
    for i in (0, 2, 4, 9, 10, 13):
        assert call(null=[i]) == INVALID, i
    assert call(null=[11]) == INVALID  # rows of a mask that is not there
    assert call(shift={0: 2}) == INVALID and call(shift={13: 1}) == INVALID
    assert call(out=P[0], os=128) == INVALID and "row stride" in _message(b)
    assert call(N=0) == OK and call(N=0, null=[0, 1, 2, 3, 4, 5, 6, 7, 8, 13]) == OK


def test_rates(b):
    """The fixed-point rates against the formulas, to float64's rounding; a rate of any size is held modulo
    a turn."""
    turns = lambda r: r.numpy().astype(np.uint64).astype(np.float64) * 2.0 ** -64
    i = np.arange(32)
    f = 10000.0 ** (-i / 32.0)
    kw = dict(device="cpu")
    np.testing.assert_allclose(turns(b.rotary_rates(64, **kw)), f / math.tau, rtol=1e-14)
    np.testing.assert_allclose(turns(b.rotary_rates(64, scaling="linear", factor=4.0, **kw)), f / 4 / math.tau, rtol=1e-14)
    np.testing.assert_allclose(turns(b.rotary_rates(64, scaling="ntk", factor=4.0, **kw)),
                               (10000.0 * 4 ** (64 / 62)) ** (-i / 32.0) / math.tau, rtol=1e-13)
    how = dict(factor=8.0, original_len=4096, low=1.0, high=32.0, **kw)
    for scaling in ("bands", "yarn"):
        got = turns(b.rotary_rates(64, scaling=scaling, **how)) * math.tau
        n = 4096 * f / math.tau
        assert np.allclose(got[n >= 40], f[n >= 40], rtol=1e-14) and np.allclose(got[n <= 0.8], f[n <= 0.8] / 8, rtol=1e-14)
        assert (np.diff(got) < 0).all() and (got <= f * (1 + 1e-14)).all() and (got >= f / 8 * (1 - 1e-14)).all()
    kept = np.clip((n - 1) / 31, 0, 1)
    np.testing.assert_allclose(turns(b.rotary_rates(64, scaling="bands", **how)) * math.tau, f * (kept + (1 - kept) / 8), rtol=1e-13)
    np.testing.assert_allclose(turns(b.rotary_rates(64, factors=[2.0] * 32, **kw)), f / 2 / math.tau, rtol=1e-14)
    big = b.rotary_rates(4, 0.25, **kw)  # f = 1, 2: still within a turn; base below 1 grows
    np.testing.assert_allclose(turns(big), [1 / math.tau, 2 / math.tau], rtol=1e-14)
    wrapped = turns(b.rotary_rates(4, 1e-4, **kw))[1]  # f = 100 radians a position
    assert abs(wrapped - math.fmod(100 / math.tau, 1.0)) < 1e-13
    assert b.rotary_rates(2, scaling="ntk", factor=3.0, **kw).numel() == 1
    assert b.rotary_magnitude(1.0) == 1.0 and abs(b.rotary_magnitude(math.e) - 1.1) < 1e-15


def test_rates_refused(b):
    for a, kw in (((0,), {}), ((3,), {}), ((-2,), {}), ((64, 0.0), {}), ((64, math.inf), {}), ((64,), dict(factor=0.0)),
                  ((64,), dict(scaling="other")), ((64,), dict(scaling="yarn")), ((64,), dict(scaling="bands", original_len=0)),
                  ((64,), dict(scaling="bands", original_len=64, low=4.0, high=4.0)), ((64,), dict(factors=[1.0])),
                  ((4,), dict(factors=[1.0, -1.0])), ((64, 0.5), dict(scaling="yarn", original_len=64))):
        with pytest.raises(b.DSparkError):
            b.rotary_rates(*a, device="cpu", **kw)


def test_tensors_that_do_not_fit(b):
    """What the marshalling refuses without a GPU: host tensors, by name."""
    t = torch.zeros((4, 2, 64))
    i = torch.zeros(4, dtype=torch.int32)
    for call, name in ((lambda: b.rotary(t, i, i.long()), "x"), (lambda: b.cache_append(t, t, t, t, t, i, i, i, i), "k"),
                       (lambda: b.chunk_attention(t, t, t, i, i, i, 1.0), "q"),
                       (lambda: b.adjust_logits(t[0], i, i), "logits")):
        with pytest.raises(b.DSparkError, match=f"{name} must be a CUDA tensor"):
            call()


def test_the_plain_forms(b):
    """The 64-bit forms that the GPU tests compare with, against independent ones."""
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((5, 2, 8)), np.array([0, 1, 77, -3, 2 ** 31 - 1])
    rates = b.rotary_rates(6, device="cpu").numpy()
    for il in (False, True):
        y, _ = ref.turned(x, pos, rates, interleaved=il, magnitude=1.5)
        for i in range(3):
            u, w = (2 * i, 2 * i + 1) if il else (i, i + 3)
            f = 10000.0 ** (-2 * i / 6)
            z = (x[:4, :, u] + 1j * x[:4, :, w]) * 1.5 * np.exp(1j * f * pos[:4])[:, None]
            np.testing.assert_allclose(y[:4, :, u] + 1j * y[:4, :, w], z, atol=1e-12)
        back, _ = ref.turned(y, pos, rates, interleaved=il, magnitude=1 / 1.5, inverse=True)
        np.testing.assert_allclose(back, x, atol=1e-12)
    from tests import serving_ref
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    q, k, v = rnd(9, 4, 16), rnd(6, 2, 4, 16), rnd(6, 2, 4, 16)
    table, lens, q_start = np.array([[3, 1, 5], [0, 2, -1]]), [11, 7], [0, 5, 9]
    for window in (0, 3):
        a, c = (m.attention(q, k, v, table, lens, q_start, 0.3, window=window) for m in (ref, serving_ref))
        for s, t in zip(a, c):
            assert torch.allclose(s, t, atol=1e-12)
    z = rng.standard_normal((3, 9))
    got, _ = ref.adjusted(z, np.array([1, 1, 4]), [0, 2, 3], history=np.array([[1, 2], [4, 8]]), history_len=[2, 1], prompt_len=[2, 0],
                          repetition=[2.0, 0.5], frequency=[0.25, 1.0], presence=[0.5, 0.0], bias_ids=np.array([[0, 0], [8, -1]]),
                          bias=np.array([[1.0, 2.0], [4.0, 9.0]]), mask=np.array([[0b11]]), mask_row=[-1, 0, -1])
    r = lambda x, rho: x / rho if x > 0 else x * rho
    want = z.copy()
    want[0, 1], want[0, 2], want[0, 0] = r(z[0, 1], 2) - 0.25 - 0.5, r(z[0, 2], 2), z[0, 0] + 3
    want[1, 1], want[1, 0], want[1, 2:] = r(z[1, 1], 2) - 0.5 - 0.5, z[1, 0] + 3, -math.inf
    want[2, 4], want[2, 8] = r(z[2, 4], 0.5) - 2.0, z[2, 8] + 4
    np.testing.assert_allclose(got, want, atol=1e-12)


def test_limits_of_adjust_logits(b):
    """The largest sizes that are taken, and the first that are refused."""
    def call(N, hw, nb):
        return b.lib.dspark_adjust_logits(N, 100, 2, 0, P[0], 100, P[1], P[2], P[3], hw, hw, P[4], P[5], P[6], P[7], P[8], nb, P[9],
                                          P[10], P[11], 4, N, None, P[13], 100, None)

    assert call(0, 50, 1024) == OK and call(0, 50, 1025) == UNSUPPORTED and "n_bias=1025" in _message(b)
    assert call(0, (1 << 29) - 1, 3) == OK and call(0, 1 << 29, 3) == UNSUPPORTED and "2^29" in _message(b)
    assert call(5, (1 << 29) - 5, 3) == UNSUPPORTED and call((1 << 31) - 1, (1 << 31) - 1, 3) == UNSUPPORTED
