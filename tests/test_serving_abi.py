"""Refusals of the serving-side entry points: arguments are checked on the host before
anything is launched, so these calls never reach the GPU (pointers are stand-ins that
validation does not follow).  Also the 64-bit gradient against differences."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import serving_ref as ref

OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
P = [ctypes.c_void_p(0x100000 + 0x1000 * i) for i in range(16)]


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import build
    build.build()
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _with(values, null=(), shift=None):
    v = list(values)
    for k in null:
        v[k] = None
    for k, by in (shift or {}).items():
        v[k] = ctypes.c_void_p(v[k].value + by)
    return v


def test_token_logprobs(b):
    def call(N=4, V=100, rs=100, dt=0, T=1.0, k=2, null=(), shift=None):
        p = _with(P[:7], null, shift)
        return b.lib.dspark_token_logprobs(N, V, rs, dt, p[0], p[1], T, k, p[2], p[3], p[4], p[5], p[6], None)

    assert call(N=-1) == INVALID and call(V=0, rs=0) == INVALID
    assert call(rs=99) == INVALID
    assert call(dt=3) == INVALID and call(dt=-1) == INVALID
    for T in (0.0, -1.0, math.nan, math.inf, 1e-45):
        assert call(T=T) == INVALID, T
    assert call(k=-1) == INVALID and call(k=101) == INVALID
    assert call(k=33) == UNSUPPORTED
    assert call(V=(1 << 20) + 1, rs=1 << 21) == UNSUPPORTED
    for i in range(7):
        assert call(null=[i]) == INVALID, i
    assert call(shift={0: 2}) == INVALID and call(dt=1, shift={0: 1}) == INVALID
    assert call(N=0, null=range(7)) == OK  # nothing to do


def test_token_logprobs_backward(b):
    def call(N=4, V=100, rs=100, gs=100, dt=0, T=1.0, null=(), shift=None, out=None):
        p = _with(P[:7], null, shift)
        return b.lib.dspark_token_logprobs_backward(N, V, rs, gs, dt, p[0], p[1], T, p[2], p[3], p[4], p[5],
                                                    out or p[6], None)

    assert call(gs=99) == INVALID and call(rs=99) == INVALID and call(T=0.0) == INVALID and call(dt=7) == INVALID
    for i in (0, 1, 2, 3, 4, 6):
        assert call(null=[i]) == INVALID, i
    assert call(shift={6: 2}) == INVALID
    assert call(out=P[0], gs=128) == INVALID  # in place, with another stride
    assert "row stride" in b.lib.dspark_last_error_message().decode()
    assert call(N=0, null=range(7)) == OK


GEOMETRY = dict(R=4, num_pages=64, page_size=16, max_pages=8, stride=8)


def _geometry_refusals(call):
    for k in ("R", "num_pages", "page_size", "max_pages"):
        assert call(**{k: 0}) == INVALID, k
    assert call(R=8193) == UNSUPPORTED
    assert call(num_pages=(1 << 22) + 1) == UNSUPPORTED
    assert call(page_size=1 << 30) == UNSUPPORTED
    assert call(stride=7) == INVALID
    assert call(ws=16) == SMALL


def _tables(kw, null=(), shift=None):
    g = dict(GEOMETRY, **{k: v for k, v in kw.items() if k in GEOMETRY})
    return (g["R"], g["num_pages"], g["page_size"], g["max_pages"], g["stride"], *_with(P[:3], null, shift))


def test_cache_fork(b):
    def call(F=2, ws=1 << 30, null=(), shift=None, **kw):
        p = _with(P, null, shift)
        return b.lib.dspark_cache_fork(F, *_tables(kw, [i for i in null if i < 3]), p[3], p[4], p[5], ws, None)

    _geometry_refusals(call)
    for i in range(6):
        assert call(null=[i]) == INVALID, i
    assert call(shift={5: 16}) == INVALID
    assert call(F=-1) == INVALID and call(F=5) == INVALID
    assert call(F=0, null=[3, 4]) == OK


def test_cache_length_limit(b):
    """Positions, rounded up to a tile, stay within 32 bits."""
    def call(max_pages, F=1):
        return b.lib.dspark_cache_fork(F, *_tables(dict(max_pages=max_pages, page_size=64, stride=1 << 25)), P[3], P[4],
                                       P[5], 1 << 30, None)

    assert call(1 << 25) == UNSUPPORTED and call((1 << 25) - 4) == UNSUPPORTED
    assert call((1 << 25) - 5, F=0) == OK


def test_cache_reserve(b):
    pools = (ctypes.c_void_p * 2)(P[10], P[11])

    def call(n=2, pb=4096, pools=pools, ws=1 << 30, null=(), **kw):
        p = _with(P, null)
        return b.lib.dspark_cache_reserve(*_tables(kw, [i for i in null if i < 3]), p[3], p[4], p[5], n, pools, pb,
                                          p[6], ws, None)

    _geometry_refusals(call)
    for i in range(7):
        assert call(null=[i]) == INVALID, i
    assert call(n=-1) == INVALID and call(n=513) == UNSUPPORTED
    assert call(pb=0) == INVALID and call(pb=24) == INVALID
    assert call(pools=None) == INVALID
    assert call(pools=(ctypes.c_void_p * 2)(P[10], None)) == INVALID
    assert call(pools=(ctypes.c_void_p * 2)(P[10], P[11].value + 8)) == INVALID


def test_cache_truncate_and_compact(b):
    def truncate(ws=1 << 30, null=(), **kw):
        p = _with(P, null)
        return b.lib.dspark_cache_truncate(*_tables(kw, [i for i in null if i < 3]), p[3], p[4], ws, None)

    _geometry_refusals(truncate)
    for i in range(5):
        assert truncate(null=[i]) == INVALID, i
    pools = (ctypes.c_void_p * 1)(P[10])

    def compact(n=1, pb=4096, ws=1 << 30, null=(), **kw):
        p = _with(P, null)
        return b.lib.dspark_cache_compact(*_tables(kw, [i for i in null if i < 3]), p[3], n, pools, pb, p[4], ws, None)

    _geometry_refusals(compact)
    for i in range(5):
        assert compact(null=[i]) == INVALID, i
    assert compact(pb=8) == INVALID
    assert b.cache_workspace_size(4, 64) > 0
    assert b.cache_workspace_size(0, 64) == 0 and b.cache_workspace_size(4, 1 << 23) == 0


def test_cache_write(b):
    def call(T=3, H=2, D=64, di=1, dk=1, it=128, ih=64, ps=(2048, 1024, 64), scales=(None, None), ws=256, null=(),
             shift=None, **kw):
        g = dict(GEOMETRY, **kw)
        p = _with(P, null, shift)
        return b.lib.dspark_cache_write(T, g["R"], H, D, g["num_pages"], g["page_size"], g["max_pages"], di, dk, p[0],
                                        p[1], it, ih, p[2], p[3], *ps, p[4], g["stride"], p[5], p[6], None, *scales,
                                        p[7], ws, None)

    _geometry_refusals(call)
    assert call(T=-1) == INVALID and call(H=0) == INVALID
    for D in (0, 8, 24, 272):
        assert call(D=D) == UNSUPPORTED, D
    assert call(di=0, dk=0) == INVALID and call(di=1, dk=2) == INVALID and call(dk=9) == INVALID
    assert call(dk=3) == INVALID  # an e4m3 cache needs its scales
    assert call(dk=3, scales=(P[8], None)) == INVALID
    assert call(scales=(P[8], P[9])) == INVALID  # and only it
    for i in range(8):
        assert call(null=[i]) == INVALID, i
    for i in (0, 1, 2, 3):
        assert call(shift={i: 8}) == INVALID, i
    assert call(shift={7: 16}) == INVALID
    assert call(it=130) == INVALID and call(ih=4) == INVALID and call(it=-128) == INVALID
    assert call(ps=(2048, 1024, 68)) == INVALID and call(ps=(2052, 1024, 64)) == INVALID
    assert call(dk=3, scales=(P[8], P[9]), ps=(2048, 1024, 72)) == INVALID
    assert call(T=0, null=[0, 1]) == OK


def test_paged_attention(b):
    need = b.paged_attention_workspace_size(3, 4, 8, 2, 64, 1)
    assert need >= 256

    def call(T=3, Hq=8, H=2, D=64, mq=1, dq=1, dk=1, qs=(512, 64), ps=(2048, 1024, 64), scale=0.1,
             scales=(None, None), window=0, ws=need, null=(), shift=None, **kw):
        g = dict(GEOMETRY, **kw)
        p = _with(P, null, shift)
        return b.lib.dspark_paged_attention(T, g["R"], Hq, H, D, g["num_pages"], g["page_size"], g["max_pages"], mq,
                                            dq, dk, p[0], *qs, p[1], p[2], *ps, p[3], g["stride"], p[4], p[5], scale,
                                            *scales, window, p[6], p[7], p[8], ws, None)

    _geometry_refusals(call)
    assert call(T=-1) == INVALID and call(Hq=7) == INVALID and call(window=-1) == INVALID
    assert call(Hq=130, H=2) == UNSUPPORTED and call(D=40) == UNSUPPORTED
    assert call(mq=0) == INVALID and call(mq=129) == UNSUPPORTED
    assert call(scale=math.nan) == INVALID and call(scale=math.inf) == INVALID
    assert call(dq=0, dk=0) == INVALID and call(dq=2, dk=1) == INVALID
    assert call(dk=3) == INVALID and call(scales=(P[9], P[10])) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 6, 8):
        assert call(null=[i]) == INVALID, i
    for i in (0, 1, 2, 6):
        assert call(shift={i: 8}) == INVALID, i
    assert call(qs=(516, 64)) == INVALID and call(ps=(2048, 1024, 60)) == INVALID
    assert call(ws=need - 1) == SMALL
    assert call(T=0, null=[0, 6]) == OK
    for bad in ((3, 0, 8, 2, 64, 1), (3, 4, 8, 3, 64, 1), (3, 4, 8, 2, 60, 1), (3, 4, 8, 2, 64, 0),
                (3, 4, 8, 2, 64, 129)):
        assert b.paged_attention_workspace_size(*bad) == 0, bad


def test_binding_refuses_host_tensors(b):
    x, t = torch.zeros((2, 8)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(b.DSparkError):
        b.token_logprobs(x, t)
    with pytest.raises(b.DSparkError):
        b.cache_pools([x])
    with pytest.raises(b.DSparkError):
        b.cache_truncate(t.view(1, 2), t, t, t, 16)


def test_reference_gradient_against_differences():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 12)) * 2
    tokens, T, gl, ge = np.array([3, 11]), 0.7, np.array([0.5, -1.2]), np.array([1.1, 0.3])

    def f(z):
        lp, H, _, _, _ = ref.token_logprobs(z, tokens, T, 0)
        return (gl * lp + ge * H).sum()

    g, h = ref.token_logprobs_grad(x, tokens, T, gl, ge), 1e-5
    for n in range(2):
        for v in range(12):
            up, dn = x.copy(), x.copy()
            up[n, v] += h
            dn[n, v] -= h
            assert abs((f(up) - f(dn)) / (2 * h) - g[n, v]) < 1e-8
