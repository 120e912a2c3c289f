"""Attention of long blocks when a bounded device wait runs out, without a fault.

The library is built a second time, as in tests/test_gpu_timeout.py, with a short wait limit (2e6 cycles, about
1 ms) and a stall switch: a call whose window is 0x5EED copies no values.  Every role that waits for them, or for
another that does, gives up; copies and products in flight end, the tensor memory is given back, and the call
returns before long.  The host reads DSPARK_TIMEOUT, and the
next call over the same workspace gives the shipped library's results."""
import ctypes
import os

import pytest
import torch

from tests.test_gpu_attention import _case, _i32

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STALL_WINDOW = 0x5EED
TIMEOUT = 5


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def short(b):
    from speculative_decoding_draft_03_gb300 import build as bld
    lib = ctypes.CDLL(bld.build(extra_flags=("-DDSPARK_TEST_WAIT_LIMIT=2000000ll",),
                                build_dir=os.path.join(ROOT, "tests", "_build", "shortwait")))
    for name in ("dspark_chunk_attention", "dspark_workspace_status"):
        getattr(lib, name).argtypes = getattr(b.lib, name).argtypes
        getattr(lib, name).restype = ctypes.c_int
    lib.dspark_workspace_status.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    return lib


def _call(b, lib, t, ws, window):
    p = b._p
    T, Hq, D = t["q"].shape
    P, H, ps, _ = t["k"].shape
    R, W = t["table"].shape
    dt = {torch.bfloat16: 1, torch.float16: 2, torch.float8_e4m3fn: 3}
    st = lib.dspark_chunk_attention(T, R, Hq, H, D, P, ps, W, dt[t["q"].dtype], dt[t["k"].dtype], p(t["q"]), Hq * D, D, p(t["k"]),
                                    p(t["v"]), H * ps * D, ps * D, D, p(t["table"]), W, p(t["lens"]), p(t["q_start"]), None, 0.1,
                                    p(t["ks"]), p(t["vs"]), window, p(t["out"]), p(t["lse"]), p(ws), ws.numel(), b._stream())
    assert st == 0


def _status(b, lib, ws):
    val = ctypes.c_int(0)
    assert lib.dspark_workspace_status(b._p(ws), 1, ctypes.byref(val), b._stream()) == 0
    return val.value


def _tensors(c):
    t = {n: c[n].cuda() for n in ("q", "k", "v")}
    t.update(table=_i32(c["table"]), lens=_i32(c["lens"]), q_start=_i32(c["q_start"]))
    t["ks"], t["vs"] = (None if s is None else s.cuda() for s in c["scales"])
    t["out"] = torch.full_like(t["q"], 77.0)
    t["lse"] = torch.full(t["q"].shape[:2], 77.0, device="cuda")
    return t


@pytest.mark.parametrize("dtype,cache,D", [(torch.bfloat16, None, 128), (torch.float16, None, 64),
                                           (torch.bfloat16, torch.float8_e4m3fn, 128)])
def test_a_wait_that_runs_out(b, short, dtype, cache, D):
    c = _case([40000], [16384], 8, 8, D, 64, dtype, cache, seed=1, garbage=False)  # some 640 tiles a CTA
    t = _tensors(c)
    ws = b.workspace(b.chunk_attention_workspace_size(16384, 1, 8, 8, D), "cuda")
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    begin.record()
    _call(b, short, t, ws, STALL_WINDOW)
    end.record()
    torch.cuda.synchronize()  # the kernels returned: no hang, no fault
    assert _status(b, short, ws) == TIMEOUT
    assert _status(b, short, ws) == 0
    assert begin.elapsed_time(end) < 100.0  # (one wait that runs out, and then some 10 us a tile)
    c = _case([700, 300, 150], [300, 300, 1], 8, 8, D, 64, dtype, cache, seed=2)
    t, u = _tensors(c), _tensors(c)
    _call(b, short, t, ws, 0)
    assert _status(b, short, ws) == 0
    _call(b, b.lib, u, ws, 0)
    assert torch.equal(t["out"], u["out"]) and torch.equal(t["lse"], u["lse"]) and not (t["out"] == 77).any()
