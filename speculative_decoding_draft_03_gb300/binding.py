"""Thin binding of ``libdspark.so`` (argument marshalling only): ctypes, and for the serving-side
calls, which run many times per token, the compiled ``_marshal`` module.

Every step of the path runs in the library's CUDA kernels; this module checks tensor
placement/dtypes, passes ``data_ptr()``s and the current CUDA stream, and owns the
caller-side buffers (outputs and workspaces) through PyTorch.  The tensors of a serving-side
call lie on one device (a call over two is refused).  If the library is missing this module raises
at import: there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import decimal
import functools
import importlib.util
import math
import os

import torch

from . import build as _build

F32, BF16, F16, E4M3 = 0, 1, 2, 3
EARLY_STOP, FULL_SEARCH, CAPACITY_K, FIXED = 0, 1, 2, 3
MAX_BLOCK = 128  # queries of a slot in one paged_attention call, at most (chunk_attention takes any number)
_DT = {torch.float32: F32, torch.bfloat16: BF16}


class DSparkError(RuntimeError):
    pass


def _load_library():
    path = _build.LIB
    if not os.path.exists(path):
        raise DSparkError(f"libdspark.so is not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, i32, u64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_float, ctypes.c_size_t
    lib.dspark_status_string.restype = ctypes.c_char_p
    lib.dspark_status_string.argtypes = [i32]
    lib.dspark_last_error_message.restype = ctypes.c_char_p
    lib.dspark_workspace_status.argtypes = [P, i32, P, P]
    lib.dspark_markov_draft_workspace_size.restype = sz
    lib.dspark_markov_draft_workspace_size.argtypes = [i32] * 5 + [i32]
    lib.dspark_markov_draft.argtypes = ([i32] * 8 + [P] * 4 + [P, f32, f32, P, f32, P, P, u64, u64]
                                        + [P] * 4 + [P, sz, P])
    lib.dspark_schedule_workspace_size.restype = sz
    lib.dspark_schedule_workspace_size.argtypes = [i32, i32]
    lib.dspark_schedule.argtypes = [i32, i32, P, P, i32, i32, P, i32, P, P, P, P, sz, P]
    lib.dspark_schedule_threshold.argtypes = [i32, i32, P, ctypes.c_double, P, P, P, P, sz, P]
    lib.dspark_schedule_threshold.restype = i32
    lib.dspark_verify_workspace_size.restype = sz
    lib.dspark_verify_workspace_size.argtypes = [i32] * 5
    lib.dspark_verify.argtypes = ([i32] * 7 + [P] * 4 + [P] * 5 + [f32, P, u64, u64] + [P] * 3 + [P, sz, P])
    lib.dspark_set_profile_events.argtypes = [P, i32]
    lib.dspark_set_profile_events.restype = None
    lib.dspark_set_verify_profile_events.argtypes = [P, i32]
    lib.dspark_set_verify_profile_events.restype = None
    lib.dspark_verify_ragged.argtypes = ([i32] * 7 + [P, i32, P] + [P] * 3 + [P] * 5 + [f32, P, u64, u64] + [P] * 3
                                         + [P, sz, P])
    lib.dspark_verify_ragged.restype = i32
    lib.dspark_verify_static.argtypes = ([i32] * 7 + [P] * 4 + [P] * 5 + [f32, P, u64, u64] + [P] * 3 + [P])
    lib.dspark_verify_static.restype = i32
    lib.dspark_verify_static_status.argtypes = [i32, P, P]
    lib.dspark_verify_static_status.restype = i32
    lib.dspark_verify_overlap_workspace_size.restype = sz
    lib.dspark_verify_overlap_workspace_size.argtypes = [i32] * 5
    lib.dspark_verify_overlap.argtypes = ([i32] * 7 + [P] * 4 + [P] * 5 + [f32, P, u64, u64] + [P] * 4
                                          + [P, sz, P])
    lib.dspark_verify_overlap.restype = i32
    lib.dspark_acceptance_overlap_workspace_size.restype = sz
    lib.dspark_acceptance_overlap_workspace_size.argtypes = [i32] * 5
    lib.dspark_acceptance_overlap.argtypes = [i32] * 7 + [P] * 4 + [P] * 4 + [f32, P, P, sz, P]
    lib.dspark_acceptance_overlap.restype = i32
    lib.dspark_rnn_draft_workspace_size.restype = sz
    lib.dspark_rnn_draft_workspace_size.argtypes = [i32] * 6
    lib.dspark_rnn_draft.argtypes = ([i32] * 9 + [P] * 7 + [P, f32, f32, P, f32, P, P, u64, u64] + [P] * 5
                                     + [P, sz, P])
    lib.dspark_rnn_draft.restype = i32
    lib.dspark_verify_rnn.argtypes = ([i32] * 7 + [P] * 4 + [P] * 5 + [f32, P, u64, u64] + [P] * 3 + [P, sz, P])
    lib.dspark_verify_rnn.restype = i32
    lib.dspark_sts_fit_workspace_size.restype = sz
    lib.dspark_sts_fit_workspace_size.argtypes = [i32] * 4
    lib.dspark_sts_fit.argtypes = [i32, i32, P, P, P, i32, i32, P, P, P, sz, P]
    lib.dspark_sts_fit.restype = i32
    i64 = ctypes.c_int64
    lib.dspark_token_logprobs.argtypes = [i32, i32, i64, i32, P, P, f32, i32] + [P] * 6
    lib.dspark_token_logprobs.restype = i32
    lib.dspark_token_logprobs_backward.argtypes = [i32, i32, i64, i64, i32, P, P, f32] + [P] * 6
    lib.dspark_token_logprobs_backward.restype = i32
    tables = [i32] * 4 + [i64] + [P] * 3
    lib.dspark_cache_workspace_size.argtypes = [i32, i32]
    lib.dspark_cache_workspace_size.restype = sz
    lib.dspark_cache_fork.argtypes = [i32] + tables + [P, P, P, sz, P]
    lib.dspark_cache_fork.restype = i32
    lib.dspark_cache_reserve.argtypes = tables + [P, P, P, i32, P, sz, P, sz, P]
    lib.dspark_cache_reserve.restype = i32
    lib.dspark_cache_write.argtypes = ([i32] * 9 + [P, P, i64, i64, P, P, i64, i64, i64, P, i64] + [P] * 5
                                       + [P, sz, P])
    lib.dspark_cache_write.restype = i32
    lib.dspark_cache_truncate.argtypes = tables + [P, P, sz, P]
    lib.dspark_cache_truncate.restype = i32
    lib.dspark_cache_compact.argtypes = tables + [P, i32, P, sz, P, sz, P]
    lib.dspark_cache_compact.restype = i32
    lib.dspark_paged_attention_workspace_size.argtypes = [i32] * 6
    lib.dspark_paged_attention_workspace_size.restype = sz
    lib.dspark_paged_attention.argtypes = ([i32] * 11 + [P, i64, i64, P, P, i64, i64, i64, P, i64, P, P, f32, P, P,
                                           i32, P, P, P, sz, P])
    lib.dspark_paged_attention.restype = i32
    lib.dspark_paged_attention_granted.argtypes = ([i32] * 11 + [P, i64, i64, P, P, i64, i64, i64, P, i64, P, P, P, f32,
                                                                 P, P, i32, P, P, P, sz, P])
    lib.dspark_paged_attention_granted.restype = i32
    lib.dspark_chunk_attention_workspace_size.argtypes = [i32] * 5
    lib.dspark_chunk_attention_workspace_size.restype = sz
    lib.dspark_chunk_attention.argtypes = ([i32] * 10 + [P, i64, i64, P, P, i64, i64, i64, P, i64, P, P, P, f32, P, P, i32,
                                                         P, P, P, sz, P])
    lib.dspark_chunk_attention.restype = i32
    lib.dspark_rotary.argtypes = [i32] * 7 + [P, i64, i64, P, P, f32, P, i64, i64, P]
    lib.dspark_rotary.restype = i32
    lib.dspark_cache_append.argtypes = ([i32] * 12 + [P, i64, i64, P, P, i64, i64, P, i64, i64, P, P, i64, i64, i64, P, i64]
                                        + [P] * 5 + [P, f32, P, sz, P])
    lib.dspark_cache_append.restype = i32
    lib.dspark_cache_append_any.argtypes = lib.dspark_cache_append.argtypes
    lib.dspark_cache_append_any.restype = i32
    lib.dspark_adjust_logits.argtypes = ([i32] * 4 + [P, i64, P, P, P, i64, i32] + [P] * 5 + [i32, P, P, P, i64, i32, P, P,
                                                                                             i64, P])
    lib.dspark_adjust_logits.restype = i32
    for fn in ("dspark_markov_draft", "dspark_schedule", "dspark_verify", "dspark_workspace_status"):
        getattr(lib, fn).restype = i32
    return lib


lib = _load_library()


def _check(status: int, what: str):
    if status != 0:
        name = lib.dspark_status_string(status).decode()
        msg = lib.dspark_last_error_message().decode()
        raise DSparkError(f"{what}: {name}: {msg}")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda(t, name, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise DSparkError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise DSparkError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise DSparkError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _dt(t, name):
    if t.dtype not in _DT:
        raise DSparkError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return _DT[t.dtype]


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def workspace(nbytes: int, device) -> torch.Tensor:
    """A caller-owned, 256-byte aligned device workspace whose status word starts at 0."""
    ws = torch.zeros(max(256, int(nbytes)) + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + max(256, int(nbytes))]


def draft_workspace_size(R, gamma, V, rank, d, w_dtype) -> int:
    return int(lib.dspark_markov_draft_workspace_size(R, gamma, V, rank, d, _DT[w_dtype]))


def schedule_workspace_size(R, gamma) -> int:
    return int(lib.dspark_schedule_workspace_size(R, gamma))


def verify_workspace_size(R, gamma, V, rank, w_dtype) -> int:
    return int(lib.dspark_verify_workspace_size(R, gamma, V, rank, _DT[w_dtype]))


def markov_draft(U, W1, W2, h, conf_w, conf_b, conf_logit_scale, conf_temp, temperature, x0, req_id,
                 seed, rnd, out=None, ws=None, stream=None):
    """Stage 1 (dspark_markov_draft).  Returns dict x, logq, lse, conf (device tensors)."""
    R, gamma, V = U.shape
    rank = W1.shape[1]
    d = h.shape[2] if h is not None else 0
    dev = U.device
    for t, n in ((U, "U"), (W1, "W1"), (W2, "W2")):
        _cuda(t, n)
    if h is not None:
        _cuda(h, "h")
    _cuda(conf_w, "conf_w", torch.float32)
    _cuda(conf_temp, "conf_temp", torch.float32)
    _cuda(x0, "x0", torch.int32)
    _cuda(req_id, "req_id", torch.int64)
    if W1.dtype != W2.dtype:
        raise DSparkError("W1 and W2 must share a dtype")
    if out is None:
        out = dict(x=torch.empty((R, gamma), dtype=torch.int32, device=dev),
                   logq=torch.empty((R, gamma), dtype=torch.float32, device=dev),
                   lse=torch.empty((R, gamma), dtype=torch.float32, device=dev),
                   conf=torch.empty((R, gamma), dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(draft_workspace_size(R, gamma, V, rank, d, W1.dtype), dev)
    st = lib.dspark_markov_draft(R, gamma, V, rank, d, _dt(U, "U"), _dt(W1, "W1"),
                                 _dt(h, "h") if h is not None else F32,
                                 _p(U), _p(W1), _p(W2), _p(h), _p(conf_w), float(conf_b),
                                 float(conf_logit_scale), _p(conf_temp), float(temperature), _p(x0),
                                 _p(req_id), int(seed), int(rnd), _p(out["x"]), _p(out["logq"]),
                                 _p(out["lse"]), _p(out["conf"]), _p(ws), ws.numel(), _stream(stream))
    _check(st, "dspark_markov_draft")
    return out


def schedule(conf, sps, mode, conf_hist=None, fixed_len=0, out=None, ws=None, stream=None):
    """Stage 2 (dspark_schedule).  Returns dict ell [R] int32, B [1] int32, tau [1] float64."""
    _cuda(conf, "conf", torch.float32)
    R, gamma = conf.shape
    dev = conf.device
    if sps is not None:
        _cuda(sps, "sps", torch.float64)
    if conf_hist is not None:
        _cuda(conf_hist, "conf_hist", torch.float32)
    if out is None:
        out = dict(ell=torch.empty(R, dtype=torch.int32, device=dev),
                   B=torch.empty(1, dtype=torch.int32, device=dev),
                   tau=torch.empty(1, dtype=torch.float64, device=dev))
    if ws is None:
        ws = workspace(schedule_workspace_size(R, gamma), dev)
    st = lib.dspark_schedule(R, gamma, _p(conf), _p(sps), 0 if sps is None else sps.numel(), int(mode),
                             _p(conf_hist), int(fixed_len), _p(out["ell"]), _p(out["B"]), _p(out["tau"]),
                             _p(ws), ws.numel(), _stream(stream))
    _check(st, "dspark_schedule")
    return out


def schedule_threshold(conf, threshold, out=None, ws=None, stream=None):
    """Stage 2 with a fixed confidence cutoff (dspark_schedule_threshold).  Returns dict
    ell [R] int32, B [1] int32, tau [1] float64."""
    _cuda(conf, "conf", torch.float32)
    R, gamma = conf.shape
    dev = conf.device
    if out is None:
        out = dict(ell=torch.empty(R, dtype=torch.int32, device=dev),
                   B=torch.empty(1, dtype=torch.int32, device=dev),
                   tau=torch.empty(1, dtype=torch.float64, device=dev))
    if ws is None:
        ws = workspace(schedule_workspace_size(R, gamma), dev)
    st = lib.dspark_schedule_threshold(R, gamma, _p(conf), float(threshold), _p(out["ell"]), _p(out["B"]),
                                       _p(out["tau"]), _p(ws), ws.numel(), _stream(stream))
    _check(st, "dspark_schedule_threshold")
    return out


def verify(target, U, W1, W2, x0, x, logq, lse_q, ell, temperature, req_id, seed, rnd, out=None,
           ws=None, stream=None):
    """Stage 3 (dspark_verify).  Returns dict n_acc [R], tokens [R,gamma+1], n_out [R]."""
    R, g1, V = target.shape
    gamma = g1 - 1
    rank = W1.shape[1]
    dev = target.device
    for t, n in ((target, "target"), (U, "U"), (W1, "W1"), (W2, "W2")):
        _cuda(t, n)
    _cuda(x0, "x0", torch.int32)
    _cuda(x, "x", torch.int32)
    _cuda(logq, "logq", torch.float32)
    _cuda(lse_q, "lse_q", torch.float32)
    _cuda(ell, "ell", torch.int32)
    _cuda(req_id, "req_id", torch.int64)
    if out is None:
        out = dict(n_acc=torch.empty(R, dtype=torch.int32, device=dev),
                   tokens=torch.empty((R, gamma + 1), dtype=torch.int32, device=dev),
                   n_out=torch.empty(R, dtype=torch.int32, device=dev))
    if ws is None:
        ws = workspace(verify_workspace_size(R, gamma, V, rank, W1.dtype), dev)
    st = lib.dspark_verify(R, gamma, V, rank, _dt(target, "target"), _dt(U, "U"), _dt(W1, "W1"),
                           _p(target), _p(U), _p(W1), _p(W2), _p(x0), _p(x), _p(logq), _p(lse_q), _p(ell),
                           float(temperature), _p(req_id), int(seed), int(rnd), _p(out["n_acc"]),
                           _p(out["tokens"]), _p(out["n_out"]), _p(ws), ws.numel(), _stream(stream))
    _check(st, "dspark_verify")
    return out


def verify_ragged(target_rows, row_offset, U, W1, W2, x0, x, logq, lse_q, ell, temperature, req_id, seed, rnd,
                  out=None, ws=None, stream=None):
    """Stage 3 on a flattened target (dspark_verify_ragged): target_rows [n_rows, V],
    request r's verify rows at row_offset[r] + t.  Returns dict n_acc, tokens, n_out."""
    n_rows, V = target_rows.shape
    R, gamma = x.shape
    rank = W1.shape[1]
    dev = target_rows.device
    for t, n in ((target_rows, "target_rows"), (U, "U"), (W1, "W1"), (W2, "W2")):
        _cuda(t, n)
    _cuda(row_offset, "row_offset", torch.int32)
    _cuda(x0, "x0", torch.int32)
    _cuda(x, "x", torch.int32)
    _cuda(logq, "logq", torch.float32)
    _cuda(lse_q, "lse_q", torch.float32)
    _cuda(ell, "ell", torch.int32)
    _cuda(req_id, "req_id", torch.int64)
    if out is None:
        out = dict(n_acc=torch.empty(R, dtype=torch.int32, device=dev),
                   tokens=torch.empty((R, gamma + 1), dtype=torch.int32, device=dev),
                   n_out=torch.empty(R, dtype=torch.int32, device=dev))
    if ws is None:
        ws = workspace(verify_workspace_size(R, gamma, V, rank, W1.dtype), dev)
    st = lib.dspark_verify_ragged(R, gamma, V, rank, _dt(target_rows, "target_rows"), _dt(U, "U"), _dt(W1, "W1"),
                                  _p(target_rows), int(n_rows), _p(row_offset), _p(U), _p(W1), _p(W2), _p(x0),
                                  _p(x), _p(logq), _p(lse_q), _p(ell), float(temperature), _p(req_id), int(seed),
                                  int(rnd), _p(out["n_acc"]), _p(out["tokens"]), _p(out["n_out"]), _p(ws),
                                  ws.numel(), _stream(stream))
    _check(st, "dspark_verify_ragged")
    return out


def verify_overlap_workspace_size(R, gamma, V, rank, w_dtype) -> int:
    return int(lib.dspark_verify_overlap_workspace_size(R, gamma, V, rank, _DT[w_dtype]))


def verify_overlap(target, U, W1, W2, x0, x, logq, lse_q, ell, temperature, req_id, seed, rnd, out=None,
                   ws=None, stream=None):
    """Stage 3 with the acceptance overlap fused in (dspark_verify_overlap).  Returns dict
    n_acc [R], tokens [R,gamma+1], n_out [R] and overlap [R,gamma] (NaN past ell[r])."""
    R, g1, V = target.shape
    gamma = g1 - 1
    rank = W1.shape[1]
    dev = target.device
    for t, n in ((target, "target"), (U, "U"), (W1, "W1"), (W2, "W2")):
        _cuda(t, n)
    _cuda(x0, "x0", torch.int32)
    _cuda(x, "x", torch.int32)
    _cuda(logq, "logq", torch.float32)
    _cuda(lse_q, "lse_q", torch.float32)
    _cuda(ell, "ell", torch.int32)
    _cuda(req_id, "req_id", torch.int64)
    if out is None:
        out = dict(n_acc=torch.empty(R, dtype=torch.int32, device=dev),
                   tokens=torch.empty((R, gamma + 1), dtype=torch.int32, device=dev),
                   n_out=torch.empty(R, dtype=torch.int32, device=dev),
                   overlap=torch.empty((R, gamma), dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(verify_overlap_workspace_size(R, gamma, V, rank, W1.dtype), dev)
    st = lib.dspark_verify_overlap(R, gamma, V, rank, _dt(target, "target"), _dt(U, "U"), _dt(W1, "W1"),
                                   _p(target), _p(U), _p(W1), _p(W2), _p(x0), _p(x), _p(logq), _p(lse_q), _p(ell),
                                   float(temperature), _p(req_id), int(seed), int(rnd), _p(out["n_acc"]),
                                   _p(out["tokens"]), _p(out["n_out"]), _p(out["overlap"]), _p(ws), ws.numel(),
                                   _stream(stream))
    _check(st, "dspark_verify_overlap")
    return out


def acceptance_overlap_workspace_size(R, gamma, V, rank, w_dtype) -> int:
    return int(lib.dspark_acceptance_overlap_workspace_size(R, gamma, V, rank, _DT[w_dtype]))


def acceptance_overlap(target, U, W1, W2, x0, x, lse_q, ell, temperature, out=None, ws=None, stream=None):
    """Expected acceptance c*[r,j] = sum_v min(q_j, p_j) of every drafted position
    (dspark_acceptance_overlap); ell None evaluates all positions.  Returns [R,gamma]
    float32, NaN past ell[r]."""
    R, g1, V = target.shape
    gamma = g1 - 1
    rank = W1.shape[1]
    dev = target.device
    for t, n in ((target, "target"), (U, "U"), (W1, "W1"), (W2, "W2")):
        _cuda(t, n)
    _cuda(x0, "x0", torch.int32)
    _cuda(x, "x", torch.int32)
    _cuda(lse_q, "lse_q", torch.float32)
    if ell is not None:
        _cuda(ell, "ell", torch.int32)
    if out is None:
        out = torch.empty((R, gamma), dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(acceptance_overlap_workspace_size(R, gamma, V, rank, W1.dtype), dev)
    st = lib.dspark_acceptance_overlap(R, gamma, V, rank, _dt(target, "target"), _dt(U, "U"), _dt(W1, "W1"),
                                       _p(target), _p(U), _p(W1), _p(W2), _p(x0), _p(x), _p(lse_q), _p(ell),
                                       float(temperature), _p(out), _p(ws), ws.numel(), _stream(stream))
    _check(st, "dspark_acceptance_overlap")
    return out


def rnn_draft_workspace_size(R, gamma, V, ns, d, w_dtype) -> int:
    return int(lib.dspark_rnn_draft_workspace_size(R, gamma, V, ns, d, _DT[w_dtype]))


def rnn_draft(U, E, Wse, Wh, bgc, Wo, h, conf_w, conf_b, conf_logit_scale, conf_temp, temperature, x0, req_id,
              seed, rnd, out=None, ws=None, stream=None):
    """Stage 1 with the recurrent head (dspark_rnn_draft).  Returns dict x, logq, lse, conf,
    state [R,gamma,ns]."""
    R, gamma, V = U.shape
    ns = Wo.shape[0]
    ne = E.shape[1] if E is not None else 0
    d = h.shape[2] if h is not None else 0
    dev = U.device
    for t, n in ((U, "U"), (Wse, "Wse"), (Wo, "Wo")):
        _cuda(t, n)
    if ne:
        _cuda(E, "E")
    if d:
        _cuda(Wh, "Wh")
        _cuda(h, "h")
    _cuda(bgc, "bgc", torch.float32)
    _cuda(conf_w, "conf_w", torch.float32)
    _cuda(conf_temp, "conf_temp", torch.float32)
    _cuda(x0, "x0", torch.int32)
    _cuda(req_id, "req_id", torch.int64)
    if out is None:
        out = dict(x=torch.empty((R, gamma), dtype=torch.int32, device=dev),
                   logq=torch.empty((R, gamma), dtype=torch.float32, device=dev),
                   lse=torch.empty((R, gamma), dtype=torch.float32, device=dev),
                   conf=torch.empty((R, gamma), dtype=torch.float32, device=dev),
                   state=torch.empty((R, gamma, ns), dtype=Wo.dtype, device=dev))
    if ws is None:
        ws = workspace(rnn_draft_workspace_size(R, gamma, V, ns, d, Wo.dtype), dev)
    st = lib.dspark_rnn_draft(R, gamma, V, ns, ne, d, _dt(U, "U"), _dt(Wo, "Wo"), _dt(h, "h") if d else F32,
                              _p(U), _p(E) if ne else None, _p(Wse), _p(Wh) if d else None, _p(bgc), _p(Wo),
                              _p(h) if d else None, _p(conf_w), float(conf_b), float(conf_logit_scale),
                              _p(conf_temp), float(temperature), _p(x0), _p(req_id), int(seed), int(rnd),
                              _p(out["x"]), _p(out["logq"]), _p(out["lse"]), _p(out["conf"]), _p(out["state"]),
                              _p(ws), ws.numel(), _stream(stream))
    _check(st, "dspark_rnn_draft")
    return out


def verify_rnn(target, U, state, Wo, x0, x, logq, lse_q, ell, temperature, req_id, seed, rnd, out=None, ws=None,
               stream=None):
    """Stage 3 for a block drafted by the recurrent head (dspark_verify_rnn)."""
    R, g1, V = target.shape
    gamma = g1 - 1
    ns = Wo.shape[0]
    dev = target.device
    for t, n in ((target, "target"), (U, "U"), (state, "state"), (Wo, "Wo")):
        _cuda(t, n)
    _cuda(x0, "x0", torch.int32)
    _cuda(x, "x", torch.int32)
    _cuda(logq, "logq", torch.float32)
    _cuda(lse_q, "lse_q", torch.float32)
    _cuda(ell, "ell", torch.int32)
    _cuda(req_id, "req_id", torch.int64)
    if out is None:
        out = dict(n_acc=torch.empty(R, dtype=torch.int32, device=dev),
                   tokens=torch.empty((R, gamma + 1), dtype=torch.int32, device=dev),
                   n_out=torch.empty(R, dtype=torch.int32, device=dev))
    if ws is None:
        ws = workspace(verify_workspace_size(R, gamma, V, ns, Wo.dtype), dev)
    st = lib.dspark_verify_rnn(R, gamma, V, ns, _dt(target, "target"), _dt(U, "U"), _dt(Wo, "Wo"), _p(target),
                               _p(U), _p(state), _p(Wo), _p(x0), _p(x), _p(logq), _p(lse_q), _p(ell),
                               float(temperature), _p(req_id), int(seed), int(rnd), _p(out["n_acc"]),
                               _p(out["tokens"]), _p(out["n_out"]), _p(ws), ws.numel(), _stream(stream))
    _check(st, "dspark_verify_rnn")
    return out


def sts_fit_workspace_size(N, gamma, G, M) -> int:
    return int(lib.dspark_sts_fit_workspace_size(N, gamma, G, M))


def sts_fit(z, acc_len, grid, M, out=None, ws=None, stream=None):
    """Per-position confidence temperatures fitted left to right on held-out samples
    (dspark_sts_fit).  z [N,gamma] fp32 logits, acc_len [N] int32, grid [G] fp32.
    Returns dict T [gamma], ece [gamma]."""
    N, gamma = z.shape
    G = grid.shape[0]
    _cuda(z, "z", torch.float32)
    _cuda(acc_len, "acc_len", torch.int32)
    _cuda(grid, "grid", torch.float32)
    dev = z.device
    if out is None:
        out = dict(T=torch.empty(gamma, dtype=torch.float32, device=dev),
                   ece=torch.empty(gamma, dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(sts_fit_workspace_size(N, gamma, G, M), dev)
    st = lib.dspark_sts_fit(N, gamma, _p(z), _p(acc_len), _p(grid), G, int(M), _p(out["T"]), _p(out["ece"]), _p(ws),
                            ws.numel(), _stream(stream))
    _check(st, "dspark_sts_fit")
    return out


def verify_static(target, U, W1, W2, x0, x, logq, lse_q, ell, temperature, req_id, seed, rnd, out=None,
                  stream=None):
    """Stage 3 through dspark_verify_static: for callers that cannot allocate device
    memory (a pooled allocator they must not bypass, allocation-free serving loops); the
    scratch is the library's own static array, so concurrent calls on one device must
    be ordered by the caller."""
    R, g1, V = target.shape
    gamma = g1 - 1
    rank = W1.shape[1]
    dev = target.device
    for t, n in ((target, "target"), (U, "U"), (W1, "W1"), (W2, "W2")):
        _cuda(t, n)
    _cuda(x0, "x0", torch.int32)
    _cuda(x, "x", torch.int32)
    _cuda(logq, "logq", torch.float32)
    _cuda(lse_q, "lse_q", torch.float32)
    _cuda(ell, "ell", torch.int32)
    _cuda(req_id, "req_id", torch.int64)
    if out is None:
        out = dict(n_acc=torch.empty(R, dtype=torch.int32, device=dev),
                   tokens=torch.empty((R, gamma + 1), dtype=torch.int32, device=dev),
                   n_out=torch.empty(R, dtype=torch.int32, device=dev))
    st = lib.dspark_verify_static(R, gamma, V, rank, _dt(target, "target"), _dt(U, "U"), _dt(W1, "W1"),
                                  _p(target), _p(U), _p(W1), _p(W2), _p(x0), _p(x), _p(logq), _p(lse_q), _p(ell),
                                  float(temperature), _p(req_id), int(seed), int(rnd), _p(out["n_acc"]),
                                  _p(out["tokens"]), _p(out["n_out"]), _stream(stream))
    _check(st, "dspark_verify_static")
    return out


def verify_static_status(reset=False, stream=None) -> int:
    """The device status word of dspark_verify_static's scratch on the current device: what
    the last call's kernels reported (0 OK, 1 bad device data, 5 a bounded wait gave up)."""
    val = ctypes.c_int(0)
    _check(lib.dspark_verify_static_status(int(reset), ctypes.byref(val), _stream(stream)),
           "dspark_verify_static_status")
    return int(val.value)


class StepTimer:
    """Times the draft stage's vocabulary-streaming step kernel (one launch per draft
    position) with CUDA events the library records around each launch."""

    def __init__(self, gamma: int):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * gamma)]
        for e in self.events:
            e.record()  # materialise the handles
        torch.cuda.synchronize()
        self._arr = (ctypes.c_void_p * len(self.events))(*[e.cuda_event for e in self.events])
        self.samples = []

    def __enter__(self):
        lib.dspark_set_profile_events(self._arr, len(self.events))
        return self

    def __exit__(self, *exc):
        lib.dspark_set_profile_events(None, 0)

    def collect(self):
        """After the stream has synchronised: append this round's per-launch times (ms)."""
        for k in range(len(self.events) // 2):
            self.samples.append(self.events[2 * k].elapsed_time(self.events[2 * k + 1]))


class VerifyTimer:
    """Times verification's two vocabulary-streaming kernels, the target-row statistics
    pass and the correction pass, with CUDA events the library records around them."""

    def __init__(self):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
        for e in self.events:
            e.record()
        torch.cuda.synchronize()
        self._arr = (ctypes.c_void_p * 4)(*[e.cuda_event for e in self.events])
        self.rows, self.correction = [], []

    def __enter__(self):
        lib.dspark_set_verify_profile_events(self._arr, 4)
        return self

    def __exit__(self, *exc):
        lib.dspark_set_verify_profile_events(None, 0)

    def collect(self):
        """After the stream has synchronised: append this round's two times (ms)."""
        self.rows.append(self.events[0].elapsed_time(self.events[1]))
        self.correction.append(self.events[2].elapsed_time(self.events[3]))


def device_status(ws, reset=False, stream=None) -> int:
    """The workspace's device status word (0 OK, 5 a bounded wait gave up, 1 bad device data)."""
    val = ctypes.c_int(0)
    _check(lib.dspark_workspace_status(_p(ws), int(reset), ctypes.byref(val), _stream(stream)),
           "dspark_workspace_status")
    return int(val.value)


class Round:
    """One DSpark round (draft -> schedule -> verify) over a fixed workload shape, with
    every output and workspace allocated once, so that repeated rounds (and CUDA-graph
    capture) launch kernels only."""

    def __init__(self, w: dict):
        self.w = w
        R, gamma, V, rank, d = w["R"], w["gamma"], w["V"], w["rank"], w["d"]
        dev = w["U"].device
        self.draft_out = dict(x=torch.empty((R, gamma), dtype=torch.int32, device=dev),
                              logq=torch.empty((R, gamma), dtype=torch.float32, device=dev),
                              lse=torch.empty((R, gamma), dtype=torch.float32, device=dev),
                              conf=torch.empty((R, gamma), dtype=torch.float32, device=dev))
        self.sched_out = dict(ell=torch.empty(R, dtype=torch.int32, device=dev),
                              B=torch.empty(1, dtype=torch.int32, device=dev),
                              tau=torch.empty(1, dtype=torch.float64, device=dev))
        self.verify_out = dict(n_acc=torch.empty(R, dtype=torch.int32, device=dev),
                               tokens=torch.empty((R, gamma + 1), dtype=torch.int32, device=dev),
                               n_out=torch.empty(R, dtype=torch.int32, device=dev))
        self.rnn = w.get("head") == "rnn"
        if self.rnn:
            self.draft_out["state"] = torch.empty((R, gamma, rank), dtype=w["Wo"].dtype, device=dev)
            self.ws_draft = workspace(rnn_draft_workspace_size(R, gamma, V, rank, d, w["Wo"].dtype), dev)
        else:
            self.ws_draft = workspace(draft_workspace_size(R, gamma, V, rank, d, w["W1"].dtype), dev)
        self.ws_sched = workspace(schedule_workspace_size(R, gamma), dev)
        wdt = w["Wo"].dtype if self.rnn else w["W1"].dtype
        self.ws_verify = workspace(verify_workspace_size(R, gamma, V, rank, wdt), dev)
        self.x0 = w["x0"].clone()

    def run(self, rnd=0, x0=None, stream=None):
        w = self.w
        x0 = self.x0 if x0 is None else x0
        if self.rnn:
            d = rnn_draft(w["U"], w["E"], w["Wse"], w["Wh"], w["bgc"], w["Wo"], w["h"], w["conf_w"], w["conf_b"],
                          w["conf_logit_scale"], w["conf_temp"], w["temperature"], x0, w["req_id"], w["seed"], rnd,
                          out=self.draft_out, ws=self.ws_draft, stream=stream)
        else:
            d = markov_draft(w["U"], w["W1"], w["W2"], w["h"], w["conf_w"], w["conf_b"], w["conf_logit_scale"],
                             w["conf_temp"], w["temperature"], x0, w["req_id"], w["seed"], rnd,
                             out=self.draft_out, ws=self.ws_draft, stream=stream)
        s = schedule(d["conf"], w["sps"], w["mode"], w.get("conf_hist"), w.get("fixed_len", 0),
                     out=self.sched_out, ws=self.ws_sched, stream=stream)
        if self.rnn:
            v = verify_rnn(w["target"], w["U"], d["state"], w["Wo"], x0, d["x"], d["logq"], d["lse"], s["ell"],
                           w["temperature"], w["req_id"], w["seed"], rnd, out=self.verify_out, ws=self.ws_verify,
                           stream=stream)
        else:
            v = verify(w["target"], w["U"], w["W1"], w["W2"], x0, d["x"], d["logq"], d["lse"], s["ell"],
                       w["temperature"], w["req_id"], w["seed"], rnd, out=self.verify_out, ws=self.ws_verify,
                       stream=stream)
        return d, s, v

    def capture(self, rnd=0, x0=None, timer=None):
        """Capture one round (round index ``rnd``) as a CUDA graph.  Replaying it launches
        the round's kernels with no host work; it writes the same output tensors as
        ``run``.  With ``timer`` (a StepTimer) the graph also records its step events."""
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream(device=self.w["U"].device)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            if timer is not None:
                with timer:
                    self.run(rnd, x0)
            else:
                self.run(rnd, x0)
        torch.cuda.current_stream().wait_stream(side)
        return g

    def status(self) -> int:
        codes = [device_status(ws) for ws in (self.ws_draft, self.ws_sched, self.ws_verify)]
        return max(codes)


# The serving-side calls: their tensors are checked and passed on by the compiled module.

def _load_marshal():
    path = _build.MARSHAL
    if not os.path.exists(path):
        raise DSparkError(f"_marshal.so is not built ({path}); run __graft_entry__.build()")
    spec = importlib.util.spec_from_file_location("_marshal", path)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        raise DSparkError(f"_marshal.so does not load ({e}); run __graft_entry__.build() with this PyTorch "
                          f"({torch.__version__})") from e
    module.set_error(DSparkError)
    return module


class _Marshal:
    """Stands for the module until the first serving-side call loads it: whoever makes none of these
    calls needs the library alone."""

    def __getattr__(self, name):
        global _m
        _m = _load_marshal()
        return getattr(_m, name)


_m = _Marshal()
_raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _raw_stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream_of is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream_of(_current_device())


def _made_on(stream):
    """Where a call makes the buffers it was not given: on the stream that it runs on (a buffer
    belongs to the stream of its making, and a workspace is cleared there)."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _on_gpu(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise DSparkError(f"{name} must be a CUDA tensor")
    return t


# ------------------------------------------------------------- token log probabilities

def token_logprobs(logits, tokens, temperature=1.0, top_k=0, out=None, stream=None):
    """Log probability of each row's token, the row's entropy and log-normaliser, and its
    ``top_k`` best alternatives (dspark_token_logprobs).  logits [N,V] float32, bfloat16 or
    float16 with any row stride; tokens [N] int32, rows with an id outside [0,V) (verification
    writes -1) are skipped and hold NaN / -1.  Returns dict logprob, entropy, lse [N] and, with
    top_k, top_ids, top_logprobs [N,top_k].  No graph is recorded, whatever the logits require: their
    gradient is token_logprobs_backward's."""
    if out is None:
        N = _on_gpu(logits, "logits").shape[0]
        f = dict(dtype=torch.float32, device=logits.device)
        with _made_on(stream):
            out = dict(logprob=torch.empty(N, **f), entropy=torch.empty(N, **f), lse=torch.empty(N, **f))
            if top_k > 0:
                out["top_ids"] = torch.empty((N, top_k), dtype=torch.int32, device=logits.device)
                out["top_logprobs"] = torch.empty((N, top_k), **f)
    st = _m.token_logprobs(logits, tokens, temperature, top_k, out["logprob"], out["entropy"], out["lse"],
                           out.get("top_ids"), out.get("top_logprobs"), _raw_stream(stream))
    if st:
        _check(st, "dspark_token_logprobs")
    return out


def token_logprobs_backward(logits, tokens, lse, entropy, grad_logprob, grad_entropy=None, temperature=1.0, out=None,
                            stream=None):
    """The gradient of sum(grad_logprob * logprob + grad_entropy * entropy) for ``logits``
    (dspark_token_logprobs_backward), from token_logprobs' lse and entropy.  ``out`` [N,V] of the
    logits' type may be the logits themselves."""
    if out is None:
        with _made_on(stream):
            out = torch.empty_like(_on_gpu(logits, "logits"), memory_format=torch.contiguous_format)
    st = _m.token_logprobs_backward(logits, tokens, lse, entropy, grad_logprob, grad_entropy, temperature, out,
                                    _raw_stream(stream))
    if st:
        _check(st, "dspark_token_logprobs_backward")
    return out


# ------------------------------------------------------------------------- paged cache

def cache_workspace_size(R, num_pages) -> int:
    return int(lib.dspark_cache_workspace_size(R, num_pages))


class CachePools:
    """The pools whose pages move together (every layer's keys and values), as the pointer
    list that dspark_cache_reserve and dspark_cache_compact take.  Keeps the tensors alive."""

    def __init__(self, pools):
        self.tensors = list(pools)
        self.n, self.page_bytes, self.num_pages = len(self.tensors), 0, None
        for i, t in enumerate(self.tensors):
            _cuda(t, f"pools[{i}]")
            if t.dim() < 2 or t.shape != self.tensors[0].shape or t.element_size() != self.tensors[0].element_size():
                raise DSparkError("pools must share one shape [num_pages, ...] and element size")
        if self.tensors:
            t = self.tensors[0]
            self.num_pages = t.shape[0]
            self.page_bytes = t.numel() // max(1, t.shape[0]) * t.element_size()
        self.array = (ctypes.c_void_p * max(1, self.n))(*[t.data_ptr() for t in self.tensors])
        self.address = ctypes.addressof(self.array)


def cache_pools(pools) -> CachePools:
    return CachePools(pools)


def _cache_ws(ws, page_table, ref_count, stream):
    if ws is None:
        with _made_on(stream):
            ws = workspace(cache_workspace_size(_on_gpu(page_table, "page_table").shape[0],
                                                _on_gpu(ref_count, "ref_count").numel()), page_table.device)
    return ws


def _page_pools(pools, ref_count):
    if not isinstance(pools, CachePools):
        pools = CachePools(pools or [])
    if pools.n and pools.num_pages != ref_count.numel():
        raise DSparkError(f"the pools have {pools.num_pages} pages, ref_count {ref_count.numel()}")
    return pools


def cache_fork(page_table, seq_len, ref_count, src, dst, page_size, ws=None, stream=None):
    """Empty slots ``dst`` become copies of slots ``src`` that share their pages
    (dspark_cache_fork).  src, dst [F] int32."""
    st = _m.cache_fork(page_table, seq_len, ref_count, src, dst, page_size, _cache_ws(ws, page_table, ref_count, stream),
                       _raw_stream(stream))
    if st:
        _check(st, "dspark_cache_fork")


def cache_reserve(page_table, seq_len, ref_count, n_new, page_size, pools, out=None, ws=None, stream=None):
    """Room for ``n_new`` [R] int32 more tokens in every slot, with a copy of each partly filled
    shared page about to be written (dspark_cache_reserve).  ``pools``: cache_pools(...), a list
    of pools, or None to change the tables only.  Returns dict granted [R], copies [R,2]."""
    if out is None:
        i32 = dict(dtype=torch.int32, device=_on_gpu(page_table, "page_table").device)
        with _made_on(stream):
            out = dict(granted=torch.empty(page_table.shape[0], **i32),
                       copies=torch.empty((page_table.shape[0], 2), **i32))
    pools = _page_pools(pools, ref_count)
    st = _m.cache_reserve(page_table, seq_len, ref_count, n_new, page_size, pools.n, pools.address, pools.page_bytes,
                          out["granted"], out["copies"], _cache_ws(ws, page_table, ref_count, stream), _raw_stream(stream))
    if st:
        _check(st, "dspark_cache_reserve")
    return out


def cache_write(k, v, k_pool, v_pool, page_table, seq_len, q_start, granted=None, k_scale=None, v_scale=None, ws=None,
                stream=None):
    """Writes the keys and values k, v [T,Hkv,D] of every slot's last tokens (rows q_start[r] ..
    q_start[r+1]-1) into one layer's pools [num_pages,Hkv,page_size,D] (dspark_cache_write), after
    cache_reserve made room.  Pools of float8_e4m3fn hold x / scale[head]."""
    if ws is None:
        with _made_on(stream):
            ws = workspace(256, _on_gpu(k_pool, "k_pool").device)
    st = _m.cache_write(k, v, k_pool, v_pool, page_table, seq_len, q_start, granted, k_scale, v_scale, ws,
                        _raw_stream(stream))
    if st:
        _check(st, "dspark_cache_write")


def cache_truncate(page_table, seq_len, ref_count, new_len, page_size, ws=None, stream=None):
    """Every slot keeps its first ``new_len`` [R] int32 tokens; pages past them are released
    (dspark_cache_truncate).  0 frees the slot."""
    st = _m.cache_truncate(page_table, seq_len, ref_count, new_len, page_size, _cache_ws(ws, page_table, ref_count, stream),
                           _raw_stream(stream))
    if st:
        _check(st, "dspark_cache_truncate")


def cache_compact(page_table, seq_len, ref_count, page_size, pools, out=None, ws=None, stream=None):
    """Moves the used pages to the lowest indexes, in the tables and in every pool
    (dspark_cache_compact).  Returns the number of pages moved, [1] int32."""
    if out is None:
        with _made_on(stream):
            out = torch.empty(1, dtype=torch.int32, device=_on_gpu(page_table, "page_table").device)
    pools = _page_pools(pools, ref_count)
    st = _m.cache_compact(page_table, seq_len, ref_count, page_size, pools.n, pools.address, pools.page_bytes, out,
                          _cache_ws(ws, page_table, ref_count, stream), _raw_stream(stream))
    if st:
        _check(st, "dspark_cache_compact")
    return out


def paged_attention_workspace_size(T, R, Hq, Hkv, D, max_q) -> int:
    return int(lib.dspark_paged_attention_workspace_size(T, R, Hq, Hkv, D, max_q))


def _attention_workspace(nbytes, device):
    """A workspace of which only the status block is cleared: the call writes the rest before it
    reads it."""
    ws = torch.empty(max(256, nbytes) + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + max(256, nbytes)]
    ws[:256].zero_()
    return ws


def paged_attention(q, k_pool, v_pool, page_table, seq_len, q_start, max_q, scale, k_scale=None, v_scale=None,
                    window=0, out=None, ws=None, stream=None, granted=None):
    """Attention of every slot's last tokens over its paged context (dspark_paged_attention).
    q [T,Hq,D] bfloat16 or float16, rows q_start[r] .. q_start[r+1]-1 for slot r, at most
    ``max_q`` a slot.  The queries of a slot whose entry of ``granted`` [R] int32 is 0 (cache_reserve
    found no room for them) see nothing.  Returns dict out [T,Hq,D], lse [T,Hq] float32."""
    if out is None or ws is None:
        T, Hq, D = _on_gpu(q, "q").shape
        with _made_on(stream):
            if out is None:
                out = dict(out=torch.empty((T, Hq, D), dtype=q.dtype, device=q.device),
                           lse=torch.empty((T, Hq), dtype=torch.float32, device=q.device))
            if ws is None:
                ws = _attention_workspace(
                    paged_attention_workspace_size(T, page_table.shape[0], Hq, k_pool.shape[1], D, max_q), q.device)
    st = _m.paged_attention(q, k_pool, v_pool, page_table, seq_len, q_start, max_q, scale, k_scale, v_scale, window,
                            out["out"], out.get("lse"), ws, _raw_stream(stream), granted)
    if st:
        _check(st, "dspark_paged_attention")
    return out


def chunk_attention_workspace_size(T, R, Hq, Hkv, D) -> int:
    return int(lib.dspark_chunk_attention_workspace_size(T, R, Hq, Hkv, D))


def chunk_attention(q, k_pool, v_pool, page_table, seq_len, q_start, scale, k_scale=None, v_scale=None, window=0, out=None,
                    ws=None, stream=None, granted=None):
    """paged_attention without a bound on a slot's queries: chunks of prompts, beside slots that
    decode (dspark_chunk_attention).  Returns dict out [T,Hq,D], lse [T,Hq] float32."""
    _here(q, "q")
    if out is None or ws is None:
        T, Hq, D = q.shape
        with _made_on(stream):
            if out is None:
                out = dict(out=torch.empty((T, Hq, D), dtype=q.dtype, device=q.device),
                           lse=torch.empty((T, Hq), dtype=torch.float32, device=q.device))
            if ws is None:
                ws = _attention_workspace(
                    chunk_attention_workspace_size(T, page_table.shape[0], Hq, k_pool.shape[1], D), q.device)
    st = _m.chunk_attention(q, k_pool, v_pool, page_table, seq_len, q_start, scale, k_scale, v_scale, window, out["out"],
                            out.get("lse"), ws, _raw_stream(stream), granted)
    if st:
        _check(st, "dspark_chunk_attention")
    return out


# ------------------------------------------------------------------- rotary positions

@functools.lru_cache(maxsize=8)
def _pi(digits):
    """Decimal of pi, by Machin's formula in whole numbers."""
    one = 10 ** (digits + 10)

    def arctan_of_inverse(n):
        power = total = one // n
        for k in range(3, 4 * digits + 40, 2):
            power //= -n * n
            total += power // k
        return total

    return decimal.Decimal(16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239)).scaleb(-(digits + 10))


def rotary_rates(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=None, low=1.0, high=32.0, factors=None,
                 device="cuda") -> torch.Tensor:
    """What rotary and cache_append take as the pairs' turns per position: int64 [rot_dim/2], units of
    2^-64 turns, from f_i = base^(-2i/rot_dim) radians per position and

      scaling="none"    f_i
      scaling="linear"  f_i / factor (positions interpolated)
      scaling="ntk"     base * factor^(rot_dim/(rot_dim-2)) in the place of base
      scaling="bands"   f_i where a pair makes more than ``high`` turns within ``original_len``
                        positions, f_i / factor where it makes fewer than ``low``, and a blend, linear
                        in the turns, between
      scaling="yarn"    the same with a blend linear in the pair's index (its magnitude is
                        rotary_magnitude(factor))

    ``factors`` [rot_dim/2], if given, divides the result pair by pair.  Computed with 60 digits and more, so that
    a rate is off by half a unit, and an angle at position p by 2^-64 p half turns, at most."""
    if rot_dim < 2 or rot_dim % 2:
        raise DSparkError(f"rot_dim={rot_dim} must be even and positive")
    if not (base > 0 and math.isfinite(base) and factor > 0 and math.isfinite(factor)):
        raise DSparkError("base and factor must be positive and finite")
    if scaling not in ("none", "linear", "ntk", "bands", "yarn"):
        raise DSparkError(f"scaling={scaling!r} must be none, linear, ntk, bands or yarn")
    pairs = rot_dim // 2
    kept = None  # of each pair: 1 as it is, 0 stretched
    if scaling in ("bands", "yarn"):
        if original_len is None or original_len <= 0 or not 0 < low < high:
            raise DSparkError(f"scaling={scaling!r} needs original_len > 0 and 0 < low < high")
        if scaling == "yarn" and base <= 1:
            raise DSparkError("scaling='yarn' needs base > 1")
    if factors is not None:
        factors = [float(x) for x in factors]
        if len(factors) != pairs or not all(x > 0 and math.isfinite(x) for x in factors):
            raise DSparkError(f"factors must hold {pairs} positive values")
    # digits before the point: of the largest rate that these can make
    digits = 60 + math.ceil(abs(math.log10(base)) + abs(math.log10(factor)) * (2 if scaling != "ntk" or rot_dim == 2 else
                            rot_dim / (rot_dim - 2)) + max([0.0] + [abs(math.log10(x)) for x in factors or ()]))
    context = decimal.Context(prec=digits, Emin=decimal.MIN_EMIN, Emax=decimal.MAX_EMAX)
    with decimal.localcontext(context):
        exact = lambda x: decimal.Decimal(float(x))
        tau, by, b = 2 * _pi(digits), exact(factor), exact(base)
        if scaling == "ntk" and rot_dim > 2:
            b *= by ** (decimal.Decimal(rot_dim) / (rot_dim - 2))
        step, f = b ** (decimal.Decimal(-2) / rot_dim), [decimal.Decimal(1)]
        for _ in range(pairs - 1):
            f.append(f[-1] * step)
        clamp = lambda x: min(decimal.Decimal(1), max(decimal.Decimal(0), x))
        if scaling == "linear":
            f = [x / by for x in f]
        elif scaling == "bands":
            n, lo, span = exact(original_len) / tau, exact(low), exact(high) - exact(low)
            kept = [clamp((n * x - lo) / span) for x in f]
        elif scaling == "yarn":
            index = lambda turns: rot_dim * math.log(original_len / (math.tau * turns)) / (2.0 * math.log(base))
            first, last = max(0, math.floor(index(high))), min(rot_dim - 1, math.ceil(index(low)))
            kept = [1 - clamp(decimal.Decimal(i - first) / max(last - first, exact(0.001))) for i in range(pairs)]
        if kept is not None:
            shrunk = 1 / by
            f = [x * (k + (1 - k) * shrunk) for x, k in zip(f, kept)]
        if factors is not None:
            f = [x / exact(y) for x, y in zip(f, factors)]
        units = 2 ** 64 / tau
        turns = [round(x * units) % (1 << 64) for x in f]
    return torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64, device=device)


def rotary_magnitude(factor) -> float:
    """The magnitude that goes with scaling="yarn"."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def _here(t, name):
    if _current_device is not None and _on_gpu(t, name).get_device() != _current_device():
        raise DSparkError(f"{name} lies on cuda:{t.get_device()}, the current device is cuda:{_current_device()}")
    return t


def rotary(x, positions, rates, interleaved=False, magnitude=1.0, inverse=False, out=None, stream=None):
    """x [T,H,D] float32, bfloat16 or float16 with the first 2 * len(rates) elements of every head
    turned by their row's position, positions [T] int32 (dspark_rotary); rates: rotary_rates(...).
    Pairs are (i, i + rot_dim/2), or neighbours where ``interleaved``.  ``inverse`` turns back: the
    gradient for x from the gradient for the result (no graph is recorded, whatever x requires).
    ``out`` may be x itself."""
    _here(x, "x")
    if out is None:
        with _made_on(stream):
            out = torch.empty_like(x, memory_format=torch.contiguous_format)
    st = _m.rotary(x, positions, rates, bool(interleaved), magnitude, bool(inverse), out, _raw_stream(stream))
    if st:
        _check(st, "dspark_rotary")
    return out


def cache_append(q, k, v, k_pool, v_pool, page_table, seq_len, q_start, rates, interleaved=False, magnitude=1.0,
                 granted=None, k_scale=None, v_scale=None, q_out=None, ws=None, stream=None):
    """cache_write with rotary positions on the way (dspark_cache_append_any): every slot's last tokens'
    keys k [T,Hkv,D] are turned by their position in the slot and stored with the values, and their
    queries q [T,Hq,D] turned into q_out (made where it is not given; q itself will do).  Any even
    number of elements may turn (2 * len(rates), up to D).  Returns q_out; None where q is."""
    _here(k, "k")
    if ws is None or (q_out is None and q is not None):
        with _made_on(stream):
            if ws is None:
                ws = workspace(256, k.device)
            if q_out is None and q is not None:
                q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    st = _m.cache_append(q, k, v, k_pool, v_pool, page_table, seq_len, q_start, rates, bool(interleaved), magnitude, granted,
                         k_scale, v_scale, q_out, ws, _raw_stream(stream))
    if st:
        _check(st, "dspark_cache_append_any")
    return q_out


# --------------------------------------------------------------- adjustment of logits

def adjust_logits(logits, tokens, q_start, history=None, history_len=None, prompt_len=None, repetition=None,
                  frequency=None, presence=None, bias_ids=None, bias=None, mask=None, mask_row=None, out=None, stream=None):
    """Logits [N,V] with penalties for repeated tokens, biases and grammar masks (dspark_adjust_logits).
    Rows q_start[r] .. q_start[r+1]-1 are slot r's, each after the token tokens[n] that was fed in for
    it: a row's sequence is history[r, :history_len[r]] and its block's tokens up to its own.
    history [R,L] int32; prompt_len [R] int32; repetition, frequency, presence [R] float32;
    bias_ids, bias [R,B] int32, float32; mask [M, (V+31)/32 or more] int32 of allowed ids' bits, row
    mask_row[n] of it for row n (none where that is negative), or row n without mask_row.  What is
    None is left out.  ``out`` may be the logits themselves.  Rows of no slot are not written (in a
    result made here they hold anything)."""
    _here(logits, "logits")
    if out is None:
        with _made_on(stream):
            out = torch.empty_like(logits, memory_format=torch.contiguous_format)
    st = _m.adjust_logits(logits, tokens, q_start, history, history_len, prompt_len, repetition, frequency, presence, bias_ids,
                          bias, mask, mask_row, out, _raw_stream(stream))
    if st:
        _check(st, "dspark_adjust_logits")
    return out


class PagedCache:
    """A paged key-value cache: the tables of ``slots`` requests over ``num_pages`` pages, and
    the pools [layers, num_pages, Hkv, page_size, D] of keys and values.  Methods launch kernels
    only (buffers are made once), so a serving step over it can be captured as a CUDA graph.  A slot
    that ``reserve`` had no room for has granted 0: nothing is written for it, and its queries see
    nothing, until the next ``reserve``."""

    def __init__(self, slots, num_pages, page_size, max_pages, layers, Hkv, D, dtype=torch.bfloat16, device="cuda",
                 k_scale=None, v_scale=None):
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = page_size
        self.page_table = torch.full((slots, max_pages), -1, **i32)
        self.seq_len = torch.zeros(slots, **i32)
        self.ref_count = torch.zeros(num_pages, **i32)
        self.k = torch.zeros((layers, num_pages, Hkv, page_size, D), dtype=dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.k_scale, self.v_scale = k_scale, v_scale
        self.pools = cache_pools([*self.k.unbind(0), *self.v.unbind(0)])
        # (until the first reserve nothing has been refused, and nothing copied)
        self.plan = dict(granted=torch.ones(slots, **i32), copies=torch.full((slots, 2), -1, **i32))
        self.not_refused = torch.ones(slots, **i32)  # by the last reserve
        self.moves = torch.empty(1, **i32)
        self.ws = workspace(cache_workspace_size(slots, num_pages), device)
        self._attention_ws = {}

    def fork(self, src, dst, stream=None):
        cache_fork(self.page_table, self.seq_len, self.ref_count, src, dst, self.page_size, ws=self.ws, stream=stream)

    def reserve(self, n_new, stream=None):
        plan = cache_reserve(self.page_table, self.seq_len, self.ref_count, n_new, self.page_size, self.pools,
                             out=self.plan, ws=self.ws, stream=stream)
        with _made_on(stream):
            torch.le(n_new, plan["granted"], out=self.not_refused)
        return plan

    def write(self, layer, k, v, q_start, stream=None):
        cache_write(k, v, self.k[layer], self.v[layer], self.page_table, self.seq_len, q_start,
                    granted=self.plan["granted"], k_scale=self.k_scale, v_scale=self.v_scale, ws=self.ws,
                    stream=stream)

    def append(self, layer, q, k, v, q_start, rates, interleaved=False, magnitude=1.0, q_out=None, stream=None):
        """``write`` with rotary positions on the way; returns the turned queries (cache_append)."""
        return cache_append(q, k, v, self.k[layer], self.v[layer], self.page_table, self.seq_len, q_start, rates,
                            interleaved=interleaved, magnitude=magnitude, granted=self.plan["granted"],
                            k_scale=self.k_scale, v_scale=self.v_scale, q_out=q_out, ws=self.ws, stream=stream)

    def attend(self, layer, q, q_start, max_q, scale, window=0, out=None, stream=None):
        """Attention of each slot's last tokens over its pages: paged_attention, or chunk_attention for
        more than 128 queries a slot (max_q).  The scratch is made on the first call of a stream and a
        size class (heads and max_q decide it, the number of rows does not) and kept: calls on one
        stream share it in order, calls on two streams never do.  Calls captured on one stream share theirs, and clear its status word:
        replays of graphs that do so must not overlap."""
        T, Hq, D = q.shape
        long = max_q > MAX_BLOCK
        n = (chunk_attention_workspace_size(T, self.seq_len.numel(), Hq, self.k.shape[2], D) if long else
             paged_attention_workspace_size(T, self.seq_len.numel(), Hq, self.k.shape[2], D, max_q))
        with _made_on(stream):
            key = (_raw_stream(None), torch.cuda.is_current_stream_capturing(), n)
            if key not in self._attention_ws:
                self._attention_ws[key] = _attention_workspace(n, q.device)
        if long:
            return chunk_attention(q, self.k[layer], self.v[layer], self.page_table, self.seq_len, q_start, scale,
                                   k_scale=self.k_scale, v_scale=self.v_scale, window=window, out=out,
                                   ws=self._attention_ws[key], stream=stream, granted=self.not_refused)
        return paged_attention(q, self.k[layer], self.v[layer], self.page_table, self.seq_len, q_start, max_q, scale,
                               k_scale=self.k_scale, v_scale=self.v_scale, window=window, out=out,
                               ws=self._attention_ws[key], stream=stream, granted=self.not_refused)

    def truncate(self, new_len, stream=None):
        cache_truncate(self.page_table, self.seq_len, self.ref_count, new_len, self.page_size, ws=self.ws,
                       stream=stream)

    def compact(self, stream=None):
        return cache_compact(self.page_table, self.seq_len, self.ref_count, self.page_size, self.pools,
                             out=self.moves, ws=self.ws, stream=stream)

    def status(self) -> int:
        """The worst device status of the cache's workspaces (0 OK, 1 bad device data, 5 a bounded wait
        gave up)."""
        codes = [device_status(w) for w in (self.ws, *self._attention_ws.values())]
        # (scratch made in a capture holds anything until the graph's first replay clears its status)
        return max(c if c in (1, 5) else 0 for c in codes)
