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
