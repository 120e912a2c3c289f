"""Rows whose statistics are out of the ordinary, through dspark_token_logprobs and its backward:
temperatures that carry the lowest value past fp32's range, likely tokens that come late in a row,
normalisers far from zero.  The 64-bit form and e = 2^-24 are those of tests/test_gpu_logprobs.py."""
import math

import numpy as np
import pytest
import torch

from tests import serving_ref as ref
from tests.test_gpu_logprobs import E, HALF_STEP, _check, _grad_case, _logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


@pytest.mark.parametrize("T", [0.25, 0.5, 0.9, 2.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_gradient_of_rows_at_the_ends_of_the_range(b, dtype, T):
    """A row full of the type's lowest (or largest) finite value is a uniform distribution whatever
    the temperature; only a row of -inf has nothing left."""
    V = 1201
    x = _logits(5, V, dtype, 12)
    x[0, :] = -math.inf
    x[1, :] = torch.finfo(dtype).min
    x[2, :] = torch.finfo(dtype).max
    x[3, 5:] = torch.finfo(dtype).min
    x[4, :] = torch.finfo(dtype).min
    x[4, 100:] = -math.inf
    tokens = np.array([3, 7, 1200, 2, 99])
    _check(b, x, tokens, T, 4)
    got, gl, ge = _grad_case(b, x, tokens, T, 3)
    g = got.double().numpy()
    want = ref.token_logprobs_grad(x.double().numpy(), tokens, T, gl, ge)
    assert (g[0] == 0).all()
    for n, ids in ((1, V), (2, V), (3, 5), (4, 100)):
        # p is off by the exponent's error, at most e (V/256 + 64 + 4 ln V), relatively; so is the
        # entropy that stands beside ln p; then the rounding to the type
        p = np.where(np.arange(V) < ids, 1.0 if n == 3 else 1.0 / ids, 0.0)
        parts = (abs(gl[n]) * p + abs(ge[n]) * p * 3 * math.log(V)) / T
        tol = E * (V / 256 + 64 + 4 * math.log(V)) * parts * 4 + HALF_STEP[dtype] * np.abs(want[n])
        tol = tol + 2.0 ** -25 * (dtype == torch.float16) + 1e-38
        tol[tokens[n]] += 4 * E * abs(gl[n]) / T
        bad = np.abs(g[n] - want[n]) > tol
        assert not bad.any(), (n, g[n][bad][:3], want[n][bad][:3], tol[bad][:3])
