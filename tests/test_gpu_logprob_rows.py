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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [3, 400])
def test_likely_ids_after_unlikely_ones(b, dtype, N):
    """The first tokens of a row are J nats less likely than the rest, which are equally likely: the
    sums must be taken about the likely ones, however late they come.

    With s = about V terms of 1, log2 s <= 15 is off by one step of it (2^-20), which is 11 e; the
    difference with the mean, the constant ln 2 (10.4 e/2), and two roundings of values up to 10.4
    (8 e each) make 32 e, and the log probability one more product's 10.4 e."""
    V = 30000
    for J in (3.0, 5.5, 8.0, 10.75):
        x = torch.full((N, V), J - 2.0)
        x[:, :4200] = -2.0
        x = x.to(dtype)
        tokens = np.full(N, V - 7)
        t = torch.as_tensor(tokens, dtype=torch.int32).cuda()
        o = b.token_logprobs(x.cuda(), t)
        lp, H, _, _, _ = ref.token_logprobs(x[:1].double().numpy(), tokens[:1], 1.0, 0)
        assert (o["entropy"].double().cpu() - H[0]).abs().max() <= 32 * E, J
        assert (o["logprob"].double().cpu() - lp[0]).abs().max() <= 43 * E, J


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_entropy_of_confident_rows(b, dtype):
    """It is never negative, and 0 where one id has all the weight."""
    V = 5000
    rng = np.random.default_rng(3)
    x = torch.full((600, V), -math.inf)
    x[:, 0] = torch.as_tensor(rng.uniform(-20, 20, 600))
    at = rng.integers(1, V, 600)
    x[np.arange(600), at] = x[:, 0] + torch.as_tensor(rng.uniform(0, 40, 600)).float()
    x[:40, 0] = -math.inf
    x = x.to(dtype)
    o = b.token_logprobs(x.cuda(), _ids(at))
    H = o["entropy"].cpu()
    assert (H >= 0).all() and (H[:40] == 0).all()
    lp, want, _, _, _ = ref.token_logprobs(x.double().numpy(), at, 1.0, 0)
    # two terms: log2 s and w / s, at most 5 each, carry a handful of roundings of 2^-24 relative
    assert np.abs(H.double().numpy() - want).max() <= 24 * E
    assert np.abs(o["logprob"].cpu().double().numpy() - lp).max() <= 24 * E + 2 * E * np.abs(lp).max()


def _ids(a):
    return torch.as_tensor(a, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shift,T", [(40.0, 1.0), (200.0, 1.0), (-900.0, 1.0), (0.0, 0.03125), (30.0, 0.0625)])
@pytest.mark.parametrize("off", [0, 3])
def test_gradient_of_rows_with_a_large_normaliser(b, dtype, shift, T, off):
    """Logits far from zero, or divided by a small temperature (a power of two, which is exact).
    Relatively, p is off by its sum's and exponent's roundings and, where it comes from a stored
    normaliser, by at most half a step of one below 64 (32 e)."""
    N, V = 12, 1003
    x = (_logits(N, V, torch.float32, 31) + shift).to(dtype)
    wide = torch.zeros((N, V + off), dtype=dtype, device="cuda")
    dev = wide[:, off:]  # (with off, rows lie otherwise on the 16-byte grid than their gradient)
    dev.copy_(x)
    tokens = np.random.default_rng(5).integers(0, V, N)
    gl, ge = (np.random.default_rng(k).standard_normal(N).astype(np.float32) for k in (6, 7))
    t = _ids(tokens)
    o = b.token_logprobs(dev, t, T)
    g = torch.empty((N, V), dtype=dtype, device="cuda")
    b.token_logprobs_backward(dev, t, o["lse"], o["entropy"], torch.from_numpy(gl).cuda(), torch.from_numpy(ge).cuda(), T, out=g)
    x64, gl, ge = x.double().numpy(), gl.astype(np.float64), ge.astype(np.float64)
    want = ref.token_logprobs_grad(x64, tokens, T, gl, ge)
    _, H, lse, _, _ = ref.token_logprobs(x64, tokens, T, 0)
    got = g.cpu().double().numpy()
    for n in range(N):
        lp = x64[n] / T - lse[n]
        p = np.exp(lp)
        parts = (abs(gl[n]) * p + abs(ge[n]) * p * (np.abs(lp) + H[n] + 1)) / T
        tol = E * (V / 256 + 64 + 32 + 4 * np.abs(lp)) * parts + HALF_STEP[dtype] * np.abs(want[n])
        tol = tol + 2.0 ** -25 * (dtype == torch.float16) + 1e-38
        tol[tokens[n]] += 4 * E * abs(gl[n]) / T
        bad = np.abs(got[n] - want[n]) > tol
        assert not bad.any(), (n, np.argmax(bad), got[n][bad][:3], want[n][bad][:3], tol[bad][:3])
    in_place = dev.clone() if off == 0 else dev
    b.token_logprobs_backward(in_place, t, o["lse"], o["entropy"], torch.from_numpy(gl).float().cuda(),
                              torch.from_numpy(ge).float().cuda(), T, out=in_place)
    if off == 0:
        assert torch.equal(in_place, g)
