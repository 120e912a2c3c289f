"""dspark_token_logprobs and its backward against a 64-bit form: types, odd sizes and strides,
vocabulary masks (rows of which nothing is left, masks of the type's lowest value), NaN and
infinities, ties, skipped rows, offsets past 32 bits, streams and graphs.

Tolerances, with e = 2^-24 (half a step of fp32): a log probability is u - ln s, where u carries
three roundings relative to itself and s at most V/256 + 32 (a thread's sequential sums, the
exponential and the joins), so |error| <= e (V/256 + 32 + 4 |u| + 4 ln s); the normaliser adds
e |lse|; the entropy's two terms carry the same relative errors.  A gradient element
multiplies p, whose relative error is that of its exponent, and is rounded once to its type
(half a step: 2^-8 bf16, 2^-11 fp16, 2^-24 fp32)."""
import math

import numpy as np
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _logits(N, V, dtype, seed, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((N, V), generator=g) * sigma).to(dtype)


def _check(b, x, tokens, T, K, stream=None, dev=None):
    """Runs the kernel on `dev` (default: x on the GPU) and compares."""
    V = x.shape[1]
    d = x.cuda() if dev is None else dev
    t = torch.as_tensor(tokens, dtype=torch.int32).cuda()
    o = b.token_logprobs(d, t, T, K, stream=stream)
    torch.cuda.synchronize()
    x64 = x.double().numpy()
    lp, H, lse, ids, top = ref.token_logprobs(x64, tokens, T, K)
    with np.errstate(over="ignore"):  # results past fp32's range are infinite
        lp, lse, top = (np.where(np.isinf(a.astype(np.float32)), a.astype(np.float32), a) for a in (lp, lse, top))
    got = {k: v.cpu().double().numpy() for k, v in o.items()}
    sums = V / 256 + 32
    for n in range(len(tokens)):
        for name, want in (("logprob", lp[n]), ("entropy", H[n]), ("lse", lse[n])):
            g = got[name][n]
            if not np.isfinite(want):
                assert (np.isnan(want) and np.isnan(g)) or g == want, (n, name, g, want)
                continue
            ln_s = math.log(V)
            u = abs(want) + ln_s
            tol = E * (sums + 4 * u + 4 * ln_s)
            if name == "entropy":
                tol = E * (sums + 8) * (1 + 2 * ln_s)
            assert abs(g - want) <= tol, (n, name, g, want, tol)
        for i in range(K):
            assert got["top_ids"][n, i] == ids[n, i], (n, i)
            w, g = top[n, i], got["top_logprobs"][n, i]
            if not np.isfinite(w):
                assert (np.isnan(w) and np.isnan(g)) or g == w, (n, i, g, w)
            else:
                assert abs(g - w) <= E * (sums + 4 * abs(w) + 8 * math.log(V) + 4 * math.log(V)), (n, i, g, w)
    return o


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 2), (2, 31, 5), (5, 255, 0), (4, 1000, 32), (7, 4099, 20),
                                   (2, 50257, 20), (40, 8200, 3), (3, 151936, 20)])
def test_matches_64_bits(b, dtype, N, V, K):
    x = _logits(N, V, dtype, 1 + N * V)
    tokens = np.random.default_rng(N + V).integers(0, V, N)
    tokens[0] = V - 1
    _check(b, x, tokens, 0.7, K)


def test_many_rows_and_few(b):
    for N in (1, 2, 17, 150, 400):
        x = _logits(N, 3001, torch.bfloat16, N)
        _check(b, x, np.arange(N) % 3001, 1.0, 4)


@pytest.mark.parametrize("dtype,N,V,K", [(torch.bfloat16, 2500, 1500, 5), (torch.float32, 900, 20011, 20),
                                         (torch.float16, 700, 40, 0), (torch.float32, 1300, 1, 1),
                                         (torch.bfloat16, 333, 70001, 32)])
def test_many_rows_in_turn(b, dtype, N, V, K):
    x = _logits(N, V, dtype, N)
    rng = np.random.default_rng(N)
    tokens = rng.integers(0, V, N)
    tokens[rng.random(N) < 0.3] = -1
    tokens[N // 3: N // 3 + 50] = V  # skipped in a run
    x[5, : V // 2] = -math.inf
    x[N - 1, :] = -math.inf
    _check(b, x, tokens, 0.9, K)
    _check(b, x, np.where(np.arange(N) == N - 2, 0, -1), 0.9, K)  # one row is left
    _check(b, x, np.full(N, -1), 0.9, K)


@pytest.mark.parametrize("N", [3, 400])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_best_ids_gathered(b, dtype, N):
    """Sorted rows, and the best in one place: more candidates pass the first threshold than fit."""
    V = 12345
    x = torch.linspace(-20, 20, V, dtype=torch.float64).expand(N, V).clone()
    x[1] = x[1].flip(0)
    x[2, 6000:6700] += 30
    x = x.to(dtype)
    tokens = np.arange(N) % V
    _check(b, x, tokens, 1.0, 32)
    _check(b, x, tokens, 1.0, 1)


def test_skipped_rows_are_not_read(b):
    x = _logits(6, 777, torch.float32, 3)
    x[1] = math.nan
    tokens = np.array([5, -1, 777, 776, -7, 0])
    o = _check(b, x, tokens, 1.0, 3)
    assert torch.isnan(o["logprob"][[1, 2, 4]]).all() and (o["top_ids"][[1, 2, 4]] == -1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_masks(b, dtype):
    V = 5003
    x = _logits(8, V, dtype, 4)
    x[0, :] = -math.inf                      # nothing is left
    x[1, 1:] = -math.inf                     # one id is left
    x[2, : V - 1] = -math.inf
    x[3, ::2] = -math.inf
    x[4, ::3] = torch.finfo(dtype).min       # masks of the lowest value
    x[5, :] = torch.finfo(dtype).min         # ... in the whole row: a uniform distribution
    x[6, 1:] = torch.finfo(dtype).min
    x[7, :] = torch.finfo(dtype).max
    _check(b, x, np.array([7, 0, V - 1, 1, 3, 9, 0, 4]), 1.0, 6)
    _check(b, x, np.array([7, 1, 0, 0, 1, 0, 5, 0]), 0.9, 32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nan_and_infinity(b, dtype):
    x = _logits(5, 600, dtype, 5)
    x[1, 599] = math.nan
    x[2, 0] = math.inf
    x[3, 5] = math.inf
    x[3, 6] = math.inf
    x[4, 77] = math.nan
    x[4, :70] = -math.inf
    _check(b, x, np.array([1, 1, 0, 5, 77]), 1.0, 4)


def test_ties_go_to_the_lowest_id(b):
    for V in (64, 700, 9001):
        x = torch.zeros((3, V))
        x[1] = torch.tensor(np.random.default_rng(V).integers(0, 3, V), dtype=torch.float32)
        x[2, ::5] = -0.0
        _check(b, x, np.array([0, V - 1, 5]), 1.0, 32)
        _check(b, x.bfloat16(), np.array([0, V - 1, 5]), 1.0, 7)


@pytest.mark.parametrize("T", [1e-3, 0.3, 50.0])
def test_temperatures(b, T):
    x = _logits(3, 2000, torch.float32, 6)
    _check(b, x, x.argmax(1).numpy(), T, 5)


@pytest.mark.parametrize("dtype,off", [(torch.float32, 1), (torch.bfloat16, 3), (torch.float16, 7)])
def test_strides_and_alignment(b, dtype, off):
    wide = _logits(5, 2111, dtype, 7)
    dev = wide.cuda()[:, off:off + 1997]
    _check(b, wide[:, off:off + 1997], np.array([0, 5, 1996, 9, 100]), 1.0, 8, dev=dev)
    dev = wide.cuda()[::2, off:off + 40]
    _check(b, wide[::2, off:off + 40], np.array([0, 5, 39]), 1.0, 8, dev=dev)


def test_offsets_past_32_bits(b):
    V, stride = 3001, 1_200_000_001  # bf16 rows 2.4 GB apart
    big = torch.empty(3 * stride, dtype=torch.bfloat16, device="cuda")
    dev = big.as_strided((3, V), (stride, 1))
    x = _logits(3, V, torch.bfloat16, 8)
    dev.copy_(x)
    tokens = np.array([1, 2, 3])
    o = _check(b, x, tokens, 1.0, 5, dev=dev)
    t = torch.as_tensor(tokens, dtype=torch.int32).cuda()
    one = torch.ones(3, device="cuda")
    want = b.token_logprobs_backward(x.cuda(), t, o["lse"], o["entropy"], one)
    b.token_logprobs_backward(dev, t, o["lse"], o["entropy"], one, out=dev)  # in place
    assert torch.equal(dev, want)


def test_deterministic_streams_and_graph(b):
    x = _logits(33, 20011, torch.bfloat16, 9).cuda()
    t = torch.arange(33, dtype=torch.int32, device="cuda")
    first = {k: v.clone() for k, v in b.token_logprobs(x, t, 1.0, 9).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = {k: torch.zeros_like(v) for k, v in first.items()}
    side.wait_stream(torch.cuda.current_stream())
    b.token_logprobs(x, t, 1.0, 9, out=out, stream=side)
    side.synchronize()
    assert all(torch.equal(out[k], first[k]) for k in first)
    grad = torch.zeros_like(x)
    gl = torch.randn(33, device="cuda")
    want = b.token_logprobs_backward(x, t, first["lse"], first["entropy"], gl, gl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.token_logprobs(x, t, 1.0, 9, out=out)
        b.token_logprobs_backward(x, t, out["lse"], out["entropy"], gl, gl, out=grad)
    for o in out.values():
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], first[k]) for k in first)
    assert torch.equal(grad, want)


def _grad_case(b, x, tokens, T, seed, entropy=True):
    N, V = x.shape
    rng = np.random.default_rng(seed)
    gl = rng.standard_normal(N).astype(np.float32)
    ge = rng.standard_normal(N).astype(np.float32) if entropy else np.zeros(N, np.float32)
    t = torch.as_tensor(tokens, dtype=torch.int32).cuda()
    d = x.cuda()
    o = b.token_logprobs(d, t, T)
    got = b.token_logprobs_backward(d, t, o["lse"], o["entropy"], torch.from_numpy(gl).cuda(),
                                    torch.from_numpy(ge).cuda() if entropy else None, T).cpu()
    return got, gl.astype(np.float64), ge.astype(np.float64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,V,T", [(1, 1, 1.0), (3, 30, 0.8), (4, 1003, 1.3), (2, 50257, 1.0), (5, 151936, 1.0)])
def test_gradient_matches_formula(b, dtype, N, V, T):
    x = _logits(N, V, dtype, 11 + V)
    if V > 8:
        x[0, 3:7] = -math.inf
    tokens = np.random.default_rng(V).integers(0, V, N)
    if N > 2:
        tokens[1] = -1
    for entropy in (True, False):
        got, gl, ge = _grad_case(b, x, tokens, T, V, entropy)
        x64 = x.double().numpy()
        want = ref.token_logprobs_grad(x64, tokens, T, gl, ge)
        _, H, lse, _, _ = ref.token_logprobs(x64, tokens, T, 0)
        g = got.double().numpy()
        for n in range(N):
            if tokens[n] < 0:
                assert (g[n] == 0).all()
                continue
            lp = np.where(x64[n] == -np.inf, -1e4, x64[n] / T - lse[n])
            p = np.exp(lp)
            parts = (abs(gl[n]) * p + abs(ge[n]) * p * (abs(lp) + H[n] + 1)) / T
            rel = E * (V / 256 + 64 + 6 * abs(lse[n]) + 4 * np.abs(lp))
            tol = rel * parts + HALF_STEP[dtype] * np.abs(want[n]) + 2.0 ** -25 * (dtype == torch.float16) + 1e-38
            tol[tokens[n]] += 4 * E * abs(gl[n]) / T
            bad = np.abs(g[n] - want[n]) > tol
            assert not bad.any(), (n, np.argmax(bad), g[n][bad][:3], want[n][bad][:3])


def test_gradient_matches_differences(b):
    # central differences of the 64-bit objective: truncation h^2/6 times the third derivative
    # (at most about 3 in these units), the kernel's own error as above
    x = _logits(2, 40, torch.float32, 21, 1.5)
    tokens = np.array([4, 39])
    T, h = 0.9, 1e-4
    got, gl, ge = _grad_case(b, x, tokens, T, 5)
    x64 = x.double().numpy()

    def objective(z):
        lp, H, _, _, _ = ref.token_logprobs(z, tokens, T, 0)
        return (gl * lp + ge * H).sum()

    for n in range(2):
        for v in range(40):
            up, dn = x64.copy(), x64.copy()
            up[n, v] += h
            dn[n, v] -= h
            d = (objective(up) - objective(dn)) / (2 * h)
            assert abs(got[n, v].item() - d) <= 1e-7 + 2e-6 * (abs(gl[n]) + abs(ge[n])), (n, v)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_gradient_of_masked_rows(b, dtype):
    V = 1201
    x = _logits(4, V, dtype, 12)
    x[0, :] = -math.inf
    x[1, :] = torch.finfo(dtype).min  # uniform
    x[2, 5:] = torch.finfo(dtype).min
    x[3, 10] = math.nan
    tokens = np.array([3, 7, 2, 1])
    got, gl, ge = _grad_case(b, x, tokens, 1.0, 3)
    g = got.double().numpy()
    want = ref.token_logprobs_grad(x.double().numpy(), tokens, 1.0, gl, ge)
    assert (g[0] == 0).all() and np.isnan(g[3]).all()
    # p = 1/V; ln p + H = 0 up to the entropy's error, e (V/256 + 40) (1 + 2 ln V)
    tol = HALF_STEP[dtype] * np.abs(want[1]) + (abs(gl[1]) + 20 * abs(ge[1])) * E * 1000 / V + 2.0 ** -25
    assert (np.abs(g[1] - want[1]) <= tol).all()
    tol = HALF_STEP[dtype] * np.abs(want[2]) + (abs(gl[2]) + 20 * abs(ge[2])) * E * 400 + 2.0 ** -25
    assert (np.abs(g[2] - want[2]) <= tol).all()


def test_empty_batch(b):
    x = torch.zeros((0, 50), device="cuda")
    t = torch.zeros(0, dtype=torch.int32, device="cuda")
    o = b.token_logprobs(x, t, 1.0, 2)
    assert o["logprob"].numel() == 0 and o["top_ids"].shape == (0, 2)
    f = torch.zeros(0, device="cuda")
    assert b.token_logprobs_backward(x, t, f, f, f).shape == (0, 50)
