"""dspark_rotary against a 64-bit form: layouts, parts of a head, types, odd sizes, strides, far and
negative positions, in place, the way back, streams and graphs.

Tolerance.  The angle is off by at most 2^-25 half turns, pi 2^-25 < 2^-23.3 radians; sincospif by an
ulp, 2^-23 at most of values up to 1; the magnitude, two products and their sum by 2^-24 each: together
less than 2^-21 of |magnitude| (|x_u| + |x_w|).  Then half a step of the stored type (subnormal fp16
numbers: half of 2^-24)."""
import numpy as np
import pytest
import torch

from tests import position_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _compare(got, x, pos, rates, **how):
    want, mag = ref.turned(x.double().cpu().numpy(), pos.cpu().numpy(), rates.cpu().numpy(), **how)
    half = torch.finfo(x.dtype).eps / 2
    tol = 2.0 ** -21 * mag + half * np.abs(want) * (mag > 0) + (2.0 ** -25 if x.dtype == torch.float16 else 0.0) * (mag > 0)
    off = np.abs(got.double().cpu().numpy() - want)
    bad = ~(off <= tol)
    assert not bad.any(), (np.argwhere(bad)[0], off[bad][0], tol[bad][0], int(bad.sum()))


def _case(T, H, D, dtype, far=200000, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, H, D), generator=g).to(dtype).cuda(), torch.randint(-far, far, (T,), generator=g).int().cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 2, 2), (1, 40, 128, 128), (7, 3, 64, 32), (5, 2, 80, 20), (3, 5, 33, 6),
                                       (700, 2, 96, 96), (3000, 1, 256, 128), (2, 1, 1024, 1024), (33, 9, 72, 72),
                                       (1, 2, 40, 8)])
def test_layouts(b, dtype, interleaved, T, H, D, rot):
    x, pos = _case(T, H, D, dtype, seed=D + rot)
    rates = b.rotary_rates(rot)
    y = b.rotary(x, pos, rates, interleaved=interleaved)
    assert torch.equal(y[..., rot:], x[..., rot:])
    _compare(y, x, pos, rates, interleaved=interleaved)
    back = b.rotary(x, pos, rates, interleaved=interleaved, inverse=True, magnitude=1.25)
    _compare(back, x, pos, rates, interleaved=interleaved, inverse=True, magnitude=1.25)
    here = x.clone()
    assert b.rotary(here, pos, rates, interleaved=interleaved, out=here) is here
    assert torch.equal(here, y)


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_over_the_whole_range(b, interleaved):
    """The angle stays exact: what one wrapping product gives, at the ends of 32 bits too."""
    x, _ = _case(9, 2, 64, torch.float32)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 20, (1 << 24) + 1, 123456789, -987654321], dtype=torch.int32).cuda()
    for how in (dict(), dict(scaling="linear", factor=4.0), dict(scaling="yarn", factor=8.0, original_len=4096)):
        rates = b.rotary_rates(64, 10000.0, **how)
        _compare(b.rotary(x, pos, rates, interleaved=interleaved), x, pos, rates, interleaved=interleaved)
    assert torch.equal(b.rotary(x, pos, rates)[0], x[0])  # position 0 turns nothing


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides(b, dtype, interleaved):
    """Queries inside a packed projection, rows off the 16-byte grid, a result with strides of its own,
    one row read for every head."""
    packed, pos = _case(50, 12, 64, dtype)
    rates = b.rotary_rates(48)
    how = dict(interleaved=interleaved)
    x = packed[:, 2:7]
    _compare(b.rotary(x, pos, rates, **how), x, pos, rates, **how)
    flat = packed.flatten()[1:1 + 49 * 9 * 70].view(49, 9, 70)[..., 3:67]
    _compare(b.rotary(flat, pos[:49], rates, **how), flat, pos[:49], rates, **how)
    out = torch.full((50, 5, 96), 7.0, dtype=dtype, device="cuda")
    b.rotary(x, pos, rates, out=out[..., 16:80], **how)
    _compare(out[..., 16:80], x, pos, rates, **how)
    assert (out[..., :16] == 7).all() and (out[..., 80:] == 7).all()
    heads_first = torch.empty((5, 50, 64), dtype=dtype, device="cuda").transpose(0, 1)
    assert torch.equal(b.rotary(x, pos, rates, out=heads_first, **how), b.rotary(x, pos, rates, **how))
    one = packed[:, :1].expand(50, 6, 64)
    _compare(b.rotary(one, pos, rates, **how), one, pos, rates, **how)
    part = packed[:, 2:7, 16:48]  # a part of the head that does not start it
    rates = b.rotary_rates(32)
    _compare(b.rotary(part, pos, rates, **how), part, pos, rates, **how)


def test_the_way_back_is_the_gradient(b):
    """<g, R x> = <R^T g, x>, and differences of <g, R x>."""
    for interleaved in (False, True):
        x, pos = _case(20, 3, 32, torch.float32, seed=3)
        gy, _ = _case(20, 3, 32, torch.float32, seed=4)
        rates = b.rotary_rates(24, scaling="ntk", factor=2.0)
        how = dict(interleaved=interleaved, magnitude=1.3)
        gx = b.rotary(gy, pos, rates, inverse=True, **how).double()
        f = lambda z: (gy.double() * torch.as_tensor(ref.turned(z.cpu().numpy(), pos.cpu().numpy(), rates.cpu().numpy(),
                                                                **how)[0]).cuda()).sum().item()
        for k in (0, 5, 23, 24, 31):
            e = torch.zeros_like(x, dtype=torch.float64)
            e[7, 1, k] = 0.5
            slope = f(x.double() + e) - f(x.double() - e)
            assert abs(slope - gx[7, 1, k].item()) < 1e-5


def test_empty_nan_and_reuse(b):
    x, pos = _case(8, 2, 64, torch.bfloat16)
    rates = b.rotary_rates(64)
    assert b.rotary(x[:0], pos[:0], rates).shape == (0, 2, 64)
    x[3, 1, 5] = float("nan")
    y = b.rotary(x, pos, rates)
    gone = torch.isnan(y)
    assert gone[3, 1, 5] and gone[3, 1, 37] and int(gone.sum()) == 2  # its pair, nothing else


def test_streams_and_graphs(b):
    x, pos = _case(64, 8, 128, torch.bfloat16)
    rates = b.rotary_rates(128)
    want = b.rotary(x, pos, rates)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.rotary(x, pos, rates, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.rotary(x, pos, rates, out=out)
    pos += 3
    g.replay()
    assert torch.equal(out, b.rotary(x, pos, rates))
