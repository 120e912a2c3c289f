"""Host-side limits of the rotary, append, long-block attention and logit-adjustment calls: what is taken and
refused before anything is launched."""
import decimal
import math

import pytest

from tests.test_serving_abi import INVALID, OK, P, SMALL, UNSUPPORTED, _with


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import build
    build.build()
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _adjust(b, N=0, hist=P[3], hw=50, mask=P[11], mr=4, mask_row=P[12]):
    return b.lib.dspark_adjust_logits(N, 100, 2, 0, P[0], 100, P[1], P[2], hist, hw, hw, P[4], P[5], P[6], P[7], P[8], 3, P[9], P[10],
                                      mask, 4, mr, mask_row, P[13], 100, None)


def test_a_mask_without_rows(b):
    """Rows may name masks where there is none: a tensor of no rows has no address."""
    assert _adjust(b, mask=None, mr=0) == OK
    assert _adjust(b, mask=None, mr=1) == INVALID
    assert _adjust(b, mask=None, mr=0, mask_row=None) == OK and _adjust(b, mr=0) == OK


def test_tokens_alone_are_counted_in_29_bits_too(b):
    """The limit on history_width + N holds without a history: the block's tokens are counted in the same words."""
    for n in (1 << 29, (1 << 31) - 1):
        assert _adjust(b, N=n, hist=None, mask=None, mr=0, mask_row=None) == UNSUPPORTED
        assert "2^29" in b.lib.dspark_last_error_message().decode()
    assert _adjust(b, hist=None, hw=1 << 30, mask=None, mr=0, mask_row=None) == OK  # (a width of no history)


def test_windows_and_rows_of_long_blocks_together(b):
    """Positions before a window are told from queries before a context in 32 bits: T + window is bounded."""
    def call(T, window, max_pages=(1 << 27) - 32, ws=1 << 40, q=P[0]):
        return b.lib.dspark_chunk_attention(T, 4, 1, 1, 64, 64, 16, max_pages, 1, 1, q, 64, 64, P[1], P[2], 1024, 1024, 64, P[3],
                                            max_pages, P[4], P[5], P[6], 0.1, None, None, window, P[9], P[10], P[11], ws, None)

    end = (1 << 31) - 1024
    for T, window in ((300, end - 300), (300, (1 << 31) - 513), (end - 5, 5), (end, 0), ((1 << 31) - 1, 0)):
        assert call(T, window) == UNSUPPORTED, (T, window)
        assert "T + window" in b.lib.dspark_last_error_message().decode()
        assert call(T, window, q=None) == UNSUPPORTED
    for T, window in ((300, end - 301), (end - 6, 5), (300, (1 << 31) - 512), (300, (1 << 31) - 1)):  # (the last two: no window)
        assert call(T, window, q=None) == INVALID and "null pointer: q" in b.lib.dspark_last_error_message().decode(), (T, window)
    assert call(0, end - 1, q=None) == OK


def test_cache_append_any(b):
    """dspark_cache_append's checks, for any even part of a row."""
    def call(T=5, R=4, Hq=4, Hkv=2, D=64, rot=20, il=0, num_pages=64, page_size=16, max_pages=8, dt=1, kv=1, qs=(256, 64),
             ins=(128, 64), os=(256, 64), strides=(2048, 1024, 64), table_stride=8, mag=1.0, ws=256, null=(), shift=None, q_out=None,
             name="dspark_cache_append_any"):
        p = _with(P[:14], set(null) | ({10, 11} if kv != 3 else set()), shift)
        return getattr(b.lib, name)(T, R, Hq, Hkv, D, rot, il, num_pages, page_size, max_pages, dt, kv, p[0], *qs, p[1], p[2], *ins,
                                    q_out or p[3], *os, p[4], p[5], *strides, p[6], table_stride, p[7], p[8], p[9], p[10], p[11], p[12],
                                    mag, p[13], ws, None)

    none = dict(T=0, null=[0, 1, 2, 3])
    for rot in (2, 6, 16, 20, 24, 40, 62, 64):
        assert call(rot=rot, **none) == OK and call(rot=rot, il=1, **none) == OK, rot
        assert call(rot=rot, name="dspark_cache_append", **none) == (UNSUPPORTED if rot % 16 else OK)
    for rot in (0, 1, 3, 63, 66, -2):
        assert call(rot=rot, **none) == INVALID, rot
    assert call(T=-1) == INVALID and call(Hq=-1) == INVALID and call(Hkv=0) == INVALID and call(ws=16) == SMALL
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 12, 13):
        assert call(null=[i]) == INVALID, i
    assert call(kv=3, null=[10]) == INVALID and call(kv=3, null=[11]) == INVALID
    assert call(D=72) == UNSUPPORTED and call(D=272) == UNSUPPORTED
    assert call(il=2) == INVALID and call(mag=math.nan) == INVALID and call(Hq=1 << 21, os=(1 << 27, 64)) == UNSUPPORTED
    for kw in (dict(strides=(0, 1024, 64)), dict(qs=(250, 64)), dict(ins=(128, 60)), dict(os=(256, 4)), dict(os=(56, 64)),
               dict(shift={0: 8}), dict(shift={4: 8}), dict(q_out=P[0], os=(512, 64))):
        assert call(**kw) == INVALID, kw


PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


@pytest.mark.parametrize("base", [10000.0, 500000.0, 3.7])
@pytest.mark.parametrize("how", [dict(), dict(scaling="linear", factor=3.0), dict(factors=[1.0 + i / 7 for i in range(32)])])
def test_rates_to_half_a_unit(b, base, how):
    """Each rate is the whole number nearest to f 2^64 / (2 pi): with f the root of f^64 = base^-2i, which is held
    by its bounds, (rate - 1/2)^64 <= (f 2^64 / 2 pi)^64 <= (rate + 1/2)^64."""
    rates = [r % (1 << 64) for r in b.rotary_rates(64, base, device="cpu", **how).tolist()]
    with decimal.localcontext(decimal.Context(prec=90)):
        for i, r in enumerate(rates):
            shrink = decimal.Decimal(how.get("factor", 1.0)) * decimal.Decimal(how["factors"][i] if "factors" in how else 1.0)
            unit = 2 * PI * shrink / 2 ** 64  # radians, before what divides them
            low, high = ((r + d) * unit for d in (decimal.Decimal("-0.50001"), decimal.Decimal("0.50001")))
            want = 1 / decimal.Decimal(base) ** (2 * i)
            assert low ** 64 <= want <= high ** 64, i


def test_rates_stretched_to_half_a_unit(b):
    """The same for a changed base, f^48 = base^-12i factor^-16i (8 elements), and for blends, by the blend's own
    formula."""
    turns = lambda t: [decimal.Decimal(r % (1 << 64)) for r in t.tolist()]
    half = decimal.Decimal("0.50001")
    with decimal.localcontext(decimal.Context(prec=90)):
        unit = 2 * PI / 2 ** 64
        for i, r in enumerate(turns(b.rotary_rates(8, 10000.0, "ntk", 5.0, device="cpu"))):
            want = 1 / (decimal.Decimal(10000) ** (12 * i) * decimal.Decimal(5) ** (16 * i))
            assert ((r - half) * unit) ** 48 <= want <= ((r + half) * unit) ** 48, i
        f = [decimal.Decimal(10000) ** (decimal.Decimal(-i) / 32) for i in range(32)]
        how = dict(factor=8.0, original_len=4096, low=1.0, high=32.0, device="cpu")
        for i, r in enumerate(turns(b.rotary_rates(64, scaling="bands", **how))):
            kept = min(decimal.Decimal(1), max(decimal.Decimal(0), (4096 * f[i] / (2 * PI) - 1) / 31))
            assert abs(r - f[i] * (kept + (1 - kept) / 8) / unit) <= half, i
        for i, r in enumerate(turns(b.rotary_rates(64, scaling="yarn", **how))):
            # ln(4096 / (64 pi)) / ln(10000) 32 = 10.46 and ln(4096 / 2 pi) / ln(10000) 32 = 22.51: from 10 to 23
            kept = 1 - min(decimal.Decimal(1), max(decimal.Decimal(0), decimal.Decimal(i - 10) / 13))
            assert abs(r - f[i] * (kept + (1 - kept) / 8) / unit) <= half, i


def test_rates_of_any_size(b):
    """Bases and factors to the ends of float64's range: held modulo a turn, or 0, and no error but the binding's."""
    for kw in (dict(base=1e300, factor=1e300, scaling="ntk"), dict(base=1e-300), dict(base=1e300), dict(factor=1e-300, scaling="linear"),
               dict(factor=1e300, scaling="linear"), dict(factors=[1e-300] * 4), dict(base=5e-324, factor=5e-324, scaling="linear")):
        assert b.rotary_rates(8, device="cpu", **kw).numel() == 4, kw
    # f = 1e300^(1/2) at the third of four pairs, modulo a turn, by whole numbers of 10^-100 turns
    got = b.rotary_rates(8, 1e-4, factors=[1.0, 1.0, 1e-60, 1.0], device="cpu")[2].item() % (1 << 64)
    with decimal.localcontext(decimal.Context(prec=140)):
        want = (decimal.Decimal(1e-4) ** decimal.Decimal("-0.5") / decimal.Decimal(1e-60) / (2 * PI)) % 1 * 2 ** 64
        assert abs(want - got) <= 1
    c = decimal.getcontext()
    before = (c.prec, c.rounding)
    b.rotary_rates(64, device="cpu")
    assert (decimal.getcontext().prec, decimal.getcontext().rounding) == before
