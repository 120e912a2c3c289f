"""Host-side limits of the rotary, append, long-block attention and logit-adjustment calls: what is taken and
refused before anything is launched."""
import pytest

from tests.test_serving_abi import INVALID, OK, P, UNSUPPORTED


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
