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
