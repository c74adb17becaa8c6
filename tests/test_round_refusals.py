"""Refusals of the gdn_round.h calls on the host, with pointers that are never followed."""

import ctypes
import os

import pytest

from gated_deltanet_speculative_amd import _lib, _round

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="library not built")


def _p(k):
    return 0x7F0000000000 + k * (1 << 34)


@pytest.mark.parametrize("scale", [2.5e38, 3.4e38, 0.0, -0.0])
def test_attention_refuses_a_scale_that_leaves_no_score(scale):
    """The scale times log2(e) is what the kernels multiply by: 2.5e38 is finite, the product is not."""
    sh = _round._CAttnShape(2, 4, 4, 4, 2, 64, 16, 20, 8, 1)
    code = _round._library().gdn_paged_attention(ctypes.byref(sh), *[_p(i) for i in range(6)], None, None, scale, None, 0, _p(9),
                                                 _p(12), 1 << 30, _p(10), None)
    assert code == _lib.GDN_ERR_SHAPE
