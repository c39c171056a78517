"""Refusals of the 4-bit store's calls that need no GPU."""
import os

import pytest

from prefix_sliding_window_b200 import binding as B
from prefix_sliding_window_b200 import build as BLD


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        BLD.build(quiet=True)
    return B.load()


@pytest.mark.parametrize("scale,code", [(2.0 ** 33, B.PS_ERR_UNSUPPORTED),
                                        (float("inf"), B.PS_ERR_INVALID_ARG),
                                        (-1.0, B.PS_ERR_INVALID_ARG)])
def test_decode_scale_refused(lib, scale, code):
    p = B.make_params(16, 2, 128, 100, 512, softmax_scale=scale)
    cache = B.PsKVCacheQ4(*[256] * 6, 4, None, 0, 0, 0)
    rc = lib.ps_decode_attn_q4(p, cache, 256, 256, 256, None, 256, 1 << 30, None, None)
    assert rc == code and B.last_error() != ""
