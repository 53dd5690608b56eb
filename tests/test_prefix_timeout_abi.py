"""The self-test of the bounded waits behind a shared prefix without a GPU: its
own refusals, and those of the call that it makes."""
import ctypes

import pytest

import attention_attn_fwd_gb300 as attn
from attention_attn_fwd_gb300 import build as cuda_build
from tests.test_prefix_abi import ALIGN, BF16, INVALID, MB, OK, cache


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return attn.load_library()


def call(lib, c, Q=64 * MB, Hq=4, Sq=1, rows=0, limit=1000,
         block=0):
    return lib.attn_selftest_prefix_timeout(
        ctypes.byref(c), Q, 65 * MB, 66 * MB, Hq, Sq, None, 0.1, 1, BF16,
        128 * MB, 256 * MB, block, rows, limit, None)


def test_refusals(lib):
    for rows in (0, 1):
        assert call(lib, cache(), rows=rows, limit=0) == INVALID
        assert call(lib, cache(), rows=rows, block=-1) == INVALID
        assert call(lib, cache(), rows=rows, Hq=3) == INVALID
        assert call(lib, cache(), rows=rows, Q=64 * MB + 8) == ALIGN
        assert call(lib, cache(B=0), rows=rows) == OK
