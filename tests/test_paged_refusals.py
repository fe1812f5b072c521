"""More of what the paged cache operators and their helpers refuse on the
host, before anything reaches a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def N():
    from speculative_decoding_verification_25_gb300 import build as b
    b.build()
    from speculative_decoding_verification_25_gb300 import _native
    _native.load()
    return _native


def test_capture_id_needs_a_place_for_it(N):
    assert N.load().spec_stream_capture_id(None, ctypes.POINTER(ctypes.c_uint64)()) == N.SV_ERR_NULL
