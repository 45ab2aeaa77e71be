"""Error words and refusals of the operators without a handle, without a GPU."""
import ctypes

import pytest

FAKE = 0x10000  # never dereferenced: the calls fail before any device access


@pytest.fixture(scope="module")
def B():
    from mixture_experts_ffn_gemv_gb300 import binding
    binding.load_library()
    return binding


def test_captured_headers_refuse(B):
    lib = B.load_library()
    assert lib.moe_captured_header(None, None) == 1 and lib.moe_captured_header(FAKE + 64, None) == 1
    assert lib.moe_captured_status(None, None) == 1
