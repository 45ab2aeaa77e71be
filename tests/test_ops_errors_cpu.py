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


def test_stall_test_refuses(B):
    lib = B.load_library()
    assert lib.moe_lora_stall_test(3) == 1 and lib.moe_lora_stall_test(-1) == 1 and lib.moe_lora_stall_test(0) == 0
    assert lib.moe_lora_set_wait_limit(0) == 0
