"""The weights', eviction's and shared plans' entry points on the CPU: NULL handles."""
import ctypes

import pytest

from int2_rotated_kv_rotate_gb300 import _native as N
from int2_rotated_kv_rotate_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.lib()


def test_null_handles_are_rejected(lib):
    one = (ctypes.c_int * 1)(0)
    assert lib.oscar_weights_stride(None) == 0
    assert lib.oscar_decode_weights_workspace_bytes(None) == 0
    assert lib.oscar_decode_weights_workspace_max_bytes(None) == 0
    assert lib.oscar_bf16_decode_weights(None, 0, 16, 16, 16, 16, 256, 1 << 20, None, None) == 1
    assert lib.oscar_evict_begin(None, one, one, 1, 0, 0, None) == 1
    assert lib.oscar_evict(None, 0, 16, 32, 48, None) == 1
    assert lib.oscar_evict_pages(None, 0, one, 1, None) == 1
    assert lib.oscar_evict_commit(None, None) == 1
    assert lib.oscar_evict_cancel(None) == 1
    assert lib.oscar_plan_shared_info(None, None, None) == 1
    assert lib.oscar_last_error()

