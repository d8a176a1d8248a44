"""The rotated append's, the window's and the 4-bit cache's entry points on the CPU: NULL handles,
configurations."""
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
    rows = ctypes.addressof(keep := N.oscar_rows(16, 128, 128))
    assert ctypes.sizeof(N.oscar_rows) == 24 and ctypes.sizeof(N.oscar_rope_tensor) == 56 and keep.row == 128
    assert len(N._pack_rows(1, 2, 3)) == 24 and bytes(N.oscar_rope_tensor(1, 2, 3, 4, 5, 6, 7)) == N._pack_rope_tensor(1, 2, 3, 4, 5, 6, 7)
    assert lib.oscar_append_rotated(None, 0, 16, 128, 1.0, 0, None, None, rows, rows, None) == 1
    assert lib.oscar_int4_append(None, 0, 16, 16, None) == 1
    assert lib.oscar_int4_read(None, 0, 0, 0, 1, 16, 16, N.OSCAR_DTYPE_BF16, None) == 1
    assert lib.oscar_int4_decode_attention(None, 0, 16, 16, 256, 1 << 20, None, None) == 1
    assert lib.oscar_plan_window(None, one, one, 1, 0, 0, None) == 1
    assert lib.oscar_plan_window_info(None, one, one, one) == 1
    assert lib.oscar_window_workspace_bytes(None) == 0
    assert lib.oscar_window_workspace_max_bytes(None) == 0
    assert lib.oscar_window_attention(None, 0, 16, 16, 256, 1 << 20, None, None) == 1
    assert lib.oscar_last_error()


def test_device_bytes_of_the_4_bit_format(lib):
    def need(group, **kw):
        base = dict(format=N.OSCAR_FORMAT_INT4, head_dim=128, n_q_heads=32, n_kv_heads=8, group=group, page=64, n_sink=0, window=0,
                    n_layers=2, max_requests=4, max_pages=100, max_pages_per_request=50)
        base.update(kw)
        c = N.oscar_config(*[base[f] for f, _ in N.oscar_config._fields_])
        return lib.oscar_cache_device_bytes(ctypes.byref(c))

    heads = 2 * 100 * 8
    assert need(32) - need(128) == heads * 64 * 2 * (16 - 4)
    assert need(128) >= heads * 64 * 2 * (64 + 4)
    for bad in (dict(group=64), dict(group=0), dict(head_dim=64), dict(n_q_heads=24), dict(page=32), dict(format=3), dict(format=5)):
        kw = dict(group=32)
        kw.update(bad)
        assert need(kw.pop("group"), **kw) == 0, bad
