"""The paged calls refuse per-row lists that are not aligned to their type
(a kernel's load of one would fault), before anything is launched."""
import ctypes as C

import pytest

import kv_cache_compression_layer_b200 as kv
from kv_cache_compression_layer_b200 import build as kvbuild


@pytest.fixture(scope="module")
def L():
    kvbuild.build()
    return kv.lib()


@pytest.mark.parametrize("name,bad", [("count", 258), ("src_off", 260), ("idx", 257), ("idx_off", 260)])
def test_append_and_compact_refuse_misaligned_lists(L, name, bad):
    sh = kv.make_paged_shape(4, 3, 2, 8, 128, kv.KV_BF16, 100, 10)
    c = kv.make_paged_cache(256, 256, 256, 256, 256, 256, 256, 1 << 40)
    a = dict(count=256, src_off=256, idx=256, idx_off=256)
    a[name] = bad
    one, two = (C.c_int32 * 1)(0), (C.c_int32 * 1)(1)
    assert L.kv_paged_append(C.byref(sh), C.byref(c), one, 1, 0, 3, 256, 256, 6, 1, a["count"], a["src_off"], a["idx"],
                             a["idx_off"], None) == kv.KV_ERR_ARG
    if name != "src_off":
        assert L.kv_paged_compact(C.byref(sh), C.byref(c), one, two, 1, a["idx"], a["idx_off"], a["count"],
                                  None) == kv.KV_ERR_ARG
