"""attn_extend and attn_decode_prefix refuse capacities whose last positions their
32-bit position arithmetic would pass.  Nothing is launched."""
import ctypes

import pytest

from int2_kv_cache_append_gb300 import oscar_kv as K

MOST = 2 ** 31 - 1 - 1024


def cfg(cap, batch=1):
    return K.KVConfig(1, batch, 8, 1, 128, 4, 8, cap)


def test_extend():
    assert K.attn_extend_workspace_bytes(cfg(MOST), 1) > 0
    big, n = ctypes.c_void_p(1 << 20), ctypes.c_uint64()
    for cap in (MOST + 1, 2 ** 31 - 1):
        with pytest.raises(K.OscarError) as e:
            K.attn_extend_workspace_bytes(cfg(cap), 1)
        assert e.value.code == -5
        rc = K.lib().attn_extend(ctypes.byref(cfg(cap).c()), big, 0, big, 1, None, big, 0, big, big, 0.0, 0, big, None, big, 1 << 40,
                                 None, None)
        assert rc == -5


@pytest.mark.parametrize("own,prefix,ok", [(MOST, MOST, True), (MOST + 1, 100, False), (100, MOST + 1, False)])
def test_prefix(own, prefix, ok):
    if ok:
        assert K.attn_decode_prefix_workspace_bytes(cfg(own, 3), cfg(prefix)) > 0
        return
    with pytest.raises(K.OscarError) as e:
        K.attn_decode_prefix_workspace_bytes(cfg(own, 3), cfg(prefix))
    assert e.value.code == -5
