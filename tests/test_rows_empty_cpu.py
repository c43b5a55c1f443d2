"""kv_read of no positions and attn_extend of no tokens do nothing, also where
the caller's tensors are empty and so have no address.  Nothing is launched."""
import ctypes

from int2_kv_cache_append_gb300 import oscar_kv as K

CFG = K.KVConfig(1, 2, 8, 2, 128, 4, 8, 64)
BIG = ctypes.c_void_p(1 << 20)


def _extend(n, q=None, out=None, ws=None, b=0, layer=0):
    return K.lib().attn_extend(ctypes.byref(CFG.c()), BIG, layer, q, n, None, BIG, 0, BIG, BIG, 0.0, 0, out, None, ws, b, None, None)


def _read(n, k=None, v=None, layer=0):
    return K.lib().kv_read(ctypes.byref(CFG.c()), BIG, layer, BIG, BIG, n, BIG, BIG, k, v, None, None)


def test_no_tokens():
    assert K.attn_extend_workspace_bytes(CFG, 0) == 0
    assert _extend(0) == 0
    assert _extend(0, layer=1) == -1 and _extend(-1) == -1
    assert [_extend(1), _extend(1, q=BIG, out=BIG), _extend(1, q=BIG, ws=BIG), _extend(1, out=BIG, ws=BIG)] == [-1] * 4


def test_no_positions():
    assert _read(0) == 0
    assert _read(0, layer=1) == -1 and _read(-1) == -1 and _read(1) == -1
