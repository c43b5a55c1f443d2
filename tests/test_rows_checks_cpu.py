"""kv_read, attn_extend and attn_decode_prefix refuse bad calls on the host,
before anything reaches the GPU: the binding by tensor type, shape and device,
the library by pointer, range, configuration and workspace size."""
import ctypes

import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K

CFG = K.KVConfig(1, 2, 8, 2, 128, 4, 8, 64)
PRE = K.KVConfig(1, 1, 8, 2, 128, 16, 8, 300)
BF, I32 = torch.bfloat16, torch.int32


def _bytes(cfg):
    return torch.zeros(K.layout_query(cfg)["total_bytes"], dtype=torch.uint8)


def _read(**over):
    args = dict(cfg=CFG, cache=_bytes(CFG), layer=0, start_pos=torch.zeros(2, dtype=I32), seq_lens=torch.zeros(2, dtype=I32),
                R_K=torch.zeros(128, 128), R_V=torch.zeros(128, 128), k_out=torch.zeros(2, 3, 2, 128, dtype=BF),
                v_out=torch.zeros(2, 3, 2, 128, dtype=BF))
    args.update(over)
    return K.kv_read(**args)


def _extend(**over):
    args = dict(cfg=CFG, cache=_bytes(CFG), layer=0, q=torch.zeros(2, 3, 8, 128, dtype=BF),
                seq_lens=torch.zeros(2, dtype=I32), R_K=torch.zeros(128, 128), R_V=torch.zeros(128, 128),
                out=torch.zeros(2, 3, 8, 128, dtype=BF), workspace=torch.zeros(256, dtype=torch.uint8),
                lse=torch.zeros(2, 3, 8), q_lens=torch.zeros(2, dtype=I32))
    args.update(over)
    return K.attn_extend(**args)


def _prefix(**over):
    args = dict(cfg=CFG, cache=_bytes(CFG), prefix_cfg=PRE, prefix_cache=_bytes(PRE), layer=0,
                q=torch.zeros(2, 8, 128, dtype=BF), seq_lens=torch.zeros(2, dtype=I32), prefix_len=torch.zeros(1, dtype=I32),
                R_K=torch.zeros(128, 128), R_V=torch.zeros(128, 128), out=torch.zeros(2, 8, 128, dtype=BF),
                workspace=torch.zeros(256, dtype=torch.uint8), lse=torch.zeros(2, 8))
    args.update(over)
    return K.attn_decode_prefix(**args)


@pytest.mark.parametrize("call", [_read, _extend, _prefix])
def test_valid_arguments_reach_the_device_check(call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        call()


@pytest.mark.parametrize("over", [
    dict(k_out=None, v_out=None),
    dict(k_out=torch.zeros(2, 3, 2, 128)),                       # fp32 without OSCAR_FLAG_OUT_FP32
    dict(v_out=torch.zeros(2, 4, 2, 128, dtype=BF)),             # K and V disagree on n
    dict(k_out=torch.zeros(2, 3, 128, dtype=BF)),
    dict(start_pos=torch.zeros(2, dtype=torch.int64)),
    dict(seq_lens=torch.zeros(1, dtype=I32)),
    dict(cache=torch.zeros(100, dtype=torch.uint8)),
    dict(R_V=torch.zeros(64, 64)),
    dict(status=torch.zeros(1)),
])
def test_read_refuses_mismatched_tensors(over):
    with pytest.raises(ValueError, match="oscar_kv"):
        _read(**over)


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(2, 3, 8, 128)),                           # fp32 q without OSCAR_FLAG_IN_FP32
    dict(q=torch.zeros(2, 8, 128, dtype=BF)),
    dict(q=torch.zeros(2, 3, 4, 128, dtype=BF)),
    dict(out=torch.zeros(2, 4, 8, 128, dtype=BF)),
    dict(out=torch.zeros(2, 3, 8, 128)),
    dict(lse=torch.zeros(2, 8, 3)),
    dict(q_lens=torch.zeros(3, dtype=I32)),
    dict(seq_lens=torch.zeros(2)),
    dict(workspace=torch.zeros(256)),
    dict(cache=torch.zeros(100, dtype=torch.uint8)),
    dict(R_K=None),
])
def test_extend_refuses_mismatched_tensors(over):
    with pytest.raises(ValueError, match="oscar_kv"):
        _extend(**over)


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(2, 1, 8, 128, dtype=BF)),
    dict(prefix_len=torch.zeros(2, dtype=I32)),
    dict(prefix_len=torch.zeros(1, dtype=torch.int64)),
    dict(prefix_cache=torch.zeros(100, dtype=torch.uint8)),
    dict(out=torch.zeros(2, 8, 128)),
    dict(lse=torch.zeros(2, 4)),
    dict(workspace=torch.zeros(256)),
])
def test_prefix_refuses_mismatched_tensors(over):
    with pytest.raises(ValueError, match="oscar_kv"):
        _prefix(**over)


@pytest.mark.parametrize("over", [
    dict(batch=2), dict(num_kv_heads=4), dict(num_q_heads=16), dict(head_dim=256), dict(flags=K.FLAG_LLOYD_MAX)])
def test_prefix_cache_has_the_shape_of_the_own(over):
    pre = K.KVConfig(**{**PRE.__dict__, **over})
    with pytest.raises(K.OscarError) as e:
        K.attn_decode_prefix_workspace_bytes(CFG, pre)
    assert e.value.code == -1
    assert K.attn_decode_prefix_workspace_bytes(CFG, PRE) > 0


def _a(x):
    return (x + 255) // 256 * 256


def test_library_checks():
    """Pointers here are never dereferenced: every call stops in the checks."""
    L, P = K.lib(), ctypes.c_void_p
    c, pc, big, odd = CFG.c(), PRE.c(), P(1 << 20), P((1 << 20) + 8)
    r = ctypes.byref

    def read(cache=big, layer=0, start=big, lens=big, n=3, rk=big, rv=big, k=big, v=big, cfg=c):
        return L.kv_read(r(cfg), cache, layer, start, lens, n, rk, rv, k, v, None, None)

    assert [read(cache=None), read(start=None), read(lens=None), read(rk=None), read(k=None, v=None)] == [-1] * 5
    assert [read(layer=1), read(layer=-1), read(n=-1), read(k=odd), read(v=odd), read(cache=odd)] == [-1] * 6
    assert read(n=0) == 0
    assert read(cfg=K.KVConfig(1, 2, 8, 2, 96, 4, 8, 64).c()) == -5

    size = 2 * 3 * 8
    ws1 = _a(size * 512) * 2 + _a(size * 8)

    def extend(cache=big, layer=0, q=big, n=3, lens=big, hint=0, rk=big, rv=big, splits=0, out=big, ws=big, b=1 << 40, cfg=c):
        return L.attn_extend(r(cfg), cache, layer, q, n, None, lens, hint, rk, rv, 0.0, splits, out, None, ws, b, None, None)

    assert [extend(cache=None), extend(q=None), extend(lens=None), extend(rv=None), extend(out=None), extend(ws=None)] == [-1] * 6
    assert [extend(layer=1), extend(n=-1), extend(hint=-1), extend(splits=-1), extend(splits=65)] == [-1] * 5
    assert [extend(ws=odd), extend(q=odd), extend(out=odd), extend(cache=odd)] == [-1] * 4
    assert [extend(n=65), extend(hint=65)] == [-2] * 2
    assert [extend(b=ws1 - 1), extend(splits=2, b=ws1), extend(b=0)] == [-3] * 3
    assert extend(n=0) == 0
    # as many rows as the row index holds, and no more
    assert extend(cfg=K.KVConfig(1, 1, 8, 1, 128, 4, 8, 1 << 28).c(), n=1 << 28) == -5

    def prefix(pcache=big, layer=0, plen=big, hint=0, phint=0, splits=0, out=big, ws=big, b=1 << 40, cache=big, lens=big, q=big,
               rk=big, pcfg=pc):
        return L.attn_decode_prefix(r(c), cache, r(pcfg), pcache, layer, q, lens, hint, plen, phint, rk, big, 0.0, splits, out,
                                    None, ws, b, None, None)

    assert [prefix(pcache=None), prefix(plen=None), prefix(out=None), prefix(ws=None), prefix(cache=None), prefix(lens=None),
            prefix(q=None), prefix(rk=None)] == [-1] * 8
    assert [prefix(layer=1), prefix(splits=65), prefix(splits=-1), prefix(phint=-1), prefix(hint=-1), prefix(ws=odd),
            prefix(pcache=odd), prefix(cache=odd), prefix(q=odd)] == [-1] * 9
    assert [prefix(phint=301), prefix(hint=65)] == [-2] * 2
    assert [prefix(b=0), prefix(b=4096)] == [-3] * 2
    n = ctypes.c_uint64()
    assert L.attn_extend_workspace_query(r(c), 65, r(n)) == -2 and L.attn_extend_workspace_query(r(c), -1, r(n)) == -1
    assert L.attn_extend_workspace_query(r(c), 3, None) == -1
    assert L.attn_extend_workspace_query(r(c), 3, r(n)) == 0 and n.value >= ws1
