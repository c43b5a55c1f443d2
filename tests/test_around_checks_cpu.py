"""qk_norm_rope, attn_prompt, kv_append_packed, attn_mass and kv_evict refuse bad calls on the host, before anything reaches
the GPU: the binding by tensor type, shape, layout and device, the library by pointer, range, configuration and workspace."""
import ctypes

import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K

CFG = K.KVConfig(1, 2, 8, 2, 128, 4, 8, 64)
OUT = K.KVConfig(2, 2, 8, 2, 128, 4, 8, 20)
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def _bytes(cfg):
    return torch.zeros(K.layout_query(cfg)["total_bytes"], dtype=U8)


def _rope(**over):
    args = dict(cfg=CFG, q=torch.zeros(5, 8, 128, dtype=BF), k=torch.zeros(5, 2, 128, dtype=BF), q_weight=torch.ones(128),
                k_weight=torch.ones(128), positions=torch.zeros(5, dtype=I32), inv_freq=torch.ones(64),
                q_out=torch.zeros(5, 8, 128, dtype=BF), k_out=torch.zeros(5, 2, 128, dtype=BF))
    return K.qk_norm_rope(**{**args, **over})


def _prompt(**over):
    args = dict(cfg=CFG, q=torch.zeros(5, 8, 128, dtype=BF), k=torch.zeros(5, 2, 128, dtype=BF), v=torch.zeros(5, 2, 128, dtype=BF),
                cu_seqlens=torch.zeros(3, dtype=I32), out=torch.zeros(5, 8, 128, dtype=BF), lse=torch.zeros(5, 8))
    return K.attn_prompt(**{**args, **over})


def _append(**over):
    args = dict(cfg=CFG, cache=_bytes(CFG), layer=0, k_new=torch.zeros(5, 2, 128, dtype=BF), v_new=torch.zeros(5, 2, 128, dtype=BF),
                cu_seqlens=torch.zeros(3, dtype=I32), start_pos=torch.zeros(2, dtype=I32), R_K=torch.zeros(128, 128),
                R_V=torch.zeros(128, 128))
    return K.kv_append_packed(**{**args, **over})


def _mass(**over):
    args = dict(cfg=CFG, cache=_bytes(CFG), layer=0, q=torch.zeros(2, 3, 8, 128, dtype=BF), seq_lens=torch.zeros(2, dtype=I32),
                R_K=torch.zeros(128, 128), lse=torch.zeros(2, 3, 8), mass_out=torch.zeros(2, 2, 64),
                workspace=torch.zeros(1 << 20, dtype=U8))
    return K.attn_mass(**{**args, **over})


def _evict(**over):
    args = dict(cfg=CFG, cache=_bytes(CFG), layer=0, mass=torch.zeros(2, 2, 64), seq_lens=torch.zeros(2, dtype=I32), keep=8,
                out_cfg=OUT, out_cache=_bytes(OUT), out_layer=1, new_lens=torch.zeros(2, dtype=I32),
                workspace=torch.zeros(1 << 16, dtype=U8))
    return K.kv_evict(**{**args, **over})


CALLS = [_rope, _prompt, _append, _mass, _evict]


@pytest.mark.parametrize("call", CALLS)
def test_valid_arguments_reach_the_device_check(call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        call()


@pytest.mark.parametrize("call,over", [
    (_rope, dict(q=torch.zeros(5, 8, 128))),                     # fp32 without OSCAR_FLAG_IN_FP32
    (_rope, dict(q=torch.zeros(5, 1024, dtype=BF))),
    (_rope, dict(q=None)),
    (_rope, dict(k=torch.zeros(4, 2, 128, dtype=BF))),
    (_rope, dict(k=torch.zeros(5, 2, 256, dtype=BF)[..., ::2])),
    (_rope, dict(q=torch.zeros(8, 5, 128, dtype=BF).transpose(0, 1))),
    (_rope, dict(q_weight=torch.ones(64))),
    (_rope, dict(k_weight=torch.ones(128, dtype=BF))),
    (_rope, dict(positions=None)),
    (_rope, dict(positions=torch.zeros(5, dtype=torch.int64))),
    (_rope, dict(q_out=torch.zeros(5, 8, 128))),
    (_rope, dict(k_out=torch.zeros(5, 8, 128, dtype=BF))),
    (_prompt, dict(q=torch.zeros(5, 8, 128))),
    (_prompt, dict(k=torch.zeros(5, 8, 128, dtype=BF))),
    (_prompt, dict(v=torch.zeros(6, 2, 128, dtype=BF))),
    (_prompt, dict(v=torch.zeros(5, 4, 128, dtype=BF)[:, :2])),
    (_prompt, dict(cu_seqlens=torch.zeros(2, dtype=I32))),
    (_prompt, dict(cu_seqlens=torch.zeros(3, dtype=torch.int64))),
    (_prompt, dict(out=torch.zeros(5, 8, 128))),
    (_prompt, dict(lse=torch.zeros(8, 5))),
    (_append, dict(k_new=torch.zeros(1, 5, 2, 128, dtype=BF))),
    (_append, dict(v_new=torch.zeros(4, 2, 128, dtype=BF))),
    (_append, dict(cu_seqlens=torch.zeros(2, dtype=I32))),
    (_append, dict(start_pos=torch.zeros(3, dtype=I32))),
    (_append, dict(R_K=None)),
    (_append, dict(cache=torch.zeros(100, dtype=U8))),
    (_mass, dict(q=torch.zeros(2, 8, 128, dtype=BF))),
    (_mass, dict(lse=torch.zeros(2, 8, 3))),
    (_mass, dict(lse=None)),
    (_mass, dict(mass_out=torch.zeros(2, 2, 63))),
    (_mass, dict(mass_in=torch.zeros(2, 64, 2))),
    (_mass, dict(q_lens=torch.zeros(3, dtype=I32))),
    (_mass, dict(workspace=torch.zeros(1 << 18))),
    (_evict, dict(mass=torch.zeros(2, 2, 20))),
    (_evict, dict(kept=torch.zeros(2, 2, 9, dtype=I32))),
    (_evict, dict(out_mass=torch.zeros(2, 2, 64))),
    (_evict, dict(new_lens=torch.zeros(2))),
    (_evict, dict(out_cache=torch.zeros(100, dtype=U8))),
])
def test_binding_refuses_mismatched_tensors(call, over):
    with pytest.raises(ValueError, match="oscar_kv"):
        call(**over)


# The library itself.  The addresses are host memory or made up: a call that is refused reads none of them.
P = 1 << 20  # an aligned address


def _c(cfg):
    return ctypes.byref(cfg.c())


def rope(cfg=CFG, q=P, qs=1024, k=P, ks=256, n=5, qw=P, kw=P, eps=1e-6, pos=P, freq=P, rot=128, qo=P, ko=P):
    return K.lib().qk_norm_rope(_c(cfg), q, qs, k, ks, n, qw, kw, eps, pos, freq, rot, 0, qo, ko, None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1), (dict(ko=None), -1), (dict(qw=None), -1), (dict(kw=None), -1),
    (dict(pos=None), -1), (dict(freq=None), -1), (dict(n=-1), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(rot=130), -1), (dict(rot=144), -1), (dict(rot=-16), -1), (dict(rot=8), -1),
    (dict(qs=1016), -1), (dict(ks=248), -1), (dict(qs=1028), -1), (dict(q=P + 8), -1), (dict(ko=P + 2), -1), (dict(qw=P + 4), -1),
    (dict(cfg=K.KVConfig(1, 2, 8, 2, 64, 4, 8, 64)), -5), (dict(cfg=K.KVConfig(1, 2, 18, 2, 128, 4, 8, 64)), -5),
    (dict(n=0, q=None, k=None, qo=None, ko=None, pos=None), 0),
])
def test_rope_refusals(over, code):
    assert rope(**over) == code


def prompt(cfg=CFG, q=P, k=P, v=P, n=5, cu=P, out=P):
    return K.lib().attn_prompt(_c(cfg), q, k, v, n, cu, 0.0, out, None, None, None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(cu=None), -1), (dict(n=-1), -1),
    (dict(q=P + 8), -1), (dict(v=P + 8), -1), (dict(out=P + 2), -1), (dict(n=1 << 28), -5),
    (dict(cfg=K.KVConfig(1, 2, 8, 2, 96, 4, 8, 64)), -5), (dict(cfg=K.KVConfig(1, 2, 8, 3, 128, 4, 8, 64)), -1),
    (dict(n=0, q=None, k=None, v=None, out=None), 0),
])
def test_prompt_refusals(over, code):
    assert prompt(**over) == code


def append(cfg=CFG, cache=P, layer=0, k=P, v=P, n=5, cu=P, start=P, rk=P, rv=P):
    return K.lib().kv_append_packed(_c(cfg), cache, layer, k, v, n, cu, start, rk, rv, None, None)


@pytest.mark.parametrize("over,code", [
    (dict(cache=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(cu=None), -1), (dict(start=None), -1), (dict(rk=None), -1),
    (dict(rv=None), -1), (dict(n=-1), -1), (dict(layer=1), -1), (dict(layer=-1), -1), (dict(cache=P + 16), -1), (dict(k=P + 8), -1),
    (dict(rv=P + 4), -1), (dict(n=0, k=None, v=None), 0),
])
def test_append_refusals(over, code):
    assert append(**over) == code


def mass(cfg=CFG, cache=P, layer=0, q=P, n=3, lens=P, hint=0, rk=P, lse=P, out=P, ws=P, size=1 << 20):
    return K.lib().attn_mass(_c(cfg), cache, layer, q, n, None, lens, hint, rk, 0.0, lse, None, out, ws, size, None, None)


@pytest.mark.parametrize("over,code", [
    (dict(cache=None), -1), (dict(q=None), -1), (dict(lens=None), -1), (dict(rk=None), -1), (dict(lse=None), -1), (dict(out=None), -1),
    (dict(ws=None), -1), (dict(ws=P + 16), -1), (dict(q=P + 8), -1), (dict(layer=1), -1), (dict(n=-1), -1), (dict(n=65), -2),
    (dict(hint=65), -2), (dict(hint=-1), -1), (dict(size=0), -3), (dict(cfg=K.KVConfig(1, 40000, 8, 2, 128, 4, 8, 64)), -5),
    (dict(cfg=K.KVConfig(1, 1, 8, 1, 128, 4, 8, 0x7fffffff)), -5),
])
def test_mass_refusals(over, code):
    assert mass(**over) == code


def test_mass_workspace_is_needed_in_full():
    need = K.attn_mass_workspace_bytes(CFG, 3)
    assert mass(size=need - 1) == -3


def evict(cfg=CFG, cache=P, layer=0, m=P, lens=P, keep=8, out_cfg=OUT, out=1 << 24, out_layer=0, out_mass=None, kept=None, new=P, ws=P,
          size=1 << 20):
    return K.lib().kv_evict(_c(cfg), cache, layer, m, lens, keep, _c(out_cfg), out, out_layer, out_mass, kept, new, ws, size, None, None)


def other(**kw):
    return K.KVConfig(**{**OUT.__dict__, **kw})


@pytest.mark.parametrize("over,code", [
    (dict(cache=None), -1), (dict(out=None), -1), (dict(m=None), -1), (dict(lens=None), -1), (dict(new=None), -1), (dict(ws=None), -1),
    (dict(keep=-1), -1), (dict(layer=1), -1), (dict(out_layer=2), -1), (dict(out=P + 16), -1), (dict(ws=P + 64), -1), (dict(size=0), -3),
    (dict(out=P), -1),                                            # the cache itself
    (dict(out=P + 256), -1),                                      # inside it
    (dict(out_mass=P), -1),                                       # mass itself
    (dict(out_cfg=other(capacity=19)), -2), (dict(keep=9), -2),
    (dict(out_cfg=other(batch=1)), -1), (dict(out_cfg=other(num_kv_heads=4)), -1), (dict(out_cfg=other(head_dim=256)), -1),
    (dict(out_cfg=other(sink=3)), -1), (dict(out_cfg=other(recent=9)), -1), (dict(out_cfg=other(flags=K.FLAG_LLOYD_MAX)), -1),
    (dict(cfg=K.KVConfig(1, 40000, 8, 2, 128, 4, 8, 64), out_cfg=other(batch=40000)), -5),
    (dict(cfg=K.KVConfig(1, 2, 8, 2, 128, 4, 8, 0x7fffffff)), -5),
])
def test_evict_refusals(over, code):
    assert evict(**over) == code


def test_two_layers_of_one_cache_may_be_read_and_written():
    """The layers must not overlap; which buffer they are in does not matter.  (The workspace is too small: refused before a launch.)"""
    cfg = K.KVConfig(2, 2, 8, 2, 128, 4, 8, 64)
    size = K.layout_query(cfg)["layer_bytes"]
    assert evict(cfg=cfg, out_cfg=cfg, layer=0, out=P, out_layer=1, size=0) == -3
    assert evict(cfg=cfg, out_cfg=cfg, layer=1, out=P + size, out_layer=0, size=0) == -1


@pytest.mark.parametrize("keep,rows", [(0, 0), (8, 8), (60, 60), (1000, 60)])
def test_evict_workspace_formula(keep, rows):
    align = lambda x: (x + 255) // 256 * 256
    assert K.kv_evict_workspace_bytes(CFG, keep) == align(2 * 4) + align(4 * rows * 4)


@pytest.mark.parametrize("n", [0, 1, 3, 64])
def test_mass_workspace_formula(n):
    align = lambda x: (x + 255) // 256 * 256
    if n * 4 > 24:  # blocks of 96 query rows: two fp16 and three bf16 parts, five constants
        parts = 2 * 2 * ((n * 4 + 95) // 96) * 96 * (128 * 10 + 5 * 4)
    else:
        parts = 2 * 2 * ((n * 4 + 3) // 4) * 4 * (128 * 12 + 16 + 4)
    assert K.attn_mass_workspace_bytes(CFG, n) == align(2 * n * 8 * 128 * 4) + align(parts)
