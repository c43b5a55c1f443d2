"""Thin ctypes binding of liboscar_kv.so (argument marshalling only).

Every computation runs in the library's CUDA kernels; this module converts
torch tensors to pointers and checks return codes.  It raises if the library
has not been built: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass, field

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liboscar_kv.so")

GROUP = 128
MAX_SPLITS = 64
FLAG_ABSORB_V = 1
FLAG_IN_FP32 = 2
FLAG_OUT_FP32 = 4
FLAG_HADAMARD = 8  # rotate by the in-quant Hadamard; R_K / R_V may be None
FLAG_V_BF16 = 16  # K-only INT2: V kept BF16 at every position
FLAG_LLOYD_MAX = 32  # INT2 codes index Lloyd-Max levels (0, rho, rho + 1, 2 rho + 1), rho = 1.16 (float32)

DEV_OVER_CAPACITY = 1
DEV_NONFINITE = 2
DEV_FP16_RANGE = 4
DEV_TIMEOUT = 8
DEV_EMPTY = 16

STATUS_NAMES = {0: "OK", -1: "INVALID", -2: "CAPACITY", -3: "WORKSPACE", -4: "LAUNCH", -5: "UNSUPPORTED"}

# every symbol include/oscar_kv.h declares
EXPORTS = ("kv_layout_query", "kv_append", "attn_decode", "decode_step", "attn_decode_static", "kv_read",
           "attn_extend_workspace_query", "attn_extend", "attn_decode_prefix_workspace_query", "attn_decode_prefix",
           "qk_norm_rope", "attn_prompt", "kv_append_packed", "attn_mass_workspace_query", "attn_mass",
           "kv_evict_workspace_query", "kv_evict",
           "oscar_kv_set_profile_events", "oscar_kv_set_wait_test", "oscar_kv_decode_kernels",
           "oscar_calibrate_workspace_query",
           "oscar_calibrate_rk",
           "oscar_calibrate_rv_workspace_query", "oscar_calibrate_rv")
STATIC_SCRATCH_BYTES = 16 << 20


class OscarError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {code} ({STATUS_NAMES.get(code, '?')})")
        self.code = code


class _Config(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("sink", ctypes.c_int32), ("recent", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("k_clip", ctypes.c_float), ("v_clip", ctypes.c_float), ("flags", ctypes.c_uint32)]


class _Layout(ctypes.Structure):
    _fields_ = [("ncap", ctypes.c_uint64), ("sink_bytes", ctypes.c_uint64), ("ring_bytes", ctypes.c_uint64),
                ("codes_bytes", ctypes.c_uint64), ("sz_bytes", ctypes.c_uint64), ("role_bytes", ctypes.c_uint64),
                ("layer_bytes", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64),
                ("decode_workspace_bytes", ctypes.c_uint64), ("max_splits", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("v_role_bytes", ctypes.c_uint64)]


@dataclass
class KVConfig:
    num_layers: int
    batch: int
    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    sink: int
    recent: int
    capacity: int
    k_clip: float = 0.96
    v_clip: float = 0.92
    flags: int = 0
    group_size: int = GROUP

    def c(self) -> _Config:
        return _Config(self.num_layers, self.batch, self.num_q_heads, self.num_kv_heads, self.head_dim,
                       self.group_size, self.sink, self.recent, self.capacity, self.k_clip, self.v_clip,
                       self.flags)


_lib = None


def lib():
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with int2_kv_cache_append_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        L.kv_layout_query.argtypes = [ctypes.POINTER(_Config), ctypes.POINTER(_Layout)]
        L.kv_layout_query.restype = ctypes.c_int
        L.kv_append.argtypes = [ctypes.POINTER(_Config), P, ctypes.c_int32, P, P, P, ctypes.c_int32, P, P, P, P, P]
        L.kv_append.restype = ctypes.c_int
        L.attn_decode.argtypes = [ctypes.POINTER(_Config), P, ctypes.c_int32, P, P, ctypes.c_int32, P, P,
                                  ctypes.c_float, ctypes.c_int32, P, P, P, ctypes.c_uint64, P, P]
        L.attn_decode.restype = ctypes.c_int
        L.attn_decode_static.argtypes = [ctypes.POINTER(_Config), P, ctypes.c_int32, P, P, ctypes.c_int32, P, P,
                                         ctypes.c_float, ctypes.c_int32, P, P, P, P]
        L.attn_decode_static.restype = ctypes.c_int
        L.decode_step.argtypes = [ctypes.POINTER(_Config), P, ctypes.c_int32, P, P, P, ctypes.c_int32, P, P,
                                  ctypes.c_int32, P, P, ctypes.c_float, ctypes.c_int32, P, P, P, ctypes.c_uint64, P, P]
        L.decode_step.restype = ctypes.c_int
        L.kv_read.argtypes = [ctypes.POINTER(_Config), P, ctypes.c_int32, P, P, ctypes.c_int32, P, P, P, P, P, P]
        L.kv_read.restype = ctypes.c_int
        L.attn_extend_workspace_query.argtypes = [ctypes.POINTER(_Config), ctypes.c_int32,
                                                  ctypes.POINTER(ctypes.c_uint64)]
        L.attn_extend_workspace_query.restype = ctypes.c_int
        L.attn_extend.argtypes = [ctypes.POINTER(_Config), P, ctypes.c_int32, P, ctypes.c_int32, P, P, ctypes.c_int32,
                                  P, P, ctypes.c_float, ctypes.c_int32, P, P, P, ctypes.c_uint64, P, P]
        L.attn_extend.restype = ctypes.c_int
        L.attn_decode_prefix_workspace_query.argtypes = [ctypes.POINTER(_Config), ctypes.POINTER(_Config),
                                                         ctypes.POINTER(ctypes.c_uint64)]
        L.attn_decode_prefix_workspace_query.restype = ctypes.c_int
        L.attn_decode_prefix.argtypes = [ctypes.POINTER(_Config), P, ctypes.POINTER(_Config), P, ctypes.c_int32, P, P,
                                         ctypes.c_int32, P, ctypes.c_int32, P, P, ctypes.c_float, ctypes.c_int32, P, P,
                                         P, ctypes.c_uint64, P, P]
        L.attn_decode_prefix.restype = ctypes.c_int
        C, I32, I64, F32, U64 = ctypes.POINTER(_Config), ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_uint64
        for name, args in (("qk_norm_rope", [C, P, I64, P, I64, I32, P, P, F32, P, P, I32, I32, P, P, P]),
                           ("attn_prompt", [C, P, P, P, I32, P, F32, P, P, P, P]),
                           ("kv_append_packed", [C, P, I32, P, P, I32, P, P, P, P, P, P]),
                           ("attn_mass_workspace_query", [C, I32, ctypes.POINTER(U64)]),
                           ("attn_mass", [C, P, I32, P, I32, P, P, I32, P, F32, P, P, P, P, U64, P, P]),
                           ("kv_evict_workspace_query", [C, I32, ctypes.POINTER(U64)]),
                           ("kv_evict", [C, P, I32, P, P, I32, C, P, I32, P, P, P, P, U64, P, P])):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = ctypes.c_int
        L.oscar_kv_set_profile_events.argtypes = [P, P]
        L.oscar_kv_set_profile_events.restype = ctypes.c_int
        L.oscar_kv_set_wait_test.argtypes = [ctypes.c_uint64, ctypes.c_int32]
        L.oscar_kv_set_wait_test.restype = ctypes.c_int
        L.oscar_kv_decode_kernels.argtypes = [ctypes.POINTER(_Config)]
        L.oscar_kv_decode_kernels.restype = ctypes.c_int
        _lib = L
    return _lib


def _ptr(t):
    """Device address of a tensor argument (None -> NULL).  The library's kernels
    read it as a dense array in device memory, so a host tensor or a strided view
    is refused here instead of reaching the GPU."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"oscar_kv: expected a CUDA tensor, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError("oscar_kv: expected a contiguous tensor")
    return t.data_ptr()


def _check(t, name: str, dtypes, shape=None, min_bytes=None, optional: bool = False):
    """Refuse, before anything reaches the GPU, a tensor whose dtype, shape or
    size does not match what the library will read or write through it."""
    if t is None:
        if optional:
            return
        raise ValueError(f"oscar_kv: {name} is required")
    if t.dtype not in dtypes:
        raise ValueError(f"oscar_kv: {name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"oscar_kv: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if min_bytes is not None and t.nbytes < min_bytes:
        raise ValueError(f"oscar_kv: {name} holds {t.nbytes} bytes, needs {min_bytes}")


_torch = None


def _dt():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


_known = {}  # (C struct, cache bytes) of the configurations in use, by their values


def _known_cfg(cfg: "KVConfig"):
    key = (cfg.num_layers, cfg.batch, cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim, cfg.sink, cfg.recent,
           cfg.capacity, cfg.k_clip, cfg.v_clip, cfg.flags, cfg.group_size)
    hit = _known.get(key)
    if hit is None:
        if len(_known) >= 256:
            _known.clear()
        hit = _known[key] = (cfg.c(), layout_query(cfg)["total_bytes"])
    return hit


def _check_cache(cfg: "KVConfig", cache, name: str = "cache"):
    """Returns the configuration for the library."""
    torch = _dt()
    c, total = _known_cfg(cfg)
    _check(cache, name, (torch.uint8,), min_bytes=total)
    return ctypes.byref(c)


def _check_rot(cfg: "KVConfig", R, name: str):
    torch = _dt()
    # with the in-quant Hadamard the matrices are not read (None allowed)
    _check(R, name, (torch.float32,), min_bytes=cfg.head_dim * cfg.head_dim * 4,
           optional=bool(cfg.flags & FLAG_HADAMARD))


def _in_dtypes(cfg: "KVConfig"):
    torch = _dt()
    return (torch.float32,) if cfg.flags & FLAG_IN_FP32 else (torch.bfloat16,)


def _check_decode_io(cfg: "KVConfig", q, seq_lens, out, lse, status):
    torch = _dt()
    B, Hq, D = cfg.batch, cfg.num_q_heads, cfg.head_dim
    _check(q, "q", _in_dtypes(cfg), shape=(B, Hq, D))
    _check(seq_lens, "seq_lens", (torch.int32,), shape=(B,))
    _check(out, "out", (torch.float32,) if cfg.flags & FLAG_OUT_FP32 else (torch.bfloat16,), shape=(B, Hq, D))
    _check(lse, "lse", (torch.float32,), min_bytes=B * Hq * 4, optional=True)
    _check(status, "status", (torch.int32,), min_bytes=4, optional=True)


def _check_append_io(cfg: "KVConfig", k_new, v_new, start_pos, debug_rot, status):
    torch = _dt()
    B, H, D = cfg.batch, cfg.num_kv_heads, cfg.head_dim
    if k_new is None or k_new.dim() != 4:
        raise ValueError("oscar_kv: k_new must be [batch][n_new][num_kv_heads][head_dim]")
    n = int(k_new.shape[1])
    _check(k_new, "k_new", _in_dtypes(cfg), shape=(B, n, H, D))
    _check(v_new, "v_new", _in_dtypes(cfg), shape=(B, n, H, D))
    _check(start_pos, "start_pos", (torch.int32,), shape=(B,))
    _check(debug_rot, "debug_rot", (torch.float32,), min_bytes=B * n * H * 2 * D * 4, optional=True)
    _check(status, "status", (torch.int32,), min_bytes=4, optional=True)


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def layout_query(cfg: KVConfig) -> dict:
    out = _Layout()
    rc = lib().kv_layout_query(ctypes.byref(cfg.c()), ctypes.byref(out))
    if rc != 0:
        raise OscarError("kv_layout_query", rc)
    return {name: getattr(out, name) for name, _ in _Layout._fields_}


def ring_rows(cfg: KVConfig, cache, layer: int):
    """The rings of a layer as views of the cache: (K, V), each [batch][num_kv_heads][recent][head_dim] bf16, position p
    in slot p % recent; V is None with FLAG_V_BF16, whose V role keeps every position.

    For a sequence that gets shorter, as by refused drafts: an append overwrites the oldest rows of the window, which the
    shorter sequence reads again.  Keep ``ring[b, :, slots]`` of the drafts' positions before the append and put back the
    refused ones' (at most ``recent`` drafts; include/oscar_kv.h, attn_extend)."""
    torch = _dt()
    _check_cache(cfg, cache)
    if not cache.is_contiguous():
        raise ValueError("oscar_kv: expected a contiguous tensor")
    if not 0 <= layer < cfg.num_layers:
        raise ValueError(f"oscar_kv: layer {layer} of {cfg.num_layers}")
    lay = layout_query(cfg)
    shape = (cfg.batch, cfg.num_kv_heads, cfg.recent, cfg.head_dim)

    def view(role):
        at = layer * lay["layer_bytes"] + role * lay["role_bytes"] + lay["sink_bytes"]
        return cache.view(-1)[at:at + 2 * math.prod(shape)].view(torch.bfloat16).view(shape)

    return view(0), None if cfg.flags & FLAG_V_BF16 else view(1)


def kv_append(cfg: KVConfig, cache, layer: int, k_new, v_new, start_pos, R_K, R_V, debug_rot=None,
              status=None, stream=None, check: bool = True) -> int:
    _check_append_io(cfg, k_new, v_new, start_pos, debug_rot, status)
    _check_cache(cfg, cache)
    _check_rot(cfg, R_K, "R_K")
    _check_rot(cfg, R_V, "R_V")
    rc = lib().kv_append(ctypes.byref(cfg.c()), _ptr(cache), layer, _ptr(k_new), _ptr(v_new), _ptr(start_pos),
                         int(k_new.shape[1]), _ptr(R_K), _ptr(R_V), _ptr(debug_rot), _ptr(status), _stream(stream))
    if check and rc != 0:
        raise OscarError("kv_append", rc)
    return rc


def attn_decode(cfg: KVConfig, cache, layer: int, q, seq_lens, R_K, R_V, out, workspace, lse=None,
                seq_len_hint: int = 0, sm_scale: float = 0.0, num_splits: int = 0, status=None, stream=None,
                check: bool = True) -> int:
    _check_decode_io(cfg, q, seq_lens, out, lse, status)
    _check_cache(cfg, cache)
    _check_rot(cfg, R_K, "R_K")
    _check_rot(cfg, R_V, "R_V")
    _check(workspace, "workspace", (_dt().uint8,))
    rc = lib().attn_decode(ctypes.byref(cfg.c()), _ptr(cache), layer, _ptr(q), _ptr(seq_lens), int(seq_len_hint),
                           _ptr(R_K), _ptr(R_V), float(sm_scale), int(num_splits), _ptr(out), _ptr(lse),
                           _ptr(workspace), int(workspace.numel() * workspace.element_size()), _ptr(status),
                           _stream(stream))
    if check and rc != 0:
        raise OscarError("attn_decode", rc)
    return rc


def decode_step(cfg: KVConfig, cache, layer: int, k_new, v_new, start_pos, q, seq_lens, R_K, R_V, out, workspace,
                lse=None, seq_len_hint: int = 0, sm_scale: float = 0.0, num_splits: int = 0, status=None,
                stream=None, check: bool = True) -> int:
    """kv_append of k_new/v_new ([B][n][Hkv][D]) at start_pos, then attn_decode, in one call."""
    _check_append_io(cfg, k_new, v_new, start_pos, None, status)
    _check_decode_io(cfg, q, seq_lens, out, lse, status)
    _check_cache(cfg, cache)
    _check_rot(cfg, R_K, "R_K")
    _check_rot(cfg, R_V, "R_V")
    _check(workspace, "workspace", (_dt().uint8,))
    n_new = int(k_new.shape[1])
    rc = lib().decode_step(ctypes.byref(cfg.c()), _ptr(cache), layer, _ptr(k_new), _ptr(v_new), _ptr(start_pos),
                           n_new, _ptr(q), _ptr(seq_lens), int(seq_len_hint), _ptr(R_K), _ptr(R_V), float(sm_scale),
                           int(num_splits), _ptr(out), _ptr(lse), _ptr(workspace),
                           int(workspace.numel() * workspace.element_size()), _ptr(status), _stream(stream))
    if check and rc != 0:
        raise OscarError("decode_step", rc)
    return rc


def attn_decode_static(cfg: KVConfig, cache, layer: int, q, seq_lens, R_K, R_V, out, lse=None,
                       seq_len_hint: int = 0, sm_scale: float = 0.0, num_splits: int = 0, status=None, stream=None,
                       check: bool = True) -> int:
    """attn_decode with the library's fixed scratch array (no workspace argument)."""
    _check_decode_io(cfg, q, seq_lens, out, lse, status)
    _check_cache(cfg, cache)
    _check_rot(cfg, R_K, "R_K")
    _check_rot(cfg, R_V, "R_V")
    rc = lib().attn_decode_static(ctypes.byref(cfg.c()), _ptr(cache), layer, _ptr(q), _ptr(seq_lens),
                                  int(seq_len_hint), _ptr(R_K), _ptr(R_V), float(sm_scale), int(num_splits),
                                  _ptr(out), _ptr(lse), _ptr(status), _stream(stream))
    if check and rc != 0:
        raise OscarError("attn_decode_static", rc)
    return rc


def _same_device(*tensors) -> None:
    """The library launches on the current device: refuse tensors that live on another one."""
    current = None
    for t in tensors:
        if t is not None and t.is_cuda:
            if current is None:
                current = _dt().cuda.current_device()
            if t.get_device() != current:
                raise ValueError(f"oscar_kv: tensor on {t.device}, current device is cuda:{current}")


def kv_read(cfg: KVConfig, cache, layer: int, start_pos, seq_lens, R_K, R_V, k_out=None, v_out=None, status=None,
            stream=None, check: bool = True) -> int:
    """Positions [start_pos[b], start_pos[b] + n) of every sequence back into k_out / v_out ([B][n][Hkv][D]; either
    may be None), in the basis the rows were appended in.  Positions outside [0, seq_lens[b]) are left as they were."""
    torch = _dt()
    B, H, D = cfg.batch, cfg.num_kv_heads, cfg.head_dim
    first = k_out if k_out is not None else v_out
    if first is None or first.dim() != 4:
        raise ValueError("oscar_kv: k_out or v_out must be [batch][n][num_kv_heads][head_dim]")
    n = int(first.shape[1])
    kind = (torch.float32,) if cfg.flags & FLAG_OUT_FP32 else (torch.bfloat16,)
    _check(k_out, "k_out", kind, shape=(B, n, H, D), optional=True)
    _check(v_out, "v_out", kind, shape=(B, n, H, D), optional=True)
    _check(start_pos, "start_pos", (torch.int32,), shape=(B,))
    _check(seq_lens, "seq_lens", (torch.int32,), shape=(B,))
    _check(status, "status", (torch.int32,), min_bytes=4, optional=True)
    c = _check_cache(cfg, cache)
    _check_rot(cfg, R_K, "R_K")
    _check_rot(cfg, R_V, "R_V")
    _same_device(cache, start_pos, seq_lens, R_K, R_V, k_out, v_out, status)
    rc = lib().kv_read(c, _ptr(cache), layer, _ptr(start_pos), _ptr(seq_lens), n, _ptr(R_K),
                       _ptr(R_V), _ptr(k_out), _ptr(v_out), _ptr(status), _stream(stream))
    if check and rc != 0:
        raise OscarError("kv_read", rc)
    return rc


def attn_extend_workspace_bytes(cfg: KVConfig, n_new: int) -> int:
    n = ctypes.c_uint64(0)
    rc = lib().attn_extend_workspace_query(ctypes.byref(cfg.c()), int(n_new), ctypes.byref(n))
    if rc != 0:
        raise OscarError("attn_extend_workspace_query", rc)
    return int(n.value)


def attn_extend(cfg: KVConfig, cache, layer: int, q, seq_lens, R_K, R_V, out, workspace, q_lens=None, lse=None,
                seq_len_hint: int = 0, sm_scale: float = 0.0, num_splits: int = 0, status=None, stream=None,
                check: bool = True) -> int:
    """Causal attention of the last q_lens[b] (None: n) tokens of every sequence, q [B][n][Hq][D], over its cache
    (append their K and V first).  Rows t >= q_lens[b] of out and lse ([B][n][Hq]) are left as they were."""
    torch = _dt()
    B, Hq, D = cfg.batch, cfg.num_q_heads, cfg.head_dim
    if q is None or q.dim() != 4:
        raise ValueError("oscar_kv: q must be [batch][n_new][num_q_heads][head_dim]")
    n = int(q.shape[1])
    _check(q, "q", _in_dtypes(cfg), shape=(B, n, Hq, D))
    _check(out, "out", (torch.float32,) if cfg.flags & FLAG_OUT_FP32 else (torch.bfloat16,), shape=(B, n, Hq, D))
    _check(lse, "lse", (torch.float32,), shape=(B, n, Hq), optional=True)
    _check(seq_lens, "seq_lens", (torch.int32,), shape=(B,))
    _check(q_lens, "q_lens", (torch.int32,), shape=(B,), optional=True)
    _check(status, "status", (torch.int32,), min_bytes=4, optional=True)
    _check(workspace, "workspace", (torch.uint8,))
    c = _check_cache(cfg, cache)
    _check_rot(cfg, R_K, "R_K")
    _check_rot(cfg, R_V, "R_V")
    _same_device(cache, q, seq_lens, q_lens, R_K, R_V, out, lse, workspace, status)
    rc = lib().attn_extend(c, _ptr(cache), layer, _ptr(q), n, _ptr(q_lens), _ptr(seq_lens),
                           int(seq_len_hint), _ptr(R_K), _ptr(R_V), float(sm_scale), int(num_splits), _ptr(out),
                           _ptr(lse), _ptr(workspace), int(workspace.numel()), _ptr(status), _stream(stream))
    if check and rc != 0:
        raise OscarError("attn_extend", rc)
    return rc


def attn_decode_prefix_workspace_bytes(cfg: KVConfig, prefix_cfg: KVConfig) -> int:
    n = ctypes.c_uint64(0)
    rc = lib().attn_decode_prefix_workspace_query(ctypes.byref(cfg.c()), ctypes.byref(prefix_cfg.c()), ctypes.byref(n))
    if rc != 0:
        raise OscarError("attn_decode_prefix_workspace_query", rc)
    return int(n.value)


def attn_decode_prefix(cfg: KVConfig, cache, prefix_cfg: KVConfig, prefix_cache, layer: int, q, seq_lens, prefix_len,
                       R_K, R_V, out, workspace, lse=None, seq_len_hint: int = 0, prefix_len_hint: int = 0,
                       sm_scale: float = 0.0, num_splits: int = 0, status=None, stream=None, check: bool = True) -> int:
    """attn_decode over a prefix that the whole batch shares (prefix_cache, one sequence of prefix_len[0] positions)
    followed by every sequence's own cache (seq_lens[b] positions, 0 allowed)."""
    torch = _dt()
    _check_decode_io(cfg, q, seq_lens, out, lse, status)
    _check(prefix_len, "prefix_len", (torch.int32,), shape=(1,))
    c = _check_cache(cfg, cache)
    pc = _check_cache(prefix_cfg, prefix_cache, "prefix_cache")
    _check_rot(cfg, R_K, "R_K")
    _check_rot(cfg, R_V, "R_V")
    _check(workspace, "workspace", (torch.uint8,))
    _same_device(cache, prefix_cache, q, seq_lens, prefix_len, R_K, R_V, out, lse, workspace, status)
    rc = lib().attn_decode_prefix(c, _ptr(cache), pc, _ptr(prefix_cache),
                                  layer, _ptr(q), _ptr(seq_lens), int(seq_len_hint), _ptr(prefix_len),
                                  int(prefix_len_hint), _ptr(R_K), _ptr(R_V), float(sm_scale), int(num_splits),
                                  _ptr(out), _ptr(lse), _ptr(workspace), int(workspace.numel()), _ptr(status),
                                  _stream(stream))
    if check and rc != 0:
        raise OscarError("attn_decode_prefix", rc)
    return rc


class _Args:
    """Checks the tensor arguments of one call and gives their addresses: type, shape, memory (dense, unless the caller says
    otherwise) and device.  The library launches on the current device, so every tensor has to be there."""

    def __init__(self, cfg: KVConfig):
        torch = _dt()
        self.device = torch.cuda.current_device() if torch.cuda.is_initialized() else -2
        self.cfg = cfg
        flags = cfg.flags
        self.kind_in = torch.float32 if flags & FLAG_IN_FP32 else torch.bfloat16
        self.kind_out = torch.float32 if flags & FLAG_OUT_FP32 else torch.bfloat16

    def place(self, t):
        d = t.get_device()
        if d != self.device:
            if d < 0:
                raise ValueError(f"oscar_kv: expected a CUDA tensor, got one on {t.device}")
            if self.device == -2:
                self.device = _dt().cuda.current_device()
                return self.place(t)
            raise ValueError(f"oscar_kv: tensor on {t.device}, current device is cuda:{self.device}")
        return t.data_ptr()

    def __call__(self, t, name: str, kind, shape, optional: bool = False):
        if t is None:
            if optional:
                return None
            raise ValueError(f"oscar_kv: {name} is required")
        if t.dtype is not kind or t.shape != shape:
            _check(t, name, (kind,), shape=shape)
        if not t.is_contiguous():
            raise ValueError("oscar_kv: expected a contiguous tensor")
        return self.place(t)

    def memory(self, t, name: str, kind, nbytes: int, optional: bool = False):
        """Any shape, nbytes at least."""
        if t is None:
            if optional:
                return None
            raise ValueError(f"oscar_kv: {name} is required")
        if t.dtype is not kind or t.nbytes < nbytes:
            _check(t, name, (kind,), min_bytes=nbytes)
        if not t.is_contiguous():
            raise ValueError("oscar_kv: expected a contiguous tensor")
        return self.place(t)

    def cache(self, cfg: KVConfig, t, name: str = "cache"):
        """The configuration for the library, and the cache's address."""
        c, total = _known_cfg(cfg)
        return ctypes.byref(c), self.memory(t, name, _dt().uint8, total)

    def rotation(self, t, name: str):
        return self.memory(t, name, _dt().float32, self.cfg.head_dim * self.cfg.head_dim * 4,
                           optional=bool(self.cfg.flags & FLAG_HADAMARD))

    def status(self, t):
        return None if t is None else self.memory(t, "status", _dt().int32, 4)

    def token_rows(self, t, name: str, shape):
        """Address of [tokens][heads][head_dim] and the elements from one token to the next, which may lie further on than the
        token's heads reach (a fused projection)."""
        _check(t, name, (self.kind_in,), shape=shape)
        at = self.place(t)
        n, heads, d = shape
        if n == 0:
            return at, heads * d
        step, head, one = t.stride()
        if one != 1 or (heads > 1 and head != d):
            raise ValueError(f"oscar_kv: the heads of a token of {name} must be contiguous")
        return at, heads * d if n == 1 else step

    def stream(self, stream):
        if stream is None:  # without the Stream object around it, a tenth of a small call's time
            return _dt()._C._cuda_getCurrentRawStream(self.device)
        return stream if isinstance(stream, int) else stream.cuda_stream


def _result(fn: str, rc: int, check: bool) -> int:
    if check and rc != 0:
        raise OscarError(fn, rc)
    return rc


def qk_norm_rope(cfg: KVConfig, q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, eps: float = 1e-6,
                 interleaved: bool = False, stream=None, check: bool = True) -> int:
    """Root-mean-square norm of every head of q [n][Hq][D] and k [n][Hkv][D] (strided over the tokens, as views of a fused
    projection), then the rotation of the first 2 * len(inv_freq) channels by positions * inv_freq (None: no rotation),
    into q_out and k_out."""
    torch = _dt()
    if q is None or q.dim() != 3:
        raise ValueError("oscar_kv: q must be [n][num_q_heads][head_dim]")
    arg, n, D = _Args(cfg), q.shape[0], cfg.head_dim
    shape_q, shape_k, f32 = (n, cfg.num_q_heads, D), (n, cfg.num_kv_heads, D), torch.float32
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    (pq, sq), (pk, sk) = arg.token_rows(q, "q", shape_q), arg.token_rows(k, "k", shape_k)
    rc = lib().qk_norm_rope(ctypes.byref(_known_cfg(cfg)[0]), pq, sq, pk, sk, n, arg(q_weight, "q_weight", f32, (D,)),
                            arg(k_weight, "k_weight", f32, (D,)), eps,
                            arg(positions, "positions", torch.int32, (n,), optional=rot == 0),
                            arg(inv_freq, "inv_freq", f32, (rot // 2,), optional=True), rot, 1 if interleaved else 0,
                            arg(q_out, "q_out", arg.kind_in, shape_q), arg(k_out, "k_out", arg.kind_in, shape_k),
                            arg.stream(stream))
    return _result("qk_norm_rope", rc, check)


def attn_prompt(cfg: KVConfig, q, k, v, cu_seqlens, out, lse=None, sm_scale: float = 0.0, status=None, stream=None,
                check: bool = True) -> int:
    """Causal attention of packed prompts, q and out [n][Hq][D], over their own k and v [n][Hkv][D]: sequence b has the
    rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1; other rows of out and lse ([n][Hq]) are left as they were."""
    torch = _dt()
    if q is None or q.dim() != 3:
        raise ValueError("oscar_kv: q must be [n][num_q_heads][head_dim]")
    arg, n, Hq, D = _Args(cfg), q.shape[0], cfg.num_q_heads, cfg.head_dim
    rows, kv = (n, Hq, D), (n, cfg.num_kv_heads, D)
    rc = lib().attn_prompt(ctypes.byref(_known_cfg(cfg)[0]), arg(q, "q", arg.kind_in, rows), arg(k, "k", arg.kind_in, kv),
                           arg(v, "v", arg.kind_in, kv), n, arg(cu_seqlens, "cu_seqlens", torch.int32, (cfg.batch + 1,)),
                           sm_scale, arg(out, "out", arg.kind_out, rows),
                           arg(lse, "lse", torch.float32, (n, Hq), optional=True), arg.status(status), arg.stream(stream))
    return _result("attn_prompt", rc, check)


def kv_append_packed(cfg: KVConfig, cache, layer: int, k_new, v_new, cu_seqlens, start_pos, R_K, R_V, status=None,
                     stream=None, check: bool = True) -> int:
    """kv_append of packed rows k_new, v_new [n][Hkv][D]: sequence b gets the rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1
    at start_pos[b]."""
    torch = _dt()
    if k_new is None or k_new.dim() != 3:
        raise ValueError("oscar_kv: k_new must be [n][num_kv_heads][head_dim]")
    arg, n = _Args(cfg), k_new.shape[0]
    rows, i32 = (n, cfg.num_kv_heads, cfg.head_dim), torch.int32
    c, at = arg.cache(cfg, cache)
    rc = lib().kv_append_packed(c, at, layer, arg(k_new, "k_new", arg.kind_in, rows), arg(v_new, "v_new", arg.kind_in, rows), n,
                                arg(cu_seqlens, "cu_seqlens", i32, (cfg.batch + 1,)),
                                arg(start_pos, "start_pos", i32, (cfg.batch,)), arg.rotation(R_K, "R_K"),
                                arg.rotation(R_V, "R_V"), arg.status(status), arg.stream(stream))
    return _result("kv_append_packed", rc, check)


def attn_mass_workspace_bytes(cfg: KVConfig, n_new: int) -> int:
    n = ctypes.c_uint64(0)
    _result("attn_mass_workspace_query", lib().attn_mass_workspace_query(ctypes.byref(cfg.c()), int(n_new), ctypes.byref(n)), True)
    return int(n.value)


def attn_mass(cfg: KVConfig, cache, layer: int, q, seq_lens, R_K, lse, mass_out, workspace, mass_in=None, q_lens=None,
              seq_len_hint: int = 0, sm_scale: float = 0.0, status=None, stream=None, check: bool = True) -> int:
    """mass_out [B][Hkv][capacity] = mass_in (None: 0) plus the attention weight that every cached position receives from
    the last q_lens[b] (None: n) tokens of its sequence, q [B][n][Hq][D] with the lse [B][n][Hq] of their attention."""
    torch = _dt()
    if q is None or q.dim() != 4:
        raise ValueError("oscar_kv: q must be [batch][n_new][num_q_heads][head_dim]")
    arg, n, B, Hq = _Args(cfg), q.shape[1], cfg.batch, cfg.num_q_heads
    whole, f32, i32 = (B, cfg.num_kv_heads, cfg.capacity), torch.float32, torch.int32
    c, at = arg.cache(cfg, cache)
    ws = arg.memory(workspace, "workspace", torch.uint8, 0)
    rc = lib().attn_mass(c, at, layer, arg(q, "q", arg.kind_in, (B, n, Hq, cfg.head_dim)), n,
                         arg(q_lens, "q_lens", i32, (B,), optional=True), arg(seq_lens, "seq_lens", i32, (B,)), seq_len_hint,
                         arg.rotation(R_K, "R_K"), sm_scale, arg(lse, "lse", f32, (B, n, Hq)),
                         arg(mass_in, "mass_in", f32, whole, optional=True), arg(mass_out, "mass_out", f32, whole), ws,
                         workspace.numel(), arg.status(status), arg.stream(stream))
    return _result("attn_mass", rc, check)


def kv_evict_workspace_bytes(cfg: KVConfig, keep: int) -> int:
    n = ctypes.c_uint64(0)
    _result("kv_evict_workspace_query", lib().kv_evict_workspace_query(ctypes.byref(cfg.c()), int(keep), ctypes.byref(n)), True)
    return int(n.value)


def kv_evict(cfg: KVConfig, cache, layer: int, mass, seq_lens, keep: int, out_cfg: KVConfig, out_cache, out_layer: int,
             new_lens, workspace, out_mass=None, kept=None, status=None, stream=None, check: bool = True) -> int:
    """A layer of `cache` without all but the `keep` positions of largest mass [B][Hkv][capacity] between sink and window
    of every KV head, into a layer of out_cache; new_lens [B] (may be seq_lens) receives the lengths, out_mass
    [B][Hkv][out capacity] the masses of what stays, kept [B][Hkv][keep] its old positions (-1 behind the last)."""
    torch = _dt()
    arg, B, H = _Args(cfg), cfg.batch, cfg.num_kv_heads
    f32, i32 = torch.float32, torch.int32
    c, at = arg.cache(cfg, cache)
    oc, out_at = arg.cache(out_cfg, out_cache, "out_cache")
    ws = arg.memory(workspace, "workspace", torch.uint8, 0)
    rc = lib().kv_evict(c, at, layer, arg(mass, "mass", f32, (B, H, cfg.capacity)), arg(seq_lens, "seq_lens", i32, (B,)), keep, oc,
                        out_at, out_layer, arg(out_mass, "out_mass", f32, (B, H, out_cfg.capacity), optional=True),
                        arg(kept, "kept", i32, (B, H, keep), optional=True), arg(new_lens, "new_lens", i32, (B,)), ws,
                        workspace.numel(), arg.status(status), arg.stream(stream))
    return _result("kv_evict", rc, check)


def set_profile_events(start=None, stop=None) -> None:
    """Record torch.cuda.Event pair around the split kernel of later attn_decode calls (None, None stops)."""
    lib().oscar_kv_set_profile_events(None if start is None else ctypes.c_void_p(start.cuda_event),
                                      None if stop is None else ctypes.c_void_p(stop.cuda_event))


def decode_kernels(cfg: KVConfig) -> int:
    """Kernels one attn_decode call launches (see oscar_kv_decode_kernels)."""
    rc = lib().oscar_kv_decode_kernels(ctypes.byref(cfg.c()))
    if rc < 0:
        raise OscarError("oscar_kv_decode_kernels", rc)
    return rc


def set_wait_test(wait_ns: int = 0, extra_bytes: int = 0) -> None:
    """Timeout-path test hook (see oscar_kv_set_wait_test); (0, 0) restores normal operation."""
    rc = lib().oscar_kv_set_wait_test(int(wait_ns), int(extra_bytes))
    if rc != 0:
        raise OscarError("oscar_kv_set_wait_test", rc)


def _calib_fns():
    L = lib()
    if not getattr(L, "_calib_ready", False):
        L.oscar_calibrate_workspace_query.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_uint64)]
        L.oscar_calibrate_workspace_query.restype = ctypes.c_int
        L.oscar_calibrate_rk.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p]
        L.oscar_calibrate_rk.restype = ctypes.c_int
        L.oscar_calibrate_rv_workspace_query.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(ctypes.c_uint64)]
        L.oscar_calibrate_rv_workspace_query.restype = ctypes.c_int
        L.oscar_calibrate_rv.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p]
        L.oscar_calibrate_rv.restype = ctypes.c_int
        L._calib_ready = True
    return L


def calibrate_workspace_bytes(head_dim: int) -> int:
    n = ctypes.c_uint64(0)
    rc = _calib_fns().oscar_calibrate_workspace_query(int(head_dim), ctypes.byref(n))
    if rc != 0:
        raise OscarError("oscar_calibrate_workspace_query", rc)
    return int(n.value)


def calibrate_rk(q, R_out, workspace, status=None, stream=None, check: bool = True) -> int:
    """R_K fitted to the float32 query rows q [n][D] (see oscar_calibrate_rk); writes R_out [D][D]."""
    torch = _dt()
    if q is None or q.dim() != 2:
        raise ValueError("oscar_kv: q must be [n_rows][head_dim] float32")
    n, d = int(q.shape[0]), int(q.shape[1])
    _check(q, "q", (torch.float32,))
    _check(R_out, "R_out", (torch.float32,), shape=(d, d))
    _check(workspace, "workspace", (torch.uint8,))
    _check(status, "status", (torch.int32,), min_bytes=4, optional=True)
    rc = _calib_fns().oscar_calibrate_rk(_ptr(q), n, d, _ptr(R_out), _ptr(workspace),
                                         int(workspace.numel() * workspace.element_size()), _ptr(status),
                                         _stream(stream))
    if check and rc != 0:
        raise OscarError("oscar_calibrate_rk", rc)
    return rc


def calibrate_rv_workspace_bytes(head_dim: int, n_kv_rows: int) -> int:
    n = ctypes.c_uint64(0)
    rc = _calib_fns().oscar_calibrate_rv_workspace_query(int(head_dim), int(n_kv_rows), ctypes.byref(n))
    if rc != 0:
        raise OscarError("oscar_calibrate_rv_workspace_query", rc)
    return int(n.value)


def calibrate_rv(q, k, v, R_out, workspace, status=None, stream=None, check: bool = True) -> int:
    """R_V fitted to the score-weighted covariance of the float32 value rows v [n][D],
    each weighted by k_t q^T q k_t^T (see oscar_calibrate_rv); writes R_out [D][D]."""
    torch = _dt()
    if q is None or q.dim() != 2 or k is None or k.dim() != 2:
        raise ValueError("oscar_kv: q and k must be [n_rows][head_dim] float32")
    nq, d = int(q.shape[0]), int(q.shape[1])
    nkv = int(k.shape[0])
    if v is None or tuple(k.shape) != tuple(v.shape) or int(k.shape[1]) != d:
        raise ValueError("k and v must both be [n_kv][head_dim] with the head_dim of q")
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, name, (torch.float32,))
    _check(R_out, "R_out", (torch.float32,), shape=(d, d))
    _check(workspace, "workspace", (torch.uint8,))
    _check(status, "status", (torch.int32,), min_bytes=4, optional=True)
    rc = _calib_fns().oscar_calibrate_rv(_ptr(q), nq, _ptr(k), _ptr(v), nkv, d, _ptr(R_out), _ptr(workspace),
                                         int(workspace.numel() * workspace.element_size()), _ptr(status),
                                         _stream(stream))
    if check and rc != 0:
        raise OscarError("oscar_calibrate_rv", rc)
    return rc
