"""The tensor-core forms that larger calls of kv_read and attn_extend take: the
same 64-bit forms, on enough rows to cross over, on every head_dim and mode, and
against the small calls' results."""
import math

import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from oracle import oscar_oracle as O
from tests import rows_ref as R
from tests.gpu_helpers import dev, dev_i32, dev_rot, kcfg
from tests.test_gpu_rows import cfg_of, filled

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


@pytest.mark.parametrize("fp32", [True, False], ids=["fp32", "bf16"])
@pytest.mark.parametrize("D,B,H,W,lens,start,n,flags", [
    (128, 2, 3, 31, [700, 333], [0, 5], 701, 0),
    (128, 1, 8, 64, [400], [3], 390, K.FLAG_LLOYD_MAX),
    (128, 2, 8, 16, [200, 0], [-3, 0], 130, K.FLAG_V_BF16 | K.FLAG_ABSORB_V),
    (128, 1, 8, 0, [300], [0], 300, K.FLAG_HADAMARD),
    (256, 1, 5, 31, [401], [0], 401, K.FLAG_LLOYD_MAX),
    (256, 2, 4, 31, [257, 140], [1, 0], 250, 0),
    (512, 2, 4, 40, [300, 150], [0, 0], 300, 0),
    (512, 1, 4, 40, [330], [0], 330, K.FLAG_LLOYD_MAX | K.FLAG_HADAMARD),
])
def test_read(D, B, H, W, lens, start, n, flags, fp32):
    c = cfg_of(D, B, H, H, 7, W, max(lens) + 2, flags | (K.FLAG_OUT_FP32 if fp32 else 0), layers=2)
    assert B * n * H >= 1024
    cache, RK, RV, _, _ = filled(c, lens, 3 * D + n, layer=1)
    kind = torch.float32 if fp32 else torch.bfloat16
    # 16-byte aligned outputs that are not 32-byte aligned
    store = [torch.full((B * n * H * D + 8,), 7.0, dtype=kind, device="cuda") for _ in range(2)]
    skip = 4 if fp32 else 8
    kv = [s[skip:skip + B * n * H * D].view(B, n, H, D) for s in store]
    rots = (None, None) if flags & K.FLAG_HADAMARD else (dev_rot(RK), dev_rot(RV))
    st, cdev = dev_i32([0]), torch.from_numpy(cache).cuda()
    K.kv_read(kcfg(c), cdev, 1, dev_i32(start), dev_i32(lens), *rots, kv[0], kv[1], status=st)
    whole = [torch.full((B, n, H, D), 7.0, dtype=kind, device="cuda") for _ in range(2)]
    K.kv_read(kcfg(c), cdev, 1, dev_i32(start), dev_i32(lens), *rots, whole[0], whole[1])
    torch.cuda.synchronize()
    seven = np.full((B, n, H, D), 7.0)
    want = R.read(c, cache, 1, start, lens, n, RK, RV, seven, seven)
    for role in (0, 1):
        assert torch.equal(kv[role], whole[role])
        size = np.linalg.norm(want[role], axis=-1)
        # Float32: D products and sums per element, the matrix and the rows as two fp16 values (2^-21 of a product
        # each; an INT2 row's middle and steps add up to at most three times the row).  bf16: the matrix and the rows in
        # one (2^-11 each, on a middle and steps of up to three times the row), and the output's rounding.
        bound = (4 * D * 2.0 ** -24 + 6 * 2.0 ** -21 if fp32 else 6 * 2.0 ** -11 + 2.0 ** -8) * size + 1e-30
        R.check_rows("kv"[role], kv[role].float().cpu().numpy().astype(np.float64), want[role], bound)
        assert (store[role][:skip] == 7).all() and (store[role][skip + B * n * H * D:] == 7).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("fp32", [True, False], ids=["fp32", "bf16"])
@pytest.mark.parametrize("D,Hq,Hkv,lens,n,q_lens,flags", [
    (128, 16, 2, [300, 210], 70, [70, 33], 0),
    (128, 8, 8, [200, 140], 130, None, K.FLAG_IN_FP32 | K.FLAG_LLOYD_MAX),
    (128, 12, 4, [150, 64], 64, None, K.FLAG_HADAMARD | K.FLAG_V_BF16),
    (128, 16, 2, [150, 64], 64, None, K.FLAG_ABSORB_V),
    (256, 8, 2, [200, 90], 80, [80, 0], 0),
    (512, 8, 1, [170, 140], 70, None, K.FLAG_IN_FP32),
])
def test_extend(D, Hq, Hkv, lens, n, q_lens, flags, fp32):
    B = 2
    c = cfg_of(D, B, Hq, Hkv, 5, 32, max(lens) + 3, flags | (K.FLAG_OUT_FP32 if fp32 else 0))
    assert B * n * Hq >= 1024
    cache, RK, RV, ch, rng = filled(c, lens, D + n)
    q = S.activations(rng, (B, n, Hq, D), ch, mag=3.0)
    if not flags & K.FLAG_IN_FP32:
        q = S.to_bf16_values(q)
    ql = [n] * B if q_lens is None else q_lens
    qdev = dev(q, torch.float32 if flags & K.FLAG_IN_FP32 else torch.bfloat16)
    for b in range(B):
        qdev[b, ql[b]:] = float("nan")
    out = torch.full((B, n, Hq, D), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    lse = torch.full((B, n, Hq), 7.0, device="cuda")
    kc, st = kcfg(c), dev_i32([0])
    ws = torch.full((K.attn_extend_workspace_bytes(kc, n),), 0xFF, dtype=torch.uint8, device="cuda")
    rots = (None, None) if flags & K.FLAG_HADAMARD else (dev_rot(RK), dev_rot(RV))
    K.attn_extend(kc, torch.from_numpy(cache).cuda(), 0, qdev, dev_i32(lens), *rots, out, ws,
                  q_lens=None if q_lens is None else dev_i32(q_lens), lse=lse, status=st)
    torch.cuda.synchronize()
    want, wlse, ob, lb = R.extend(c, cache, 0, q, ql, lens, RK, RV, 1 / math.sqrt(D), np.full(q.shape, 7.0),
                                  np.full(q.shape[:3], 7.0), fp32)
    if not fp32:
        # the merged rows and the matrix of the un-rotation in fp16: 2^-11 each
        ob = ob + 2 * 2.0 ** -11 * np.linalg.norm(want, axis=-1)
    else:
        ob = ob + 6 * 2.0 ** -21 * np.linalg.norm(want, axis=-1)
    R.check_rows("out", out.float().cpu().numpy().astype(np.float64), want, ob)
    R.check_lse(lse.cpu().numpy().astype(np.float64), wlse, lb)
    assert int(st.item()) == 0


def test_non_finite_query_rows_are_flagged_and_stay_alone():
    c = cfg_of(128, 1, 16, 2, 5, 32, 300)
    cache, RK, RV, ch, rng = filled(c, [300], 4)
    q = dev(S.activations(rng, (1, 80, 16, 128), ch), torch.bfloat16)
    kc, cdev, rk, rv = kcfg(c), torch.from_numpy(cache).cuda(), dev_rot(RK), dev_rot(RV)
    ws = torch.empty(K.attn_extend_workspace_bytes(kc, 80), dtype=torch.uint8, device="cuda")
    res = []
    for bad in (False, True):
        if bad:
            q[0, 40, 3, 7] = float("inf")
        out, st = torch.empty(1, 80, 16, 128, dtype=torch.bfloat16, device="cuda"), dev_i32([0])
        K.attn_extend(kc, cdev, 0, q, dev_i32([300]), rk, rv, out, ws, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == (K.DEV_NONFINITE if bad else 0)
        res.append(out)
    assert res[1][0, 40, 3].isnan().all()
    res[1][0, 40, 3] = res[0][0, 40, 3]
    assert torch.equal(res[0], res[1])
