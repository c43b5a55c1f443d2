"""attn_decode_prefix against its 64-bit form: a prefix shared by the batch and
every sequence's own cache, with either of them empty, the windows of each its
own, every mode and head_dim; then a run of append, extend, prefix decode and
read together."""
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


def refill(c, lens, RK, RV, seed):
    """A second cache with the first one's rotations."""
    rng = np.random.default_rng(seed)
    top = max(1, max(lens))
    k, v = (S.to_bf16_values(S.activations(rng, (c.batch, top, c.num_kv_heads, c.head_dim), [3, 50], mag=3.0))
            for _ in range(2))
    cache = np.full(O.layout(c)["total_bytes"], 0xFF, np.uint8)
    O.append(c, cache, 0, k, v, [n - top for n in lens], RK, RV)
    return cache


@pytest.mark.parametrize("fp32", [True, False], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", [
    # D, B, Hq, Hkv, (S, W) own, (S, W) prefix, lens, prefix, flags, splits
    (128, 2, 8, 2, (4, 8), (4, 8), [30, 1], 200, 0, 0),
    (128, 1, 4, 1, (0, 8), (64, 256), [3], 1, 0, 0),                       # a prefix of one
    (128, 3, 6, 2, (0, 0), (4, 16), [40, 0, 129], 130, 0, 3),              # a sequence with nothing of its own
    (128, 3, 8, 2, (4, 8), (4, 8), [40, 0, 9], 0, 0, 0),                   # no prefix: one sequence has nothing
    (128, 33, 8, 2, (2, 4), (4, 8), [5] * 33, 300, 0, 0),                  # more rows than a tile
    (128, 5, 14, 2, (4, 8), (4, 8), [7, 5, 3, 2, 90], 700, K.FLAG_LLOYD_MAX, 0),
    (128, 2, 8, 2, (4, 8), (4, 8), [30, 21], 150, K.FLAG_V_BF16, 0),
    (128, 2, 8, 2, (4, 8), (4, 8), [30, 21], 300, K.FLAG_HADAMARD | K.FLAG_IN_FP32, 2),
    (256, 3, 8, 4, (4, 8), (4, 40), [30, 11, 140], 260, K.FLAG_ABSORB_V, 0),
    (512, 2, 8, 2, (4, 8), (4, 8), [30, 21], 140, 0, 0),
    (512, 2, 8, 1, (4, 8), (4, 8), [30, 21], 200, K.FLAG_LLOYD_MAX, 4),
    # own caches of more than 1024 positions go through attn_decode's kernels
    (128, 3, 8, 2, (4, 64), (4, 8), [1500, 20, 0], 150, 0, 0),
    (128, 2, 16, 2, (4, 64), (4, 8), [1100, 1030], 0, K.FLAG_HADAMARD | K.FLAG_V_BF16, 0),
    (256, 2, 4, 2, (4, 64), (4, 8), [1100, 7], 90, K.FLAG_LLOYD_MAX, 0),
    (128, 600, 16, 2, (0, 4), (4, 8), [2] * 600, 40, 0, 0),                # rows of query beyond 4096
], ids=lambda x: "-".join(map(str, x[:4])) + f"-{x[7]}-{x[8]}-{x[9]}")
def test_prefix(case, fp32):
    D, B, Hq, Hkv, own, pre, lens, plen, flags, splits = case
    flags |= K.FLAG_OUT_FP32 if fp32 else 0
    c = cfg_of(D, B, Hq, Hkv, *own, max(lens) + 3, flags)
    pc = cfg_of(D, 1, Hq, Hkv, *pre, plen + 5, flags)
    cache, RK, RV, ch, rng = filled(c, lens, 5 * D + B)
    pcache = refill(pc, [plen], RK, RV, 99)
    q = S.activations(rng, (B, Hq, D), ch, mag=3.0)
    if not flags & K.FLAG_IN_FP32:
        q = S.to_bf16_values(q)
    kc, pk, st = kcfg(c), kcfg(pc), dev_i32([0])
    out = torch.full((B, Hq, D), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq), 7.0, device="cuda")
    ws = torch.full((K.attn_decode_prefix_workspace_bytes(kc, pk),), 0xFF, dtype=torch.uint8, device="cuda")
    rots = (None, None) if flags & K.FLAG_HADAMARD else (dev_rot(RK), dev_rot(RV))
    args = (kc, torch.from_numpy(cache).cuda(), pk, torch.from_numpy(pcache).cuda(), 0,
            dev(q, torch.float32 if flags & K.FLAG_IN_FP32 else torch.bfloat16), dev_i32(lens), dev_i32([plen]), *rots, out, ws)
    kw = dict(lse=lse, num_splits=splits, status=st)
    K.attn_decode_prefix(*args, **kw)
    torch.cuda.synchronize()
    want, wlse, ob, lb = R.prefix(c, cache, pc, pcache, 0, q, lens, plen, RK, RV, 1 / math.sqrt(D), fp32)
    # the own caches' part runs through attn_decode, whose probabilities are fp16 pairs and whose values are
    # exact codes: 2^-11 covers it
    ob = ob + 2.0 ** -11 * np.linalg.norm(want, axis=-1)
    lb = lb + 1e-4
    R.check_rows("out", out.float().cpu().numpy().astype(np.float64), want, ob)
    R.check_lse(lse.cpu().numpy().astype(np.float64), wlse, lb)
    assert int(st.item()) == (K.DEV_EMPTY if plen == 0 and 0 in lens else 0)
    first = out.clone(), lse.clone()
    K.attn_decode_prefix(*args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)


def test_status_of_both_caches():
    c, pc = cfg_of(128, 2, 4, 2, 4, 8, 30), cfg_of(128, 1, 4, 2, 4, 8, 60)
    cache, RK, RV, ch, rng = filled(c, [30, 20], 1)
    pcache = refill(pc, [60], RK, RV, 2)
    q = dev(S.activations(rng, (2, 4, 128), ch), torch.bfloat16)
    kc, pk = kcfg(c), kcfg(pc)
    ws = torch.empty(K.attn_decode_prefix_workspace_bytes(kc, pk), dtype=torch.uint8, device="cuda")
    res = []
    for lens, plen, want in (([30, 20], 60, 0), ([31, 20], 60, K.DEV_OVER_CAPACITY), ([30, 20], 61, K.DEV_OVER_CAPACITY),
                             ([30, 0], 60, 0)):
        out, st = torch.empty(2, 4, 128, dtype=torch.bfloat16, device="cuda"), dev_i32([0])
        K.attn_decode_prefix(kc, torch.from_numpy(cache).cuda(), pk, torch.from_numpy(pcache).cuda(), 0, q, dev_i32(lens),
                             dev_i32([plen]), dev_rot(RK), dev_rot(RV), out, ws, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == want, (lens, plen)
        res.append(out)
    assert torch.equal(res[0], res[1]) and torch.equal(res[0], res[2])  # clamped to the capacities


def test_a_run_together():
    """A prompt appended and attended in two chunks, then decoded by a batch that
    shares it, each sequence appending its own tokens; at last the rows read back."""
    D, B, Hq, Hkv, P, chunk, steps = 128, 3, 8, 2, 300, 170, 4
    pc, c = cfg_of(D, 1, Hq, Hkv, 8, 32, 320), cfg_of(D, B, Hq, Hkv, 0, 8, 16)
    rng = np.random.default_rng(8)
    RK, RV = S.qr_rotation(rng, D).astype(np.float32), S.qr_rotation(rng, D).astype(np.float32)
    kc, pk, rk, rv = kcfg(c), kcfg(pc), dev_rot(RK), dev_rot(RV)
    pcache = torch.zeros(K.layout_query(pk)["total_bytes"], dtype=torch.uint8, device="cuda")
    cache = torch.zeros(K.layout_query(kc)["total_bytes"], dtype=torch.uint8, device="cuda")
    rows = lambda *s: S.to_bf16_values(S.activations(rng, s, [4, 90], mag=3.0))
    scale = 1 / math.sqrt(D)
    k, v, q = rows(1, P, Hkv, D), rows(1, P, Hkv, D), rows(1, P, Hq, D)
    ws = torch.empty(max(K.attn_extend_workspace_bytes(pk, chunk), K.attn_decode_prefix_workspace_bytes(kc, pk)),
                     dtype=torch.uint8, device="cuda")
    for t0 in range(0, P, chunk):
        t1 = min(P, t0 + chunk)
        K.kv_append(pk, pcache, 0, dev(k[:, t0:t1]), dev(v[:, t0:t1]), dev_i32([t0]), rk, rv)
        out = torch.empty(1, t1 - t0, Hq, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(1, t1 - t0, Hq, device="cuda")
        K.attn_extend(pk, pcache, 0, dev(q[:, t0:t1]), dev_i32([t1]), rk, rv, out, ws, lse=lse)
        torch.cuda.synchronize()
        want, wlse, ob, lb = R.extend(pc, pcache.cpu().numpy(), 0, q[:, t0:t1], [t1 - t0], [t1], RK, RV, scale,
                                      np.zeros(out.shape), np.zeros(lse.shape), False)
        R.check_rows("chunk", out.float().cpu().numpy().astype(np.float64), want, ob)
        R.check_lse(lse.cpu().numpy().astype(np.float64), wlse, lb)
    for t in range(steps):
        K.kv_append(kc, cache, 0, dev(rows(B, 1, Hkv, D)), dev(rows(B, 1, Hkv, D)), dev_i32([t] * B), rk, rv)
        qs = rows(B, Hq, D)
        out, lse = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hq, device="cuda")
        K.attn_decode_prefix(kc, cache, pk, pcache, 0, dev(qs), dev_i32([t + 1] * B), dev_i32([P]), rk, rv, out, ws, lse=lse)
        torch.cuda.synchronize()
        want, wlse, ob, lb = R.prefix(c, cache.cpu().numpy(), pc, pcache.cpu().numpy(), 0, qs, [t + 1] * B, P, RK, RV, scale,
                                      False)
        R.check_rows("step", out.float().cpu().numpy().astype(np.float64), want,
                     ob + 2.0 ** -11 * np.linalg.norm(want, axis=-1))
        R.check_lse(lse.cpu().numpy().astype(np.float64), wlse, lb + 1e-4)
    ko, vo = (torch.empty(1, P, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K.kv_read(pk, pcache, 0, dev_i32([0]), dev_i32([P]), rk, rv, ko, vo)
    torch.cuda.synchronize()
    # the windows come back to the rounding of BF16 rows and outputs
    for got, x in ((ko, k), (vo, v)):
        g = got.double().cpu().numpy()
        for part in (slice(0, 8), slice(P - 32, P)):
            err = np.linalg.norm(g[:, part] - x[:, part], axis=-1)
            assert (err <= 2.05 * 2.0 ** -8 * np.linalg.norm(x[:, part], axis=-1)).all()
