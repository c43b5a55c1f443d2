"""kv_read and attn_extend against their 64-bit forms over the oracle's cached
rows: head_dims, shared heads, windows of zero and of the whole sequence, ragged
lengths and query counts (zero and one among them), splits, modes, types; rows
that belong to no token and memory that belongs to no position are garbage."""
import math

import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from oracle import oscar_oracle as O
from tests import rows_ref as R
from tests.gpu_helpers import dev, dev_i32, dev_rot, kcfg

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def filled(c, lens, seed, layer=0):
    """(cache bytes, R_K, R_V): rows [0, lens[b]) appended by the oracle over
    memory full of NaN patterns."""
    rng = np.random.default_rng(seed)
    D, top = c.head_dim, max(1, max(lens))
    RK, RV = S.qr_rotation(rng, D).astype(np.float32), S.qr_rotation(rng, D).astype(np.float32)
    ch = rng.choice(D, 3, replace=False)
    shape = (c.batch, top, c.num_kv_heads, D)
    k, v = (S.to_bf16_values(S.activations(rng, shape, ch, mag=3.0)) for _ in range(2))
    cache = np.full(O.layout(c)["total_bytes"], 0xFF, np.uint8)
    # positions below zero are not stored: every sequence ends at its own length
    O.append(c, cache, layer, k, v, [n - top for n in lens], RK, RV)
    return cache, RK, RV, ch, rng


def cfg_of(D, B, Hq, Hkv, S_, W, cap, flags=0, layers=1):
    return O.Config(layers, B, Hq, Hkv, D, S_, W, cap, 0.96, 0.92, flags)


EXTEND = [
    # D, B, Hq, Hkv, S, W, lens, n, q_lens, flags, splits
    (128, 1, 4, 1, 4, 8, [1], 1, None, 0, 0),                                   # one position
    (128, 3, 8, 2, 4, 8, [300, 5, 77], 5, [5, 5, 3], 0, 0),
    (128, 2, 8, 8, 16, 32, [200, 130], 7, None, 0, 1),                          # a KV head per query head
    (128, 2, 6, 2, 0, 0, [129, 128], 33, None, 0, 0),                           # no windows; G = 3
    (128, 1, 8, 1, 64, 256, [250], 250, None, 0, 0),                            # windows hold everything; G = 8
    (128, 4, 10, 2, 8, 16, [40, 0, 7, 1], 6, [6, 2, 0, 6], 0, 0),               # empty rows, no tokens, q_len > length
    (128, 1, 14, 2, 5, 100, [700], 129, None, 0, 3),                            # G = 7; odd sizes
    (128, 2, 8, 2, 4, 8, [600, 513], 150, [150, 1], K.FLAG_LLOYD_MAX, 0),
    (128, 2, 8, 2, 4, 8, [300, 64], 20, None, K.FLAG_V_BF16, 0),
    (128, 2, 4, 1, 4, 8, [260, 64], 20, None, K.FLAG_V_BF16 | K.FLAG_LLOYD_MAX, 5),
    (128, 2, 8, 2, 4, 8, [300, 64], 20, None, K.FLAG_HADAMARD, 0),
    (128, 2, 8, 2, 4, 8, [300, 64], 9, None, K.FLAG_ABSORB_V | K.FLAG_IN_FP32, 2),
    (256, 2, 8, 4, 16, 32, [500, 90], 11, None, 0, 0),
    (256, 1, 5, 1, 3, 64, [333], 200, None, K.FLAG_LLOYD_MAX, 2),
    (256, 1, 4, 2, 0, 64, [200], 3, None, K.FLAG_V_BF16 | K.FLAG_HADAMARD, 0),
    (512, 2, 4, 2, 16, 32, [260, 33], 9, None, 0, 0),
    (512, 1, 8, 1, 4, 40, [400], 50, None, K.FLAG_LLOYD_MAX, 3),
    (512, 1, 6, 2, 4, 40, [150], 40, None, K.FLAG_V_BF16, 0),
]


@pytest.mark.parametrize("fp32", [True, False], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", EXTEND, ids=lambda x: "-".join(map(str, x[:6])) + f"-{x[9]}-{x[10]}")
def test_extend(case, fp32):
    D, B, Hq, Hkv, S_, W, lens, n, q_lens, flags, splits = case
    c = cfg_of(D, B, Hq, Hkv, S_, W, max(lens) + 3, flags | (K.FLAG_OUT_FP32 if fp32 else 0), layers=2)
    cache, RK, RV, ch, rng = filled(c, lens, 11 * D + n, layer=1)
    q = S.activations(rng, (B, n, Hq, D), ch, mag=3.0)
    if not flags & K.FLAG_IN_FP32:
        q = S.to_bf16_values(q)
    ql = [n] * B if q_lens is None else q_lens
    qdev = dev(q, torch.float32 if flags & K.FLAG_IN_FP32 else torch.bfloat16)
    for b in range(B):
        qdev[b, max(0, ql[b]):] = float("nan")  # rows of no token are not read
    kind = torch.float32 if fp32 else torch.bfloat16
    out = torch.full((B, n, Hq, D), 7.0, dtype=kind, device="cuda")
    lse = torch.full((B, n, Hq), 7.0, device="cuda")
    kc, st = kcfg(c), dev_i32([0])
    rows = B * n * Hq
    al = lambda x: (x + 255) // 256 * 256
    size = al(rows * D * 4) + al(rows * splits * D * 4) + al(rows * splits * 8) if splits else \
        K.attn_extend_workspace_bytes(kc, n)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    rots = (None, None) if flags & K.FLAG_HADAMARD else (dev_rot(RK), dev_rot(RV))
    cdev = torch.from_numpy(cache).cuda()
    args = (kc, cdev, 1, qdev, dev_i32(lens), *rots, out, ws)
    kw = dict(q_lens=None if q_lens is None else dev_i32(q_lens), lse=lse, seq_len_hint=max(lens), num_splits=splits,
              status=st)
    K.attn_extend(*args, **kw)
    torch.cuda.synchronize()
    want, wlse, ob, lb = R.extend(c, cache, 1, q, ql, lens, RK, RV, 1 / math.sqrt(D), np.full(q.shape, 7.0),
                                  np.full(q.shape[:3], 7.0), fp32)
    first = out.clone(), lse.clone()
    R.check_rows("out", out.float().cpu().numpy().astype(np.float64), want, ob)
    R.check_lse(lse.cpu().numpy().astype(np.float64), wlse, lb)
    empty = any(T - m + t < 0 for T, m in zip(lens, ql) for t in range(min(m, n)))
    assert int(st.item()) == (K.DEV_EMPTY if empty else 0)
    assert np.array_equal(cdev.cpu().numpy(), cache)
    K.attn_extend(*args, **kw)  # the same bits again
    torch.cuda.synchronize()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)


@pytest.mark.parametrize("fp32", [True, False], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", [
    # D, B, Hkv, S, W, lens, start, n, flags
    (128, 1, 1, 4, 8, [1], [0], 1, 0),
    (128, 3, 3, 4, 8, [300, 5, 77], [0, -2, 70], 301, 0),
    (128, 2, 2, 0, 0, [130, 64], [3, 63], 40, 0),
    (128, 2, 8, 64, 256, [200, 321], [0, 0], 321, K.FLAG_HADAMARD),
    (128, 2, 2, 4, 16, [300, 0], [17, 0], 283, K.FLAG_LLOYD_MAX),
    (128, 2, 2, 4, 16, [200, 40], [0, 0], 210, K.FLAG_V_BF16 | K.FLAG_ABSORB_V),
    (256, 2, 3, 7, 31, [257, 90], [0, 20], 257, 0),
    (256, 1, 2, 7, 31, [150], [1], 140, K.FLAG_LLOYD_MAX | K.FLAG_V_BF16),
    (512, 2, 2, 16, 32, [140, 33], [2, 0], 130, 0),
    (512, 1, 1, 3, 5, [70], [0], 70, K.FLAG_HADAMARD | K.FLAG_LLOYD_MAX),
], ids=lambda x: "-".join(map(str, x[:5])) + f"-{x[8]}")
def test_read(case, fp32):
    D, B, H, S_, W, lens, start, n, flags = case
    c = cfg_of(D, B, H, H, S_, W, max(lens) + 2, flags | (K.FLAG_OUT_FP32 if fp32 else 0), layers=2)
    cache, RK, RV, _, _ = filled(c, lens, 7 * D + n, layer=1)
    kind = torch.float32 if fp32 else torch.bfloat16
    kv = [torch.full((B, n, H, D), 7.0, dtype=kind, device="cuda") for _ in range(2)]
    rots = (None, None) if flags & K.FLAG_HADAMARD else (dev_rot(RK), dev_rot(RV))
    st = dev_i32([0])
    cdev = torch.from_numpy(cache).cuda()
    K.kv_read(kcfg(c), cdev, 1, dev_i32(start), dev_i32(lens), *rots, kv[0], kv[1], status=st)
    torch.cuda.synchronize()
    seven = np.full((B, n, H, D), 7.0)
    want = R.read(c, cache, 1, start, lens, n, RK, RV, seven, seven)
    for role in (0, 1):
        size = np.linalg.norm(want[role], axis=-1)
        # D float32 products and sums per element (as sums over a row: the norm of x' is that of the result),
        # and the rounding of the output
        bound = (4 * D * 2.0 ** -24 + (0 if fp32 else 2.0 ** -8)) * size + 1e-30
        R.check_rows("kv"[role], kv[role].float().cpu().numpy().astype(np.float64), want[role], bound)
    assert int(st.item()) == 0
    # one role alone
    alone = torch.full_like(kv[1], 7.0)
    K.kv_read(kcfg(c), cdev, 1, dev_i32(start), dev_i32(lens), *rots, None, alone)
    assert torch.equal(alone, kv[1])


def test_read_clamps_a_length_above_capacity():
    c = cfg_of(128, 1, 2, 2, 4, 8, 40, K.FLAG_OUT_FP32)
    cache, RK, RV, _, _ = filled(c, [40], 3)
    cdev, st = torch.from_numpy(cache).cuda(), dev_i32([0])
    k = [torch.full((1, 40, 2, 128), 7.0, device="cuda") for _ in range(2)]
    K.kv_read(kcfg(c), cdev, 0, dev_i32([10]), dev_i32([40]), dev_rot(RK), dev_rot(RV), k[0])
    K.kv_read(kcfg(c), cdev, 0, dev_i32([10]), dev_i32([4000]), dev_rot(RK), dev_rot(RV), k[1], status=st)
    assert torch.equal(k[0], k[1]) and int(st.item()) == K.DEV_OVER_CAPACITY
    assert (k[0][:, 30:] == 7).all()


@pytest.mark.parametrize("fp32", [True, False], ids=["fp32", "bf16"])
@pytest.mark.parametrize("D", [128, 256, 512])
def test_extend_hidden_rows_may_hold_anything(D, fp32):
    """A token does not see later positions, whatever their rows hold: with NaN
    and infinities in the rows of the last positions, earlier tokens' results
    stay as they were, bit for bit, and the tokens that see them get NaN."""
    c = cfg_of(D, 1, 4, 2, 2, 6, 64, K.FLAG_OUT_FP32 if fp32 else 0)
    cache, RK, RV, ch, rng = filled(c, [50], 5)
    q = dev(S.activations(rng, (1, 12, 4, D), ch), torch.bfloat16)
    bad = cache.copy()
    for role, value in ((0, 0x7F80), (1, 0x7FC0)):  # +inf in K, NaN in V, at positions 46 and 47 (ring)
        view = O.CacheView(c, bad, 0, role)
        view.ring[0, :, 46 % 6, 5] = value
        view.ring[0, :, 47 % 6, :] = value
    res = []
    for x in (cache, bad):
        out = torch.empty(1, 12, 4, D, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        lse = torch.empty(1, 12, 4, device="cuda")
        ws = torch.empty(K.attn_extend_workspace_bytes(kcfg(c), 12), dtype=torch.uint8, device="cuda")
        K.attn_extend(kcfg(c), torch.from_numpy(x).cuda(), 0, q, dev_i32([50]), dev_rot(RK), dev_rot(RV), out, ws, lse=lse)
        torch.cuda.synchronize()
        res.append((out.cpu(), lse.cpu()))
    # tokens sit at positions 38 .. 49
    assert torch.equal(res[0][0][:, :8], res[1][0][:, :8]) and torch.equal(res[0][1][:, :8], res[1][1][:, :8])
    assert torch.isfinite(res[0][0].float()).all()
    assert res[1][0][:, 9:].isnan().any(-1).all()


def test_extend_values_beyond_fp16():
    """BF16 rows may be far outside the fp16 range: outputs scale with the values."""
    for power in (-40, 20, 60):
        c = cfg_of(128, 1, 4, 2, 8, 64, 64)
        cache, RK, RV, ch, rng = filled(c, [50], 9)
        q = dev(S.activations(rng, (1, 5, 4, 128), ch), torch.bfloat16)
        eye = torch.eye(128, device="cuda")
        res = []
        for p in (0, power):
            x = cache.copy()
            for part in (O.CacheView(c, x, 0, 1).sink, O.CacheView(c, x, 0, 1).ring):
                part[...] = O.f32_to_bf16_bits(O.bf16_bits_to_f32(part) * np.float32(2.0 ** p))
            out = torch.empty(1, 5, 4, 128, dtype=torch.bfloat16, device="cuda")
            ws = torch.empty(K.attn_extend_workspace_bytes(kcfg(c), 5), dtype=torch.uint8, device="cuda")
            K.attn_extend(kcfg(c), torch.from_numpy(x).cuda(), 0, q, dev_i32([50]), eye, eye, out, ws)
            torch.cuda.synchronize()
            res.append(out.double().cpu() * 2.0 ** -p)
        # The rows' power of two joins the scores' exponents before they are rounded to float32 (|score + power| < 2^7:
        # off by 2^-18, which moves a probability by less than 2^-17 of itself) and moves the reference of the
        # probabilities, so either result has fp16 roundings of its own: 2^-12 of each probability, 2 * 2^-12 of the
        # largest value between the two.  Then one bf16 rounding each (2^-8).
        vmax = float(np.abs(np.concatenate([O.dequant_history(c, cache, 0, 1, 0, h, 50) for h in range(2)])).max())
        lim = 2 * 2.0 ** -8 * res[0].abs() + (2.0 ** -11 + 2 * 2.0 ** -17) * vmax
        assert ((res[0] - res[1]).abs() <= lim).all(), power


@pytest.mark.parametrize("fp32", [True, False], ids=["fp32", "bf16"])
def test_extend_of_one_token_is_decode(fp32):
    """n_new = 1 computes what attn_decode computes."""
    c = cfg_of(128, 3, 16, 4, 16, 64, 1500, K.FLAG_OUT_FP32 if fp32 else 0)
    lens = [1500, 3, 700]
    cache, RK, RV, ch, rng = filled(c, lens, 17)
    q = dev(S.activations(rng, (3, 1, 16, 128), ch), torch.bfloat16)
    kc, cdev, rk, rv = kcfg(c), torch.from_numpy(cache).cuda(), dev_rot(RK), dev_rot(RV)
    kind = torch.float32 if fp32 else torch.bfloat16
    a, b = (torch.empty(3, 1, 16, 128, dtype=kind, device="cuda") for _ in range(2))
    la, lb = (torch.empty(3, 1, 16, device="cuda") for _ in range(2))
    ws = torch.empty(max(K.attn_extend_workspace_bytes(kc, 1), K.layout_query(kc)["decode_workspace_bytes"]),
                     dtype=torch.uint8, device="cuda")
    K.attn_extend(kc, cdev, 0, q, dev_i32(lens), rk, rv, a, ws, lse=la)
    K.attn_decode(kc, cdev, 0, q[:, 0], dev_i32(lens), rk, rv, b[:, 0], ws, lse=lb)
    torch.cuda.synchronize()
    # both are within their own bounds of the exact result; outputs are of order one
    assert (a.double() - b.double()).norm() <= (2e-4 if fp32 else 8e-3) * b.double().norm()
    # log-sum-exps reach 150 here: each side is within the bound of its scores' float32 sums (rows_ref.score_error)
    x = q.float().cpu().numpy()
    lim = 2 * R.extend(c, cache, 0, x, [1] * 3, lens, RK, RV, 1 / math.sqrt(128), x, x[..., 0], fp32)[3]
    assert (np.abs((la - lb).double().cpu().numpy()) <= lim + 8 * 2.0 ** -24 * la.abs().cpu().numpy()).all()


def test_extend_splits_agree_and_graphs_replay():
    c = cfg_of(128, 2, 8, 2, 16, 64, 2000)
    lens = [1999, 1500]
    cache, RK, RV, ch, rng = filled(c, lens, 23)
    q = dev(S.activations(rng, (2, 24, 8, 128), ch), torch.bfloat16)
    kc, cdev, rk, rv, sl = kcfg(c), torch.from_numpy(cache).cuda(), dev_rot(RK), dev_rot(RV), dev_i32(lens)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    outs = []
    for splits in (0, 1, 2, 13, 64):
        out = torch.empty(2, 24, 8, 128, dtype=torch.bfloat16, device="cuda")
        K.attn_extend(kc, cdev, 0, q, sl, rk, rv, out, ws, num_splits=splits)
        outs.append(out)
    torch.cuda.synchronize()
    for o in outs[1:]:  # two bf16 roundings of results that differ by the fp16 roundings
        assert (o.double() - outs[0].double()).norm() <= (2 * 2.0 ** -8 + 4 * 2.0 ** -11) * outs[0].double().norm()
    # captured on a side stream, replayed twice with another query in the same buffer
    q2 = dev(S.activations(rng, (2, 24, 8, 128), ch), torch.bfloat16)
    want = torch.empty_like(outs[0])
    K.attn_extend(kc, cdev, 0, q2, sl, rk, rv, want, ws)
    out, qg = torch.empty_like(want), q.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.attn_extend(kc, cdev, 0, qg, sl, rk, rv, out, ws)
    qg.copy_(q2)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
