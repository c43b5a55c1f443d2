"""attn_extend and attn_decode_prefix on configurations drawn from seeds, against
the bounds of rows_bounds.py: head_dims, shared heads, windows, modes, lengths,
split counts, and keys, values and queries of sizes far from one.
OSCAR_ROWS_SEEDS=a-b widens it for a stress run."""
import math
import os

import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from oracle import oscar_oracle as O
from tests import rows_bounds as B
from tests.gpu_helpers import dev, dev_i32, dev_rot, kcfg
from tests.test_gpu_rows_accuracy import check

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]
A, Z = (int(x) for x in os.environ.get("OSCAR_ROWS_SEEDS", "0-24").split("-"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def fill(c, rng, lens, ksize, vsize):
    eye, top = np.eye(c.head_dim, dtype=np.float32), max(1, max(lens))
    shape = (c.batch, top, c.num_kv_heads, c.head_dim)
    k, v = (S.to_bf16_values(s * rng.standard_normal(shape)) for s in (ksize, vsize))
    cache = np.full(O.layout(c)["total_bytes"], 0xFF, np.uint8)
    O.append(c, cache, 0, k, v, [n - top for n in lens], eye, eye)
    return cache


@pytest.mark.parametrize("seed", range(A, Z))
def test_extend(seed):
    rng = np.random.default_rng(seed)
    D, flags = int(rng.choice([128, 128, 256, 512])), int(rng.choice([0, 0, K.FLAG_LLOYD_MAX, K.FLAG_V_BF16]))
    H, G, batch = int(rng.integers(1, 4)), int(rng.integers(1, 9)), int(rng.integers(1, 4))
    T, n = int(2 ** rng.uniform(0, 9.5)), int(2 ** rng.uniform(0, 6.5))
    lens = [T] + [int(rng.integers(1, T + 1)) for _ in range(batch - 1)]
    ksize, vsize = 10.0 ** rng.uniform(-5, 3), 10.0 ** rng.uniform(-4, 3)
    c = O.Config(1, batch, H * G, H, D, int(rng.integers(0, 70)), int(rng.integers(0, 300)), T + int(rng.integers(0, 9)), 0.96, 0.92, flags)
    cache = fill(c, rng, lens, ksize, vsize)
    n = min(n, c.capacity)
    # scores of some 4; every query row of a size of its own, which the softmax scale makes up for on the average
    q = S.to_bf16_values(4 / ksize * 2.0 ** rng.uniform(-2, 2, (batch, n, H * G, 1)) * rng.standard_normal((batch, n, H * G, D)))
    kc, eye, splits = kcfg(c), dev_rot(np.eye(D, dtype=np.float32)), int(rng.choice([0, 0, 1, 3]))
    out = torch.empty(batch, n, H * G, D, dtype=torch.bfloat16, device="cuda")
    lse, st = torch.empty(batch, n, H * G, device="cuda"), dev_i32([0])
    ws = torch.empty(max(K.attn_extend_workspace_bytes(kc, n), 16 * batch * n * H * G * (D + 64) + 4096), dtype=torch.uint8, device="cuda")
    K.attn_extend(kc, torch.from_numpy(cache).cuda(), 0, dev(q), dev_i32(lens), eye, eye, out, ws, lse=lse, num_splits=splits, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == (K.DEV_EMPTY if min(lens) < n else 0)
    lm = bool(flags & K.FLAG_LLOYD_MAX)
    for b in range(batch):
        t0 = max(0, n - lens[b])  # tokens before the first position
        assert (out[b, :t0] == 0).all() and torch.isneginf(lse[b, :t0]).all()
        hidden = np.arange(lens[b])[None, :] > (lens[b] - n + np.arange(t0, n))[:, None]
        for h in range(H * G):
            mid, steps, _, factor = B.pieces(c, cache, 0, b, h // G, lens[b])
            V, floor = B.values(c, cache, 0, b, h // G, lens[b])
            want, wlse, ob, lb = B.attend(q[b, t0:, h].astype(np.float64), mid, steps, factor, V, floor, hidden, D ** -0.5, lm)
            check("lse", lse[b, t0:, h].double().cpu().numpy(), wlse, lb)
            check("out", out[b, t0:, h].double().cpu().numpy(), want, ob)


@pytest.mark.parametrize("seed", range(A, Z))
def test_prefix(seed):
    rng = np.random.default_rng(10 ** 6 + seed)
    D, flags = int(rng.choice([128, 128, 256, 512])), int(rng.choice([0, 0, K.FLAG_LLOYD_MAX, K.FLAG_V_BF16]))
    H, G, batch = int(rng.integers(1, 4)), int(rng.integers(1, 9)), int(2 ** rng.uniform(0, 5))
    P, T = int(2 ** rng.uniform(0, 9.5)), int(2 ** rng.uniform(0, 8))
    lens = [T] + [int(rng.integers(0, T + 1)) for _ in range(batch - 1)]
    ksize, vsize = 10.0 ** rng.uniform(-5, 3), 10.0 ** rng.uniform(-4, 3)
    window = lambda: (int(rng.integers(0, 70)), int(rng.integers(0, 300)))
    c, pc = (O.Config(1, b, H * G, H, D, *window(), cap, 0.96, 0.92, flags) for b, cap in ((batch, T + 2), (1, P + 3)))
    cache, pcache = fill(c, rng, lens, ksize, vsize), fill(pc, rng, [P], ksize, vsize)
    q = S.to_bf16_values(4 / ksize * 2.0 ** rng.uniform(-2, 2, (batch, H * G, 1)) * rng.standard_normal((batch, H * G, D)))
    kc, pk, eye = kcfg(c), kcfg(pc), dev_rot(np.eye(D, dtype=np.float32))
    out, lse = torch.empty(batch, H * G, D, dtype=torch.bfloat16, device="cuda"), torch.empty(batch, H * G, device="cuda")
    st = dev_i32([0])
    ws = torch.empty(K.attn_decode_prefix_workspace_bytes(kc, pk), dtype=torch.uint8, device="cuda")
    K.attn_decode_prefix(kc, torch.from_numpy(cache).cuda(), pk, torch.from_numpy(pcache).cuda(), 0, dev(q), dev_i32(lens), dev_i32([P]),
                         eye, eye, out, ws, lse=lse, num_splits=int(rng.choice([0, 0, 2, 7])), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    lm, got, glse = bool(flags & K.FLAG_LLOYD_MAX), out.double().cpu().numpy(), lse.double().cpu().numpy()
    for h in range(H * G):
        pre = B.pieces(pc, pcache, 0, 0, h // G, P)
        pv = B.values(pc, pcache, 0, 0, h // G, P)
        for b in range(batch):
            parts, rows = [pre], [pv]
            if lens[b]:
                parts.append(B.pieces(c, cache, 0, b, h // G, lens[b]))
                rows.append(B.values(c, cache, 0, b, h // G, lens[b]))
            mid, steps, factor = (np.concatenate([x[i] for x in parts]) for i in (0, 1, 3))
            V, floor = (np.concatenate(x) for x in zip(*rows))
            want, wlse, ob, lb = B.attend(q[b, h:h + 1].astype(np.float64), mid, steps, factor, V, floor,
                                          np.zeros((1, len(mid)), bool), D ** -0.5, lm)
            check("lse", glse[b, h:h + 1], wlse, lb)
            check("out", got[b, h:h + 1], want, ob)
