"""attn_extend and attn_decode_prefix with a bf16 output against bounds that follow
their arithmetic (rows_bounds.py), tight enough that a part left out would show;
and the accuracy that the header states."""
import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from oracle import oscar_oracle as O
from tests import rows_bounds as B
from tests.gpu_helpers import dev, dev_i32, dev_rot, kcfg

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def inputs(D, batch, T, n, flags, seed=0):
    """A cache of normal rows without rotations and queries that give scores of some 5."""
    c = O.Config(1, batch, 8, 2, D, 4, 40, T, 0.96, 0.92, flags)
    rng = np.random.default_rng(1000 * seed + D + T)
    eye = np.eye(D, dtype=np.float32)
    k, v, q = (S.to_bf16_values(2.2 * rng.standard_normal(s)) for s in ((batch, T, 2, D), (batch, T, 2, D), (batch, n, 8, D)))
    cache = O.new_cache(c)
    O.append(c, cache, 0, k, v, [0] * batch, eye, eye)
    return c, cache, q


def check(name, got, want, bound):
    err = np.abs(got - want)
    assert (err <= bound).all(), f"{name}: {(err / bound).max():.2f} of the bound at {np.unravel_index((err / bound).argmax(), err.shape)}"


@pytest.mark.parametrize("D,n,T,flags", [
    (128, 3, 500, 0), (128, 40, 300, 0), (128, 90, 1000, 0), (256, 40, 300, 0), (512, 3, 300, 0), (512, 40, 300, 0),
    (128, 3, 500, K.FLAG_LLOYD_MAX), (128, 90, 300, K.FLAG_LLOYD_MAX), (256, 3, 300, K.FLAG_LLOYD_MAX),
    (512, 40, 300, K.FLAG_LLOYD_MAX), (128, 90, 300, K.FLAG_V_BF16), (512, 40, 300, K.FLAG_V_BF16),
])
def test_extend(D, n, T, flags):
    c, cache, q = inputs(D, 1, T, n, flags)
    kc, eye = kcfg(c), dev_rot(np.eye(D, dtype=np.float32))
    out, lse = torch.empty(1, n, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, 8, device="cuda")
    ws = torch.empty(K.attn_extend_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
    K.attn_extend(kc, torch.from_numpy(cache).cuda(), 0, dev(q), dev_i32([T]), eye, eye, out, ws, lse=lse)
    torch.cuda.synchronize()
    hidden = np.arange(T)[None, :] > (T - n + np.arange(n))[:, None]
    lm = bool(flags & K.FLAG_LLOYD_MAX)
    for h in range(8):
        mid, steps, _, factor = B.pieces(c, cache, 0, 0, h // 4, T)
        V, floor = B.values(c, cache, 0, 0, h // 4, T)
        want, wlse, ob, lb = B.attend(q[0, :, h].astype(np.float64), mid, steps, factor, V, floor, hidden, D ** -0.5, lm)
        check("lse", lse[0, :, h].double().cpu().numpy(), wlse, lb)
        check("out", out[0, :, h].double().cpu().numpy(), want, ob)


@pytest.mark.parametrize("D,batch,flags", [(128, 3, 0), (128, 20, 0), (256, 12, K.FLAG_LLOYD_MAX), (512, 3, 0), (128, 20, K.FLAG_V_BF16)])
def test_prefix(D, batch, flags):
    P, T = 400, 150
    pc, pcache, _ = inputs(D, 1, P, 1, flags, seed=1)
    c, cache, q = inputs(D, batch, T, 1, flags)
    kc, pk, eye = kcfg(c), kcfg(pc), dev_rot(np.eye(D, dtype=np.float32))
    lens = [1 + (37 * b) % T for b in range(batch)]
    out, lse = torch.empty(batch, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(batch, 8, device="cuda")
    ws = torch.empty(K.attn_decode_prefix_workspace_bytes(kc, pk), dtype=torch.uint8, device="cuda")
    K.attn_decode_prefix(kc, torch.from_numpy(cache).cuda(), pk, torch.from_numpy(pcache).cuda(), 0, dev(q[:, 0]), dev_i32(lens),
                         dev_i32([P]), eye, eye, out, ws, lse=lse)
    torch.cuda.synchronize()
    lm = bool(flags & K.FLAG_LLOYD_MAX)
    for b in range(batch):
        for h in range(8):
            parts = [B.pieces(pc, pcache, 0, 0, h // 4, P), B.pieces(c, cache, 0, b, h // 4, lens[b])]
            mid, steps, factor = (np.concatenate([x[i] for x in parts]) for i in (0, 1, 3))
            V, floor = (np.concatenate(x) for x in zip(B.values(pc, pcache, 0, 0, h // 4, P), B.values(c, cache, 0, b, h // 4, lens[b])))
            want, wlse, ob, lb = B.attend(q[b, :, h].astype(np.float64), mid, steps, factor, V, floor,
                                          np.zeros((1, P + lens[b]), bool), D ** -0.5, lm)
            check("lse", lse[b, h].double().cpu().numpy(), wlse[0], lb[0])
            check("out", out[b, h].double().cpu().numpy(), want[0], ob[0])
