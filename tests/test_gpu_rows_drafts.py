"""Drafted tokens end to end: appended, attended by attn_extend, some refused and
their ring slots put back; the sequences then decode the bits that sequences
give which never saw the refused drafts."""
import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from tests.gpu_helpers import dev, dev_i32, dev_rot, kcfg
from tests.test_gpu_rows import cfg_of, filled

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


@pytest.mark.parametrize("D,flags", [(128, 0), (128, K.FLAG_V_BF16), (256, 0)])
def test_refused_drafts(D, flags):
    lens, n, keep, steps, W = [200, 133], 5, 2, 4, 16
    c = cfg_of(D, 2, 8, 2, 4, W, 220, flags)
    start, RK, RV, ch, rng = filled(c, lens, D)
    kc, R, st = kcfg(c), (dev_rot(RK), dev_rot(RV)), dev_i32([0])
    rows = lambda m, h: dev(S.activations(rng, (2, m, h, D), ch, mag=3.0))
    dk, dv, dq = rows(n, 2), rows(n, 2), rows(n, 8)
    after = [(rows(1, 2), rows(1, 2), rows(1, 8)[:, 0].contiguous()) for _ in range(steps)]
    ws = torch.empty(max(K.attn_extend_workspace_bytes(kc, n), K.layout_query(kc)["decode_workspace_bytes"]), dtype=torch.uint8,
                     device="cuda")
    got = []
    for drafts in (True, False):
        cache = torch.from_numpy(start).cuda()
        if drafts:
            rings = [r for r in K.ring_rows(kc, cache, 0) if r is not None]
            at = torch.tensor(lens, device="cuda")[:, None] + torch.arange(n, device="cuda")
            b, slots = torch.arange(2, device="cuda")[:, None], at % W
            saved = [r[b, :, slots].clone() for r in rings]
            K.kv_append(kc, cache, 0, dk, dv, dev_i32(lens), *R)
            out = torch.empty_like(dq)
            K.attn_extend(kc, cache, 0, dq, dev_i32([t + n for t in lens]), *R, out, ws, status=st)
            for r, s in zip(rings, saved):
                r[b, :, slots[:, keep:]] = s[:, keep:]
        else:
            K.kv_append(kc, cache, 0, dk[:, :keep].contiguous(), dv[:, :keep].contiguous(), dev_i32(lens), *R)
        res = []
        for i, (k, v, q) in enumerate(after):
            pos = [t + keep + i for t in lens]
            K.kv_append(kc, cache, 0, k, v, dev_i32(pos), *R)
            out, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
            K.attn_decode(kc, cache, 0, q, dev_i32([p + 1 for p in pos]), *R, out, ws, lse=lse, status=st)
            res += [out, lse]
        torch.cuda.synchronize()
        got.append(res)
    assert int(st.item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(*got))
