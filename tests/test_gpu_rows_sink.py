"""One dominant position and many weak ones: the weak ones' weights, each below
fp16's smallest number beside the dominant one's, add up and have to stay."""
import math

import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from oracle import oscar_oracle as O
from tests.gpu_helpers import dev_i32, dev_rot, kcfg
from tests.test_gpu_rows import cfg_of

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


@pytest.mark.parametrize("gap", [24, 26, 30])
@pytest.mark.parametrize("D,n,T", [(128, 2, 700), (128, 60, 700), (128, 60, 40000), (128, 2, 40000), (256, 20, 700), (512, 2, 700)])
def test_weak_positions_keep_their_weight(D, n, T, gap):
    """Position 0 scores `gap` ln 2 above all others and has a value row of zero; the others' value rows are ones.  All in
    BF16 rows without rotations, so the result is W / (1 + W) with W = T' 2^-gap, T' the other positions seen."""
    Hq, Hkv = 4, 2
    c = cfg_of(D, 1, Hq, Hkv, 1, T, T, K.FLAG_V_BF16)
    cache = O.new_cache(c)
    key, val = O.CacheView(c, cache, 0, 0), O.CacheView(c, cache, 0, 1)
    bf = lambda x: O.f32_to_bf16_bits(np.float32(x))
    key.sink[...] = 0
    key.sink[..., 0] = bf(gap)
    key.ring[...] = 0
    val.full[...] = bf(1.0)
    val.full[:, :, 0] = 0
    q = torch.zeros(1, n, Hq, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    eye = dev_rot(np.eye(D, dtype=np.float32))
    kc = kcfg(c)
    out, lse = torch.empty_like(q), torch.empty(1, n, Hq, device="cuda")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    for splits in (1, 0):
        K.attn_extend(kc, torch.from_numpy(cache).cuda(), 0, q, dev_i32([T]), eye, eye, out, ws, lse=lse, sm_scale=math.log(2.0),
                      num_splits=splits)
        torch.cuda.synchronize()
        others = T - n + np.arange(n, dtype=np.float64)
        weight = others * 2.0 ** -gap
        want = np.broadcast_to((weight / (1 + weight))[None, :, None, None], out.shape)
        got = out.double().cpu().numpy()
        # Scores: off by 2^-19 of `gap` (float32 products, the scale and the base change) on either end, so a weight by
        # 2^-18 gap.  A weight is at least 2^-30 of the largest, which is 2^8 in fp16, and off by 2^-25 at the most there;
        # one share more or less; the output's rounding.
        rel = gap * 2.0 ** -18 + 2.0 ** -25 / 2.0 ** (8 - gap) + 2.0 ** -8 + 4 * 2.0 ** -11
        assert (np.abs(got - want) <= rel * want).all(), np.abs(got / want - 1).max()
        # The sum is float32.  A share takes one addition per tile of 128 positions to each of its partial sums, every one
        # off by 2^-24 of a sum that the dominant position fills; some 64 more within a tile and between the partial sums.
        top = gap * math.log(2.0)
        lim = 2.0 ** -18 * top + (T / 128 + 64) * 2.0 ** -24
        assert (np.abs(lse.double().cpu().numpy() - (top + np.log1p(weight))[None, :, None]) <= lim).all()
