"""attn_prompt's weights in bf16: what all of a row's weight has in common does not change its output.  The products take the
rounded weights, so the output has to be divided by their sum."""
import math

import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from tests.gpu_helpers import dev_i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def attend(D, q, k, v):
    """One sequence, one KV head: q [T][G][D], k and v [T][1][D]: out and lse."""
    T, G, _ = q.shape
    out, lse = torch.empty_like(q), torch.empty(T, G, device="cuda")
    status = dev_i32([0])
    K.attn_prompt(K.KVConfig(1, 1, G, 1, D, 0, 0, 1), q, k, v, dev_i32([0, T]), out, lse=lse, sm_scale=math.log(2.0), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out, lse


def rows(D, T, heavy):
    """Scores in log2 units are q[t, g, 0] k[p, 0, 0]: 0 at position 0, -8 q elsewhere and q, between 14 and 20, at the heavy
    positions: a growth that the softmax's reference does not follow, so that the heavy weights are not powers of two."""
    g = torch.Generator().manual_seed(D + T)
    q, k = torch.zeros(T, 4, D), torch.zeros(T, 1, D)
    q[:, :, 0] = 14 + 6 * torch.rand(T, 4, generator=g)
    k[:, 0, 0] = -8
    k[0, 0, 0] = 0
    k[heavy, 0, 0] = 1
    v = torch.randint(128, 256, (T, 1, D), generator=g) / 128.0  # [1, 2), exact in bf16
    return (x.bfloat16().cuda() for x in (q, k, v))


@pytest.mark.parametrize("D", [128, 256, 512])
@pytest.mark.parametrize("T,at", [(300, 130), (700, 128), (700, 511)])
def test_a_dominant_weight_leaves_its_value(D, T, at):
    """The weights beside the heavy one are 2^-14 of it in all, so the output is off from its value by 2^-14 before it is
    rounded to bf16: half a step there is 2^-9 of the value at least, so it is that value."""
    q, k, v = rows(D, T, [at])
    out, lse = attend(D, q, k, v)
    assert torch.equal(out[at:], v[at].expand(T - at, 4, D))
    # log2 (2^q + 1 + T 2^-8q): its sum is not that of the rounded weights (2^-9)
    want = q[at:, :, 0].double() + torch.log2(1 + torch.exp2(-q[at:, :, 0].double()))
    assert float((lse[at:].double() / math.log(2.0) - want).abs().max()) < (T + 64) * 2.0 ** -24 + 32 * 2.0 ** -22


@pytest.mark.parametrize("D", [128, 256, 512])
def test_equal_weights_give_the_mean(D):
    """Two, then four heavy positions with values m / 16 in [1, 2): their mean, a multiple of 1 / 64, is a bf16 number, and
    what position 0 adds (2^-14) is far below half a step."""
    T, at = 640, [130, 200, 390, 391]
    q, k, v = rows(D, T, at)
    v[at] = (torch.randint(16, 32, (4, 1, D), generator=torch.Generator().manual_seed(1)) / 16.0).bfloat16().cuda()
    out, _ = attend(D, q, k, v)
    assert torch.equal(out[200:390], v[at[:2]].float().mean(0).bfloat16().expand(190, 4, D))
    assert torch.equal(out[391:], v[at].float().mean(0).bfloat16().expand(T - 391, 4, D))
