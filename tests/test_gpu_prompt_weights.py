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


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [128, 256, 512])
@pytest.mark.parametrize("size", [1e5, 1e7, 1e9, 1e12, 1e20, 1e31, 1e37])
@pytest.mark.parametrize("sign", ["any", "negative"])
def test_scores_of_any_size(D, kind, size, sign):
    """Scores q k_p of one channel, exact in float32 and further apart (2^-8 of them) than weights reach: a token's output is
    the value of the largest score that it sees, or the mean of those that share it, also where all of them are far below
    zero.  lse is that score, to its own last bits."""
    T, flags = 333, K.FLAG_IN_FP32 | K.FLAG_OUT_FP32 if kind == "fp32" else 0
    dtype = torch.float32 if flags else torch.bfloat16
    g = torch.Generator().manual_seed(D)
    q, k = torch.zeros(T, 2, D), torch.zeros(T, 1, D)
    k[:, 0, 0] = -(1 + torch.randint(0, 128, (T,), generator=g) / 128.0)
    if sign == "any":
        k[::2] *= -1
    root = 2.0 ** int(math.log2(size) / 2)
    k *= root
    q[:, 0, 0], q[:, 1, 0] = root, root * 1.5
    v = torch.randint(1, 32, (T, 1, D), generator=g) / 1.0
    q, k, v = (x.to(dtype).cuda() for x in (q, k, v))
    out, lse = torch.empty_like(q), torch.empty(T, 2, device="cuda")
    K.attn_prompt(K.KVConfig(1, 1, 2, 1, D, 0, 0, 1, flags=flags), q, k, v, dev_i32([0, T]), out, lse=lse)
    torch.cuda.synchronize()
    score = q[:, :, 0].double()[:, :, None] * k[:, 0, 0].double()  # [T][2][T]
    score = torch.where(torch.ones(T, T, dtype=torch.bool, device="cuda").tril()[:, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    w = (score == top).double()
    want = (w / w.sum(-1, keepdim=True)) @ v[:, 0].double()
    bound = want.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else 0) + 32 * 8 * 2.0 ** -24
    assert bool(((out.double() - want).abs() <= bound).all())
    want = top[..., 0] / math.sqrt(D) + torch.log(w.sum(-1))
    assert bool(((lse.double() - want).abs() <= want.abs() * 2.0 ** -21 + 1e-5).all())


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [128, 256, 512])
def test_a_score_at_the_end_of_the_range(D, kind):
    """-3.24e38 in log2 units, for one token and for two."""
    flags = K.FLAG_IN_FP32 | K.FLAG_OUT_FP32 if kind == "fp32" else 0
    dtype = torch.float32 if flags else torch.bfloat16
    q, k, v = (torch.zeros(2, 1, D) for _ in range(3))
    q[:, 0, 0], k[:, 0, 0] = 1.8e19, -1.8e19
    v[0], v[1] = 3, 5
    q, k, v = (x.to(dtype).cuda() for x in (q, k, v))
    out = torch.empty_like(q)
    K.attn_prompt(K.KVConfig(1, 1, 1, 1, D, 0, 0, 1, flags=flags), q, k, v, dev_i32([0, 2]), out, sm_scale=math.log(2.0))
    torch.cuda.synchronize()
    assert bool((out[0] == 3).all()) and bool((out[1] == 4).all())
