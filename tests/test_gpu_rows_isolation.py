"""No row of attn_extend and attn_decode_prefix depends on finite values that are
none of its business, however large: on another row's query, or on a key that
its mask hides.  All comparisons are of bits."""
import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from oracle import oscar_oracle as O
from tests.gpu_helpers import dev, dev_i32, dev_rot, kcfg
from tests.test_gpu_rows import cfg_of, filled
from tests.test_gpu_rows_streams import Prefix

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def bits(x):
    return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("size", [1e8, 1e12, 1e30])
@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D,n,flags", [(128, 3, 0), (128, 80, 0), (128, 80, K.FLAG_LLOYD_MAX), (256, 40, 0), (512, 3, 0),
                                       (512, 40, K.FLAG_V_BF16)])
def test_a_large_query_leaves_the_others_alone(D, n, flags, fp32, size):
    c = cfg_of(D, 1, 8, 2, 4, 40, 300, flags | (K.FLAG_OUT_FP32 if fp32 else 0))
    cache, RK, RV, ch, rng = filled(c, [300], D + n)
    kc, cdev, R = kcfg(c), torch.from_numpy(cache).cuda(), (dev_rot(RK), dev_rot(RV))
    q = dev(S.activations(rng, (1, n, 8, D), ch, mag=3.0), torch.bfloat16)
    ws = torch.empty(K.attn_extend_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
    res, st = [], dev_i32([0])
    for large in (False, True):
        if large:
            q[0, n // 2, 3] *= size
        out = torch.empty(1, n, 8, D, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        lse = torch.empty(1, n, 8, device="cuda")
        K.attn_extend(kc, cdev, 0, q, dev_i32([300]), *R, out, ws, lse=lse, status=st)
        torch.cuda.synchronize()
        res.append((bits(out).clone(), bits(lse).clone()))
    assert int(st.item()) == 0
    for a, b in zip(*res):
        b[0, n // 2, 3] = a[0, n // 2, 3]
        assert torch.equal(a, b)


@pytest.mark.parametrize("size", [1e8, 1e12, 1e30])
@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D,B,cap", [(128, 5, 64), (128, 40, 64), (512, 5, 64), (128, 5, 1500)])
def test_a_large_query_leaves_its_batch_alone(D, B, cap, fp32, size):
    p = Prefix(D, B, [1 + i % 40 for i in range(B)], 500, D + B, cap=cap, fp32=fp32)
    a = p.alone()
    p.q[2, 5] *= size
    b = p.alone()
    assert int(p.st.item()) in (0, K.DEV_FP16_RANGE)  # of attn_decode's kernels, for long own caches
    for x, y in zip(a, b):
        x, y = bits(x), bits(y)
        y[2, 5] = x[2, 5]
        assert torch.equal(x, y)


@pytest.mark.parametrize("D,n", [(128, 2), (128, 90), (256, 40), (512, 2)])
def test_results_scale_with_a_query(D, n):
    """A query times 2^k and a softmax scale times 2^-k: the same scores, to the bit."""
    c = cfg_of(D, 1, 8, 2, 4, 40, 300)
    cache, RK, RV, ch, rng = filled(c, [300], D + n)
    kc, cdev, R = kcfg(c), torch.from_numpy(cache).cuda(), (dev_rot(RK), dev_rot(RV))
    q = dev(S.activations(rng, (1, n, 8, D), ch, mag=3.0), torch.bfloat16)
    ws = torch.empty(K.attn_extend_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
    res = []
    for k in (0, 60, -60):
        out, lse = torch.empty(1, n, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, 8, device="cuda")
        K.attn_extend(kc, cdev, 0, q * 2.0 ** k, dev_i32([300]), *R, out, ws, lse=lse, sm_scale=D ** -0.5 * 2.0 ** -k)
        torch.cuda.synchronize()
        res.append((out, lse))
    for out, lse in res[1:]:
        assert torch.equal(out, res[0][0]) and torch.equal(lse, res[0][1])


@pytest.mark.parametrize("size", [1e8, 1e12, 1e30])
@pytest.mark.parametrize("D,n,W,flags", [(128, 3, 40, 0), (128, 80, 200, 0), (128, 80, 200, K.FLAG_LLOYD_MAX), (256, 40, 100, 0),
                                         (512, 12, 40, 0), (512, 40, 100, K.FLAG_V_BF16)])
def test_a_large_hidden_key_or_value_row_leaves_earlier_tokens_alone(D, n, W, flags, size):
    """The last position's BF16 rows times 1e8 to 1e30: the tokens before it do not see them."""
    T = 300
    c = cfg_of(D, 1, 8, 2, 4, W, T, flags)
    cache, RK, RV, ch, rng = filled(c, [T], D + n)
    kc, R = kcfg(c), (dev_rot(RK), dev_rot(RV))
    q = dev(S.activations(rng, (1, n, 8, D), ch, mag=3.0), torch.bfloat16)
    ws = torch.empty(K.attn_extend_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
    large = cache.copy()
    for role in (0, 1):
        view = O.CacheView(c, large, 0, role)
        row = view.full[0, :, T - 1] if role and flags & K.FLAG_V_BF16 else view.ring[0, :, (T - 1) % W]
        row[...] = O.f32_to_bf16_bits(O.bf16_bits_to_f32(row) * np.float32(size))
    res = []
    for x in (cache, large):
        out, lse = torch.empty(1, n, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, 8, device="cuda")
        K.attn_extend(kc, torch.from_numpy(x).cuda(), 0, q, dev_i32([T]), *R, out, ws, lse=lse)
        torch.cuda.synchronize()
        res.append((out[:, :-1], lse[:, :-1]))
    assert torch.equal(bits(res[0][0]), bits(res[1][0])) and torch.equal(bits(res[0][1]), bits(res[1][1]))


@pytest.mark.parametrize("D,n,flags", [(128, 3, 0), (128, 80, 0), (128, 80, K.FLAG_LLOYD_MAX), (256, 40, 0), (512, 3, K.FLAG_LLOYD_MAX),
                                       (512, 40, 0)])
@pytest.mark.parametrize("size", [1e-3, 1e-5])
def test_small_keys_keep_their_bits(D, n, flags, size):
    """Keys of 1e-3 and 1e-5 against queries that bring the scores to ordinary size.  Without rotations a score is off
    by some 2^-18 of the sum of its products' magnitudes (two fp16 parts of the query, sums that are cut off); 2^-14 is
    allowed.  A middle or step that has lost its bits to fp16's smallest number is off by 2^-10 and more."""
    T = 300
    c = cfg_of(D, 1, 8, 2, 4, 40, T, flags)
    rng = np.random.default_rng(D)
    k, v = (S.to_bf16_values(S.activations(rng, (1, T, 2, D), [3, 70], mag=3.0)) for _ in range(2))
    k = S.to_bf16_values(k * np.float32(size))
    eye = np.eye(D, dtype=np.float32)
    cache = O.new_cache(c)
    O.append(c, cache, 0, k, v, [0], eye, eye)
    q = S.to_bf16_values(S.activations(rng, (1, n, 8, D), [3, 70], mag=3.0) / np.float32(size))
    kc = kcfg(c)
    ws = torch.empty(K.attn_extend_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(1, n, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, 8, device="cuda")
    K.attn_extend(kc, torch.from_numpy(cache).cuda(), 0, dev(q), dev_i32([T]), dev_rot(eye), dev_rot(eye), out, ws, lse=lse)
    torch.cuda.synchronize()
    got = lse.cpu().numpy().astype(np.float64)
    for h in range(8):
        x = O.dequant_history(c, cache, 0, 0, 0, h // 4, T).astype(np.float64)
        s = q[0, :, h].astype(np.float64) @ x.T / D ** 0.5
        s[np.arange(T)[None, :] > (T - n + np.arange(n))[:, None]] = -np.inf
        top = s.max(1)
        want = top + np.log(np.exp(s - top[:, None]).sum(1))
        lim = 2.0 ** -14 * (np.abs(q[0, :, h]).astype(np.float64) @ np.abs(x).T).max(1) / D ** 0.5
        assert (np.abs(got[0, :, h] - want) <= lim).all(), (h, np.abs(got[0, :, h] - want).max(), lim.min())
