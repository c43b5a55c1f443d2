"""qk_norm_rope against its 64-bit form: head_dims, head counts that do not fill a warp, one token and many, partial and no
rotation, both pair orders, far positions, strided inputs, outputs over their inputs, float32."""
import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from tests import around_ref as R
from tests.gpu_helpers import dev_i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def make(D, Hq, Hkv, n, fp32, seed, size=2.0):
    g = torch.Generator().manual_seed(seed)
    kind = torch.float32 if fp32 else torch.bfloat16
    fused = (torch.randn(n, (Hq + 2 * Hkv) * D, generator=g) * size).to(kind).cuda()
    q, k = fused[:, :Hq * D].view(n, Hq, D), fused[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2)]
    return fused, q, k, w


def cfg(D, Hq, Hkv, fp32):
    return K.KVConfig(1, 1, Hq, Hkv, D, 0, 0, 1, flags=K.FLAG_IN_FP32 if fp32 else 0)


def freqs(rot, theta=1e6):
    return (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def compare(q, k, w, pos, freq, inter, fp32, q_out, k_out, eps):
    f = None if freq is None else freq.cpu().double().numpy()
    for name, x, y, wt in (("q", q, q_out, w[0]), ("k", k, k_out, w[1])):
        want, bound = R.norm_rope(x.cpu().double().numpy(), wt.cpu().double().numpy(), eps, pos, f, inter, fp32)
        R.check(name, y.cpu().double().numpy(), want, bound)


@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("D,Hq,Hkv,n,rot,first", [
    (128, 4, 1, 1, 128, 0), (128, 32, 8, 7, 128, 131072), (128, 5, 5, 3, 64, 1000), (128, 3, 1, 4000, 128, 5),
    (128, 8, 2, 33, 16, 77), (128, 8, 2, 33, 112, 77), (128, 8, 2, 5, 0, 0), (256, 6, 2, 9, 256, 1048576), (256, 7, 1, 40, 32, 3),
    (512, 3, 3, 11, 512, 1000003), (512, 8, 1, 2, 496, 12), (128, 64, 8, 700, 128, 2 ** 20)])
def test_against_64_bits(D, Hq, Hkv, n, rot, first, inter, fp32):
    _, q, k, w = make(D, Hq, Hkv, n, fp32, D + n)
    kind = q.dtype
    out = [torch.full((n, h, D), 7.0, dtype=kind, device="cuda") for h in (Hq, Hkv)]
    pos = np.arange(first, first + n)
    freq = freqs(rot) if rot else None
    K.qk_norm_rope(cfg(D, Hq, Hkv, fp32), q, k, *w, dev_i32(pos) if rot else None, freq, *out, eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    compare(q, k, w, pos, freq, inter, fp32, *out, 1e-5)


def test_positions_in_any_order_and_repeated():
    n = 50
    _, q, k, w = make(128, 8, 2, n, True, 1)
    pos = np.random.default_rng(0).integers(0, 10 ** 6, n)
    pos[3] = pos[4]
    out = [torch.empty(n, h, 128, device="cuda") for h in (8, 2)]
    K.qk_norm_rope(cfg(128, 8, 2, True), q, k, *w, dev_i32(pos), freqs(128), *out)
    torch.cuda.synchronize()
    compare(q, k, w, pos, freqs(128), False, True, *out, 1e-6)


def test_positions_below_zero_and_frequencies_above_a_turn():
    n = 40
    _, q, k, w = make(128, 4, 2, n, True, 2)
    pos = np.arange(n) * 13 - 300
    freq = torch.linspace(-7.0, 30.0, 64, device="cuda")
    out = [torch.empty(n, h, 128, device="cuda") for h in (4, 2)]
    K.qk_norm_rope(cfg(128, 4, 2, True), q, k, *w, dev_i32(pos), freq, *out)
    torch.cuda.synchronize()
    compare(q, k, w, pos, freq, False, True, *out, 1e-6)


@pytest.mark.parametrize("n", [3, 3000])
@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
def test_outputs_over_their_dense_inputs(fp32, n):
    _, q, k, w = make(128, 12, 3, n, fp32, 5)
    c, pos = cfg(128, 12, 3, fp32), dev_i32(np.arange(n))
    q, k = q.contiguous(), k.contiguous()
    out = [torch.empty_like(x) for x in (q, k)]
    K.qk_norm_rope(c, q, k, *w, pos, freqs(128), *out)
    K.qk_norm_rope(c, q, k, *w, pos, freqs(128), q, k)
    torch.cuda.synchronize()
    assert torch.equal(q, out[0]) and torch.equal(k, out[1])


def test_small_and_zero_rows():
    """A row of zeros stays zero; eps counts where the squares are as small."""
    _, q, k, w = make(128, 4, 2, 6, True, 9, size=1e-3)
    q, k = q.contiguous(), k.contiguous()
    q[2] = 0
    out = [torch.empty_like(x) for x in (q, k)]
    K.qk_norm_rope(cfg(128, 4, 2, True), q, k, *w, dev_i32(np.arange(6)), freqs(128), *out, eps=1e-6)
    torch.cuda.synchronize()
    assert bool((out[0][2] == 0).all())
    compare(q, k, w, np.arange(6), freqs(128), False, True, *out, 1e-6)


def test_a_bad_row_leaves_the_others_alone():
    _, q, k, w = make(128, 8, 2, 20, False, 3)
    q, k = q.contiguous(), k.contiguous()
    c, pos = cfg(128, 8, 2, False), dev_i32(np.arange(20))
    want = [torch.empty_like(x) for x in (q, k)]
    K.qk_norm_rope(c, q, k, *w, pos, freqs(128), *want)
    q[7, 3, 11] = float("nan")
    q[8, 4, 0] = float("inf")
    got = [torch.empty_like(x) for x in (q, k)]
    K.qk_norm_rope(c, q, k, *w, pos, freqs(128), *got)
    torch.cuda.synchronize()
    assert bool(torch.isnan(got[0][7, 3]).any()) and bool(torch.isnan(got[0][8, 4]).any())
    got[0][7, 3], got[0][8, 4] = want[0][7, 3], want[0][8, 4]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_rows():
    e = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, device="cuda")
    assert K.qk_norm_rope(cfg(128, 8, 2, False), e, k, w, w, dev_i32([]), freqs(128), e, k) == 0
