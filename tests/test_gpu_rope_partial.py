"""qk_norm_rope with a partial rotation: channels behind it are normed each by itself, also beside one that is not finite."""
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from tests.gpu_helpers import dev_i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("D,rot", [(128, 0), (128, 64), (128, 16), (256, 32), (512, 496)])
def test_an_infinite_channel_behind_the_rotation(D, rot, inter, fp32):
    """x / sqrt(mean x^2) is NaN for it and 0 for all others."""
    kind = torch.float32 if fp32 else torch.bfloat16
    g = torch.Generator().manual_seed(D)
    q, k = (torch.randn(D - rot, 1, D, generator=g).to(kind).cuda() for _ in range(2))
    n = D - rot
    at = torch.arange(n, device="cuda")
    q[at, 0, rot + at] = float("inf")
    k[at, 0, rot + at] = float("-inf")
    w, out = torch.ones(D, device="cuda"), [torch.empty(n, 1, D, dtype=kind, device="cuda") for _ in range(2)]
    cfg = K.KVConfig(1, 1, 1, 1, D, 0, 0, 1, flags=K.FLAG_IN_FP32 if fp32 else 0)
    freq = torch.rand(rot // 2, generator=g).cuda() if rot else None
    K.qk_norm_rope(cfg, q, k, w, w, dev_i32(range(n)) if rot else None, freq, *out, interleaved=inter)
    torch.cuda.synchronize()
    for x in out:
        own = torch.zeros(n, D, dtype=torch.bool, device="cuda")
        own[at, rot + at] = True
        assert bool(x[:, 0][own].isnan().all()) and bool((x[:, 0][~own] == 0).all())


@pytest.mark.parametrize("n", [1, 5])
def test_outputs_beside_and_over_their_inputs(n):
    """In place where that is dense (one token of a fused projection is), and directly behind an input."""
    D, Hq, Hkv = 128, 8, 2
    cfg = K.KVConfig(1, 1, Hq, Hkv, D, 0, 0, 1)
    w, freq, pos = torch.ones(D, device="cuda"), torch.rand(D // 2, device="cuda"), dev_i32(range(n))
    flat = torch.randn(n * (2 * Hq + 2 * Hkv) * D, device="cuda").bfloat16()
    at = [0, n * Hq * D, n * (Hq + Hkv) * D, n * (2 * Hq + Hkv) * D, len(flat)]
    q, k, qo, ko = (flat[a:b].view(n, -1, D) for a, b in zip(at, at[1:]))
    K.qk_norm_rope(cfg, q, k, w, w, pos, freq, qo, ko)
    a, b = q.clone(), k.clone()
    K.qk_norm_rope(cfg, a, b, w, w, pos, freq, a, b)
    torch.cuda.synchronize()
    assert torch.equal(a, qo) and torch.equal(b, ko)
    if n == 1:
        row = torch.cat((q.view(-1), k.view(-1), k.view(-1))).view(1, -1)
        x, y = row[:, :Hq * D].view(1, Hq, D), row[:, Hq * D:(Hq + Hkv) * D].view(1, Hkv, D)
        K.qk_norm_rope(cfg, x, y, w, w, pos, freq, x, y)
        torch.cuda.synchronize()
        assert torch.equal(x, qo) and torch.equal(y, ko) and torch.equal(row[0, -Hkv * D:], k.view(-1))
