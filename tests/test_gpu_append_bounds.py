"""kv_append_packed with bounds that are not those of its rows: flagged on every kernel path, and what lies beyond the rows is
clamped to them, so that the window holds the last rows that there are."""
import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from tests.gpu_helpers import dev_i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


PATHS = [(128, 20, 0), (256, 20, 0),                                                 # row-parallel, clusters
         (128, 1500, 0), (128, 1500, K.FLAG_IN_FP32), (256, 1500, 0),                # tensor cores, tiles
         (128, 1500, K.FLAG_LLOYD_MAX), (128, 1500, K.FLAG_V_BF16),                  # row-parallel, many
         (128, 20, K.FLAG_HADAMARD), (128, 1500, K.FLAG_HADAMARD), (512, 600, K.FLAG_HADAMARD | K.FLAG_IN_FP32)]


def append(D, n, flags, cu, B=2):
    c = K.KVConfig(1, B, 2, 1, D, 3, 8, n + 10, flags=flags)
    g = torch.Generator().manual_seed(D + n)
    k, v = (torch.randn(n, 1, D, generator=g).to(torch.float32 if flags & K.FLAG_IN_FP32 else torch.bfloat16).cuda() for _ in range(2))
    R = (None, None) if flags & K.FLAG_HADAMARD else (torch.eye(D, device="cuda"),) * 2
    size = K.layout_query(c)["total_bytes"]
    base = torch.full((size + 8192,), 0xEE, dtype=torch.uint8, device="cuda")
    status = dev_i32([0])
    K.kv_append_packed(c, base[4096:4096 + size], 0, k, v, dev_i32(cu), dev_i32([0] * B), *R, status=status)
    torch.cuda.synchronize()
    assert bool((base[:4096] == 0xEE).all()) and bool((base[4096 + size:] == 0xEE).all())
    return base[4096:4096 + size], int(status.item())


@pytest.mark.parametrize("D,n,flags", PATHS)
def test_bounds_beyond_the_rows_are_clamped(D, n, flags):
    want, status = append(D, n, flags, [0, n // 2, n])
    assert status == 0
    for cu in ([0, n // 2, n + 37], [-5, n // 2, n], [-2 ** 31, n // 2, 2 ** 31 - 1]):
        got, status = append(D, n, flags, cu)
        assert status == K.DEV_OVER_CAPACITY, cu
        assert torch.equal(got, want), cu


@pytest.mark.parametrize("D,n,flags", PATHS)
@pytest.mark.parametrize("cu", [(0, 2, 1), (1, 0, 2), (2, 1, 0), (2, 3, 4)], ids=str)
def test_bounds_out_of_order_are_flagged(D, n, flags, cu):
    """In halves of the rows; the last lies behind all of them."""
    assert append(D, n, flags, [x * (n // 2) for x in cu])[1] == K.DEV_OVER_CAPACITY


@pytest.mark.parametrize("D,n,flags", PATHS)
def test_many_sequences_are_looked_at(D, n, flags):
    """More than a warp's lanes; one bound of them out of order."""
    cu = np.linspace(0, n, 71).astype(int)
    assert append(D, n, flags, cu, B=70)[1] == 0
    cu[45] = cu[46] + 1
    assert append(D, n, flags, cu, B=70)[1] == K.DEV_OVER_CAPACITY
