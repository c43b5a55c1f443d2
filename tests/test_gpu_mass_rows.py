"""attn_mass where its query rows are of no weight, and at the borders of its forms."""
import math

import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from tests.test_gpu_mass import Mass

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


@pytest.mark.parametrize("strange", [math.nan, math.inf, 3e38])
@pytest.mark.parametrize("D,n,flags", [(128, 3, 0), (128, 1, K.FLAG_HADAMARD), (256, 3, K.FLAG_LLOYD_MAX), (512, 2, 0), (128, 20, 0),
                                       (128, 40, K.FLAG_HADAMARD | K.FLAG_LLOYD_MAX)])
def test_a_token_without_weight_may_hold_anything(D, n, flags, strange):
    """lse -inf: the token is a batch's padding, say, and its query whatever lies there."""
    m = Mass(D, 8, 2, 4, 8, [300, 64], n, flags=flags)
    m.lse[0, 0] = m.lse[1, n - 1, 3] = -math.inf
    m.q[0, 0] = m.q[1, n - 1, 3] = 0
    want = m.run().clone()
    m.q[0, 0] = m.q[1, n - 1, 3] = strange
    got = m.run(out=torch.full_like(m.out, 5.0))
    assert bool(torch.isfinite(got).all()) and torch.equal(got, want)


@pytest.mark.parametrize("Hq,Hkv,n,flags", [
    (8, 1, 1, K.FLAG_LLOYD_MAX), (10, 2, 1, K.FLAG_LLOYD_MAX), (3, 1, 3, K.FLAG_LLOYD_MAX),  # two tiles of four rows; more
    (8, 1, 2, 0), (4, 1, 4, K.FLAG_LLOYD_MAX), (1, 1, 17, 0), (2, 2, 17, K.FLAG_LLOYD_MAX),  # 16 and 17 rows: both forms
    (8, 1, 3, 0), (8, 1, 3, K.FLAG_LLOYD_MAX), (5, 1, 5, 0), (5, 1, 5, K.FLAG_LLOYD_MAX)])   # 24 and 25
def test_forms_and_their_borders_at_head_dim_128(Hq, Hkv, n, flags):
    m = Mass(128, Hq, Hkv, 4, 40, [400, 64, 33], n, flags=flags)
    m.run()
    m.check()
