"""kv_read of no positions and attn_extend of no tokens through the binding."""
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from tests.gpu_helpers import dev_i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def test_empty_tensors():
    cfg = K.KVConfig(1, 2, 8, 2, 128, 4, 8, 64)
    cache = torch.zeros(K.layout_query(cfg)["total_bytes"], dtype=torch.uint8, device="cuda")
    R, lens, st = torch.eye(128, device="cuda"), dev_i32([5, 7]), dev_i32([0])
    q, kv = (torch.empty(2, 0, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 2))
    ws = torch.empty(K.attn_extend_workspace_bytes(cfg, 0), dtype=torch.uint8, device="cuda")
    K.attn_extend(cfg, cache, 0, q, lens, R, R, torch.empty_like(q), ws, lse=torch.empty(2, 0, 8, device="cuda"), status=st)
    K.kv_read(cfg, cache, 0, dev_i32([0, 0]), lens, R, R, kv, torch.empty_like(kv), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
