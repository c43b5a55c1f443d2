"""attn_decode_prefix: the own caches' attention runs beside the prefix's and reads
the queries that a kernel before both has rotated.  Calls queued one after the
other on one workspace, each with other queries, give the bits that each gives
alone; no older queries are read, and nothing is left behind in the workspace."""
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from tests.gpu_helpers import dev
from tests.test_gpu_rows_streams import Prefix

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D,B,plen", [(128, 3, 700), (128, 40, 300), (256, 12, 260), (512, 2, 1)])
def test_queued_calls_read_their_own_queries(D, B, plen, fp32):
    import numpy as np
    p = Prefix(D, B, [1 + i % 40 for i in range(B)], plen, D + B, fp32=fp32)
    rng = np.random.default_rng(1)
    qs = [dev(S.activations(rng, (B, 8, D), [5, 60], mag=3.0), torch.bfloat16) for _ in range(4)]
    want = []
    for q in qs:
        p.ws.fill_(0xFF)
        p.q.copy_(q)
        want.append(p.alone())
    outs = [[(torch.empty_like(p.out), torch.empty_like(p.lse)) for _ in qs] for _ in range(8)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for row in outs:
            for q, (out, lse) in zip(qs, row):
                K.attn_decode_prefix(p.kc, p.cache, p.pk, p.pcache, 0, q, p.lens, p.plen, *p.R, out, p.ws, lse=lse, status=p.st)
    torch.cuda.synchronize()
    for row in outs:
        for got, w in zip(row, want):
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    assert int(p.st.item()) == 0


def test_a_prefix_block_with_nothing_to_see_still_releases_the_queries():
    """No prefix: every block of the first attention ends early, the first one with the queries released."""
    p = Prefix(128, 3, [40, 9, 21], 5, 2)
    ref = p.alone(seq_len_hint=40)
    p.plen.zero_()
    for _ in range(3):
        got = p.alone(seq_len_hint=40)
        assert int(p.st.item()) == 0
        assert torch.isfinite(got[0].float()).all() and not torch.equal(got[0], ref[0])
