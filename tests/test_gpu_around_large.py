"""kv_append_packed, attn_mass and kv_evict over a cache whose offsets pass 32 bits: one sequence of 2^27 positions (4.8 GB of K
and as much of V), of which the last ones are written, weighed and kept."""
import math

import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from oracle import oscar_oracle as O
from tests.gpu_helpers import dev_i32
from tests.test_gpu_append_packed import region_views

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


@pytest.mark.parametrize("flags", [0, K.FLAG_HADAMARD])
def test_at_the_end_of_a_long_cache(flags):
    T, n, S, W, keep = 1 << 27, 1500, 4, 64, 1000
    c = K.KVConfig(1, 1, 4, 1, 128, S, W, T + 64, flags=flags)
    oc = K.KVConfig(1, 1, 4, 1, 128, S, W, S + W + keep, flags=flags)
    lay = K.layout_query(c)
    cache = torch.zeros(lay["total_bytes"], dtype=torch.uint8, device="cuda")
    R = (None, None) if flags else (torch.eye(128, device="cuda"),) * 2
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(n, 1, 128, generator=g).bfloat16().cuda() for _ in range(2))
    st = dev_i32([0])
    K.kv_append_packed(c, cache, 0, k, v, dev_i32([0, n]), dev_i32([T - n]), *R, status=st)
    # the same rows in a short cache
    sc = K.KVConfig(1, 1, 4, 1, 128, 0, W, n, flags=flags)
    short = torch.zeros(K.layout_query(sc)["total_bytes"], dtype=torch.uint8, device="cuda")
    K.kv_append(sc, short, 0, k[None], v[None], dev_i32([0]), *R)
    big = region_views(O.Config(1, 1, 4, 1, 128, S, W, T + 64, flags=flags), lay, cache)
    small = region_views(O.Config(1, 1, 4, 1, 128, 0, W, n, flags=flags), K.layout_query(sc), short)
    for name, each in (("codes", 32), ("sz", 4)):
        for role in "kv":
            at = (T - n - S) * each
            assert torch.equal(big[role + name][0, 0, at:at + n * each], small[role + name][0, 0, :n * each])
    # weights: a query equal to a late key, everything before it zero rows
    q = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    q[0, 0, :] = k[777, 0] * 2
    lse, out = torch.empty(1, 4, device="cuda"), torch.empty(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(lay["decode_workspace_bytes"], K.attn_mass_workspace_bytes(c, 1), K.kv_evict_workspace_bytes(c, keep)),
                     dtype=torch.uint8, device="cuda")
    K.attn_decode(c, cache, 0, q[0], dev_i32([T]), *R, out, ws, lse=lse, status=st)
    mass = torch.zeros(1, 1, T + 64, device="cuda")
    K.attn_mass(c, cache, 0, q, dev_i32([T]), R[0], lse[:, None], mass, ws, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert math.isclose(float(mass.double().sum()), 4.0, rel_tol=1e-3)
    assert int(mass[0, 0].argmax()) == T - n + 777 and bool((mass[0, 0, T:] == 0).all())
    # the late rows are heavier than the zero rows where their score is positive; all of them are kept that way
    late = torch.arange(T - n, T - W, device="cuda")
    mass.zero_()
    pick = late[torch.randperm(len(late), generator=g)[:keep].cuda()]
    mass[0, 0, pick] = 1.0
    small_cache = torch.zeros(K.layout_query(oc)["total_bytes"], dtype=torch.uint8, device="cuda")
    kept, new = torch.zeros(1, 1, keep, dtype=torch.int32, device="cuda"), dev_i32([0])
    K.kv_evict(c, cache, 0, mass, dev_i32([T]), keep, oc, small_cache, 0, new, ws, kept=kept, status=st)
    torch.cuda.synchronize()
    assert int(new.item()) == S + W + keep and int(st.item()) == 0
    assert torch.equal(kept[0, 0].long(), pick.sort().values)
    got = region_views(O.Config(1, 1, 4, 1, 128, S, W, S + W + keep, flags=flags), K.layout_query(oc), small_cache)
    rows = (kept[0, 0].long() - (T - n)).cpu().numpy()
    want = small["kcodes"][0, 0].cpu().numpy().reshape(-1, 32)[rows]
    assert np.array_equal(got["kcodes"][0, 0].cpu().numpy().reshape(-1, 32)[:keep], want)
