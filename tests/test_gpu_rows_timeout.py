"""The bounded waits of the tensor-core kernels behind kv_read, attn_extend and
attn_decode_prefix: when one runs out the kernel flags OSCAR_DEV_TIMEOUT, waits
for its own products and copies, frees its tensor memory and returns, and the
next call is right.  The wait is made to run out by the hook that shortens the
limit to 1 ms and has one barrier expect an arrival that never comes; nothing
faults and nothing hangs.  The whole call must end within a small multiple of
the limit: a warp that has given up once does not wait again."""
import time

import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from tests.gpu_helpers import dev, dev_i32, dev_rot, kcfg
from tests.test_gpu_rows import cfg_of, filled
from tests.test_gpu_rows_streams import Prefix

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def times_out_and_recovers(call, results, status):
    """call() normally, with the hook, and normally again."""
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in results]
    assert int(status.item()) == 0
    K.set_wait_test(1_000_000, 16)
    try:
        t0 = time.perf_counter()
        call()
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    finally:
        K.set_wait_test(0, 0)
    assert int(status.item()) & K.DEV_TIMEOUT
    assert took < 0.5  # some ten waits of 1 ms one behind the other at the most
    status.zero_()
    for x in results:
        x.fill_(7.0)
    call()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(want, results))


@pytest.mark.parametrize("D,n,T,flags", [
    (128, 2, 600, 0),                       # tokens in the TMEM lanes
    (128, 2, 100, K.FLAG_LLOYD_MAX),        # one tile
    (128, 90, 600, 0),                      # query rows in the TMEM lanes
    (128, 90, 600, K.FLAG_LLOYD_MAX),
    (256, 30, 400, 0),
    (512, 2, 400, 0),
    (512, 30, 400, K.FLAG_LLOYD_MAX),
])
def test_extend(D, n, T, flags):
    c = cfg_of(D, 2, 8, 2, 4, 40, T, flags)
    cache, RK, RV, ch, rng = filled(c, [T, T - 9], D + n)
    kc, st = kcfg(c), dev_i32([0])
    cdev, R, sl = torch.from_numpy(cache).cuda(), (dev_rot(RK), dev_rot(RV)), dev_i32([T, T - 9])
    q = dev(S.activations(rng, (2, n, 8, D), ch, mag=3.0), torch.bfloat16)
    out, lse = torch.empty(2, n, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, n, 8, device="cuda")
    ws = torch.empty(K.attn_extend_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
    times_out_and_recovers(lambda: K.attn_extend(kc, cdev, 0, q, sl, *R, out, ws, lse=lse, status=st), [out, lse], st)


@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D,n,flags", [(128, 1400, 0), (256, 600, 0), (512, 300, K.FLAG_LLOYD_MAX)])
def test_read(D, n, flags, fp32):
    c = cfg_of(D, 2, 4, 4, 4, 40, n, flags | (K.FLAG_OUT_FP32 if fp32 else 0))
    cache, RK, RV, _, _ = filled(c, [n, n], D)
    st = dev_i32([0])
    cdev, R = torch.from_numpy(cache).cuda(), (dev_rot(RK), dev_rot(RV))
    k, v = (torch.empty(2, n, 4, D, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda") for _ in range(2))
    times_out_and_recovers(lambda: K.kv_read(kcfg(c), cdev, 0, dev_i32([0, 0]), dev_i32([n, n]), *R, k, v, status=st), [k, v], st)


def test_rotations_of_many_rows():
    """Query rotation, attention, merge and un-rotation of one call, each with a wait that runs out."""
    n, T = 1100, 1200
    c = cfg_of(128, 1, 8, 1, 4, 40, T)
    cache, RK, RV, ch, rng = filled(c, [T], 3)
    kc, st = kcfg(c), dev_i32([0])
    cdev, R = torch.from_numpy(cache).cuda(), (dev_rot(RK), dev_rot(RV))
    q = dev(S.activations(rng, (1, n, 8, 128), ch, mag=3.0), torch.bfloat16)
    out, lse = torch.empty(1, n, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, 8, device="cuda")
    ws = torch.zeros(K.attn_extend_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
    times_out_and_recovers(lambda: K.attn_extend(kc, cdev, 0, q, dev_i32([T]), *R, out, ws, lse=lse, status=st), [out, lse], st)


@pytest.mark.parametrize("B", [3, 40])
def test_prefix_with_the_own_caches_beside_it(B):
    p = Prefix(128, B, [1 + i % 40 for i in range(B)], 700, 5)
    times_out_and_recovers(p.run, [p.out, p.lse], p.st)
