"""kv_read, attn_extend and attn_decode_prefix as a serving program queues them:
many calls on one workspace without a wait between them, on another stream than
the default one, captured once and replayed with other lengths, two captured
graphs at once.  Within a call the kernels overlap their launches, so every
comparison is of bits against a call that had the GPU to itself."""
import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from tests.gpu_helpers import dev, dev_i32, dev_rot, kcfg
from tests.test_gpu_prefix import refill
from tests.test_gpu_rows import cfg_of, filled

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


class Prefix:
    """A prefix decode with its own outputs and workspace."""

    def __init__(self, D, B, lens, plen, seed, cap=64, fp32=False):
        flags = K.FLAG_OUT_FP32 if fp32 else 0
        self.c, self.pc = cfg_of(D, B, 8, 2, 4, 8, cap, flags), cfg_of(D, 1, 8, 2, 4, 40, plen + 5, flags)
        cache, RK, RV, ch, rng = filled(self.c, lens, seed)
        self.kc, self.pk = kcfg(self.c), kcfg(self.pc)
        self.cache, self.pcache = (torch.from_numpy(x).cuda() for x in (cache, refill(self.pc, [plen], RK, RV, seed + 1)))
        self.q = dev(S.activations(rng, (B, 8, D), ch, mag=3.0), torch.bfloat16)
        self.lens, self.plen, self.R = dev_i32(lens), dev_i32([plen]), (dev_rot(RK), dev_rot(RV))
        self.out = torch.empty(B, 8, D, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        self.lse = torch.empty(B, 8, device="cuda")
        self.ws = torch.empty(K.attn_decode_prefix_workspace_bytes(self.kc, self.pk), dtype=torch.uint8, device="cuda")
        self.st = dev_i32([0])

    def run(self, **kw):
        K.attn_decode_prefix(self.kc, self.cache, self.pk, self.pcache, 0, self.q, self.lens, self.plen, *self.R, self.out,
                             self.ws, lse=self.lse, status=self.st, **kw)

    def alone(self, **kw):
        torch.cuda.synchronize()
        self.run(**kw)
        torch.cuda.synchronize()
        return self.out.clone(), self.lse.clone()


def same(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D", [128, 512])
def test_prefix_replays_with_other_lengths(D, fp32):
    p = Prefix(D, 3, [40, 9, 21], 300, 7, fp32=fp32)
    settings = [([40, 9, 21], 300), ([3, 0, 1], 300), ([40, 9, 21], 1), ([0, 0, 5], 0), ([17, 9, 0], 131)]
    want = []
    for lens, plen in settings:
        p.lens.copy_(dev_i32(lens)), p.plen.copy_(dev_i32([plen]))
        want.append(p.alone())
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        p.run()
    for (lens, plen), w in zip(settings, want):
        p.lens.copy_(dev_i32(lens)), p.plen.copy_(dev_i32([plen]))
        p.out.fill_(7.0)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert same((p.out, p.lse), w), (lens, plen)


def test_two_graphs_at_once():
    ps = [Prefix(128, 4, [40, 30, 20, 10], 700, 1), Prefix(128, 70, [5] * 70, 900, 2)]
    want = [p.alone() for p in ps]
    graphs = []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run()
        graphs.append((g, torch.cuda.Stream()))
    for p in ps:
        p.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(same((p.out, p.lse), w) for p, w in zip(ps, want))


def test_hints_and_lengths_of_every_kind_fit_the_workspace():
    # own caches up to 1024 positions and longer ones go different ways; the hint is only an upper bound
    p = Prefix(128, 2, [1500, 900], 200, 3, cap=1600)
    p.lens.copy_(dev_i32([5, 1]))
    ref = p.alone()
    for hint in (5, 127, 128, 129, 500, 1023, 1024, 1025, 1600):
        for splits in (0, 1, 3, K.MAX_SPLITS):
            got = p.alone(seq_len_hint=hint, num_splits=splits)
            # two roundings to bf16 and the parts' to fp16
            assert torch.allclose(got[0].float(), ref[0].float(), rtol=2 ** -7, atol=2 ** -7 * float(ref[0].abs().max()))
            assert torch.allclose(got[1], ref[1], rtol=1e-5, atol=1e-4)
    assert int(p.st.item()) == 0


@pytest.mark.parametrize("D,n", [(128, 3), (128, 90), (512, 20)])
def test_queued_extends_share_a_workspace(D, n):
    B, lens = 2, [400, 333]
    c = cfg_of(D, B, 8, 2, 4, 40, 420)
    cache, RK, RV, ch, rng = filled(c, lens, D + n)
    kc = kcfg(c)
    cache, R = torch.from_numpy(cache).cuda(), (dev_rot(RK), dev_rot(RV))
    qs = [dev(S.activations(rng, (B, n, 8, D), ch, mag=3.0), torch.bfloat16) for _ in range(4)]
    ws = torch.empty(K.attn_extend_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
    outs = [[torch.empty(B, n, 8, D, dtype=torch.bfloat16, device="cuda") for _ in qs] for _ in range(6)]
    lses = [[torch.empty(B, n, 8, device="cuda") for _ in qs] for _ in range(6)]
    sl, st = dev_i32(lens), dev_i32([0])

    def call(i, o, l):
        K.attn_extend(kc, cache, 0, qs[i], sl, *R, o, ws, lse=l, status=st)

    torch.cuda.synchronize()
    for i in range(4):
        call(i, outs[0][i], lses[0][i])
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for k in range(1, 6):
            for i in range(4):
                call(i, outs[k][i], lses[k][i])
    torch.cuda.synchronize()
    for k in range(1, 6):
        assert all(torch.equal(a, b) for a, b in zip(outs[0] + lses[0], outs[k] + lses[k]))
    assert int(st.item()) == 0


@pytest.mark.parametrize("n", [1, 400])
def test_append_extend_read_on_a_side_stream(n):
    """What an append has just queued is what the others see, on the appending stream."""
    B, D, old = 2, 128, 100
    c = cfg_of(D, B, 8, 4, 4, 40, old + n)
    cache, RK, RV, ch, rng = filled(c, [old] * B, 5)
    kc = kcfg(c)
    start = torch.from_numpy(cache).cuda()
    R, pos, sl = (dev_rot(RK), dev_rot(RV)), dev_i32([old] * B), dev_i32([old + n] * B)
    k, v = (dev(S.activations(rng, (B, n, 4, D), [3], mag=3.0), torch.bfloat16) for _ in range(2))
    q = dev(S.activations(rng, (B, n, 8, D), ch, mag=3.0), torch.bfloat16)
    ws = torch.empty(K.attn_extend_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
    res = []
    side = torch.cuda.Stream()
    for wait in (True, False, False):
        mem = start.clone()
        out = torch.empty(B, n, 8, D, dtype=torch.bfloat16, device="cuda")
        ko, vo = (torch.zeros(B, n, 4, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        done = torch.cuda.synchronize if wait else (lambda: None)
        with torch.cuda.stream(side):
            K.kv_append(kc, mem, 0, k, v, pos, *R)
            done()
            K.attn_extend(kc, mem, 0, q, sl, *R, out, ws)
            done()
            K.kv_read(kc, mem, 0, pos, sl, *R, k_out=ko, v_out=vo)
        torch.cuda.synchronize()
        res.append((out, ko, vo))
    for r in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(res[0], r))
    err = (res[0][1].float() - k.float()).norm() / k.float().norm()
    assert np.isfinite(float(err)) and float(err) < 0.8  # 2-bit rows and BF16 ones: it is these tokens that came back


@pytest.mark.parametrize("n", [3, 1500])
@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
def test_read_of_one_role(n, fp32):
    """Either role alone gives the bits that it has beside the other."""
    c = cfg_of(128, 2, 8, 2, 4, 40, 1600, K.FLAG_OUT_FP32 if fp32 else 0)
    cache, RK, RV, _, _ = filled(c, [1600, 1510], 11)
    kc, R = kcfg(c), (dev_rot(RK), dev_rot(RV))
    cache, pos, sl = torch.from_numpy(cache).cuda(), dev_i32([100, 10]), dev_i32([1600, 1510])

    def empty():
        return torch.zeros(2, n, 2, 128, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")

    k, v, k1, v1 = empty(), empty(), empty(), empty()
    K.kv_read(kc, cache, 0, pos, sl, *R, k_out=k, v_out=v)
    K.kv_read(kc, cache, 0, pos, sl, *R, k_out=k1)
    K.kv_read(kc, cache, 0, pos, sl, *R, v_out=v1)
    torch.cuda.synchronize()
    assert torch.equal(k, k1) and torch.equal(v, v1)
    assert not torch.equal(k, v) and float(k.abs().sum()) > 0
