"""attn_prompt against its 64-bit form: head_dims, shared heads (a tile's rows full and not), packed lengths of zero, one,
around every tile border and long, rows of no sequence, types; what is not finite reaches only the tokens that see it."""
import math

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


KINDS = {"bf16": 0, "fp32": K.FLAG_IN_FP32 | K.FLAG_OUT_FP32, "fp32-in": K.FLAG_IN_FP32, "fp32-out": K.FLAG_OUT_FP32}


class Prompt:
    def __init__(self, D, Hq, Hkv, lens, kind="bf16", before=0, behind=3, seed=0, gaps=0.0):
        g = torch.Generator().manual_seed(seed + D + sum(lens))
        self.flags = KINDS[kind]
        self.cfg = K.KVConfig(1, len(lens), Hq, Hkv, D, 0, 0, 1, flags=self.flags)
        self.lens, self.first = lens, before + np.concatenate(([0], np.cumsum(lens)))
        n = int(self.first[-1]) + behind
        t = torch.float32 if self.flags & K.FLAG_IN_FP32 else torch.bfloat16
        self.q, self.k, self.v = (torch.randn(n, h, D, generator=g).to(t).cuda() for h in (Hq, Hkv, Hkv))
        self.q[:, 0] *= 4  # one head with sharp attention
        self.cu = dev_i32(self.first)
        self.out = torch.full((n, Hq, D), 7.0, dtype=torch.float32 if self.flags & K.FLAG_OUT_FP32 else torch.bfloat16, device="cuda")
        self.lse = torch.full((n, Hq), 7.0, device="cuda")
        self.st = dev_i32([0])

    def run(self, scale=0.0):
        K.attn_prompt(self.cfg, self.q, self.k, self.v, self.cu, self.out, lse=self.lse, sm_scale=scale, status=self.st)
        torch.cuda.synchronize()
        assert int(self.st.item()) == 0

    def check(self, scale=None):
        exact = self.flags != 0
        f = lambda x: x.cpu().double().numpy()
        want = R.prompt(f(self.q), f(self.k), f(self.v), self.lens, self.first[:-1], scale or 1 / math.sqrt(self.cfg.head_dim), exact)
        rounding = R.F32 if self.flags & K.FLAG_OUT_FP32 else R.BF16
        R.check("out", f(self.out), want[0], want[2] + np.abs(want[0]) * rounding)
        R.check("lse", f(self.lse), want[1], want[3])


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("D,Hq,Hkv,lens", [
    (128, 1, 1, [1]), (128, 4, 1, [1, 1, 1]), (128, 8, 2, [64, 65, 63]), (128, 2, 2, [127, 128, 129]), (128, 3, 1, [84, 85, 43]),
    (128, 10, 2, [0, 200, 0, 0, 7, 51]), (128, 6, 1, [130]), (128, 7, 1, [19, 300]), (128, 8, 1, [33, 31, 16, 15, 17]),
    (128, 16, 8, [257]), (256, 4, 2, [1, 64, 200]), (256, 5, 1, [26, 130]), (256, 3, 3, [129, 128]), (512, 2, 1, [65, 0, 140]),
    (512, 8, 1, [16, 33]), (512, 3, 3, [130])])
def test_against_64_bits(D, Hq, Hkv, lens, kind):
    p = Prompt(D, Hq, Hkv, lens, kind)
    p.run()
    p.check()


@pytest.mark.parametrize("D,Hq,Hkv,lens", [(128, 8, 2, [1100, 700]), (128, 5, 1, [900]), (128, 1, 1, [1500]), (256, 4, 1, [800]),
                                           (512, 2, 1, [700])])
def test_longer_ones(D, Hq, Hkv, lens):
    p = Prompt(D, Hq, Hkv, lens)
    p.run()
    p.check()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [128, 256, 512])
def test_rows_around_the_sequences_and_other_scales(D, kind):
    p = Prompt(D, 4, 2, [50, 90], kind, before=37, behind=200)
    p.run(scale=0.05)
    p.check(0.05)


@pytest.mark.parametrize("D,kind", [(128, "bf16"), (256, "bf16"), (512, "bf16"), (128, "fp32")])
def test_scores_of_a_wide_range(D, kind):
    """Maxima that grow and fall by hundreds along a row, and keys far below them: the reference follows."""
    p = Prompt(D, 4, 2, [400], kind)
    size = torch.linspace(0.01, 6, 400, device="cuda")
    p.k[:400] *= size[torch.randperm(400, device="cuda")][:, None, None].to(p.k.dtype)
    p.run()
    p.check()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("D,G", [(128, 1), (128, 2), (128, 3), (128, 4), (128, 8), (256, 2), (256, 5), (512, 1), (512, 4)])
def test_what_is_not_finite_reaches_only_who_sees_it(D, G, kind):
    """Infinite values and NaN in V and K of single tokens, and everywhere behind the sequences, which is nobody's."""
    a, b = (Prompt(D, 2 * G, 2, [301, 140], kind, behind=70) for _ in range(2))
    nan, inf = float("nan"), float("inf")
    bad = [(100, 0, 3, inf), (101, 0, 3, -inf), (130, 0, 5, nan), (290, 0, 7, -inf), (300, 0, 1, nan)]
    for t, h, c, x in bad:
        b.v[t, h, c] = x
    b.k[200, 1, 2] = nan
    for x in (b.q, b.k, b.v):
        x[441:] = nan
    a.run(), b.run()
    want, got = a.out.float(), b.out.float()
    clean = torch.ones_like(want, dtype=torch.bool)
    for t, h, c, x in bad:
        clean[t:301, h * G:(h + 1) * G, c] = False
        assert not bool(torch.isfinite(got[t:301, h * G:(h + 1) * G, c]).any())
    clean[200:301, G:] = False
    assert bool(torch.isnan(got[200:301, G:]).all())
    assert bool((got[100, :G, 3] == inf).all()) and bool(torch.isnan(got[101, :G, 3]).all()) and bool((got[290, :G, 7] == -inf).all())
    assert torch.equal(got[clean], want[clean])  # bit for bit


@pytest.mark.parametrize("size", [1e4, 1e18, 1e30])
@pytest.mark.parametrize("D,kind", [(128, "bf16"), (512, "bf16"), (128, "fp32")])
def test_a_large_query_leaves_the_others_alone(D, kind, size):
    a, b = (Prompt(D, 8, 2, [200, 77], kind) for _ in range(2))
    b.q[90, 3] *= size
    a.run(), b.run()
    b.out[90, 3], b.lse[90, 3] = a.out[90, 3], a.lse[90, 3]
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


@pytest.mark.parametrize("D", [128, 256, 512])
def test_a_sequence_does_not_depend_on_its_batch(D):
    """Bit for bit: packed with others, alone, at another place."""
    p = Prompt(D, 8, 2, [90, 333, 5])
    p.run()
    for i, T in enumerate(p.lens):
        at = slice(int(p.first[i]), int(p.first[i]) + T)
        c = K.KVConfig(1, 1, 8, 2, D, 0, 0, 1)
        out, lse = torch.empty_like(p.out[at]), torch.empty_like(p.lse[at])
        K.attn_prompt(c, p.q[at].contiguous(), p.k[at].contiguous(), p.v[at].contiguous(), dev_i32([0, T]), out, lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(out, p.out[at]) and torch.equal(lse, p.lse[at])


@pytest.mark.parametrize("D,lens", [(128, [4000, 3, 900, 1500] * 2), (256, [2000, 300, 1200]), (512, [1500, 700, 90])])
def test_repeated_calls_give_the_same_bits(D, lens):
    """Many items a block, run after run, with other work on the GPU beside every other one."""
    p = Prompt(D, 16, 4, lens)
    p.run()
    want, lse = p.out.clone(), p.lse.clone()
    other, x = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    for i in range(40):
        p.out.fill_(7.0)
        if i % 2:
            with torch.cuda.stream(other):
                x @ x
        p.run()
        assert torch.equal(p.out, want) and torch.equal(p.lse, lse), i


@pytest.mark.parametrize("D,kind", [(128, "bf16"), (256, "bf16"), (512, "bf16"), (128, "fp32")])
def test_many_sequences(D, kind):
    """More than a warp's lanes, empty ones among them, in any order of length."""
    rng = np.random.default_rng(D)
    lens = [int(x) for x in rng.integers(0, 40, 70)]
    lens[13], lens[40] = 300, 0
    p = Prompt(D, 2, 1, lens, kind)
    p.run()
    p.check()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_bounds_out_of_range_are_clamped_and_flagged(kind):
    for cu in ([-5, 20, 40], [0, 30, 20], [0, 20, 4000], [50, 60, 70]):
        p = Prompt(128, 4, 2, [20, 20], kind, behind=0)
        p.cu = dev_i32(cu)
        K.attn_prompt(p.cfg, p.q, p.k, p.v, p.cu, p.out, lse=p.lse, status=p.st)
        torch.cuda.synchronize()
        assert int(p.st.item()) == K.DEV_OVER_CAPACITY
        assert bool(torch.isfinite(p.out.float()).all())


def test_no_sequences_with_rows():
    p = Prompt(128, 4, 2, [0, 0], behind=9)
    p.run()
    assert bool((p.out == 7).all()) and bool((p.lse == 7).all())


@pytest.mark.parametrize("D", [128, 256, 512])
def test_without_lse(D):
    p = Prompt(D, 4, 2, [150])
    p.run()
    out = torch.empty_like(p.out)
    K.attn_prompt(p.cfg, p.q, p.k, p.v, p.cu, out)
    torch.cuda.synchronize()
    assert torch.equal(out[:150], p.out[:150])


@pytest.mark.parametrize("D", [128, 256, 512])
def test_an_output_at_any_16_bytes(D):
    p = Prompt(D, 4, 2, [150, 41])
    p.run()
    flat = torch.full((p.out.numel() + 16,), 7.0, dtype=p.out.dtype, device="cuda")
    out = flat[8:8 + p.out.numel()].view(p.out.shape)
    K.attn_prompt(p.cfg, p.q, p.k, p.v, p.cu, out)
    torch.cuda.synchronize()
    assert out.data_ptr() % 32 == 16 and torch.equal(out, p.out)
    assert bool((flat[:8] == 7).all()) and bool((flat[-8:] == 7).all())


@pytest.mark.parametrize("D,lens", [(128, [600, 33]), (128, [1]), (256, [400]), (512, [300, 300])])
def test_a_wait_that_runs_out(D, lens):
    from tests.test_gpu_rows_timeout import times_out_and_recovers
    p = Prompt(D, 8, 2, lens, behind=0)
    times_out_and_recovers(lambda: K.attn_prompt(p.cfg, p.q, p.k, p.v, p.cu, p.out, lse=p.lse, status=p.st), [p.out, p.lse], p.st)
