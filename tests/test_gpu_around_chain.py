"""The operators around the cache as a serving program runs them: prompts normed and rotated, attended and appended packed,
decode steps whose weights are added up, an eviction, further steps; against the same in 64 bits from the caches' bytes, eagerly,
on another stream and captured into a graph and replayed on other inputs."""
import math

import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from oracle import oscar_oracle as O
from tests import around_ref as R
from tests import rows_ref
from tests.gpu_helpers import dev_i32, dev_rot, kcfg

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


class Program:
    """One layer of a model's serving loop over prompts of the lengths `lens`, `steps` tokens, an eviction to `keep` and `steps` more."""

    def __init__(self, D, Hq, Hkv, S_, W, lens, steps, keep, flags=0, seed=0, stream=None):
        B = len(lens)
        self.lens, self.steps, self.keep, self.stream, self.D = lens, steps, keep, stream, D
        cap = max(lens) + steps
        self.c = O.Config(1, B, Hq, Hkv, D, S_, W, cap, 0.96, 0.92, flags)
        self.oc = O.Config(1, B, Hq, Hkv, D, S_, W, min(cap, S_ + W + keep) + steps, 0.96, 0.92, flags)
        self.kc, self.koc = kcfg(self.c), kcfg(self.oc)
        rng = np.random.default_rng(seed)
        self.R = (None, None) if flags & K.FLAG_HADAMARD else tuple(S.qr_rotation(rng, D).astype(np.float32) for _ in range(2))
        self.rk, self.rv = (dev_rot(x) for x in self.R)
        self.n, self.width = sum(lens), (Hq + 2 * Hkv) * D
        self.w = [dev_rot(1 + 0.2 * rng.standard_normal(D)) for _ in range(2)]
        self.freq = dev_rot(1e4 ** (-np.arange(0, D, 2) / D))
        self.cu = dev_i32(np.concatenate(([0], np.cumsum(lens))))
        self.pos = dev_i32(np.concatenate([np.arange(x) for x in lens]))
        self.zero = dev_i32([0] * B)
        self.fused = torch.zeros(self.n, self.width, dtype=torch.bfloat16, device="cuda")
        self.token = torch.zeros(2 * steps, B, self.width, dtype=torch.bfloat16, device="cuda")
        e = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")
        f32 = torch.float32
        self.q, self.k, self.v = e(self.n, Hq, D), e(self.n, Hkv, D), e(self.n, Hkv, D)
        self.out, self.lse = e(self.n, Hq, D), e(self.n, Hq, t=f32)
        self.cache, self.cache2 = (e(K.layout_query(x)["total_bytes"], t=torch.uint8) for x in (self.kc, self.koc))
        self.tq, self.tk, self.tout, self.tlse = e(2 * steps, B, Hq, D), e(2 * steps, B, Hkv, D), e(2 * steps, B, Hq, D), e(2 * steps, B, Hq, t=f32)
        self.mass, self.mass2 = e(B, Hkv, cap, t=f32), e(B, Hkv, self.oc.capacity, t=f32)
        self.seq, self.start, self.length = dev_i32([0] * B), dev_i32([0] * B), dev_i32([0] * B)
        self.kept = e(B, Hkv, keep, t=torch.int32)
        need = max(K.layout_query(self.kc)["decode_workspace_bytes"], K.layout_query(self.koc)["decode_workspace_bytes"])
        self.ws = e(max(need, K.attn_mass_workspace_bytes(self.kc, 1), K.kv_evict_workspace_bytes(self.kc, keep)), t=torch.uint8)
        self.st = dev_i32([0])
        self.lens_dev = dev_i32(lens)
        self.draw(seed)

    def draw(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.fused.copy_(torch.randn(self.fused.shape, generator=g).bfloat16())
        self.token.copy_(torch.randn(self.token.shape, generator=g).bfloat16())

    def split(self, x):
        Hq, H, D = self.c.num_q_heads, self.c.num_kv_heads, self.D
        n = x.shape[0]
        return x[:, :Hq * D].view(n, Hq, D), x[:, Hq * D:(Hq + H) * D].view(n, H, D), x[:, (Hq + H) * D:].view(n, H, D)

    def step(self, i, kc, cache, mass):
        """Token i of every sequence: its position counts on, its place in the cache is the length."""
        q, k, v = self.split(self.token[i])
        s = self.stream
        K.qk_norm_rope(self.kc, q, k, *self.w, self.seq, self.freq, self.tq[i], self.tk[i], stream=s)
        self.start.copy_(self.length)
        self.length.add_(1)
        self.seq.add_(1)
        K.decode_step(kc, cache, 0, self.tk[i][:, None], v[:, None].contiguous(), self.start, self.tq[i], self.length, self.rk, self.rv,
                      self.tout[i], self.ws, lse=self.tlse[i], status=self.st, stream=s)
        K.attn_mass(kc, cache, 0, self.tq[i][:, None], self.length, self.rk, self.tlse[i][:, None], mass, self.ws, mass_in=mass,
                    status=self.st, stream=s)

    def run(self):
        s = self.stream
        q, k, v = self.split(self.fused)
        self.mass.zero_()
        self.length.copy_(self.lens_dev)
        self.seq.copy_(self.lens_dev)
        K.qk_norm_rope(self.kc, q, k, *self.w, self.pos, self.freq, self.q, self.k, stream=s)
        self.v.copy_(v)
        K.attn_prompt(self.kc, self.q, self.k, self.v, self.cu, self.out, lse=self.lse, status=self.st, stream=s)
        K.kv_append_packed(self.kc, self.cache, 0, self.k, self.v, self.cu, self.zero, self.rk, self.rv, status=self.st, stream=s)
        for i in range(self.steps):
            self.step(i, self.kc, self.cache, self.mass)
        K.kv_evict(self.kc, self.cache, 0, self.mass, self.length, self.keep, self.koc, self.cache2, 0, self.length, self.ws,
                   out_mass=self.mass2, kept=self.kept, status=self.st, stream=s)
        for i in range(self.steps, 2 * self.steps):
            self.step(i, self.koc, self.cache2, self.mass2)

    def results(self):
        return [self.out, self.lse, self.tout, self.tlse, self.mass, self.mass2, self.kept, self.length, self.cache, self.cache2]


def f64(x):
    return x.cpu().double().numpy()


@pytest.mark.parametrize("D,Hq,Hkv,S_,W,lens,steps,keep,flags", [
    (128, 8, 2, 4, 16, [150, 61], 3, 40, 0), (128, 4, 1, 4, 16, [90, 200, 33], 2, 30, K.FLAG_HADAMARD | K.FLAG_LLOYD_MAX),
    (256, 4, 2, 4, 8, [70, 100], 2, 25, K.FLAG_V_BF16), (512, 4, 1, 4, 8, [64], 2, 25, 0)])
def test_program_against_64_bits(D, Hq, Hkv, S_, W, lens, steps, keep, flags):
    p = Program(D, Hq, Hkv, S_, W, lens, steps, keep, flags, seed=D + keep)
    p.run()
    torch.cuda.synchronize()
    assert int(p.st.item()) == 0
    w, freq = [f64(x) for x in p.w], f64(p.freq)
    q, k, v = (f64(x) for x in p.split(p.fused))
    pos = f64(p.pos)
    for name, x, wt, got in (("q", q, w[0], p.q), ("k", k, w[1], p.k)):
        R.check(name, f64(got), *R.norm_rope(x, wt, 1e-6, pos, freq, False, False))
    first = np.concatenate(([0], np.cumsum(lens)))
    scale = 1 / math.sqrt(D)
    out, lse, ob, lb = R.prompt(f64(p.q), f64(p.k), f64(p.v), lens, first[:-1], scale, False)
    R.check("out", f64(p.out), out, ob + np.abs(out) * R.BF16)
    R.check("lse", f64(p.lse), lse, lb)
    # steps: attn_decode's own tests hold its tolerances; here the caches' bytes after the last step of each half
    RK, RV = p.R
    for half, (c, cache) in enumerate(((p.c, p.cache), (p.oc, p.cache2))):
        i = half * steps + steps - 1
        T = [x + steps for x in lens] if half == 0 else p.length.tolist()
        want, _ = O.decode(c, cache.cpu().numpy(), 0, f64(p.tq[i]).astype(np.float32), T, RK, RV)
        err = np.linalg.norm(f64(p.tout[i]) - want) / np.linalg.norm(want)
        assert err < 2.0 ** -8 + 1e-3
    # the last step's weights before the eviction, and the choice made from them
    mass, kept, new = p.mass.cpu().numpy(), p.kept.cpu().numpy(), [x - steps for x in p.length.tolist()]
    for b, x in enumerate(lens):
        assert abs(mass[b, :, :x + steps].sum() - steps * Hq) < 2e-3 * steps * Hq
        assert bool((mass[b, :, x + steps:] == 0).all())
        for h in range(Hkv):
            body, N = R.evict_choice(mass[b, h], x + steps, S_, W, keep)
            assert N == new[b] and kept[b, h].tolist() == body + [-1] * (keep - len(body))
            # the rows that stayed are the ones that they were
            a = rows_ref.rows64(p.c, p.cache.cpu().numpy(), 0, 0, b, h, x + steps)
            z = rows_ref.rows64(p.oc, p.cache2.cpu().numpy(), 0, 0, b, h, N + steps)
            if len(body) and S_ + len(body) <= max(S_, N + steps - W):
                assert np.array_equal(z[S_:S_ + len(body)], a[body])


@pytest.mark.parametrize("D,flags", [(128, 0), (256, 0), (512, K.FLAG_HADAMARD)])
def test_repeated_on_another_stream_and_replayed(D, flags):
    p = Program(D, 8, 2, 4, 16, [150, 61, 7], 2, 40, flags, seed=1)
    p.run()
    torch.cuda.synchronize()
    eager = {1: [x.clone() for x in p.results()]}
    p.draw(2)
    p.run()
    torch.cuda.synchronize()
    eager[2] = [x.clone() for x in p.results()]

    other = torch.cuda.Stream()
    p.draw(1)
    torch.cuda.synchronize()
    p.stream = other
    with torch.cuda.stream(other):
        p.run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager[1], p.results()))

    p.stream = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for seed in (2, 1, 2):
        p.draw(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager[seed], p.results())), seed
    assert int(p.st.item()) == 0


def test_two_programs_at_once():
    """Buffers of their own, streams of their own: neither sees the other."""
    ps = [Program(128, 8, 2, 4, 16, [400, 61, 7], 2, 40, seed=s) for s in (1, 2)]
    want = []
    for p in ps:
        p.run()
        torch.cuda.synchronize()
        want.append([x.clone() for x in p.results()])
    for p in ps:
        p.stream = torch.cuda.Stream()
    for _ in range(3):
        for p in ps:
            with torch.cuda.stream(p.stream):
                p.run()
        torch.cuda.synchronize()
        for p, w in zip(ps, want):
            assert all(torch.equal(a, b) for a, b in zip(w, p.results()))
