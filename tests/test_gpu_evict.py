"""kv_evict: which positions stay (ties, equal masses, NaN, infinities, negative ones), what the other cache, masses and lengths
are, byte for byte, over head_dims, modes, windows, ragged lengths and budgets; memory of no position is not written."""
import math

import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from oracle import oscar_oracle as O
from tests import around_ref as R
from tests.gpu_helpers import dev_i32, kcfg
from tests.test_gpu_append_packed import region_views

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


class Evict:
    def __init__(self, D, B, Hkv, S_, W, lens, keep, flags=0, cap=None, out_cap=None, mass=None, layers=(1, 0, 1, 0)):
        cap = cap or max(max(lens), 1) + 7
        out_cap = out_cap or min(cap, S_ + W + keep) + 5
        in_layers, self.layer, out_layers, self.out_layer = layers
        self.c = O.Config(in_layers, B, 2 * Hkv, Hkv, D, S_, W, cap, 0.96, 0.92, flags)
        self.oc = O.Config(out_layers, B, 2 * Hkv, Hkv, D, S_, W, out_cap, 0.9, 0.8, flags)
        self.kc, self.koc, self.lens, self.keep = kcfg(self.c), kcfg(self.oc), lens, keep
        g = torch.Generator().manual_seed(D + keep + sum(lens))
        self.cache = torch.randint(0, 256, (K.layout_query(self.kc)["total_bytes"],), generator=g, dtype=torch.uint8).cuda()
        if mass is None:  # heavy tails on a grid: many are equal
            mass = (torch.exp(2 * torch.randn(B, Hkv, cap, generator=g)) * 4).round() / 4
        self.mass = mass.cuda()
        self.out = torch.full((K.layout_query(self.koc)["total_bytes"],), 0xA5, dtype=torch.uint8, device="cuda")
        self.out_mass = torch.full((B, Hkv, out_cap), 9.0, device="cuda")
        self.kept = torch.full((B, Hkv, keep), 9, dtype=torch.int32, device="cuda")
        self.new = torch.full((B,), 9, dtype=torch.int32, device="cuda")
        self.ws = torch.full((K.kv_evict_workspace_bytes(self.kc, keep) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        self.st = dev_i32([0])

    def run(self, lens=None, new=None, out_mass=True, kept=True):
        size = K.kv_evict_workspace_bytes(self.kc, self.keep)
        K.kv_evict(self.kc, self.cache, self.layer, self.mass, dev_i32(self.lens) if lens is None else lens, self.keep, self.koc, self.out,
                   self.out_layer, self.new if new is None else new, self.ws[:size], out_mass=self.out_mass if out_mass else None,
                   kept=self.kept if kept else None, status=self.st)
        torch.cuda.synchronize()
        assert bool((self.ws[size:] == 0xFF).all())

    def layer_of(self, c, cache, layer):
        size = K.layout_query(kcfg(c))["layer_bytes"]
        return region_views(c, K.layout_query(kcfg(c)), cache[layer * size:(layer + 1) * size])

    def check(self):
        c, oc = self.c, self.oc
        S_, W, D, cap, ocap = c.sink, c.recent, c.head_dim, c.capacity, oc.capacity
        src = {k: v.cpu().numpy() for k, v in self.layer_of(c, self.cache, self.layer).items()}
        dst = {k: v.cpu().numpy() for k, v in self.layer_of(oc, self.out, self.out_layer).items()}
        mass, out_mass, kept, new = (x.cpu().numpy() for x in (self.mass, self.out_mass, self.kept, self.new))
        for b, T in enumerate(self.lens):
            T = max(0, min(T, cap))
            for h in range(c.num_kv_heads):
                body, N = R.evict_choice(mass[b, h], T, S_, W, self.keep)
                old = list(range(min(S_, T))) + body + list(range(max(S_, T - W) if T > S_ else T, T))
                assert len(old) == N
                assert new[b] == N
                assert kept[b, h].tolist() == body + [-1] * (self.keep - len(body))
                want = np.zeros(ocap, np.float32)
                want[:N] = mass[b, h, old]
                assert np.array_equal(out_mass[b, h], want, equal_nan=True)
                for name, was in src.items():
                    each = {"sink": 2 * D, "ring": 2 * D, "codes": D // 4, "sz": D // 32, "full": 2 * D}[name[1:]]
                    x, y = was[b, h].reshape(-1, each), dst[name][b, h].reshape(-1, each)
                    want = np.full_like(y, 0xA5)
                    for p, o in enumerate(old):
                        if name[1:] == "full":
                            want[p] = x[o]
                        elif name[1:] == "sink" and p < S_:
                            want[p] = x[o]
                        elif name[1:] == "ring" and p >= max(S_, N - W):
                            want[p % W] = x[o % W]
                        elif name[1:] in ("codes", "sz") and p >= S_:
                            want[p - S_] = x[o - S_]
                    assert np.array_equal(y, want), (name, b, h)


@pytest.mark.parametrize("D,B,Hkv,S_,W,lens,keep,flags", [
    (128, 3, 2, 4, 8, [100, 12, 50], 10, 0),                       # one without anything between the windows
    (128, 4, 1, 4, 8, [0, 1, 3, 13], 1, 0),                        # shorter than the windows; one position between
    (128, 2, 2, 4, 8, [70, 300], 0, 0),                            # nothing stays
    (128, 2, 2, 4, 8, [70, 300], 1000, 0),                         # everything
    (128, 2, 2, 4, 8, [70, 300], 288, 0),
    (128, 2, 1, 0, 0, [200, 129], 40, 0),                          # no windows
    (128, 2, 1, 0, 33, [200, 20], 40, K.FLAG_LLOYD_MAX),
    (128, 2, 3, 17, 0, [200, 16], 40, 0),
    (128, 2, 2, 4, 50, [90, 300], 20, K.FLAG_V_BF16),
    (128, 1, 1, 64, 256, [5000], 1000, 0),                         # several blocks' pieces
    (256, 2, 2, 5, 9, [130, 64], 33, 0),
    (256, 2, 1, 5, 9, [130, 64], 33, K.FLAG_V_BF16 | K.FLAG_LLOYD_MAX),
    (512, 2, 1, 3, 20, [100, 44], 25, 0),
    (512, 1, 2, 3, 20, [400], 130, K.FLAG_V_BF16),
])
def test_bytes(D, B, Hkv, S_, W, lens, keep, flags):
    e = Evict(D, B, Hkv, S_, W, lens, keep, flags)
    e.run()
    e.check()
    assert int(e.st.item()) == 0


@pytest.mark.parametrize("T,Hkv,keep", [(9000, 1, 4000), (40000, 2, 5), (40000, 1, 39000), (70001, 3, 20011), (8200, 40, 100)])
def test_long_ones_over_several_blocks(T, Hkv, keep):
    e = Evict(128, 1, Hkv, 4, 30, [T], keep)
    e.run()
    e.check()


@pytest.mark.parametrize("kind", ["equal", "zeros", "signs", "nan", "inf", "tiny", "all-nan"])
@pytest.mark.parametrize("T", [60, 9000])
def test_masses_that_compare_oddly(kind, T):
    rng = np.random.default_rng(3)
    m = rng.standard_normal((1, 2, T + 7)).astype(np.float32)
    if kind == "equal":
        m[:] = 0.25
    elif kind == "zeros":  # +0 and -0 are equal
        m = np.where(rng.random(m.shape) < 0.5, np.float32(-0.0), np.float32(0.0))
    elif kind == "nan":
        m[rng.random(m.shape) < 0.7] = np.nan
    elif kind == "inf":
        m[rng.random(m.shape) < 0.4] = np.inf
        m[rng.random(m.shape) < 0.4] = -np.inf
        m[rng.random(m.shape) < 0.4] = np.nan
    elif kind == "tiny":
        m = (m * np.float32(1e-42)).astype(np.float32)  # below the normal range
    elif kind == "all-nan":
        m[:] = np.nan
    e = Evict(128, 1, 2, 4, 8, [T], T // 3, mass=torch.from_numpy(m))
    e.run()
    e.check()


def test_layers_of_two_caches_and_of_one():
    e = Evict(128, 2, 2, 4, 8, [100, 40], 30, layers=(3, 2, 2, 1))
    e.run()
    e.check()
    size = K.layout_query(e.koc)["layer_bytes"]
    assert bool((e.out[:size] == 0xA5).all())
    # from one layer of a cache into another of the same
    e = Evict(128, 2, 2, 4, 8, [100, 40], 30, layers=(3, 2, 3, 0), out_cap=107)
    size = K.layout_query(e.kc)["layer_bytes"]
    e.oc.k_clip, e.oc.v_clip = e.c.k_clip, e.c.v_clip
    e.koc = e.kc
    both = e.cache
    both[:size] = 0xA5
    e.out = both
    e.run()
    e.check()


def test_lengths_in_place_and_without_the_optional_outputs():
    e = Evict(128, 3, 2, 4, 8, [100, 12, 50], 10)
    e.run()
    want, lens = e.out.clone(), dev_i32(e.lens)
    e.out.fill_(0xA5)
    e.run(lens=lens, new=lens, out_mass=False, kept=False)
    assert torch.equal(lens, e.new) and torch.equal(want, e.out)


def test_lengths_out_of_range():
    e = Evict(128, 3, 2, 4, 8, [500, -4, 50], 10, cap=90)
    e.run()
    e.check()
    assert int(e.st.item()) == K.DEV_OVER_CAPACITY


def test_of_the_smallest_capacity_that_is_allowed():
    e = Evict(128, 2, 2, 4, 8, [100, 15], 10, out_cap=22)
    e.run()
    e.check()
