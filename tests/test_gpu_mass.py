"""attn_mass against its 64-bit form over the oracle's cached rows: head_dims, shared heads, query rows that do and do not fill
the kernel's tiles, windows of zero and of everything, ragged lengths and query counts (zero and one among them), modes; rows
of no token and memory of no position are garbage.  The weights of a decode step add up to the query heads."""
import math

import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from tests import around_ref as R
from tests import rows_ref
from tests.gpu_helpers import dev, dev_i32, dev_rot, kcfg
from tests.test_gpu_rows import cfg_of, filled

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def f64(x):
    return x.cpu().double().numpy()


class Mass:
    def __init__(self, D, Hq, Hkv, S_, W, lens, n, q_lens=None, flags=0, extra=9, layers=1, layer=0, scale=0.0):
        B, cap = len(lens), max(lens) + extra
        self.c = cfg_of(D, B, Hq, Hkv, S_, W, cap, flags, layers)
        self.cache, self.RK, self.RV, ch, rng = filled(self.c, lens, D + n + sum(lens), layer)
        self.kc, self.layer, self.lens, self.n = kcfg(self.c), layer, lens, n
        self.q_lens = [n] * B if q_lens is None else q_lens
        fp32 = bool(flags & K.FLAG_IN_FP32)
        q = S.activations(rng, (B, n, Hq, D), ch, mag=3.0)
        for b, m in enumerate(self.q_lens):
            q[b, m:] = np.nan
        self.q = dev(q, torch.float32 if fp32 else torch.bfloat16)
        self.scale, self.given = scale or 1 / math.sqrt(D), scale
        self.cdev = torch.from_numpy(self.cache).cuda()
        self.R = None if flags & K.FLAG_HADAMARD else dev_rot(self.RK)
        # the rows' log-sum-exp, in 64 bits
        Rk = np.asarray(rows_ref.O.rotations_of(self.c, self.RK, self.RV)[0], np.float64)
        lse = np.full((B, n, Hq), np.nan)
        for b in range(B):
            T = max(0, min(lens[b], cap))
            for t in range(min(self.q_lens[b], n)):
                last = T - min(self.q_lens[b], n) + t
                for i in range(Hq):
                    lse[b, t, i] = -np.inf
                    if last >= 0:
                        x = rows_ref.rows64(self.c, self.cache, layer, 0, b, i // self.c.G, T)[:last + 1] @ (f64(self.q)[b, t, i] @ Rk)
                        x = x * self.scale
                        lse[b, t, i] = x.max() + math.log(np.exp(x - x.max()).sum())
        self.lse = torch.from_numpy(lse.astype(np.float32)).cuda()
        self.before = torch.rand(B, Hkv, cap, generator=torch.Generator().manual_seed(1)).cuda()
        self.out = torch.full_like(self.before, 5.0)
        self.ws = torch.full((K.attn_mass_workspace_bytes(self.kc, n) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        self.st = dev_i32([0])

    def run(self, before=True, out=None, hint=0, stream=None):
        out = self.out if out is None else out
        size = K.attn_mass_workspace_bytes(self.kc, self.n)
        K.attn_mass(self.kc, self.cdev, self.layer, self.q, dev_i32(self.lens), self.R, self.lse, out, self.ws[:size],
                    mass_in=(self.before if before is True else before) if before is not None else None,
                    q_lens=dev_i32(self.q_lens), seq_len_hint=hint, sm_scale=self.given, status=self.st, stream=stream)
        torch.cuda.synchronize()
        assert bool((self.ws[size:] == 0xFF).all())
        return out

    def check(self, out=None, before=None):
        out = self.out if out is None else out
        start = f64(self.before) if before is None else before
        want, bound = R.mass(self.c, self.cache, self.layer, f64(self.q), self.q_lens, self.lens, self.RK, self.scale, f64(self.lse), start)
        for b, T in enumerate(self.lens):
            T = min(max(T, 0), self.c.capacity)
            R.check("mass", f64(out)[b, :, :T], want[b, :, :T], bound[b, :, :T])
            assert bool((out[b, :, T:] == 5.0).all())


CASES = [
    # D, Hq, Hkv, S, W, lens, n, q_lens, flags
    (128, 4, 1, 4, 8, [1], 1, None, 0),
    (128, 8, 2, 4, 8, [300, 5, 77, 0], 1, None, 0),
    (128, 8, 8, 64, 256, [600, 330], 1, None, 0),                          # a KV head per query head
    (128, 16, 2, 0, 0, [129, 128, 31, 32, 33], 1, None, 0),                # no windows; G = 8
    (128, 10, 2, 16, 32, [700, 50], 1, None, 0),                           # G = 5
    (128, 6, 2, 3, 500, [400, 503, 520], 1, None, K.FLAG_LLOYD_MAX),       # windows hold (almost) everything
    (128, 4, 1, 5, 31, [290, 1000], 5, [5, 2], 0),                         # 20 rows: tiles and a half
    (128, 8, 1, 4, 8, [100, 7, 300], 9, [9, 9, 0], 0),                     # tokens before the sequence; none
    (128, 7, 1, 4, 8, [333], 33, None, K.FLAG_LLOYD_MAX),
    (128, 8, 2, 4, 8, [300, 64], 20, None, K.FLAG_V_BF16),
    (128, 8, 2, 4, 8, [300, 64], 3, None, K.FLAG_HADAMARD | K.FLAG_IN_FP32),
    (256, 8, 2, 16, 32, [500, 90], 1, None, 0),
    (256, 5, 1, 3, 64, [333], 7, None, K.FLAG_LLOYD_MAX),
    (256, 16, 2, 3, 64, [333, 70], 1, None, K.FLAG_HADAMARD),
    (512, 4, 1, 7, 40, [260, 30], 1, None, 0),
    (512, 8, 1, 7, 40, [260, 30], 1, None, K.FLAG_LLOYD_MAX),
    (512, 6, 2, 0, 40, [200], 11, None, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_against_64_bits(case):
    m = Mass(*case)
    m.run()
    m.check()
    assert int(m.st.item()) == 0


@pytest.mark.parametrize("case", [CASES[1], CASES[6], CASES[11], CASES[16]])
def test_without_masses_before_and_in_place(case):
    m = Mass(*case)
    m.run(before=None)
    m.check(before=np.zeros(m.out.shape))
    first = m.run(out=torch.full_like(m.out, 5.0)).clone()
    m.before[:, :, max(m.lens):] = 5.0
    for b, T in enumerate(m.lens):
        m.before[b, :, T:] = 5.0
    m.run(out=m.before, before=m.before)
    assert torch.equal(first, m.before)  # the same bits where it is added to itself


@pytest.mark.parametrize("hint", [1, 40, 300])
def test_any_hint(hint):
    m = Mass(128, 8, 2, 4, 8, [300, 5, 77], 2)
    want = m.run().clone()
    assert torch.equal(m.run(out=torch.full_like(m.out, 5.0), hint=hint), want)


def test_other_layer_and_scale():
    m = Mass(128, 8, 2, 4, 8, [300, 64], 2, layers=3, layer=2, scale=0.05)
    m.run()
    m.check()


def test_length_above_capacity_is_clamped_and_flagged():
    m = Mass(128, 8, 2, 4, 8, [100, 64], 1, extra=0)
    want = m.run().clone()
    m.lens = [1000, 64]
    got = m.run(out=torch.full_like(m.out, 5.0))
    assert int(m.st.item()) == K.DEV_OVER_CAPACITY and torch.equal(got, want)


@pytest.mark.parametrize("D,G,T,n", [(128, 4, 3000, 1), (128, 8, 1500, 1), (512, 2, 700, 1), (128, 4, 900, 30)])
def test_weights_of_a_token_add_up_to_its_query_heads(D, G, T, n):
    """With the library's own log-sum-exp: attn_decode's and attn_extend's rows, all positions' weights sum to one a row."""
    c = cfg_of(D, 1, 2 * G, 2, 16, 64, T + 3)
    cache, RK, RV, ch, rng = filled(c, [T], D + T)
    kc, cdev, rk, rv = kcfg(c), torch.from_numpy(cache).cuda(), dev_rot(RK), dev_rot(RV)
    q = dev(S.activations(rng, (1, n, 2 * G, D), ch, mag=3.0))
    out, lse = torch.empty_like(q), torch.empty(1, n, 2 * G, device="cuda")
    if n == 1:
        ws = torch.empty(K.layout_query(kc)["decode_workspace_bytes"], dtype=torch.uint8, device="cuda")
        K.attn_decode(kc, cdev, 0, q[:, 0], dev_i32([T]), rk, rv, out[:, 0], ws, lse=lse[:, 0])
    else:
        ws = torch.empty(K.attn_extend_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
        K.attn_extend(kc, cdev, 0, q, dev_i32([T]), rk, rv, out, ws, lse=lse)
    mass = torch.zeros(1, 2, T + 3, device="cuda")
    ws = torch.empty(K.attn_mass_workspace_bytes(kc, n), dtype=torch.uint8, device="cuda")
    K.attn_mass(kc, cdev, 0, q, dev_i32([T]), rk, lse, mass, ws)
    torch.cuda.synchronize()
    # scores of both sides within 1e-6 of the largest magnitudes (up to about 40): 1e-4 of a weight
    assert np.allclose(f64(mass.double().sum(-1)), n * G, rtol=2e-4)


def test_rows_without_weight_add_nothing():
    m = Mass(128, 8, 2, 4, 8, [300], 4)
    want = m.run().clone()
    lse = m.lse.clone()
    m.lse[0, 2] = -math.inf
    less = m.run(out=torch.full_like(m.out, 5.0)).clone()
    m.lse[0, :] = -math.inf
    none = m.run(out=torch.full_like(m.out, 5.0))
    assert torch.equal(none[0, :, :300], m.before[0, :, :300])
    assert bool((less <= want).all()) and bool((less < want).any())
    m.lse.copy_(lse)


def test_no_tokens_copies():
    m = Mass(128, 8, 2, 4, 8, [300, 20], 1)
    q, lse = torch.empty(2, 0, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 0, 8, device="cuda")
    K.attn_mass(m.kc, m.cdev, 0, q, dev_i32([300, 20]), m.R, lse, m.out, m.ws[:0], mass_in=m.before)
    torch.cuda.synchronize()
    for b, T in enumerate((300, 20)):
        assert torch.equal(m.out[b, :, :T], m.before[b, :, :T]) and bool((m.out[b, :, T:] == 5).all())


@pytest.mark.parametrize("size", [1e4, 1e18])
@pytest.mark.parametrize("n", [1, 6])
def test_a_large_query_leaves_other_heads_alone(n, size):
    m = Mass(128, 8, 2, 4, 8, [300, 64], n)
    want = m.run().clone()
    m.q[0, 0, 1] *= size
    got = m.run(out=torch.full_like(m.out, 5.0))
    assert torch.equal(got[0, 1], want[0, 1]) and torch.equal(got[1], want[1])


MANY = [  # more than 32 query rows a KV head at head_dim 128: positions in the tensor memory's lanes
    (128, 8, 1, 0, 0, [255, 256, 257, 1, 0], 16, None, 0),                     # 128 rows, tiles full and not
    (128, 8, 2, 4, 8, [700, 30, 4, 11], 33, [33, 9, 33, 1], 0),                # 132 rows; before the sequence; a window only
    (128, 6, 2, 100, 300, [900, 399, 250], 43, [43, 0, 20], K.FLAG_LLOYD_MAX),  # 129 rows; windows over two tiles; no row
    (128, 5, 1, 3, 600, [590, 1200], 90, None, K.FLAG_HADAMARD | K.FLAG_IN_FP32),  # rows hidden inside the codes and the ring
    (128, 16, 2, 64, 0, [520, 64, 65], 60, None, K.FLAG_V_BF16),               # 480 rows; no ring
    (128, 8, 2, 0, 4, [300, 600], 290, None, 0),                               # hidden rows among codes
]


@pytest.mark.parametrize("case", MANY, ids=[f"{i}" for i in range(len(MANY))])
def test_many_rows_against_64_bits(case):
    m = Mass(*case)
    m.run()
    m.check()
    assert int(m.st.item()) == 0
    again = torch.full_like(m.out, 5.0)
    for hint in (1, 200):
        assert torch.equal(m.run(out=again.fill_(5.0), hint=hint), m.out)
    in_place = m.before.clone()
    for b, T in enumerate(m.lens):
        in_place[b, :, max(T, 0):] = 5.0
    assert torch.equal(m.run(out=in_place, before=in_place), m.out)


@pytest.mark.parametrize("case", [MANY[1], MANY[2], MANY[3]])
def test_a_wait_that_runs_out(case):
    from tests.test_gpu_rows_timeout import times_out_and_recovers
    m = Mass(*case)

    def call():
        m.out.fill_(5.0)
        K.attn_mass(m.kc, m.cdev, 0, m.q, dev_i32(m.lens), m.R, m.lse, m.out, m.ws[:K.attn_mass_workspace_bytes(m.kc, m.n)],
                    q_lens=dev_i32(m.q_lens), status=m.st)
    times_out_and_recovers(call, [m.out], m.st)


def test_many_rows_whose_query_or_weight_is_strange():
    """What is not finite stays with its KV head; a row without weight adds nothing."""
    m = Mass(128, 8, 2, 4, 8, [300, 64], 20)
    want = m.run().clone()
    m.q[0, 3, 1] = math.inf
    m.q[1, 2, 5] *= 1e18
    got = m.run(out=torch.full_like(m.out, 5.0))
    assert torch.equal(got[0, 1], want[0, 1]) and torch.equal(got[1, 0], want[1, 0])
    m = Mass(128, 8, 2, 4, 8, [300, 64], 20)
    m.lse[0, :] = -math.inf
    got = m.run(out=torch.full_like(m.out, 5.0))
    assert torch.equal(got[0, :, :300], m.before[0, :, :300]) and torch.equal(got[1], want[1])


def test_many_rows_captured_and_on_two_streams():
    """Replays give the bits of a plain call, also while another call with a workspace of its own runs on a second stream."""
    a, b = Mass(*MANY[1]), Mass(*MANY[3])
    want = [m.run().clone() for m in (a, b)]
    sizes = [K.attn_mass_workspace_bytes(m.kc, m.n) for m in (a, b)]
    given = [(dev_i32(m.lens), dev_i32(m.q_lens)) for m in (a, b)]

    def call(i, m, stream=None):
        K.attn_mass(m.kc, m.cdev, 0, m.q, given[i][0], m.R, m.lse, m.out, m.ws[:sizes[i]], mass_in=m.before, q_lens=given[i][1],
                    status=m.st, stream=stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0, a)
    other = torch.cuda.Stream()
    for m in (a, b):
        m.out.fill_(5.0)
    torch.cuda.synchronize()
    for _ in range(20):
        graph.replay()
        with torch.cuda.stream(other):
            call(1, b)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    assert int(a.st.item()) == int(b.st.item()) == 0
