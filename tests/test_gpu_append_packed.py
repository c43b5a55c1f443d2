"""kv_append_packed writes what kv_append of every sequence's own rows writes, byte for byte, in every mode and on every kernel
path (sizes on both sides of the paths' borders; rotations that are exact in any arithmetic), and nothing else."""
import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from oracle import oscar_oracle as O
from tests.gpu_helpers import dev, dev_i32, dev_rot, kcfg

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def region_views(c, lay, cache):
    """Every region of a one-layer cache as bytes [B][Hkv][..]."""
    B, H, D = c.batch, c.num_kv_heads, c.head_dim
    out = {}
    for role, name in enumerate("kv"):
        at = role * lay["role_bytes"]
        parts = (("sink", c.sink * D * 2, lay["sink_bytes"]), ("ring", c.recent * D * 2, lay["ring_bytes"]),
                 ("codes", lay["ncap"] * (D // 4), lay["codes_bytes"]), ("sz", lay["ncap"] * (D // 32), lay["sz_bytes"]))
        if role and c.flags & K.FLAG_V_BF16:
            parts = (("full", c.capacity * D * 2, lay["v_role_bytes"]),)
        for part, each, whole in parts:
            out[name + part] = cache[at:at + B * H * each].view(B, H, each)
            at += whole
    return out


@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D,Hkv,S_,W,lens,starts,flags", [
    (128, 2, 4, 8, [5, 0, 1, 40], [0, 3, 7, 0], 0),                    # row-parallel
    (128, 4, 64, 256, [300, 17, 555], [0, 0, 20], 0),                   # tensor cores (bf16), tiled (float32)
    (128, 3, 0, 0, [700, 0, 201], [0, 0, 0], 0),
    (128, 2, 5, 31, [900, 300], [0, 11], K.FLAG_HADAMARD),              # eight rows to a warp
    (128, 1, 5, 31, [9, 300], [2, 11], K.FLAG_HADAMARD),
    (128, 8, 16, 32, [400, 77], [0, 0], K.FLAG_HADAMARD | K.FLAG_LLOYD_MAX),
    (128, 2, 4, 8, [600, 130], [0, 0], K.FLAG_V_BF16),
    (128, 2, 4, 8, [600, 130], [0, 9], K.FLAG_HADAMARD | K.FLAG_V_BF16),
    (128, 2, 4, 8, [50, 600], [0, 9], K.FLAG_LLOYD_MAX),
    (256, 2, 7, 20, [30, 2, 11], [0, 0, 100], 0),                       # clusters
    (256, 4, 7, 20, [300, 99], [0, 0], 0),
    (256, 4, 7, 20, [300, 99], [0, 0], K.FLAG_HADAMARD),
    (512, 2, 7, 20, [30, 2], [0, 0], 0),
    (512, 4, 64, 128, [300, 90], [0, 50], K.FLAG_HADAMARD | K.FLAG_LLOYD_MAX),
    (512, 4, 3, 600, [300, 90], [0, 50], 0),
])
def test_bytes_of_every_sequence(D, Hkv, S_, W, lens, starts, flags, fp32):
    rng = np.random.default_rng(D + sum(lens))
    B, cap = len(lens), max(a + n for a, n in zip(starts, lens)) + 5
    flags |= K.FLAG_IN_FP32 if fp32 else 0
    kind = torch.float32 if fp32 else torch.bfloat16
    c = O.Config(1, B, 2 * Hkv, Hkv, D, S_, W, cap, 0.96, 0.92, flags)
    one = O.Config(1, 1, 2 * Hkv, Hkv, D, S_, W, cap, 0.96, 0.92, flags)
    had = bool(flags & K.FLAG_HADAMARD)
    R = (None, None) if had else tuple(dev_rot(S.signed_permutation(rng, D)) for _ in range(2))
    before, behind = 3, 4
    n = before + sum(lens) + behind
    k, v = (dev(S.activations(rng, (n, Hkv, D), rng.choice(D, 3, replace=False), mag=3.0), kind) for _ in range(2))
    k[:before], v[n - behind:] = float("nan"), float("nan")  # rows of no sequence
    cu = before + np.concatenate(([0], np.cumsum(lens)))
    total = K.layout_query(kcfg(c))["total_bytes"]
    cache, st = torch.full((total,), 0x5A, dtype=torch.uint8, device="cuda"), dev_i32([0])
    K.kv_append_packed(kcfg(c), cache, 0, k, v, dev_i32(cu), dev_i32(starts), *R, status=st)
    got = region_views(c, K.layout_query(kcfg(c)), cache)
    for b in range(B):
        mine = torch.full((K.layout_query(kcfg(one))["total_bytes"],), 0x5A, dtype=torch.uint8, device="cuda")
        at = slice(int(cu[b]), int(cu[b + 1]))
        if lens[b]:  # kv_append takes no empty tensors; nothing is written then
            K.kv_append(kcfg(one), mine, 0, k[at][None].contiguous(), v[at][None].contiguous(), dev_i32([starts[b]]), *R)
        torch.cuda.synchronize()
        for name, want in region_views(one, K.layout_query(kcfg(one)), mine).items():
            assert torch.equal(got[name][b], want[0]), (name, b)
    assert int(st.item()) == 0


@pytest.mark.parametrize("rows,flags", [(20, 0), (2000, 0), (2000, K.FLAG_HADAMARD), (20, K.FLAG_HADAMARD)])
def test_positions_outside_are_skipped_and_flagged(rows, flags):
    c = K.KVConfig(1, 2, 4, 1, 128, 2, 4, 50, flags=flags)
    R = (None, None) if flags else (torch.eye(128, device="cuda"),) * 2
    lay = K.layout_query(c)
    k = torch.randn(rows, 1, 128, device="cuda").bfloat16()
    cu = dev_i32([0, rows // 2, rows])
    base = torch.zeros(lay["total_bytes"] + 4096, dtype=torch.uint8, device="cuda")
    base[lay["total_bytes"]:] = 0xEE
    st = dev_i32([0])
    K.kv_append_packed(c, base[:lay["total_bytes"]], 0, k, k, cu, dev_i32([-3, 45]), *R, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == K.DEV_OVER_CAPACITY
    assert bool((base[lay["total_bytes"]:] == 0xEE).all())


@pytest.mark.parametrize("cu", [[0, 900, 300], [-7, 5, 2 ** 31 - 1], [500, 400, 300], [2 ** 30, 2 ** 30 + 5, 2 ** 31 - 1]])
@pytest.mark.parametrize("flags", [0, K.FLAG_HADAMARD])
@pytest.mark.parametrize("rows", [20, 1500])
def test_bounds_out_of_order_write_nothing_outside(rows, flags, cu):
    c = K.KVConfig(1, 2, 4, 1, 128, 2, 4, 50, flags=flags)
    R = (None, None) if flags else (torch.eye(128, device="cuda"),) * 2
    lay = K.layout_query(c)
    k = torch.randn(rows, 1, 128, device="cuda").bfloat16()
    base = torch.full((lay["total_bytes"] + 8192,), 0xEE, dtype=torch.uint8, device="cuda")
    K.kv_append_packed(c, base[4096:4096 + lay["total_bytes"]], 0, k, k, dev_i32(cu), dev_i32([0, 0]), *R)
    torch.cuda.synchronize()
    assert bool((base[:4096] == 0xEE).all()) and bool((base[4096 + lay["total_bytes"]:] == 0xEE).all())


@pytest.mark.parametrize("D", [128, 256, 512])
@pytest.mark.parametrize("n", [1, 300, 3000])
def test_hadamard_rows_as_the_oracle_codes_them(D, n):
    """Large Hadamard appends against the oracle's codec on the kernel's own rotated rows, non-finite rows among them."""
    rng = np.random.default_rng(n)
    c = O.Config(1, 1, 2, 1, D, 4, 16, n + 3, 0.96, 0.92, K.FLAG_HADAMARD)
    k, v = (dev(S.activations(rng, (1, n, 1, D), rng.choice(D, 3, replace=False), mag=3.0)) for _ in range(2))
    if n > 100:
        k[0, 50, 0, 3], v[0, 60, 0, 4], k[0, 70] = float("nan"), float("inf"), 0
    cache = torch.zeros(K.layout_query(kcfg(c))["total_bytes"], dtype=torch.uint8, device="cuda")
    rot, st = torch.empty(1, n, 1, 2, D, device="cuda"), dev_i32([0])
    K.kv_append(kcfg(c), cache, 0, k, v, dev_i32([0]), None, None, debug_rot=rot, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == (K.DEV_NONFINITE | K.DEV_FP16_RANGE if n > 100 else 0)
    lay = K.layout_query(kcfg(c))
    views = region_views(c, lay, cache)
    rows = rot.cpu().numpy()
    for role, name in enumerate("kv"):
        r = rows[0, 4:, 0, role]
        if not len(r):
            continue
        fine = np.isfinite(r).all(1)
        codes, scale, zero = O.quantize_rows(r[fine], (0.96, 0.92)[role])
        got = views[name + "codes"][0, 0].cpu().numpy().reshape(-1, D // 4)[:n - 4][fine]
        assert np.array_equal(got, O.pack_codes(codes, role).view(np.uint8).reshape(got.shape))
        sz = views[name + "sz"][0, 0].cpu().numpy().view(np.float16).reshape(-1, D // 128, 2)[:n - 4][fine]
        assert np.array_equal(sz[..., 0], scale) and np.array_equal(sz[..., 1], zero)
