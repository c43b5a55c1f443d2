"""Refused drafts: the ring slots that their append overwrote have to be put back,
or the shorter sequence reads the refused rows as the oldest ones of its window."""
import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from oracle import oscar_oracle as O
from tests.gpu_helpers import kcfg


def drafted(flags, lens, n, keep, W, restore):
    """History of every role, batch and head after `n` drafts of which `keep[b]` stay, and the one of a cache that only
    ever saw the kept ones."""
    D, B, H = 128, len(lens), 2
    c = O.Config(2, B, H, H, D, 3, W, max(lens) + n + 2, 0.96, 0.92, flags)
    rng = np.random.default_rng(n)
    R = S.qr_rotation(rng, D).astype(np.float32)
    rows = lambda m: S.to_bf16_values(S.activations(rng, (B, m, H, D), [3], mag=3.0))
    top = max(lens)
    prompt, drafts = [rows(top) for _ in range(2)], [rows(n) for _ in range(2)]
    caches = [O.new_cache(c) for _ in range(2)]
    for x in caches:
        O.append(c, x, 1, *prompt, [t - top for t in lens], R, R)
    # the one that never saw the others: each sequence appends its own kept ones
    want = []
    for b in range(B):
        x = caches[1].copy()
        if keep[b]:
            O.append(c, x, 1, *[d[:, :keep[b]] for d in drafts], lens, R, R)
        want.append(x)
    t = torch.from_numpy(caches[0])
    rings = [r for r in K.ring_rows(kcfg(c), t, 1) if r is not None]
    assert len(rings) == (1 if flags & K.FLAG_V_BF16 else 2)
    at = torch.tensor(lens)[:, None] + torch.arange(n)
    b, slots = torch.arange(B)[:, None], at % W
    saved = [r[b, :, slots].clone() for r in rings]
    O.append(c, caches[0], 1, *drafts, lens, R, R)
    if restore:
        refused = at >= (torch.tensor(lens) + torch.tensor(keep))[:, None]
        for r, s in zip(rings, saved):
            r[b.expand_as(at)[refused], :, slots[refused]] = s[refused]
    got = [[O.dequant_history(c, caches[0], 1, role, b, h, lens[b] + keep[b]) for role in (0, 1) for h in range(H)] for b in range(B)]
    ref = [[O.dequant_history(c, want[b], 1, role, b, h, lens[b] + keep[b]) for role in (0, 1) for h in range(H)] for b in range(B)]
    return all(np.array_equal(x, y) for g, r in zip(got, ref) for x, y in zip(g, r))


@pytest.mark.parametrize("flags", [0, K.FLAG_V_BF16, K.FLAG_LLOYD_MAX])
@pytest.mark.parametrize("lens,n,keep,W", [([40, 33], 5, [5, 2], 8), ([40, 9], 8, [0, 3], 8), ([6, 2], 4, [1, 0], 16), ([20, 21], 1, [0, 1], 1)])
def test_rings_put_back(lens, n, keep, W, flags):
    assert drafted(flags, lens, n, keep, W, True)


def test_not_put_back_the_refused_rows_are_read():
    assert not drafted(0, [40, 33], 5, [5, 2], 8, False)


def test_arguments():
    cfg = K.KVConfig(2, 1, 2, 2, 128, 3, 8, 40)
    cache = torch.zeros(K.layout_query(cfg)["total_bytes"], dtype=torch.uint8)
    k, v = K.ring_rows(cfg, cache, 1)
    assert k.shape == v.shape == (1, 2, 8, 128) and k.dtype == torch.bfloat16
    k.fill_(1.0)
    assert int((cache != 0).sum()) == 2 * 8 * 128 * 2
    for bad in (dict(cache=cache[:-1]), dict(cache=cache.to(torch.int32)), dict(layer=2), dict(layer=-1)):
        with pytest.raises(ValueError, match="oscar_kv"):
            K.ring_rows(**{**dict(cfg=cfg, cache=cache, layer=0), **bad})
    k, _ = K.ring_rows(K.KVConfig(1, 1, 2, 2, 128, 3, 0, 40), torch.zeros(10 ** 6, dtype=torch.uint8), 0)
    assert k.numel() == 0
