"""The bounds of rows_bounds.py hold for the arithmetic that the kernels use and
not for it with a part left out: without the low part of the query, without
those of the rank-one middles, without the Lloyd-Max residues."""
import numpy as np
import pytest

from int2_kv_cache_append_gb300 import oscar_kv as K
from oracle import oscar_oracle as O
from tests import rows_bounds as B
from tests.test_gpu_rows_accuracy import inputs


def lse_of(s):
    top = s.max(1)
    return top + np.log(np.exp(s - top[:, None]).sum(1))


@pytest.mark.parametrize("D,flags,parts", [(128, 0, ["q", "middle"]), (256, 0, ["q", "middle"]), (512, 0, ["q", "middle"]),
                                           (128, K.FLAG_LLOYD_MAX, ["q", "middle", "residue"]),
                                           (512, K.FLAG_LLOYD_MAX, ["q", "middle", "residue"])])
def test_bounds(D, flags, parts):
    T, n = 300, 40
    c, cache, q = inputs(D, 1, T, n, flags)
    lm, scale = bool(flags), D ** -0.5
    worst = {d: 0.0 for d in ["", *parts]}
    for h in range(c.num_q_heads):
        mid, steps, s, factor = B.pieces(c, cache, 0, 0, h // c.G, T)
        V, floor = B.values(c, cache, 0, 0, h // c.G, T)
        x = q[0, :, h].astype(np.float64)
        hidden = np.zeros((n, T), bool)
        _, lse, _, lb = B.attend(x, mid, steps, factor, V, floor, hidden, scale, lm)
        bound = B.score_bound(x, mid, steps, factor, scale, lm)
        exact = scale * (x @ (steps + np.repeat(mid, 128, axis=1)).T)
        for d in worst:
            got = B.emulated_scores(x, mid, steps, s, scale, lm, d)
            if not d:
                assert (np.abs(got - exact) <= bound).all()
            worst[d] = max(worst[d], (np.abs(lse_of(got) - lse) / lb).max())
    assert worst[""] <= 1
    assert all(worst[d] > 1.5 for d in parts), worst
