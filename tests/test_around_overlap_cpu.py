"""Outputs over inputs that others still read are refused on the host.  Addresses are made up: a refused call reads none."""
import pytest

from int2_kv_cache_append_gb300 import oscar_kv as K
from tests.test_around_checks_cpu import CFG, P, _c

INVALID = -1


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


@pytest.mark.parametrize("flags", [0, K.FLAG_IN_FP32, K.FLAG_OUT_FP32, K.FLAG_IN_FP32 | K.FLAG_OUT_FP32])
def test_attn_prompt(flags):
    """5 tokens of 8 and 2 heads of 128: q, k and v one behind the other, and the output over one's last or first 16 bytes."""
    cfg = K.KVConfig(1, 2, 8, 2, 128, 4, 8, 64, flags=flags)
    size_in, size_out = 4 if flags & K.FLAG_IN_FP32 else 2, 4 if flags & K.FLAG_OUT_FP32 else 2
    q, kv, out = 5 * 8 * 128 * size_in, 5 * 2 * 128 * size_in, 5 * 8 * 128 * size_out
    far = 1 << 30
    for at in (P, P + q - 16, P + q, P + q + kv - 16, P + q + kv, P + q + 2 * kv - 16, P - out + 16):
        assert K.lib().attn_prompt(_c(cfg), P, P + q, P + q + kv, 5, P, 0.0, at, None, None, None) == INVALID
    for i in range(3):  # one input alone
        args = [far + i * (1 << 20) for i in range(3)]
        args[i] = P
        assert K.lib().attn_prompt(_c(cfg), *args, 5, P, 0.0, P, None, None, None) == INVALID


def rope(n=5, q=P, qs=8 * 128, k=P + (1 << 24), ks=2 * 128, qo=P + (2 << 24), ko=P + (3 << 24), fp32=False):
    cfg = K.KVConfig(1, 2, 8, 2, 128, 4, 8, 64, flags=K.FLAG_IN_FP32 if fp32 else 0)
    return K.lib().qk_norm_rope(_c(cfg), q, qs, k, ks, n, P, P, 1e-6, P, P, 128, 0, qo, ko, None)


@pytest.mark.parametrize("fp32", [False, True])
def test_qk_norm_rope(fp32):
    size = 4 if fp32 else 2
    q, k = 5 * 8 * 128 * size, 5 * 2 * 128 * size
    for over in (dict(qo=P + 16), dict(qo=P - 16), dict(ko=P + q - 16), dict(qo=P + (1 << 24) + k - 16), dict(ko=P + (2 << 24) + q - 16),
                 dict(ko=P + (1 << 24) + 16), dict(qs=8 * 128 + 8, qo=P), dict(ks=3 * 128, ko=P + (1 << 24)),
                 dict(q=P, qs=12 * 128, k=P + 8 * 128 * size, ks=12 * 128, qo=P + 10 * 128 * size)):
        assert rope(fp32=fp32, **over) == INVALID
