"""kv_read of rows of small magnitude: INT2 rows are scale and zero in fp16, which
the tensor-core form must not push further down; what it gives agrees with the
64-bit form and with the few-row form whatever the rows' size."""
import numpy as np
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from int2_kv_cache_append_gb300 import synth as S
from oracle import oscar_oracle as O
from tests import rows_ref as R
from tests.gpu_helpers import dev_i32, dev_rot, kcfg
from tests.test_gpu_rows import cfg_of

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


@pytest.mark.parametrize("size", [1e-5, 1e-3, 1.0, 1e4])
@pytest.mark.parametrize("fp32", [True, False], ids=["fp32", "bf16"])
@pytest.mark.parametrize("D,H,T,flags", [(128, 4, 400, 0), (128, 4, 400, K.FLAG_LLOYD_MAX), (256, 4, 300, K.FLAG_LLOYD_MAX),
                                         (256, 4, 300, 0), (512, 4, 200, 0), (512, 4, 200, K.FLAG_LLOYD_MAX)])
def test_read(D, H, T, flags, fp32, size):
    c = cfg_of(D, 1, H, H, 5, 20, T, flags | (K.FLAG_OUT_FP32 if fp32 else 0))
    rng = np.random.default_rng(D + T)
    RK, RV = S.qr_rotation(rng, D).astype(np.float32), S.qr_rotation(rng, D).astype(np.float32)
    # rows of one call differ in size as well: every fourth is another 2^-6 smaller
    k, v = (S.to_bf16_values(S.activations(rng, (1, T, H, D), [3, 70], mag=3.0) * np.float32(size)) for _ in range(2))
    k[:, ::4] *= np.float32(2.0 ** -6)
    cache = O.new_cache(c)
    O.append(c, cache, 0, k, v, [0], RK, RV)
    cdev, R_, kind = torch.from_numpy(cache).cuda(), (dev_rot(RK), dev_rot(RV)), torch.float32 if fp32 else torch.bfloat16
    assert T * H * D >= 1 << 17  # the tensor-core form
    kv = [torch.empty((1, T, H, D), dtype=kind, device="cuda") for _ in range(2)]
    K.kv_read(kcfg(c), cdev, 0, dev_i32([0]), dev_i32([T]), *R_, *kv)
    few = [torch.empty((1, 8, H, D), dtype=kind, device="cuda") for _ in range(2)]
    K.kv_read(kcfg(c), cdev, 0, dev_i32([64]), dev_i32([T]), *R_, *few)
    torch.cuda.synchronize()
    zero = np.zeros((1, T, H, D))
    want = R.read(c, cache, 0, [0], [T], T, RK, RV, zero, zero)
    for role in (0, 1):
        got, part = kv[role].double().cpu().numpy(), few[role].double().cpu().numpy()
        # rows that left fp16's range when they were appended (scale or zero infinite) come back as no numbers
        lost = ~np.isfinite(want[role]).all(-1)
        assert (size > 1 or not lost.any()) and not np.isfinite(got[lost]).any() and not np.isfinite(part[lost[:, 64:72]]).any()
        got[lost], part[lost[:, 64:72]], want[role][lost] = 0, 0, 0
        norm = np.linalg.norm(want[role], axis=-1)
        # float32: D products and sums per element, matrix and rows in two fp16 values (2^-21 of a product each, on a middle
        # and steps of up to three times the row); bf16: in one (2^-11 each), and the output's rounding
        bound = (4 * D * 2.0 ** -24 + 6 * 2.0 ** -21 if fp32 else 6 * 2.0 ** -11 + 2.0 ** -8) * norm + 1e-30
        R.check_rows("kv"[role], got, want[role], bound)
        R.check_rows("few", part, want[role][:, 64:72], bound[:, 64:72])
