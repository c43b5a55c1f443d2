"""The binding keeps the C form of the configurations in use by their fields, whatever else a program keeps in them."""
import dataclasses

import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from tests.test_binding_checks_cpu import _append_args, _decode_args


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def test_attributes_that_cannot_be_hashed():
    cfg = dataclasses.replace(_append_args()["cfg"])
    cfg.layers, cfg.names = [1, 2], {"a": 1}
    with pytest.raises(ValueError, match="CUDA tensor"):
        K.kv_append(**_append_args(cfg=cfg))
    with pytest.raises(ValueError, match="CUDA tensor"):
        K.attn_decode(**_decode_args(cfg=cfg))
    with pytest.raises(ValueError, match="CUDA tensor"):
        K.kv_append_packed(cfg, torch.zeros(K.layout_query(cfg)["total_bytes"], dtype=torch.uint8), 0,
                           torch.zeros(5, 2, 128, dtype=torch.bfloat16), torch.zeros(5, 2, 128, dtype=torch.bfloat16),
                           torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(128, 128), torch.zeros(128, 128))


def test_the_order_in_which_fields_were_set():
    """Two configurations whose fields' values, in the order of their last assignment, are the same."""
    a, b = (K.KVConfig(1, 2, 8, 2, 128, 4, 8, 64) for _ in range(2))
    names = [{"sink": "recent", "recent": "sink"}.get(f.name, f.name) for f in dataclasses.fields(b)]
    values = list(vars(b).values())
    vars(b).clear()
    for name, value in zip(names, values):
        setattr(b, name, value)
    assert (b.sink, b.recent) == (8, 4)
    for c in (a, b):
        got, total = K._known_cfg(c)
        assert (got.sink, got.recent, got.capacity) == (c.sink, c.recent, c.capacity)
        assert total == K.layout_query(c)["total_bytes"]
