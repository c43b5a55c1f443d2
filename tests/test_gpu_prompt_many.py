"""attn_prompt where a block has many items one behind the other: every sequence and KV head as it is alone, bit for bit."""
import math

import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K
from tests.gpu_helpers import dev_i32
from tests.test_gpu_prompt import Prompt

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


def items_of(D, G, heads, lens):
    """Items of a call: a block has 128 // G tokens with their G heads, twice that at head_dim 128; at 512 two share them."""
    tokens = 128 // G * (2 if D == 128 else 1)
    return sum(math.ceil(T / tokens) for T in lens) * heads * (2 if D == 512 else 1)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def each_as_alone(p, which=None):
    """Every sequence (or those in `which`) and query head in a call of its own, which has at most one item a block."""
    D, G = p.cfg.head_dim, p.cfg.num_q_heads // p.cfg.num_kv_heads
    for i in range(len(p.lens)) if which is None else which:
        T, at = p.lens[i], slice(int(p.first[i]), int(p.first[i + 1]))
        assert items_of(D, 1, 1, [T]) <= sms()
        for h in range(p.cfg.num_q_heads):
            q, k, v = (x[at, j:j + 1].contiguous() for x, j in ((p.q, h), (p.k, h // G), (p.v, h // G)))
            out, lse = torch.empty_like(q), torch.empty(T, 1, device="cuda")
            K.attn_prompt(K.KVConfig(1, 1, 1, 1, D, 0, 0, 1), q, k, v, dev_i32([0, T]), out, lse=lse, status=p.st)
            torch.cuda.synchronize()
            assert int(p.st.item()) == 0
            assert torch.equal(lse[:, 0], p.lse[at, h]), (i, h)
            assert torch.equal(out[:, 0].isnan(), p.out[at, h].isnan()), (i, h)
            assert torch.equal(out[:, 0].nan_to_num(nan=0.0), p.out[at, h].nan_to_num(nan=0.0)), (i, h)


@pytest.mark.parametrize("D,G,heads,lens", [(256, 6, 4, [2300, 1408]), (256, 6, 8, [1408] * 20), (256, 5, 4, [3000, 3000, 2176]),
                                            (512, 6, 2, [2300, 1408, 1408]), (512, 5, 2, [3000, 3000, 2176])])
def test_items_with_nothing_to_look_through(D, G, heads, lens):
    """The last token of 1408 (6 query heads a KV head, tiles of 21 tokens) or 2176 (5, 25) is a tile of its own and the end of
    a position tile: no position is hidden from any of its rows.  Longer sequences, or enough of them, put such an item
    behind others of its block."""
    tokens = 128 // G
    assert lens[-1] % tokens == 1 and lens[-1] % 128 == 0
    before = sum(max(0, math.ceil(T / tokens) - math.ceil(lens[-1] / tokens)) for T in lens) * heads * (D // 256)
    assert before + sum(T == lens[-1] for T in lens) * heads * (D // 256) > sms()  # later tiles come first
    p = Prompt(D, G * heads, heads, lens)
    p.run()
    each_as_alone(p, None if len(lens) < 5 else (0, 7, len(lens) - 1))


LENS = [2500, 1700, 900, 1, 130, 257, 0, 640] * 2


@pytest.mark.parametrize("D", [128, 256, 512])
@pytest.mark.parametrize("G", [3, 5, 6, 7])
def test_many_items_a_block(D, G):
    assert items_of(D, G, 4, LENS) > 2 * sms()
    p = Prompt(D, 4 * G, 4, LENS)
    p.run()
    each_as_alone(p)


@pytest.mark.parametrize("D", [128, 256, 512])
@pytest.mark.parametrize("G", [1, 4, 5])
def test_what_is_not_finite_stays_with_its_item(D, G):
    """Values that are infinite or not numbers all over the longest sequences, whose items come first: those of the others,
    behind them in the same blocks, are as they are alone."""
    heads = 8 if D == 128 else 4
    assert items_of(D, G, heads, LENS) > sms()
    p = Prompt(D, heads * G, heads, LENS)
    g = torch.Generator().manual_seed(G)
    for i in (0, 1, 8, 9):
        n = p.lens[i]
        t, h, c = (torch.randint(0, x, (60,), generator=g).cuda() for x in (n, heads, D))
        x = torch.tensor([math.nan, math.inf, -math.inf]).repeat(20).bfloat16().cuda()
        p.v[int(p.first[i]) + t, h, c] = x
    p.run()
    each_as_alone(p)
    for i, T in enumerate(p.lens):
        if T < 1700:
            assert bool(torch.isfinite(p.out[int(p.first[i]):int(p.first[i + 1])].float()).all())
