"""Decode steps of large batches with the in-quant Hadamard: the append and the kernels around it are launched before the ones
ahead of them end, so every layer's rows are made from the layer before, and the results compared with calls that are waited
for one by one."""
import pytest
import torch

from int2_kv_cache_append_gb300 import oscar_kv as K

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs CUDA")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from int2_kv_cache_append_gb300 import build
    build.build()


class Model:
    def __init__(self, B, Hq, Hkv, D, T, flags, layers=5):
        self.c = K.KVConfig(layers, B, Hq, Hkv, D, 4, 32, T + 8, flags=K.FLAG_HADAMARD | flags)
        lay = K.layout_query(self.c)
        g = torch.Generator().manual_seed(D + B)
        self.prompt = [torch.randn(B, T, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2)]
        self.q = torch.randn(B, Hq, D, generator=g).bfloat16().cuda()
        self.start = torch.full((B,), T, dtype=torch.int32, device="cuda")
        self.lens = self.start + 1
        self.cache = torch.zeros(lay["total_bytes"], dtype=torch.uint8, device="cuda")
        self.out = torch.empty_like(self.q)
        self.ws = torch.empty(lay["decode_workspace_bytes"], dtype=torch.uint8, device="cuda")
        self.T, self.layers, self.Hkv, self.G = T, layers, Hkv, Hq // Hkv

    def fill(self):
        self.cache.zero_()
        zero = torch.zeros_like(self.start)
        for layer in range(self.layers):
            K.kv_append(self.c, self.cache, layer, *self.prompt, zero, None, None)
        torch.cuda.synchronize()

    def run(self, step, apart):
        """The layers one behind the other; `apart`: every call by itself, waited for."""
        q, outs = self.q, []
        for layer in range(self.layers):
            x = q.view(q.shape[0], self.Hkv, self.G, -1)
            k, v = x[:, None, :, 0].contiguous(), x[:, None, :, -1].contiguous() * 0.5
            out = torch.empty_like(q)
            if apart:
                torch.cuda.synchronize()
            if step:
                K.decode_step(self.c, self.cache, layer, k, v, self.start, q, self.lens, None, None, out, self.ws)
            else:
                K.kv_append(self.c, self.cache, layer, k, v, self.start, None, None)
                if apart:
                    torch.cuda.synchronize()
                K.attn_decode(self.c, self.cache, layer, q, self.lens, None, None, out, self.ws)
            if apart:
                torch.cuda.synchronize()
            outs.append(out)
            q = out + self.q
        return torch.stack(outs)


@pytest.mark.parametrize("B,Hq,Hkv,D,T,flags", [(160, 16, 8, 128, 90, 0), (160, 16, 8, 128, 90, K.FLAG_LLOYD_MAX), (300, 8, 4, 128, 40, K.FLAG_V_BF16),
                                                (80, 16, 8, 256, 50, 0), (40, 8, 8, 512, 50, 0)])
def test_layers_behind_each_other(B, Hq, Hkv, D, T, flags):
    assert B * Hkv * D > 1024 * 128  # beyond the row-parallel kernel
    m = Model(B, Hq, Hkv, D, T, flags)
    m.fill()
    want = m.run(step=False, apart=True)
    cache = m.cache.clone()
    assert bool(torch.isfinite(want.float()).all())
    for step in (False, True):
        m.fill()
        got = m.run(step, apart=False)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(m.cache, cache), step
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.run(step=True, apart=False)
    for _ in range(5):
        m.fill()
        graph.replay()
        graph.replay()  # the same rows again
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(m.cache, cache)
