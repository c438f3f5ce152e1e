"""Expert layers one after another on the stream, nothing waited for in between (GPU)."""
import pytest
import torch

import bit_weight_quantized_tgemm_b200 as tg
from ep_reference import pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E", [(3, 2, 8), (61, 2, 8), (3000, 2, 8)])  # few rows, many rows, a sort over several CTAs
def test_layers_whose_buffers_are_handed_on(T, k, E):
    """Each kernel may start before the one ahead of it ends, and reads plans, activations and operands
    that it has just written into memory that earlier layers used: the bits of layers run one by one."""
    D, F, layers = 256, 384, 24
    g = torch.Generator().manual_seed(T)
    up, dn = pack("q4", (E, F, D), 1, "cuda"), pack("q4", (E, D, F), 2, "cuda")
    bias = torch.randn(E, F, generator=g).cuda()
    ids = [torch.rand(T, E, generator=g).topk(k).indices.int().cuda() for _ in range(layers)]
    wts = [torch.rand(T, k, generator=g).cuda() for _ in range(layers)]
    x0 = (torch.randn(T, D, generator=g) / 4).bfloat16().cuda()

    def layer(x, i):
        offsets, rows, pos = tg.expert_sort(ids[i], E)
        h = tg.gemm_q4_grouped(x, up[0], up[1], offsets, rows=rows, bias=bias, act=tg.ACT_RELU)
        o = tg.gemm_q4_grouped(h, dn[0], dn[1], offsets)
        return tg.expert_combine(o, pos, wts[i], residual=x)

    want = [x0]
    for i in range(layers):
        want.append(layer(want[-1], i))
        torch.cuda.synchronize()
    for _ in range(4):
        x = x0
        for i in range(layers):
            x = layer(x, i)
        assert torch.equal(x, want[-1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x = x0
        for i in range(layers):
            x = layer(x, i)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want[-1])
    assert tg.device_error() == 0
