"""Epilogue and expert calls on no tokens (GPU)."""
import pytest
import torch

import bit_weight_quantized_tgemm_b200 as tg
from ep_reference import pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["q2", "q4"])
def test_expert_layer_of_no_tokens(fmt):
    E, D, F = 4, 256, 384
    grouped = tg.gemm_q2_grouped if fmt == "q2" else tg.gemm_q4_grouped
    up, dn = pack(fmt, (E, F, D), 1, "cuda"), pack(fmt, (E, D, F), 2, "cuda")
    x = torch.empty(0, D, device="cuda").bfloat16()
    ids, wts = torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")

    def layer():
        plan = tg.expert_sort(ids, E)
        h = grouped(x, up[0], up[1], plan[0], rows=plan[1], act=tg.ACT_SILU)
        o = grouped(h, dn[0], dn[1], plan[0], out_dtype=tg.OUT_F32)
        return (*plan, h, o, tg.expert_combine(o, plan[2], wts, residual=x))

    offsets, rows, pos, h, o, y = layer()
    assert offsets.tolist() == [0] * (E + 1) and rows.shape == (0,) and pos.shape == (0, 2)
    assert h.shape == (0, F) and h.dtype == torch.bfloat16 and o.shape == (0, D) and o.dtype == torch.float32
    assert y.shape == (0, D) and y.dtype == torch.bfloat16
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = layer()
    kept[0].fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert kept[0].tolist() == [0] * (E + 1)


@pytest.mark.parametrize("fmt", ["q2", "q4"])
def test_epilogue_matmul_of_no_tokens(fmt):
    N, K = 72, 256
    wq, sc, _ = pack(fmt, (N, K), 1, "cuda")
    fn = tg.gemm_q2_ep if fmt == "q2" else tg.gemm_q4_ep
    x, res = torch.empty(0, K, device="cuda").bfloat16(), torch.empty(0, N, device="cuda")
    y = fn(x, wq, sc, bias=torch.ones(N, device="cuda"), residual=res, out_dtype=tg.OUT_F32)
    assert y.shape == (0, N) and y.dtype == torch.float32
    assert fn(x, wq, sc, residual=res, out_dtype=tg.OUT_F32, y=res) is res


def test_no_tokens_with_other_shapes_wrong_are_refused():
    wq, sc, _ = pack("q2", (72, 256), 1, "cuda")
    x = torch.empty(0, 256, device="cuda").bfloat16()
    with pytest.raises(ValueError):
        tg.gemm_q2_ep(x, wq, sc, bias=torch.ones(71, device="cuda"))
    with pytest.raises(ValueError):
        tg.gemm_q2_ep(x[:, :128], wq, sc)
    with pytest.raises(TypeError):
        tg.expert_combine(x, torch.empty(0, 2, dtype=torch.int64, device="cuda"), torch.empty(0, 2, device="cuda"))
    with pytest.raises(ValueError):
        tg.expert_sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), tg.MAX_EXPERTS + 1)
