"""What the epilogue and expert calls refuse, and their workspace sizes (no GPU): every check
returns before any CUDA call."""
import ctypes

import pytest
import torch

import bit_weight_quantized_tgemm_b200 as tg
from bit_weight_quantized_tgemm_b200 import binding

P = ctypes.c_void_p
MB = 1 << 20


def at(i):
    """The i-th of a set of made-up device addresses far from each other."""
    return (i + 1) * 256 * MB


def ep(**kw):
    return ctypes.addressof(ep_keep.setdefault(str(kw), binding._Epilogue(**kw)))


ep_keep = {}


def call_ep(fn="tgemm_q2_ep", x=at(0), wq=at(1), sc=at(2), e=None, y=at(3), M=96, N=64, K=256, out=1, ws=at(4),
            nbytes=MB, **_):
    return getattr(tg.lib(), fn)(x, wq, sc, e, y, M, N, K, out, ws, nbytes, None)


def call_grouped(fn="tgemm_q2_grouped", x=at(0), x_rows=20, wq=at(1), sc=at(2), off=at(5), rows=None, e=None, y=at(3),
                 R=20, E=3, N=64, K=256, out=1, ws=at(4), nbytes=MB):
    return getattr(tg.lib(), fn)(x, x_rows, wq, sc, off, rows, e, y, R, E, N, K, out, ws, nbytes, None)


@pytest.mark.parametrize("fn", ["tgemm_q2_ep", "tgemm_q4_ep"])
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), tg.EINVAL), (dict(wq=None), tg.EINVAL), (dict(sc=None), tg.EINVAL), (dict(y=None), tg.EINVAL),
    (dict(M=0), tg.EINVAL), (dict(N=0), tg.EINVAL), (dict(K=0), tg.EINVAL), (dict(K=96), tg.EINVAL), (dict(M=-1), tg.EINVAL),
    (dict(out=2), tg.EINVAL), (dict(N=2 ** 31 - 1), tg.ETOOLARGE),
    (dict(x=at(0) + 8), tg.EALIGN), (dict(wq=at(1) + 4), tg.EALIGN), (dict(sc=at(2) + 1), tg.EALIGN), (dict(y=at(3) + 8), tg.EALIGN),
    (dict(ws=None), tg.EWORKSPACE), (dict(nbytes=100), tg.EWORKSPACE), (dict(ws=at(4) + 16), tg.EALIGN),
    (dict(e=dict(act=5)), tg.EINVAL), (dict(e=dict(act=-1)), tg.EINVAL),
    (dict(e=dict(bias=at(6), bias_dtype=2)), tg.EINVAL), (dict(e=dict(residual=at(6), residual_dtype=7)), tg.EINVAL),
    (dict(e=dict(gate=at(6), gate_rows=2)), tg.EINVAL),
    (dict(e=dict(bias=at(6) + 2)), tg.EALIGN), (dict(e=dict(bias=at(6) + 1, bias_dtype=1)), tg.EALIGN),
    (dict(e=dict(gate=at(6) + 2)), tg.EALIGN), (dict(e=dict(residual=at(6) + 8)), tg.EALIGN),
    # y over an input: x, the weights, the workspace, a part of the residual, a residual or gate of another type or shape
    (dict(y=at(0) + 256), tg.EINVAL), (dict(y=at(1)), tg.EINVAL), (dict(y=at(2)), tg.EINVAL), (dict(y=at(4)), tg.EINVAL),
    # the workspace over an input
    (dict(ws=at(0)), tg.EINVAL), (dict(ws=at(1) + 256), tg.EINVAL), (dict(ws=at(2)), tg.EINVAL),
    (dict(e=dict(bias=at(4))), tg.EINVAL), (dict(e=dict(gate=at(4) + 256)), tg.EINVAL), (dict(e=dict(residual=at(4))), tg.EINVAL),
    (dict(e=dict(residual=at(3) + 128, residual_dtype=1)), tg.EINVAL), (dict(e=dict(residual=at(3), residual_dtype=0)), tg.EINVAL),
    (dict(e=dict(gate=at(3), gate_rows=0)), tg.EINVAL), (dict(e=dict(gate=at(3) + 16, gate_rows=1)), tg.EINVAL),
    (dict(e=dict(gate=at(3), gate_rows=1), out=0), tg.EINVAL), (dict(e=dict(bias=at(3))), tg.EINVAL),
], ids=str)
def test_ep_refuses(fn, kw, status):
    kw = dict(kw)
    if "e" in kw:
        kw["e"] = ep(**kw["e"])
    assert call_ep(fn, **kw) == status


@pytest.mark.parametrize("fn", ["tgemm_q2_grouped", "tgemm_q4_grouped"])
@pytest.mark.parametrize("kw,status", [
    (dict(off=None), tg.EINVAL), (dict(x_rows=19), tg.EINVAL), (dict(x_rows=0, rows=at(6)), tg.EINVAL), (dict(R=0), tg.EINVAL),
    (dict(E=0), tg.EINVAL), (dict(E=1025), tg.EINVAL), (dict(off=at(5) + 2), tg.EALIGN), (dict(rows=at(6) + 1), tg.EALIGN),
    (dict(e=dict(gate=at(6), gate_rows=0)), tg.EINVAL), (dict(E=1024, N=2 ** 21), tg.ETOOLARGE),
    (dict(y=at(5)), tg.EINVAL), (dict(rows=at(6), y=at(6)), tg.EINVAL), (dict(nbytes=255), tg.EWORKSPACE),
    (dict(ws=at(5)), tg.EINVAL), (dict(rows=at(4)), tg.EINVAL), (dict(ws=at(0)), tg.EINVAL),
], ids=str)
def test_grouped_refuses(fn, kw, status):
    kw = dict(kw)
    if "e" in kw:
        kw["e"] = ep(**kw["e"])
    assert call_grouped(fn, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), tg.EINVAL), (dict(T=0), tg.EINVAL), (dict(k=0), tg.EINVAL), (dict(E=0), tg.EINVAL), (dict(E=1025), tg.EINVAL),
    (dict(T=2 ** 26, k=2), tg.ETOOLARGE), (dict(T=2 ** 31 - 1, k=2 ** 31 - 1), tg.ETOOLARGE), (dict(ids=at(0) + 2), tg.EALIGN),
    (dict(rows=at(0)), tg.EINVAL), (dict(pos=at(2)), tg.EINVAL), (dict(off=at(3)), tg.EINVAL),
    (dict(T=100000, ws=at(0)), tg.EINVAL), (dict(T=100000, ws=at(1)), tg.EINVAL), (dict(T=100000, rows=at(4)), tg.EINVAL),
    (dict(T=100000, pos=at(4)), tg.EINVAL), (dict(T=100000, ws=None), tg.EWORKSPACE), (dict(T=100000, nbytes=64), tg.EWORKSPACE), (dict(T=100000, ws=at(4) + 4), tg.EALIGN),
], ids=str)
def test_sort_refuses(kw, status):
    a = dict(ids=at(0), T=50, k=2, E=8, off=at(1), rows=at(2), pos=at(3), ws=at(4), nbytes=MB)
    a.update(kw)
    assert tg.lib().tgemm_expert_sort(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(h=None), tg.EINVAL), (dict(pos=None), tg.EINVAL), (dict(w=None), tg.EINVAL), (dict(y=None), tg.EINVAL),
    (dict(T=0), tg.EINVAL), (dict(k=0), tg.EINVAL), (dict(N=0), tg.EINVAL), (dict(R=0), tg.EINVAL), (dict(hd=3), tg.EINVAL),
    (dict(rd=3), tg.EINVAL), (dict(out=-1), tg.EINVAL), (dict(h=at(0) + 8), tg.EALIGN), (dict(y=at(4) + 2), tg.EALIGN),
    (dict(res=at(3) + 8), tg.EALIGN), (dict(pos=at(1) + 2), tg.EALIGN), (dict(y=at(0)), tg.EINVAL), (dict(y=at(1)), tg.EINVAL),
    (dict(y=at(3) + 16), tg.EINVAL), (dict(y=at(3), rd=0), tg.EINVAL),
], ids=str)
def test_combine_refuses(kw, status):
    a = dict(h=at(0), hd=1, pos=at(1), w=at(2), res=at(3), rd=1, y=at(4), T=5, k=2, N=64, R=12, out=1)
    a.update(kw)
    assert tg.lib().tgemm_expert_combine(*a.values(), None) == status


def test_workspace_sizes():
    L = tg.lib()
    for f in (lambda M, N, K, op: L.tgemm_ep_workspace_size(op, M, N, K), lambda M, N, K, op: L.tgemm_grouped_workspace_size(op, M, 4, N, K)):
        assert f(300, 64, 256, tg.OP_Q2) >= 300 * 256 * 2
        assert f(300, 64, 256, tg.OP_Q2) % 256 == 0
        assert f(0, 64, 256, tg.OP_Q2) == 0 and f(300, 64, 256, tg.OP_Q2_LORA) == 0
        assert f(2 ** 20, 64, 2 ** 16, tg.OP_Q4) >= 2 ** 37  # past 32 bits
    assert L.tgemm_expert_sort_workspace_size(1, 8, 64) == 0
    assert L.tgemm_expert_sort_workspace_size(2 ** 20, 8, 64) > 0
    assert L.tgemm_expert_sort_workspace_size(2 ** 20, 8, 1025) == 0


def test_binding_checks_types_and_shapes():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    wq, d = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tg.gemm_q2_ep(x, wq, d)
    with pytest.raises(TypeError, match="bfloat16"):
        tg.gemm_q2_ep(x.float(), wq, d)
    with pytest.raises(TypeError, match="int32"):
        tg.expert_sort(torch.zeros(4, 2, dtype=torch.int64), 8)
    with pytest.raises(TypeError, match="float32 or"):
        tg.expert_combine(torch.zeros(4, 8, dtype=torch.float16), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))
