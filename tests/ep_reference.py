"""The epilogue and expert operators in 64 bits, and how far f32 kernels may be from them.

The error bound of one output follows the steps of the computation.  With S = sum_k |w x|:
  product   bf16 activations are exact in f16 down to 2^-14, below that off by at most 2^-25
            each; ternary weights are exact in f16; 4-bit weights take two f16 roundings of half a
            step when y is bf16, f16(q s - f16(z s)) or f16(f16(q - z) s): 2^-11 of |w| and 2^-11
            of |z s| or |w|, so at most 2^-11 (2 |w| + |z s|) (2^-25 each where subnormal); they
            are a high and a low f16 part (error of the low part's rounding 2^-22, and 2^-25
            absolute where it is subnormal) when y is f32; the f32 sum over k is at most K / 16 + 16
            accumulations, each off by at most a whole step 2^-23 of S
  bias      one f32 rounding
  act       slope at most 1.13 for the four activations; its own steps at most 8 f32 steps of
            |v| + 1
  gate and  one f32 rounding each
  residual
  store     half a step of y's type
"""
import math

import torch

import bit_weight_quantized_tgemm_b200 as tg

ACTS = {"none": tg.ACT_NONE, "silu": tg.ACT_SILU, "gelu": tg.ACT_GELU, "gelu_tanh": tg.ACT_GELU_TANH,
        "relu": tg.ACT_RELU}
F32 = 2.0 ** -23


def pack(fmt, shape, seed, device, z_lo=7.0):
    """Random packed weights [*, N, K] by plain byte arithmetic: (wq, scales, W in f64)."""
    g = torch.Generator().manual_seed(seed)
    *lead, K = shape
    if fmt == "q2":
        q = torch.randint(0, 3, shape, generator=g)
        b = q.view(*lead, K // 4, 4)
        wq = b[..., 0] + 4 * b[..., 1] + 16 * b[..., 2] + 64 * b[..., 3]
        sc = (torch.randn(*lead, K // 128, generator=g).abs() * 0.02).half()
        w = (q.double() - 1) * sc.double().repeat_interleave(128, -1)
    else:
        q = torch.randint(0, 16, shape, generator=g)
        b = q.view(*lead, K // 2, 2)
        wq = b[..., 0] + 16 * b[..., 1]
        s = (torch.randn(*lead, K // 64, generator=g).abs() * 0.01).half()
        z = (z_lo + torch.rand(*lead, K // 64, generator=g)).half()
        sc = torch.stack([s, z], -1)
        w = (q.double() - z.double().repeat_interleave(64, -1)) * s.double().repeat_interleave(64, -1)
    return wq.to(torch.uint8).to(device), sc.to(device), w.to(device)


def act64(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * 0.5 * torch.special.erfc(-v / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "relu":
        return v.clamp_min(0)
    return v


def reference(fmt, x, w, bias, act, gate, residual, out_f32, sc=None):
    """(y in f64, bound on |error|) of the rows x [M, K] times w [N, K]; bias [N], gate broadcasts;
    sc: the 4-bit (s, z) [N, K/64, 2]."""
    K = x.shape[1]
    x, aw = x.double(), w.abs()
    S = x.abs() @ aw.T
    dv = (K / 16 + 16) * F32 * S + 2.0 ** -25 * aw.sum(1)
    if fmt == "q4":
        ax = x.abs().sum(1, keepdim=True)
        if out_f32:
            dv = dv + 2.0 ** -22 * S + 2.0 ** -25 * ax
        else:
            zs = (sc[..., 0].double() * sc[..., 1].double()).abs().repeat_interleave(64, -1)
            dv = dv + 2.0 ** -11 * (2 * S + x.abs() @ zs.T) + 2 * 2.0 ** -25 * ax
    v = x @ w.T
    if bias is not None:
        v = v + bias.double()
        dv = dv + F32 * v.abs()
    y = act64(v, act)
    dy = 1.13 * dv + (8 * F32 * (v.abs() + 1) if act != "none" else 0)
    if gate is not None:
        y = y * gate.double()
        dy = dy * gate.double().abs() + F32 * y.abs()
    if residual is not None:
        y = y + residual.double()
        dy = dy + F32 * y.abs()
    half = 2.0 ** -24 if out_f32 else 2.0 ** -8
    return y, dy + half * (y.abs() + dy)


def check(y, ref, bound, what):
    err = (y.double() - ref).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = int((err / bound).nan_to_num(float("inf")).argmax())
        m, n = divmod(i, ref.shape[1])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outputs off; worst [{m}, {n}]: "
                             f"{y[m, n].item()} against {ref[m, n].item()}, bound {bound[m, n].item():.3g}")


def epilogue(case, M, N, groups, seed, device):
    """bias [*groups, N], gate, residual of a case string such as 'bias:f32 gate:row residual:bf16'."""
    g = torch.Generator().manual_seed(seed + 1000)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    out = dict(bias=None, gate=None, residual=None)
    for word in case.split():
        k, v = word.split(":")
        if k == "bias":
            out[k] = torch.randn(*groups, N, generator=g).to(dt[v]).to(device)
        elif k == "gate":
            out[k] = torch.randn(*((N,) if v == "row" else (M, N)), generator=g).bfloat16().to(device)
        else:
            out[k] = torch.randn(M, N, generator=g).to(dt[v]).to(device)
    return out
