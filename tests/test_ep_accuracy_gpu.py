"""How far the epilogue and expert matmuls are from 64 bits as a whole (GPU): norms of the error, which
a worst-case bound on each output is too wide to hold.

The steps of the bounds, each relative to the norm of y:
  a rounding off by at most half a step h is taken as spread evenly over [-h, h], mean square h^2 / 3;
  roundings of different values are independent, so that mean squares add up; equal values have
  equal errors, and the activations that meet them are summed first.
"""
import pytest
import torch

import bit_weight_quantized_tgemm_b200 as tg
from ep_reference import pack

pytestmark = pytest.mark.gpu

PATHS = {"small": tg.PATH_SMALL_M, "tensor": tg.PATH_TENSOR}


@pytest.fixture
def path():
    prev = tg.set_path(tg.PATH_AUTO)
    yield tg.set_path
    tg.set_path(prev)


def activations(kind, M, K):
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(5))
    return {"zero_mean": x, "rectified": x.relu(), "around_one": 1 + 0.1 * x}[kind].bfloat16().cuda()


def pack4(codes, s, z):
    """Packed 4-bit weights from codes [N, K] and scales and zero points [N, K / 64]: (wq, sz, W in f64)."""
    s, z = s.half(), z.half()
    wq = (codes[:, 0::2] + 16 * codes[:, 1::2]).to(torch.uint8)
    w = (codes.double() - z.double().repeat_interleave(64, -1)) * s.double().repeat_interleave(64, -1)
    return wq.cuda(), torch.stack([s, z], -1).cuda(), w.cuda()


def weight_rounding(x, codes, w, s):
    """Mean square of each output's error, summed over the outputs, from 4-bit weights as one f16
    rounding of (q - z) s (half a step is at most 2^-11 |w|) after a first one, the same for a group,
    of at most half a step of s / 2 (the rounding of z - c, for the code c next to z, times s)."""
    M, K = x.shape
    N, G = w.shape[0], K // 64
    xg, cg, wg = x.double().view(M, G, 64), codes.cuda().view(N, G, 64), w.view(N, G, 64)
    total = torch.einsum("mg,ng->", xg.sum(-1) ** 2, (2.0 ** -12 * s.cuda().double()) ** 2 / 3)
    for v in range(16):
        hit = (cg == v).double()
        wv = (wg * hit).sum(-1) / hit.sum(-1).clamp_min(1)  # this code's weight in each group
        total += ((torch.einsum("mgk,ngk->mng", xg, hit) * (2.0 ** -11 * wv)) ** 2).sum() / 3
    return float(total)


def f32_sums(x, w, sz):
    """Norm of the error of f32 sums: each of K / 16 steps is off by at most 2^-23 of the sum so far
    and of its own products, and the sums that carry the codes' centre by as much of s (8 + |z - 8|) |x|."""
    x, total = x.double(), 0.0
    acc = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    for k in range(0, x.shape[1], 16):
        acc += x[:, k:k + 16] @ w[:, k:k + 16].T
        total += float(acc.norm() + (x[:, k:k + 16].abs() @ w[:, k:k + 16].abs().T).norm())
    centre = ((8 + (sz[..., 1].double() - 8).abs()) * sz[..., 0].double()).repeat_interleave(64, -1)
    return 2.0 ** -23 * (total + float((x.abs() @ centre.T).norm()))


@pytest.mark.parametrize("pname", list(PATHS))
@pytest.mark.parametrize("kind", ["zero_mean", "rectified", "around_one"])
@pytest.mark.parametrize("z_lo,z_hi", [(7, 8), (0, 1), (0, 15), (12, 13), (-3, -2), (20, 21)])
def test_4bit_weights_of_a_bf16_y(path, pname, kind, z_lo, z_hi):
    """4-bit weights of a bf16 y are as good as f16((q - z) s), whatever the activations' mean and the
    zero points.  The residual -y (f32) leaves the error itself, so that the store's rounding is one
    of the error, 2^-8 of it."""
    path(PATHS[pname])
    M, N, K = 40, 136, 2560
    g = torch.Generator().manual_seed(int(10 * z_lo + z_hi + 100))
    codes = torch.randint(0, 16, (N, K), generator=g)
    s = (0.01 * torch.randn(N, K // 64, generator=g).abs()).half()
    wq, sz, w = pack4(codes, s, z_lo + (z_hi - z_lo) * torch.rand(N, K // 64, generator=g))
    x = activations(kind, M, K)
    ref = x.double() @ w.T
    y = tg.gemm_q4_ep(x, wq, sz, residual=-ref.float())
    torch.cuda.synchronize()
    got = float((y.double() + ref.float().double() - ref).norm() / ref.norm())
    bound = (weight_rounding(x, codes, w, s) ** 0.5 + f32_sums(x, w, sz)) * (1 + 2.0 ** -8) / float(ref.norm())
    assert got <= bound, f"{got:.3g} of the norm, at most {bound:.3g}"


def test_4bit_weights_of_grouped_rows(path):
    """The same of a grouped call, for activations of one sign."""
    path(tg.PATH_TENSOR)
    M, N, K, E = 60, 136, 2560, 3
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 16, (E * N, K), generator=g)
    s = (0.01 * torch.randn(E * N, K // 64, generator=g).abs()).half()
    wq, sz, w = pack4(codes, s, 7 + torch.rand(E * N, K // 64, generator=g))
    x = activations("around_one", M, K)
    ends = [0, 13, 13, 60]
    ref = torch.cat([x[a:b].double() @ w[e * N:(e + 1) * N].T for e, (a, b) in enumerate(zip(ends, ends[1:]))])
    y = tg.gemm_q4_grouped(x, wq.view(E, N, -1), sz.view(E, N, -1, 2), torch.tensor(ends).int().cuda(),
                           residual=-ref.float())
    torch.cuda.synchronize()
    bound = 0.0
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        own = slice(e * N, (e + 1) * N)
        if b > a:
            bound += weight_rounding(x[a:b], codes[own], w[own], s[own]) ** 0.5 + f32_sums(x[a:b], w[own], sz[own])
    got = float((y.double() + ref.float().double() - ref).norm())
    assert got <= bound * (1 + 2.0 ** -8)


@pytest.mark.parametrize("pname", list(PATHS))
@pytest.mark.parametrize("out", [tg.OUT_F32, tg.OUT_BF16])
@pytest.mark.parametrize("s,z,lo,hi", [(6000, 15, 8, 15), (4300, 0, 0, 15), (10000, 0, 0, 6), (8000, 15, 7, 15), (60000, 8, 7, 9),
                                       (1, 60000, 0, 15), (0.99, -60000, 0, 15), (5000, 24, 12, 15)])
def test_4bit_weights_up_to_the_f16_range(path, pname, out, s, z, lo, hi):
    """Weights that f16 holds, whose q s, z s or (z - 8) s it does not."""
    path(PATHS[pname])
    M, N, K = 20, 72, 320
    g = torch.Generator().manual_seed(int(s) + int(z))
    codes = torch.randint(lo, hi + 1, (N, K), generator=g)
    wq, sz, w = pack4(codes, torch.full((N, K // 64), float(s)), torch.full((N, K // 64), float(z)))
    assert w.abs().max() <= 65504
    x = (torch.randn(M, K, generator=g) / 64).bfloat16().cuda()
    ref = x.double() @ w.T
    y = tg.gemm_q4_ep(x, wq, sz, out_dtype=out)
    torch.cuda.synchronize()
    S = x.double().abs() @ w.abs().T
    # q - z to 11 bits and its product with s; the f32 sums; the store
    bound = 2.0 ** -10 * S + (K / 16 + K / 64) * 2.0 ** -23 * S
    bound = bound + 2.0 ** -8 * (ref.abs() + bound)
    assert ((y.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("pname", list(PATHS))
@pytest.mark.parametrize("out", [tg.OUT_F32, tg.OUT_BF16])
def test_ternary_weights_up_to_the_f16_range(path, pname, out):
    path(PATHS[pname])
    M, N, K = 20, 72, 384
    wq, d, w = pack("q2", (N, K), 2, "cuda")
    scale = 60000 / d.float().max()
    d2 = (d.float() * scale).half()
    w2 = w.sign() * d2.double().repeat_interleave(128, -1)
    x = (torch.randn(M, K, generator=torch.Generator().manual_seed(3)) / 64).bfloat16().cuda()
    ref = x.double() @ w2.T
    y = tg.gemm_q2_ep(x, wq, d2, out_dtype=out)
    torch.cuda.synchronize()
    bound = (K / 16 + K / 64) * 2.0 ** -23 * (x.double().abs() @ w2.abs().T)
    bound = bound + (2.0 ** -24 if out == tg.OUT_F32 else 2.0 ** -8) * (ref.abs() + bound)
    assert ((y.double() - ref).abs() <= bound).all()


# The tensor core cuts each K = 16 step's sum off, by 1.5e-8 (2^-26) of it on average, and running sums
# are taken every 48 steps, so that a segment's partial sums grow as the root of the steps: the cuts
# come to 2 / 3 * 48 * 2^-26 of the segment, and, the segments' signs being independent, of y.  Twice
# that is allowed.  One accumulator for all of K would be 2.3e-6 off at K = 2560 and 8e-6 at 9728.
SUMS = 2 * (2 / 3 * 48) * 2.0 ** -26


@pytest.mark.parametrize("pname", list(PATHS))
@pytest.mark.parametrize("M,K", [(20, 2560), (130, 2560), (20, 9728), (130, 9728), (60, 9664)])
@pytest.mark.parametrize("fmt,size", [("q2", 0.02), ("q2", 0.0002), ("q4", 0.01), ("q4", 0.001), ("q4", 0.0001)])
def test_f32_y(path, pname, M, K, fmt, size):
    """f32 outputs, for ordinary and small scales.  4-bit weights are two f16 parts on the tensor path:
    the low one is off by at most 2^-22 |w| and where it is subnormal by 2^-25, whatever the scale."""
    if fmt == "q2" and K % 128:
        K += 64
    path(PATHS[pname])
    N = 136
    wq, sc, w = pack(fmt, (N, K), K + M, "cuda")
    f = size / (0.02 if fmt == "q2" else 0.01)
    if fmt == "q2":
        sc = (sc.float() * f).half()
        w = w.sign() * sc.double().repeat_interleave(128, -1)
    else:
        q = (w / sc[..., 0].double().repeat_interleave(64, -1) + sc[..., 1].double().repeat_interleave(64, -1)).round()
        sc[..., 0] = (sc[..., 0].float() * f).half()
        w = (q - sc[..., 1].double().repeat_interleave(64, -1)) * sc[..., 0].double().repeat_interleave(64, -1)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(K)).bfloat16().cuda()
    ref = x.double() @ w.T
    y = (tg.gemm_q2_ep if fmt == "q2" else tg.gemm_q4_ep)(x, wq, sc, out_dtype=tg.OUT_F32)
    torch.cuda.synchronize()
    low = 0.0
    if fmt == "q4" and pname == "tensor":
        low = float(((x.double() ** 2) @ (((2.0 ** -22 * w) ** 2 + 2.0 ** -50) / 3).T).sum()) ** 0.5
    got, bound = float((y.double() - ref).norm()), float(ref.norm()) * (SUMS + 2.0 ** -24) + low
    assert got <= bound, f"{got / float(ref.norm()):.3g} of the norm, at most {bound / float(ref.norm()):.3g}"
