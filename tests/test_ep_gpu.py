"""Matmuls with an epilogue against their definition in 64 bits (GPU)."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import bit_weight_quantized_tgemm_b200 as tg
from ep_reference import ACTS, check, epilogue, pack, reference
from helpers import canary_intact, nan_filled

pytestmark = pytest.mark.gpu

PATHS = {"auto": tg.PATH_AUTO, "small": tg.PATH_SMALL_M, "tensor": tg.PATH_TENSOR}


@pytest.fixture
def path():
    prev = tg.set_path(tg.PATH_AUTO)
    yield tg.set_path
    tg.set_path(prev)


def fn(fmt):
    return tg.gemm_q2_ep if fmt == "q2" else tg.gemm_q4_ep


def run(fmt, M, N, K, act, ep, out, seed=0, x_scale=1.0, **kw):
    wq, sc, w = pack(fmt, (N, K), seed, "cuda", **kw)
    x = (torch.randn(M, K, generator=torch.Generator().manual_seed(seed + 7)) * x_scale).bfloat16().cuda()
    e = epilogue(ep, M, N, (), seed, "cuda")
    dt = torch.float32 if out == "f32" else torch.bfloat16
    y, buf = nan_filled((M, N), dt)
    got = fn(fmt)(x, wq, sc, act=ACTS[act], out_dtype=tg.OUT_F32 if out == "f32" else tg.OUT_BF16, y=y, **e)
    assert got is y
    torch.cuda.synchronize()
    assert canary_intact(buf, M * N)
    check(y, *reference(fmt, x, w, e["bias"], act, e["gate"], e["residual"], out == "f32", sc),
          f"{fmt} {M}x{N}x{K} {act} {ep} {out}")


SHAPES = [(1, 8, 128), (1, 640, 2560), (3, 41, 256), (8, 128, 384), (9, 200, 1152), (16, 128, 640), (17, 300, 384),
          (33, 129, 512), (65, 127, 256), (100, 256, 512), (128, 520, 640), (129, 1000, 1024), (300, 260, 896)]


@pytest.mark.parametrize("pname", list(PATHS))
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fmt,out", [("q2", "f32"), ("q2", "bf16"), ("q4", "f32"), ("q4", "bf16")])
def test_shapes(path, pname, M, N, K, fmt, out):
    path(PATHS[pname])
    run(fmt, M, N, K, "silu", "bias:f32 gate:full residual:bf16", out, seed=M + N)


@pytest.mark.parametrize("fmt,M,N,K", [("q4", 1, 8, 64), ("q4", 5, 33, 192), ("q4", 20, 300, 320), ("q4", 200, 96, 448),
                                       ("q2", 2, 5, 9728), ("q4", 40, 130, 9728), ("q2", 700, 64, 256)])
@pytest.mark.parametrize("pname", list(PATHS))
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_odd_widths(path, pname, fmt, M, N, K, out):
    """K of half a stage, long K, a few weight rows, many token tiles."""
    path(PATHS[pname])
    run(fmt, M, N, K, "none", "residual:f32", out, seed=K)


@pytest.mark.parametrize("M,N,K", [(17, 128, 9728), (70, 72, 2176), (33, 301, 1152), (100, 250, 4096), (128, 640, 9728),
                                   (40, 1408, 2048), (17, 2560, 2560), (130, 1279, 4224), (256, 2560, 9728)])
@pytest.mark.parametrize("fmt,out", [("q2", "f32"), ("q2", "bf16"), ("q4", "f32"), ("q4", "bf16")])
def test_few_tiles(path, M, N, K, fmt, out):
    """Long rows and few tiles, whose units CTAs share: odd unit counts, ragged tiles, odd widths."""
    path(tg.PATH_TENSOR)
    run(fmt, M, N, K, "gelu", "bias:f32 gate:full residual:bf16", out, seed=K + M)


@pytest.mark.parametrize("M,N,K", [(1, 512, 9728), (3, 1408, 9728), (8, 41, 5120), (16, 300, 9728), (13, 1408, 4096), (1, 2560, 9728),
                                   (40, 70, 9728)])
@pytest.mark.parametrize("fmt,out", [("q2", "f32"), ("q2", "bf16"), ("q4", "f32"), ("q4", "bf16")])
def test_few_items(path, M, N, K, fmt, out):
    """Few rows, few weight rows and long K, which CTAs share; twice the same bits."""
    path(tg.PATH_SMALL_M)
    run(fmt, M, N, K, "silu", "bias:bf16 gate:full residual:f32", out, seed=K + M)
    wq, sc, _ = pack(fmt, (N, K), 9, "cuda")
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    ys = [fn(fmt)(x, wq, sc) for _ in range(5)]
    assert all(torch.equal(ys[0], y) for y in ys)


@pytest.mark.parametrize("K", [1088, 3136])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_few_tiles_of_half_units(path, K, out):
    path(tg.PATH_TENSOR)
    run("q4", 50, 200, K, "none", "gate:row", out, seed=K)


def test_few_tiles_repeat_and_replay(path):
    """Shared tiles: the same bits each time, on two streams at once and from a graph."""
    path(tg.PATH_TENSOR)
    wq, sc, _ = pack("q2", (1408, 4096), 1, "cuda")
    x = torch.randn(90, 4096, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    want = tg.gemm_q2_ep(x, wq, sc)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            got.append(tg.gemm_q2_ep(x, wq, sc))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        kept = [tg.gemm_q2_ep(x, wq, sc) for _ in range(3)]
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want, y) for y in got + kept)


def test_first_call_in_a_capture():
    """A process whose first calls are captured: nothing in them may need to run before."""
    code = """
import torch
import bit_weight_quantized_tgemm_b200 as tg
wq = torch.zeros(1408, 512, dtype=torch.uint8, device="cuda")
d = torch.ones(1408, 16, dtype=torch.float16, device="cuda")
x = torch.ones(200, 2048, dtype=torch.bfloat16, device="cuda")
ids = torch.zeros(3000, 2, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    ys = [tg.gemm_q2_ep(x[:m], wq, d) for m in (1, 20, 100, 200)]
    offsets, rows, pos = tg.expert_sort(ids, 4)
g.replay()
torch.cuda.synchronize()
assert all((y == -2048).all() for y in ys)
assert offsets.tolist() == [0, 6000, 6000, 6000, 6000]
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


EPILOGUES = ["", "bias:bf16", "gate:row", "gate:full", "residual:bf16", "residual:f32", "bias:f32 gate:row residual:f32"]


@pytest.mark.parametrize("M", [2, 70])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("ep", EPILOGUES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_every_epilogue(M, act, ep, out):
    run("q2", M, 136, 256, act, ep, out, seed=5)


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("M,N,K", [(2600, 3500, 256), (2305, 4099, 128), (1281, 9300, 384)])
@pytest.mark.parametrize("act,ep", [("gelu_tanh", "bias:bf16"), ("none", "bias:f32 gate:row"), ("silu", "gate:full"),
                                    ("none", "residual:f32"), ("gelu", "bias:bf16 gate:full residual:bf16")])
def test_many_tiles(fmt, M, N, K, act, ep):
    """Several tiles for each SM, ragged in both directions, odd widths (no pairs of outputs)."""
    run(fmt, M, N, K, act, ep, "bf16", seed=N)


@pytest.mark.parametrize("fmt", ["q2", "q4"])
def test_many_tiles_with_the_smallest_workspace(fmt):
    M, N, K = 2600, 3500, 256
    wq, sc, w = pack(fmt, (N, K), 3, "cuda")
    x = torch.randn(M, K, device="cuda").bfloat16()
    ws = torch.empty(M * K * 2, dtype=torch.uint8, device="cuda")
    y = fn(fmt)(x, wq, sc, act=tg.ACT_RELU, workspace=ws)
    torch.cuda.synchronize()
    check(y, *reference(fmt, x, w, None, "relu", None, None, False, sc), fmt)


@pytest.mark.parametrize("M", [4, 70])
@pytest.mark.parametrize("fmt", ["q2", "q4"])
def test_large_and_small_activations(M, fmt):
    """Pre-activations far out on both tails, and activations down to f16's subnormals."""
    run(fmt, M, 72, 512, "gelu_tanh", "", "f32", x_scale=1000.0)
    run(fmt, M, 72, 512, "silu", "", "f32", x_scale=1000.0)
    run(fmt, M, 72, 512, "none", "", "f32", x_scale=1e-5)


@pytest.mark.parametrize("M", [4, 70])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_zero_points_of_any_size(M, out):
    """Zero points near 0, where q - z takes more bits than f16 has."""
    run("q4", M, 72, 512, "none", "", out, z_lo=0.0)


@pytest.mark.parametrize("M", [3, 50])
@pytest.mark.parametrize("N,K", [(70, 256), (40, 384), (130, 1024)])
def test_scales_on_any_16_bit_address(M, N, K):
    """Ternary scales that start between two words, with rows of an even and an odd number."""
    wq, sc, w = pack("q2", (N, K), 12, "cuda")
    d = torch.empty(N * K // 128 + 1, dtype=torch.float16, device="cuda")[1:].view(N, K // 128)
    d.copy_(sc)
    assert d.data_ptr() % 4 == 2
    x = torch.randn(M, K, device="cuda").bfloat16()
    y = tg.gemm_q2_ep(x, wq, d, out_dtype=tg.OUT_F32)
    torch.cuda.synchronize()
    assert torch.equal(y, tg.gemm_q2_ep(x, wq, sc, out_dtype=tg.OUT_F32))
    check(y, *reference("q2", x, w, None, "none", None, None, True), "shifted scales")


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("K", [20480, 32768, 33792])
def test_very_long_rows(fmt, K):
    """Longer than the small path keeps activations for, and than it takes at all."""
    run(fmt, 3, 40, K, "none", "bias:f32", "f32")
    run(fmt, 13, 40, K, "none", "", "bf16")


@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("M", [3, 50])
def test_large_scales(fmt, M):
    """Scales up to f16's range, where the offsets of the unpacked codes must not overflow."""
    N, K = 72, 256
    wq, sc, w = pack(fmt, (N, K), 2, "cuda")
    big = 2.0 ** 11
    s2, w2 = sc.clone(), w * big
    (s2 if fmt == "q2" else s2[..., 0]).mul_(big)
    x = torch.randn(M, K, device="cuda").bfloat16()
    for out in ("f32", "bf16"):
        y = fn(fmt)(x, wq, s2, out_dtype=tg.OUT_F32 if out == "f32" else tg.OUT_BF16)
        torch.cuda.synchronize()
        check(y, *reference(fmt, x, w2, None, "none", None, None, out == "f32", s2), f"{fmt} {M} {out}")


@pytest.mark.parametrize("M", [3, 50, 260])
@pytest.mark.parametrize("out", [tg.OUT_F32, tg.OUT_BF16])
def test_in_place_on_the_residual(M, out):
    N, K = 264, 512
    wq, sc, w = pack("q2", (N, K), 3, "cuda")
    x = torch.randn(M, K, device="cuda").bfloat16()
    r = torch.randn(M, N, device="cuda").to(torch.float32 if out == tg.OUT_F32 else torch.bfloat16)
    apart = tg.gemm_q2_ep(x, wq, sc, residual=r, out_dtype=out)
    y = r.clone()
    tg.gemm_q2_ep(x, wq, sc, residual=y, out_dtype=out, y=y)
    torch.cuda.synchronize()
    assert torch.equal(y, apart)


@pytest.mark.parametrize("M", [3, 50])
def test_nan_and_infinity_pass_through_where_they_belong(M):
    """A NaN or infinite bias, gate or residual reaches its own outputs and no others."""
    N, K = 136, 256
    wq, sc, w = pack("q2", (N, K), 4, "cuda")
    x = torch.randn(M, K, device="cuda").bfloat16()
    bias, res = torch.zeros(N, device="cuda"), torch.zeros(M, N, device="cuda")
    gate = torch.ones(M, N, device="cuda").bfloat16()
    plain = tg.gemm_q2_ep(x, wq, sc, out_dtype=tg.OUT_F32)
    bias[5], res[1, 7], gate[2, 9] = float("nan"), float("inf"), float("nan")
    y = tg.gemm_q2_ep(x, wq, sc, bias=bias, gate=gate, residual=res, out_dtype=tg.OUT_F32)
    torch.cuda.synchronize()
    assert y[:, 5].isnan().all() and y[1, 7] == float("inf") and y[2, 9].isnan()
    keep = torch.ones(M, N, dtype=torch.bool, device="cuda")
    keep[:, 5] = keep[1, 7] = keep[2, 9] = False
    assert torch.equal(y[keep], plain[keep])


def test_calls_repeat_bit_for_bit_and_on_other_streams():
    """Two streams at once with workspaces of their own, and the default stream: the same bits."""
    N, K, M = 1100, 1280, 90
    wq, sc, w = pack("q4", (N, K), 6, "cuda")
    x = torch.randn(M, K, device="cuda").bfloat16()
    first = tg.gemm_q4_ep(x, wq, sc, act=tg.ACT_GELU)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                ys.append(tg.gemm_q4_ep(x, wq, sc, act=tg.ACT_GELU))
    torch.cuda.synchronize()
    assert all(torch.equal(y, first) for y in ys)
    assert tg.device_error() == 0


@pytest.mark.parametrize("M", [2, 80])
def test_captured_and_replayed(M):
    """Two graphs, each with its own workspace, replayed at once on new inputs."""
    N, K = 512, 768
    wq, sc, w = pack("q2", (N, K), 8, "cuda")
    xs = [torch.zeros(M, K, device="cuda").bfloat16() for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tg.gemm_q2_ep(xs[0], wq, sc, act=tg.ACT_SILU)
    torch.cuda.current_stream().wait_stream(s)
    graphs, ys = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            h = tg.gemm_q2_ep(x, wq, sc, act=tg.ACT_SILU)
        graphs.append(g)
        ys.append(h)
    new = [torch.randn(M, K, device="cuda").bfloat16() for _ in range(2)]
    for x, v in zip(xs, new):
        x.copy_(v)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for v, y in zip(new, ys):
        assert torch.equal(y, tg.gemm_q2_ep(v, wq, sc, act=tg.ACT_SILU))


def test_no_device_error():
    assert tg.device_error() == 0
