"""Matmuls grouped by expert, the expert sort and combine, and a run of them (GPU)."""
import pytest
import torch

import bit_weight_quantized_tgemm_b200 as tg
from ep_reference import ACTS, F32, check, epilogue, pack, reference

pytestmark = pytest.mark.gpu

PATHS = {"auto": tg.PATH_AUTO, "small": tg.PATH_SMALL_M, "tensor": tg.PATH_TENSOR}


@pytest.fixture
def path():
    prev = tg.set_path(tg.PATH_AUTO)
    yield tg.set_path
    tg.set_path(prev)


def grouped(fmt):
    return tg.gemm_q2_grouped if fmt == "q2" else tg.gemm_q4_grouped


def run(fmt, counts, N, K, act="none", ep="", out="bf16", gather=None, first=0, spare=0, seed=0):
    """Groups of the given sizes after `first` rows and before `spare` ones that belong to no
    expert; gather: rows of x that the sorted rows are drawn from (None: x is sorted)."""
    E, R = len(counts), first + sum(counts) + spare
    g = torch.Generator().manual_seed(seed)
    offsets = torch.tensor([first] + counts).cumsum(0).int().cuda()
    wq, sc, w = pack(fmt, (E, N, K), seed, "cuda")
    x = torch.randn(gather or R, K, generator=g).bfloat16().cuda()
    rows = torch.randint(0, gather, (R,), generator=g).int().cuda() if gather else None
    e = epilogue(ep, R, N, (E,), seed, "cuda")
    y = torch.full((R, N), 77.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    grouped(fmt)(x, wq, sc, offsets, rows=rows, act=ACTS[act], y=y,
                 out_dtype=tg.OUT_F32 if out == "f32" else tg.OUT_BF16, **e)
    torch.cuda.synchronize()
    at = first
    for i, n in enumerate(counts):
        sl = slice(at, at + n)
        if n:
            xs = x[sl] if rows is None else x[rows[sl].long()]
            check(y[sl], *reference(fmt, xs, w[i], None if e["bias"] is None else e["bias"][i], act,
                                    None if e["gate"] is None else e["gate"][sl],
                                    None if e["residual"] is None else e["residual"][sl], out == "f32", sc[i]),
                  f"{fmt} expert {i} of {counts}")
        at += n
    assert (y[:first] == 77).all() and (y[at:] == 77).all(), "rows of no expert were written"


COUNTS = [[1], [0, 1, 0], [5, 0, 3, 1], [16, 17, 1, 0, 15], [128, 129, 0, 1], [1] * 20, [0, 0, 300, 2], [33, 64, 65, 8, 9]]


@pytest.mark.parametrize("pname", list(PATHS))
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("fmt,out", [("q2", "f32"), ("q2", "bf16"), ("q4", "f32"), ("q4", "bf16")])
def test_group_sizes(path, pname, counts, fmt, out):
    path(PATHS[pname])
    run(fmt, counts, 200, 384, "silu", "bias:bf16 gate:full", out, seed=len(counts))


@pytest.mark.parametrize("pname", list(PATHS))
@pytest.mark.parametrize("gather", [None, 7])
@pytest.mark.parametrize("first,spare", [(0, 0), (3, 0), (0, 40), (5, 131)])
def test_rows_of_no_expert_stay(path, pname, gather, first, spare):
    path(PATHS[pname])
    run("q2", [4, 0, 19, 1], 129, 256, ep="residual:f32", gather=gather, first=first, spare=spare)


@pytest.mark.parametrize("pname", list(PATHS))
@pytest.mark.parametrize("fmt,N,K", [("q4", 5, 64), ("q4", 260, 448), ("q2", 1000, 128), ("q2", 127, 2560), ("q4", 130, 4096)])
def test_widths(path, pname, fmt, N, K):
    path(PATHS[pname])
    run(fmt, [9, 1, 40], N, K, "gelu", "bias:f32 residual:bf16", "f32", gather=50)


def test_no_rows_at_all():
    run("q2", [0, 0, 0], 128, 256, spare=20)


def test_many_experts():
    run("q2", [i % 3 for i in range(1024)], 40, 128)


@pytest.mark.parametrize("E", [33, 64, 100])
def test_expert_counts_around_a_warp(E):
    run("q4", [(7 * i) % 5 for i in range(E)], 72, 128)


def test_rows_outside_x_read_zeros():
    wq, sc, w = pack("q2", (1, 64, 256), 1, "cuda")
    x = torch.randn(4, 256, device="cuda").bfloat16()
    bias = torch.randn(1, 64, device="cuda")
    off = torch.tensor([0, 4]).int().cuda()
    for R in (4, 40):
        rows = torch.tensor(([-1, 4, 2, 2 ** 30] * 10)[:R]).int().cuda()
        off = torch.tensor([0, R]).int().cuda()
        y = tg.gemm_q2_grouped(x, wq, sc, off, rows=rows, bias=bias, out_dtype=tg.OUT_F32)
        torch.cuda.synchronize()
        for i in (0, 1, 3):
            assert torch.equal(y[i], bias[0])
        check(y[2:3], *reference("q2", x[2:3], w[0], bias[0], "none", None, None, True), "row 2")


def test_bad_offsets_stay_inside_the_buffers():
    """Offsets out of range or out of order are clamped: nothing outside y is written and no
    error is raised; a later call on the same inputs is right."""
    N, K, R = 136, 256, 50
    wq, sc, w = pack("q2", (3, N, K), 2, "cuda")
    x = torch.randn(R, K, device="cuda").bfloat16()
    buf = torch.full((R + 40, N), 5.0, device="cuda")
    for bad in ([-5, 10, 2 ** 31 - 1, 60], [0, 40, 20, 50], [60, 70, 80, 90], [0, -1, -2, -3]):
        tg.gemm_q2_grouped(x, wq, sc, torch.tensor(bad).int().cuda(), out_dtype=tg.OUT_F32, y=buf[:R])
        torch.cuda.synchronize()
        assert (buf[R:] == 5).all()
    assert tg.device_error() == 0
    run("q2", [10, 20, 20], N, K)


def test_graph_replayed_with_other_group_sizes():
    E, N, K, R = 6, 200, 512, 96
    wq, sc, w = pack("q2", (E, N, K), 9, "cuda")
    x = torch.randn(R, K, device="cuda").bfloat16()
    off = torch.tensor([0, 96, 96, 96, 96, 96, 96]).int().cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tg.gemm_q2_grouped(x, wq, sc, off)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = tg.gemm_q2_grouped(x, wq, sc, off)
    for counts in ([96, 0, 0, 0, 0, 0], [1, 2, 3, 40, 50, 0], [16] * 6, [0, 0, 0, 0, 0, 0]):
        off.copy_(torch.tensor([0] + counts).cumsum(0).int())
        y.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        at = 0
        for i, n in enumerate(counts):
            if n:
                check(y[at:at + n], *reference("q2", x[at:at + n], w[i], None, "none", None, None, False), f"replay {counts}")
            at += n
        assert (y[at:] == 3).all()


# ---- sort --------------------------------------------------------------------------------

def sort_reference(ids, E):
    flat = ids.flatten().cpu().tolist()
    k = ids.shape[1]
    groups = [[i for i, e in enumerate(flat) if e == x] for x in range(E)]
    rows, pos, offsets = [], [-1] * len(flat), [0]
    for grp in groups:
        for i in grp:
            pos[i] = len(rows)
            rows.append(i // k)
        offsets.append(len(rows))
    rows += [-1] * (len(flat) - len(rows))
    return offsets, rows, pos


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (7, 3, 5), (33, 2, 2), (500, 6, 64), (4096, 1, 8), (683, 6, 30),
                                   (1200, 8, 128), (2500, 4, 1024), (5000, 2, 3)])
@pytest.mark.parametrize("stray", [False, True])
def test_sort(T, k, E, stray):
    g = torch.Generator().manual_seed(T + k + E)
    ids = torch.randint(0, E, (T, k), generator=g).int()
    if stray:  # ids of no expert among them
        m = torch.rand(T, k, generator=g) < 0.3
        ids[m] = torch.randint(0, 4, (T, k), generator=g)[m].int().mul(2 ** 29).sub(2 ** 30 + 1)
        ids[0, 0] = E
    offsets, rows, pos = tg.expert_sort(ids.cuda(), E)
    torch.cuda.synchronize()
    o, r, p = sort_reference(ids, E)
    assert offsets.tolist() == o and rows.tolist() == r and pos.flatten().tolist() == p


def test_sort_one_expert_gets_all():
    for T in (100, 9000):
        ids = torch.full((T, 1), 3, dtype=torch.int32, device="cuda")
        offsets, rows, pos = tg.expert_sort(ids, 5)
        torch.cuda.synchronize()
        assert offsets.tolist() == [0, 0, 0, 0, T, T]
        assert torch.equal(rows.cpu(), torch.arange(T).int()) and torch.equal(pos[:, 0].cpu(), torch.arange(T).int())


# ---- combine -----------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 2048), (5, 3, 77), (40, 6, 520), (300, 2, 1028), (17, 9, 256)])
@pytest.mark.parametrize("h_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("res", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out", [tg.OUT_F32, tg.OUT_BF16])
def test_combine(T, k, N, h_dt, res, out):
    g = torch.Generator().manual_seed(N)
    R = T * k + 3
    h = torch.randn(R, N, generator=g).to(h_dt).cuda()
    pos = torch.randint(-1, R + 1, (T, k), generator=g).int().cuda()
    wts = torch.randn(T, k, generator=g).cuda()
    r = None if res is None else torch.randn(T, N, generator=g).to(res).cuda()
    y = tg.expert_combine(h, pos, wts, residual=r, out_dtype=out)
    torch.cuda.synchronize()
    ok = (pos >= 0) & (pos < R)
    terms = h.double()[pos.clamp(0, R - 1).long()] * (wts.double() * ok)[..., None]
    ref = terms.sum(1) + (0 if r is None else r.double())
    # k products and k sums in f32, then the residual's, then the store's half step
    mag = terms.abs().sum(1) + (0 if r is None else r.double().abs())
    bound = (k + 2) * F32 * mag
    check(y, ref, bound + (2.0 ** -24 if out == tg.OUT_F32 else 2.0 ** -8) * (ref.abs() + bound), "combine")


def test_combine_in_place_and_of_nothing():
    h = torch.randn(4, 264, device="cuda").bfloat16()
    pos = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    r = torch.randn(6, 264, device="cuda")
    y = r.clone()
    tg.expert_combine(h, pos, torch.full((6, 2), float("nan"), device="cuda"), residual=y, y=y, out_dtype=tg.OUT_F32)
    torch.cuda.synchronize()
    assert torch.equal(y, r)
    y = tg.expert_combine(h, pos, torch.ones(6, 2, device="cuda"))
    assert (y == 0).all()


# ---- together ----------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["q2", "q4"])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_expert_mlp(fmt, T):
    """sort, up, gate, down, combine: a whole expert layer against the same in 64 bits."""
    E, k, D, F = 8, 2, 256, 384
    g = torch.Generator().manual_seed(T)
    up, gt, dn = (pack(fmt, s, i, "cuda") for i, s in enumerate([(E, F, D), (E, F, D), (E, D, F)]))
    x = torch.randn(T, D, generator=g).bfloat16().cuda()
    ids = torch.rand(T, E, generator=g).topk(k).indices.int().cuda()
    wts = torch.rand(T, k, generator=g).cuda()
    offsets, rows, pos = tg.expert_sort(ids, E)
    u = grouped(fmt)(x, up[0], up[1], offsets, rows=rows)
    h = grouped(fmt)(x, gt[0], gt[1], offsets, rows=rows, act=tg.ACT_SILU, gate=u)
    o = grouped(fmt)(h, dn[0], dn[1], offsets, out_dtype=tg.OUT_F32)
    y = tg.expert_combine(o, pos, wts, residual=x, out_dtype=tg.OUT_F32)
    torch.cuda.synchronize()
    ref = x.double()
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            a = x[t].double() @ up[2][e].T
            b = x[t].double() @ gt[2][e].T
            ref[t] += float(wts[t, j]) * ((a * b * torch.sigmoid(b)) @ dn[2][e].T)
    # u and h are rounded to bf16 in between (half a step 2^-8 each, twice), and 4-bit weights to
    # f16: relative errors of independent terms, so the norm of the difference is within them
    rel = float((y.double() - ref).norm() / (ref - x.double()).norm())
    assert rel <= 2 * 2.0 ** -8 + 3 * 2.0 ** -10, rel
    assert tg.device_error() == 0
