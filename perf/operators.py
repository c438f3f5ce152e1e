"""The expert and epilogue matmuls of the library, as measured work.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the
calls a user makes of the library:

``ep``       y = residual + gate * act(x W^T + bias) for packed ternary or 4-bit weights
``grouped``  the same epilogue on matmuls grouped by expert: rows [o_e, o_{e+1}) of the
             sorted activations times the packed weights of expert e
``sort``     the plan of the grouped matmul: (token, choice) pairs sorted by expert
``combine``  the weighted sum of each token's expert outputs, plus a residual

Widths are the library's text encoder's (2560 and 9728) and its MLP width 12288, or generic
expert widths.
"""
from __future__ import annotations

import math

import torch

own = False

# The smallest to the largest of these stand for serving (one token, a few, a batch of
# single tokens) and for prefill (hundreds to thousands of tokens).
_LISTED = [
    # one token through a square ternary projection that adds onto the residual stream
    dict(name="ep_q2_one_token", op="ep", fmt="q2", M=1, N=2560, K=2560, act="none", bias="bf16",
         gate="", residual="bf16", out="bf16"),
    # a batch of single tokens through the encoder's gated 4-bit MLP-up: silu(x Wg^T) * up
    dict(name="ep_q4_twelve_tokens", op="ep", fmt="q4", M=12, N=9728, K=2560, act="silu", bias="",
         gate="full", residual="", out="bf16"),
    # image and text tokens together through the ternary MLP-up with a tanh-GELU
    dict(name="ep_q2_image_tokens", op="ep", fmt="q2", M=1536, N=12288, K=2560, act="gelu_tanh",
         bias="bf16", gate="", residual="", out="bf16"),
    # a prompt through the encoder's 4-bit MLP-down: a gated residual add
    dict(name="ep_q4_prompt", op="ep", fmt="q4", M=509, N=2560, K=9728, act="none", bias="f32",
         gate="row", residual="f32", out="f32"),
    # one token's eight experts of sixty-four, ternary
    dict(name="grouped_q2_one_token", op="grouped", fmt="q2", T=1, k=8, E=64, N=1408, K=2048,
         gather=True, act="none", bias="", gate=False, residual="", out="bf16"),
    # a batch of single tokens: a few rows for each of sixty-four experts, gated, 4-bit
    dict(name="grouped_q4_batch", op="grouped", fmt="q4", T=61, k=6, E=64, N=1408, K=2048,
         gather=True, act="silu", bias="", gate=True, residual="", out="bf16"),
    # a prompt over eight wide experts: ragged groups of hundreds of rows
    dict(name="grouped_q4_prompt", op="grouped", fmt="q4", T=1021, k=2, E=8, N=4864, K=2560,
         gather=True, act="gelu", bias="bf16", gate=False, residual="", out="bf16"),
    # the largest: long prefill over sixty-four ternary experts, already in expert order
    dict(name="grouped_q2_prefill", op="grouped", fmt="q2", T=4096, k=4, E=64, N=2048, K=2560,
         gather=False, act="none", bias="f32", gate=False, residual="", out="f32"),
    # routing plans: a batch of single tokens, and a long prefill
    dict(name="sort_batch", op="sort", T=61, k=6, E=64),
    dict(name="sort_prefill", op="sort", T=32749, k=8, E=128),
    # combining expert outputs: a batch of single tokens, and a long prefill
    dict(name="combine_batch", op="combine", T=61, k=6, N=2048, h="bf16", residual="bf16", out="bf16"),
    dict(name="combine_prefill", op="combine", T=8191, k=8, N=2560, h="bf16", residual="f32", out="f32"),
]


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ep", "ep", "ep", "grouped", "grouped", "grouped", "sort", "combine"])
    if op == "sort":
        E = _log(rng, 2, 512)
        return dict(op=op, T=_log(rng, 1, 32768), k=rng.randint(1, min(8, E)), E=E)
    if op == "combine":
        return dict(op=op, T=_log(rng, 1, 8192), k=rng.randint(1, 8), N=8 * _log(rng, 16, 320) + rng.choice([0, 0, 0, 4, 3]),
                    h=rng.choice(["bf16", "bf16", "f32"]), residual=rng.choice(["", "bf16", "f32"]),
                    out=rng.choice(["bf16", "f32"]))
    fmt = rng.choice(["q2", "q4"])
    block = 128 if fmt == "q2" else 64
    act = rng.choice(["none", "silu", "gelu", "gelu_tanh"])
    out = rng.choice(["bf16", "bf16", "f32"])
    bias = rng.choice(["", "bf16", "f32"])
    K = block * _log(rng, 256 // block, 9728 // block)
    if op == "ep":
        while True:
            M, N = _log(rng, 1, 4096), _log(rng, 256, 12288)
            if rng.random() < 0.7:
                N = (N + 7) // 8 * 8
            if M * N * K <= 1536 * 12288 * 2560:
                return dict(op=op, fmt=fmt, M=M, N=N, K=K, act=act, bias=bias,
                            gate=rng.choice(["", "row", "full"]), residual=rng.choice(["", "bf16", "f32"]), out=out)
    while True:
        E = _log(rng, 2, 128)
        T, k, N = _log(rng, 1, 8192), rng.randint(1, min(8, E)), _log(rng, 256, 5632)
        if rng.random() < 0.7:
            N = (N + 7) // 8 * 8
        if T * k * N * K <= 4096 * 4 * 2048 * 2560 and E * N * K <= 64 * 2560 * 2560:
            return dict(op=op, fmt=fmt, T=T, k=k, E=E, N=N, K=K, gather=rng.random() < 0.5, act=act, bias=bias,
                        gate=rng.random() < 0.4, residual=rng.choice(["", "", "bf16", "f32"]), out=out)


# ---- inputs ----------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _popularity(E):
    """The share of the pairs that each expert gets, near enough: some are twice as popular as others."""
    p = [2.0 ** math.sin(1.7 * e) for e in range(E)]
    s = sum(p)
    return [v / s for v in p]


def _weights(fmt, N, K, g):
    """Packed weights of N rows: ternary codes with a scale for each 128, or 4-bit codes with
    scale and zero point for each 64 (codes and scales as the library's packers lay them out)."""
    if fmt == "q2":
        codes = torch.randint(0, 3, (N, K // 4, 4), dtype=torch.uint8, device="cuda", generator=g)
        wq = codes[..., 0] | codes[..., 1] << 2 | codes[..., 2] << 4 | codes[..., 3] << 6
        return wq.contiguous(), (torch.randn(N, K // 128, device="cuda", generator=g).abs() * 0.02).half()
    wq = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.randn(N, K // 64, device="cuda", generator=g).abs() * 0.01
    z = 7 + torch.rand(N, K // 64, device="cuda", generator=g)
    return wq, torch.stack([s, z], -1).half()


def _routing(T, k, E, g):
    """ids [T, k]: k different experts for each token, some experts more popular than others."""
    logp = torch.tensor(_popularity(E), device="cuda").log()
    u = torch.rand(T, E, device="cuda", generator=g).clamp_min(1e-20)
    return (logp - (-u.log()).log()).topk(k, dim=1).indices.int()


def _epilogue(case, M, N, groups, g):
    def rnd(*shape):
        return torch.randn(*shape, device="cuda", generator=g)
    st = dict(bias=None, gate=None, residual=None)
    if case["bias"]:
        st["bias"] = (0.5 * rnd(*groups, N)).to(_DT[case["bias"]])
    if case["gate"]:
        st["gate"] = rnd(N).bfloat16() if case["gate"] == "row" else rnd(M, N).bfloat16()
    if case["residual"]:
        st["residual"] = rnd(M, N).to(_DT[case["residual"]])
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "sort":
        return dict(case=case, ids=_routing(case["T"], case["k"], case["E"], g))
    if op == "combine":
        T, k, N = case["T"], case["k"], case["N"]
        st = dict(case=case, h=torch.randn(T * k, N, device="cuda", generator=g).to(_DT[case["h"]]),
                  pos=torch.randperm(T * k, device="cuda", generator=g).int().view(T, k),
                  weights=torch.softmax(torch.randn(T, k, device="cuda", generator=g), 1), residual=None)
        if case["residual"]:
            st["residual"] = torch.randn(T, N, device="cuda", generator=g).to(_DT[case["residual"]])
        return st
    N, K = case["N"], case["K"]
    if op == "ep":
        M = case["M"]
        wq, sc = _weights(case["fmt"], N, K, g)
        x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
        return dict(case=case, x=x, wq=wq, sc=sc, **_epilogue(case, M, N, (), g))
    T, k, E = case["T"], case["k"], case["E"]
    ids = _routing(T, k, E, g).flatten().long()
    order = ids.sort(stable=True).indices
    counts = ids.bincount(minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    wq, sc = _weights(case["fmt"], E * N, K, g)
    x = torch.randn(T if case["gather"] else T * k, K, device="cuda", generator=g).bfloat16()
    return dict(case=case, x=x, wq=wq.view(E, N, -1), sc=sc.view(E, N, *sc.shape[1:]), offsets=offsets,
                rows=(order // k).int() if case["gather"] else None, counts=counts.tolist(),
                **_epilogue(case, T * k, N, (E,), g))


# ---- one pass --------------------------------------------------------------------------

def _dequant(fmt, wq, sc):
    """The weights that packed rows [N, bytes] stand for, f32 [N, K]."""
    N = wq.shape[0]
    if fmt == "q2":
        q = torch.stack([(wq >> s) & 3 for s in (0, 2, 4, 6)], -1).view(N, -1, 128).float()
        return ((q - 1) * sc.float()[..., None]).view(N, -1)
    q = torch.stack([wq & 15, wq >> 4], -1).view(N, -1, 64).float()
    return ((q - sc[..., 1:].float()) * sc[..., :1].float()).view(N, -1)


def _activate(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_rows(st, x, wq, sc, bias, rows):
    """The plain form of some rows of a matmul with its epilogue, in the output's type."""
    c = st["case"]
    v = x.float() @ _dequant(c["fmt"], wq, sc).T
    if bias is not None:
        v = v + bias.float()
    v = _activate(v, c["act"])
    if st["gate"] is not None:
        v = v * (st["gate"] if st["gate"].dim() == 1 else st["gate"][rows]).float()
    if st["residual"] is not None:
        v = v + st["residual"][rows].float()
    return v.to(_DT[c["out"]])


def _plain(st):
    c = st["case"]
    if c["op"] == "ep":
        return _plain_rows(st, st["x"], st["wq"], st["sc"], st["bias"], slice(None))
    if c["op"] == "grouped":
        x = st["x"] if st["rows"] is None else st["x"][st["rows"].long()]
        y = torch.empty(c["T"] * c["k"], c["N"], dtype=_DT[c["out"]], device=x.device)
        at = 0
        for e, n in enumerate(st["counts"]):
            if n:
                rows = slice(at, at + n)
                y[rows] = _plain_rows(st, x[rows], st["wq"][e], st["sc"][e],
                                      None if st["bias"] is None else st["bias"][e], rows)
            at += n
        return y
    if c["op"] == "sort":
        ids = st["ids"].flatten().long()
        order = ids.sort(stable=True).indices
        offsets = torch.zeros(c["E"] + 1, dtype=torch.int32, device=ids.device)
        offsets[1:] = (ids[:, None] == torch.arange(c["E"], device=ids.device)).sum(0).cumsum(0)
        pos = torch.empty_like(order)
        pos[order] = torch.arange(order.numel(), device=ids.device)
        return offsets, (order // c["k"]).int(), pos.int().view(c["T"], c["k"])
    y = (st["h"][st["pos"].long()].float() * st["weights"][..., None]).sum(1)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(_DT[c["out"]])


def _own(st):
    import bit_weight_quantized_tgemm_b200 as tg

    c = st["case"]
    out = {"bf16": tg.OUT_BF16, "f32": tg.OUT_F32}[c["out"]] if "out" in c else None
    if c["op"] == "sort":
        return tg.expert_sort(st["ids"], c["E"])
    if c["op"] == "combine":
        return tg.expert_combine(st["h"], st["pos"], st["weights"], residual=st["residual"], out_dtype=out)
    act = {"none": tg.ACT_NONE, "silu": tg.ACT_SILU, "gelu": tg.ACT_GELU, "gelu_tanh": tg.ACT_GELU_TANH}[c["act"]]
    ep = dict(bias=st["bias"], act=act, gate=st["gate"], residual=st["residual"], out_dtype=out)
    if c["op"] == "ep":
        return (tg.gemm_q2_ep if c["fmt"] == "q2" else tg.gemm_q4_ep)(st["x"], st["wq"], st["sc"], **ep)
    fn = tg.gemm_q2_grouped if c["fmt"] == "q2" else tg.gemm_q4_grouped
    return fn(st["x"], st["wq"], st["sc"], st["offsets"], rows=st["rows"], **ep)


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -------------------------------------------------------

_SIZE = {"": 0, "bf16": 2, "f32": 4}


def work(case):
    c = case
    if c["op"] == "sort":
        pairs = c["T"] * c["k"]
        return dict(bytes=4 * (3 * pairs + c["E"] + 1), flops=pairs)
    if c["op"] == "combine":
        T, k, N = c["T"], c["k"], c["N"]
        return dict(bytes=T * k * (N * _SIZE[c["h"]] + 8) + T * N * (_SIZE[c["residual"]] + _SIZE[c["out"]]),
                    flops=2 * T * k * N)
    N, K = c["N"], c["K"]
    per_row = K // 4 + K // 128 * 2 if c["fmt"] == "q2" else K // 2 + K // 64 * 4  # packed bytes of a weight row
    if c["op"] == "ep":
        M, experts, x_rows = c["M"], 1, c["M"]
        gate = {"": 0, "row": 2 * N, "full": 2 * M * N}[c["gate"]]
    else:
        M = c["T"] * c["k"]
        # the experts that get a row at all, on average
        experts = sum(1 - (1 - min(1.0, c["k"] * p)) ** c["T"] for p in _popularity(c["E"]))
        x_rows = c["T"] if c["gather"] else M
        gate = 2 * M * N if c["gate"] else 0
    return dict(bytes=int(experts * N * (per_row + _SIZE[c["bias"]]) + 2 * x_rows * K + gate
                          + M * N * (_SIZE[c["residual"]] + _SIZE[c["out"]])), flops=2 * M * N * K)


# ---- the definitions in 64 bits ------------------------------------------------------------

def _w64(fmt, wq, sc):
    """Weight by weight: code j of a row sits in byte j / 4 at bit 2 (j % 4) (ternary) or in
    byte j / 2 at bit 4 (j % 2); ternary (q - 1) d, 4-bit (q - z) s."""
    bits = 2 if fmt == "q2" else 4
    per = 8 // bits
    j = torch.arange(wq.shape[1] * per, device=wq.device)
    q = (wq.long()[:, j // per] >> (bits * (j % per))) & (2 ** bits - 1)
    if fmt == "q2":
        return (q.double() - 1) * sc.double()[:, j // 128]
    return (q.double() - sc.double()[:, j // 64, 1]) * sc.double()[:, j // 64, 0]


def _phi64(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        # (1 + tanh(u)) / 2 is the logistic function of 2 u
        return v * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    return v


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "sort":
        # whole numbers: they have one right value, which the plain form gives
        return None
    if c["op"] == "combine":
        y = torch.zeros(c["T"], c["N"], dtype=torch.float64, device="cuda")
        if st["residual"] is not None:
            y += st["residual"].double()
        for j in range(c["k"]):
            y += st["weights"][:, j, None].double() * st["h"].double()[st["pos"][:, j].long()]
        return y
    if c["op"] == "ep":
        y = torch.einsum("mk,nk->mn", st["x"].double(), _w64(c["fmt"], st["wq"], st["sc"]))
        if st["bias"] is not None:
            y += st["bias"].double()[None]
    else:
        y = torch.zeros(c["T"] * c["k"], c["N"], dtype=torch.float64, device="cuda")
        ends = st["offsets"].tolist()
        for e in range(c["E"]):
            lo, hi = ends[e], ends[e + 1]
            if lo == hi:
                continue
            src = st["x"][lo:hi] if st["rows"] is None else st["x"].index_select(0, st["rows"][lo:hi].long())
            y[lo:hi] = torch.einsum("mk,nk->mn", src.double(), _w64(c["fmt"], st["wq"][e], st["sc"][e]))
            if st["bias"] is not None:
                y[lo:hi] += st["bias"][e].double()
    y = _phi64(y, c["act"])
    if st["gate"] is not None:
        y = y * st["gate"].double()
    if st["residual"] is not None:
        y = st["residual"].double() + y
    return y
