"""Measured cases of the experts' FP8 linear layers and of the 8-bit integer
linear layers: their inputs, their plain form in elementary torch operations,
the calls of this package's entry points, and the exact results in 64 bits.

Operators (``case["op"]``):

  experts_fwd   Y[t] = X8[t] W8[e]^T / (sx sw[e]) (+ b[e]) for the rows t of
                expert e; rows sorted by expert, offsets on the device
  experts_bwd   the gradients of that layer: dX, dW per expert, db per expert
  int8          Y = (Xq Wq^T) / (sx[m] sw[n]) (+ b[n]); X quantized to 8-bit
                integers row by row inside the call
  int8_experts  the same, with a weight matrix per expert

The routing of an experts' case (how many rows each expert has) is drawn once
from the case's sizes; the seed decides which expert gets which share.
"""

import math

import numpy as np
import torch

own = False

E4M3_MAX, E5M2_MAX = 448.0, 57344.0


# ---------------------------------------------------------------- cases

def _experts(name, op, rows, experts, K, N, **kw):
    return {"name": name, "op": op, "rows": rows, "experts": experts, "K": K, "N": N, **kw}


def listed():
    return [
        # a training step of a few wide experts: the largest products, the
        # matrix rate bounds them
        _experts("experts fwd wide", "experts_fwd", 16384, 8, 4096, 11008, bias=False),
        # a training step of many experts with few rows each: tiles end
        # inside most groups, every expert's weights are read
        _experts("experts fwd many", "experts_fwd", 8190, 64, 1536, 6912, bias=True),
        # decoding: a handful of tokens spread over the experts, bound by
        # reading the weights of those that were hit
        _experts("experts fwd decode", "experts_fwd", 24, 64, 1536, 6912, bias=True),
        # the gradients for already quantized output gradients
        _experts("experts bwd wide", "experts_bwd", 16384, 8, 1536, 6912, grad="e5m2"),
        # the gradients from bf16, quantized in the call with a scale of its own
        _experts("experts bwd many", "experts_bwd", 4093, 32, 1024, 4096, grad="bf16"),
        # a small layer's gradients, where the launches count
        _experts("experts bwd small", "experts_bwd", 130, 4, 256, 256, grad="bf16"),
        # one token of one sequence through one projection
        {"name": "int8 one token", "op": "int8", "M": 1, "K": 4096, "N": 11008, "type": "bf16",
         "bias": True},
        # a decoding batch of an odd number of sequences
        {"name": "int8 batch", "op": "int8", "M": 33, "K": 11008, "N": 4096, "type": "fp16",
         "bias": False},
        # a prompt
        {"name": "int8 prompt", "op": "int8", "M": 4096, "K": 4096, "N": 11008, "type": "bf16",
         "bias": True},
        # sizes that no vector width divides
        {"name": "int8 odd sizes", "op": "int8", "M": 511, "K": 1003, "N": 777, "type": "fp16",
         "bias": True},
        # decoding through the experts
        _experts("int8 experts decode", "int8_experts", 16, 16, 4096, 11008, type="bf16",
                 bias=False),
        # a prompt through the experts
        _experts("int8 experts prompt", "int8_experts", 8200, 16, 1536, 6912, type="bf16",
                 bias=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["experts_fwd", "experts_bwd", "int8", "int8_experts"])
    K, N = _spread(rng, 128, 11008), _spread(rng, 128, 11008)
    if rng.random() < 0.8:  # most layers' sizes are multiples of 32
        K, N = max(32, K // 32 * 32), max(32, N // 32 * 32)
    most = 700_000_000_000 // (K * N)  # rows: no more products than the listed cases have
    if op == "int8":
        return {"op": op, "M": _spread(rng, 1, min(8192, most)), "K": K, "N": N,
                "type": rng.choice(["bf16", "fp16"]), "bias": rng.random() < 0.5}
    rows = _spread(rng, 1, min(12000, most // 2 if op == "experts_bwd" else most))
    experts = _spread(rng, 2, 128)
    experts = max(1, min(experts, (1 << 29) // (K * N)))  # one card's share of the experts
    case = {"op": op, "rows": rows, "experts": experts, "K": K, "N": N}
    if op == "experts_bwd":
        case["grad"] = rng.choice(["e5m2", "bf16"])
    else:
        case["bias"] = rng.random() < 0.5
    if op == "int8_experts":
        case["type"] = rng.choice(["bf16", "fp16"])
    return case


def _shares(case):
    """Rows of each expert, largest first: a multinomial draw over unequal
    shares, the same for every seed of a case."""
    E = case["experts"]
    p = 1.0 / (4.0 + np.arange(E))
    r = np.random.RandomState(case["rows"] * 131 + E)
    return np.sort(r.multinomial(case["rows"], p / p.sum()))[::-1]


# ---------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _codes(v, top, f8):
    """v as FP8 codes (bytes) with the scale top / max |v|."""
    s = (top / v.abs().amax()).reshape(1)
    return (v * s).clamp(-top, top).to(f8).view(torch.uint8), s


def _rows8(v):
    """v [.., N, K] as 8-bit integers with one scale for each row."""
    s = 127.0 / v.abs().amax(-1)
    return (v * s[..., None]).round().to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    K, N, dev = case["K"], case["N"], "cuda"
    if case["op"] == "int8":
        M, E = case["M"], 1
    else:
        M, E = case["rows"], case["experts"]
        sizes = torch.from_numpy(_shares(case).copy())
        cpu = torch.Generator()
        cpu.manual_seed(seed)
        sizes = sizes[torch.randperm(E, generator=cpu)]
        st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(
            torch.int32).to(dev)
        st["sizes"] = sizes.tolist()
    dt = _TYPES.get(case.get("type"), torch.bfloat16)
    if case.get("bias"):
        st["b"] = (_randn(g, *((E, N) if "experts" in case else (N,))) * 0.1).to(dt)
    else:
        st["b"] = None
    if case["op"].startswith("int8"):
        # activations with a few large channels, as linear layers meet them
        x = _randn(g, M, K)
        st["x"] = (x * (1.0 + 20.0 * (torch.rand(K, generator=g, device=dev) < 0.002))).to(dt)
        w = [_rows8(_randn(g, N, K) * 0.02) for _ in range(E)]
        st["w"], st["sw"] = torch.stack([q for q, _ in w]), torch.stack([s for _, s in w])
        if case["op"] == "int8":
            st["w"], st["sw"] = st["w"][0], st["sw"][0]
        st["y"] = torch.empty(M, N, dtype=dt, device=dev)
        st["x8"] = torch.empty(M, K, dtype=torch.int8, device=dev)
        st["sx"] = torch.empty(M, dtype=torch.float32, device=dev)
        return st
    st["x"], st["sx"] = _codes(_randn(g, M, K), E4M3_MAX, torch.float8_e4m3fn)
    w = [_codes(_randn(g, N, K) * 0.02, E4M3_MAX, torch.float8_e4m3fn) for _ in range(E)]
    st["w"], st["sw"] = torch.stack([q for q, _ in w]), torch.cat([s for _, s in w])
    if case["op"] == "experts_fwd":
        st["y"] = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
        return st
    gr = _randn(g, M, N) * 1e-3
    if case["grad"] == "bf16":
        st["g"] = gr.to(torch.bfloat16)
    else:
        st["g"], st["sg"] = _codes(gr, E5M2_MAX, torch.float8_e5m2)
    st["g8"] = torch.empty(M, N, dtype=torch.uint8, device=dev)
    st["sg_used"], st["amax"] = (torch.empty(1, dtype=torch.float32, device=dev)
                                 for _ in range(2))
    st["dx"] = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    st["dw"] = torch.empty(E, N, K, dtype=torch.bfloat16, device=dev)
    st["db"] = torch.empty(E, N, dtype=torch.bfloat16, device=dev)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    import scaled_quantize_fp8_amd as F

    case = st["case"]
    if case["op"] == "int8":
        F.fp8_i8_linear_fwd(st["x"], F.QuantizedRows(st["w"], st["sw"]), st["b"], st["y"],
                            st["x8"], st["sx"])
        return st["y"]
    if case["op"] == "int8_experts":
        F.fp8_i8_grouped_linear_fwd(st["x"], F.QuantizedRows(st["w"], st["sw"]), st["b"],
                                    st["offsets"], st["y"], st["x8"], st["sx"])
        return st["y"]
    x8 = F.Quantized(st["x"], F.FP8_E4M3, st["sx"])
    w8 = F.Quantized(st["w"], F.FP8_E4M3, st["sw"])
    if case["op"] == "experts_fwd":
        F.fp8_grouped_linear_fwd(x8, w8, st["b"], st["offsets"], F.FP8_E4M3, st["y"])
        return st["y"]
    gr = st["g"] if case["grad"] == "bf16" else F.Quantized(st["g"], F.FP8_E5M2, st["sg"])
    ws = torch.empty(F.fp8_grouped_db_workspace_bytes(case["rows"], case["experts"], case["N"]),
                     dtype=torch.uint8, device="cuda")
    F.fp8_grouped_linear_bwd(gr, F.FP8_E5M2, st["offsets"], x8, w8, st["dx"], st["dw"], st["db"],
                             ws, g8_out=st["g8"], sg_used=st["sg_used"], amax_g=st["amax"])
    return {"dx": st["dx"], "dw": st["dw"], "db": st["db"]}


def _quantize_rows(x):
    """Row-wise 8-bit integers: s = 127 / max |x|, q = rint(x s), in 32 bits."""
    s = 127.0 / x.abs().amax(1)
    return (x * s[:, None]).round(), s


class _Rows:
    """The experts that have rows, and their rows padded to the longest group:
    [A, longest] row numbers, and where a place holds a row."""

    def __init__(self, st):
        sizes = st["sizes"]
        off = st["offsets"].long()
        self.live = torch.tensor([e for e, n in enumerate(sizes) if n], device="cuda")
        place = torch.arange(max(sizes), device="cuda")
        self.row = off[self.live][:, None] + place
        self.here = self.row < off[self.live + 1][:, None]
        self.row = self.row.clamp(max=st["x"].shape[0] - 1)

    def gather(self, m):
        return m[self.row] * self.here[..., None]

    def scatter(self, padded):
        return padded[self.here]  # groups in order, rows in order


def _plain(st):
    case, dt = st["case"], _TYPES.get(st["case"].get("type"), torch.bfloat16)
    if case["op"] == "int8":
        q, s = _quantize_rows(st["x"].float())
        y = (q @ st["w"].float().T) * ((1.0 / s)[:, None] * (1.0 / st["sw"])[None])
        return (y if st["b"] is None else y + st["b"].float()).to(dt)
    r = _Rows(st)
    if case["op"] == "int8_experts":
        q, s = _quantize_rows(st["x"].float())
        y = torch.bmm(r.gather(q), st["w"][r.live].float().transpose(1, 2))
        y = y * ((1.0 / s)[r.row][..., None] * (1.0 / st["sw"][r.live])[:, None])
        if st["b"] is not None:
            y = y + st["b"][r.live].float()[:, None]
        return r.scatter(y).to(dt)
    w = st["w"].view(torch.float8_e4m3fn)[r.live].float() / st["sw"][r.live][:, None, None]
    x = r.gather(st["x"].view(torch.float8_e4m3fn).float() / st["sx"])
    if case["op"] == "experts_fwd":
        y = torch.bmm(x, w.transpose(1, 2))
        if st["b"] is not None:
            y = y + st["b"][r.live].float()[:, None]
        return r.scatter(y).to(dt)
    if case["grad"] == "bf16":
        gb = st["g"].float()
        s = E5M2_MAX / gb.abs().amax()
        gr = (gb * s).clamp(-E5M2_MAX, E5M2_MAX).to(torch.float8_e5m2).float() / s
    else:
        gb = gr = st["g"].view(torch.float8_e5m2).float() / st["sg"]
    gp = r.gather(gr)
    E, N, K = case["experts"], case["N"], case["K"]
    dw = torch.zeros(E, N, K, dtype=dt, device="cuda")
    dw[r.live] = torch.bmm(gp.transpose(1, 2), x).to(dt)
    db = torch.zeros(E, N, dtype=dt, device="cuda")
    db[r.live] = r.gather(gb).sum(1).to(dt)
    return {"dx": r.scatter(torch.bmm(gp, w)).to(dt), "dw": dw, "db": db}


# ---------------------------------------------------------------- what it takes

def work(case):
    K, N = case["K"], case["N"]
    if case["op"] == "int8":
        M = case["M"]
        return {"bytes": 2 * M * K + N * K + 4 * N + (2 * N if case["bias"] else 0) + 2 * M * N,
                "flops": 2 * M * N * K}
    T, E = case["rows"], case["experts"]
    live = int((_shares(case) > 0).sum())
    if case["op"] == "int8_experts":
        return {"bytes": 2 * T * K + live * (N * K + 4 * N + (2 * N if case["bias"] else 0))
                + 2 * T * N + 4 * (E + 1), "flops": 2 * T * N * K}
    if case["op"] == "experts_fwd":
        return {"bytes": T * K + live * (N * K + 4 + (2 * N if case["bias"] else 0)) + 2 * T * N
                + 4 * (E + 1), "flops": 2 * T * N * K}
    gb = 2 if case["grad"] == "bf16" else 1
    return {"bytes": T * K + gb * T * N + live * (N * K + 4) + 2 * T * K + 2 * E * N * K
            + 2 * E * N + 4 * (E + 1), "flops": 4 * T * N * K}


# ---------------------------------------------------------------- exact results

def _decoded(codes, fmt):
    """FP8 codes as 64-bit values, from the formats' fields: E4M3 is
    sign.4.3 with bias 7, E5M2 sign.5.2 with bias 15 (finite codes)."""
    man = 3 if fmt == "e4m3" else 2
    bias = 7 if fmt == "e4m3" else 15
    c = np.arange(256)
    e, m = (c & 0x7F) >> man, c & ((1 << man) - 1)
    mag = np.where(e == 0, m * 2.0 ** (1 - bias - man),
                   (m + (1 << man)) * 2.0 ** (e - bias - man))
    table = torch.from_numpy(np.where(c & 0x80, -mag, mag)).to("cuda")
    return table[codes.long()]


def _encoded_e5m2(v):
    """The E5M2 value nearest to each v (|v| <= 57344), ties to the even code."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(ex - 3, min=-16))
    return torch.round(v / step) * step


def _int8_rows_exact(x):
    """Codes and scales of the row-wise quantize: both the scale 127 / max |x|
    and the product x s are 32-bit numbers by definition."""
    x = x.double()
    s = (127.0 / x.abs().amax(1)).float().double()
    return torch.round((x * s[:, None]).float().double()), s


def exact(case, seed):
    st = prepare(case, seed)
    b = st["b"]
    if case["op"] == "int8":
        q, s = _int8_rows_exact(st["x"])
        y = q @ st["w"].double().T / (s[:, None] * st["sw"].double()[None])
        return y if b is None else y + b.double()
    off = st["offsets"].tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(case["experts"]) if off[e + 1] > off[e]]
    if case["op"] == "int8_experts":
        q, s = _int8_rows_exact(st["x"])
        y = torch.empty(case["rows"], case["N"], dtype=torch.float64, device="cuda")
        for e, i, j in spans:
            y[i:j] = q[i:j] @ st["w"][e].double().T / (s[i:j, None] * st["sw"][e].double()[None])
            if b is not None:
                y[i:j] += b[e].double()
        return y
    x = _decoded(st["x"], "e4m3") / st["sx"].double()
    sw = st["sw"].double()
    if case["op"] == "experts_fwd":
        y = torch.empty(case["rows"], case["N"], dtype=torch.float64, device="cuda")
        for e, i, j in spans:
            y[i:j] = x[i:j] @ (_decoded(st["w"][e], "e4m3") / sw[e]).T
            if b is not None:
                y[i:j] += b[e].double()
        return y
    if case["grad"] == "bf16":
        gb = st["g"].double()
        s = (E5M2_MAX / gb.abs().amax()).float().double()
        gr = _encoded_e5m2((gb * s).float().double().clamp(-E5M2_MAX, E5M2_MAX)) / s
    else:
        gb = gr = _decoded(st["g"], "e5m2") / st["sg"].double()
    E, N, K = case["experts"], case["N"], case["K"]
    dx = torch.empty(case["rows"], K, dtype=torch.float64, device="cuda")
    dw = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    db = torch.zeros(E, N, dtype=torch.float64, device="cuda")
    for e, i, j in spans:
        dx[i:j] = gr[i:j] @ (_decoded(st["w"][e], "e4m3") / sw[e])
        dw[e] = gr[i:j].T @ x[i:j]
        db[e] = gb[i:j].sum(0)
    return {"dx": dx, "dw": dw, "db": db}
