"""Measured cases of the routing to experts, of the exchange of rows with them,
and of the linear layers in microscaled 4-bit floating point: their inputs,
their plain form in elementary torch operations, the calls of this package's
entry points, and the exact results in 64 bits.

Operators (``case["op"]``):

  route        scores of T tokens for E experts (softmax or sigmoid of the
               logits), the k best by score + bias inside the best groups,
               their weights, and where each row goes when rows are sorted by
               expert; with ``train`` also the gradient of the logits
  exchange     rows copied into expert order, and the experts' rows back as
               weighted sums; with ``train`` both backward passes
  mx4_quantize blocks of 32 values to 4-bit floating point (sign, two exponent
               bits, one of significand) with a power of two for each block,
               and back
  mx4          Y = X W^T (+ b), both operands in that format, X quantized
               inside the call
  mx4_experts  the same with a weight matrix per expert, rows sorted by expert

A tie goes to the lowest index.  The choice of experts is that of scores held
in 64 bits.
"""

import math

import numpy as np
import torch

own = False

# ---------------------------------------------------------------- cases

def _route(name, T, E, k, **kw):
    case = {"name": name, "op": "route", "T": T, "E": E, "k": k, "type": "fp32",
            "score": "sigmoid", "bias": True, "groups": 1, "kept": 1, "group_top": 1,
            "renorm": True, "scale": 1.0, "train": False}
    return {**case, **kw}


def listed():
    return [
        # decoding: one token finds its experts; nothing but latency
        _route("route one token", 1, 64, 4),
        # a prompt over many experts in groups, a bias that balances them
        _route("route prompt", 16384, 256, 8, groups=8, kept=4, group_top=2, scale=2.5),
        # a training step, an odd number of experts and tokens, some of them
        # padding (no expert may be chosen)
        _route("route train", 4093, 96, 6, type="bf16", score="softmax", bias=False,
               renorm=False, train=True),
        # decoding: a few tokens' rows to their experts and back
        {"name": "exchange decode", "op": "exchange", "T": 24, "E": 64, "k": 4, "D": 1536,
         "type": "bf16", "train": False},
        # a training step's rows, and both backward passes
        {"name": "exchange train", "op": "exchange", "T": 4096, "E": 64, "k": 8, "D": 4096,
         "type": "bf16", "train": True},
        # a projection's weights, quantized when a trained layer is taken over
        {"name": "mx4 quantize weights", "op": "mx4_quantize", "rows": 11008, "K": 4096,
         "type": "bf16"},
        # rows that no block size divides
        {"name": "mx4 quantize odd", "op": "mx4_quantize", "rows": 511, "K": 1003, "type": "fp16"},
        # one token of one sequence through one projection
        {"name": "mx4 one token", "op": "mx4", "M": 1, "K": 4096, "N": 11008, "type": "bf16",
         "bias": True},
        # a decoding batch of an odd number of sequences
        {"name": "mx4 batch", "op": "mx4", "M": 33, "K": 11008, "N": 4096, "type": "fp16",
         "bias": False},
        # a prompt
        {"name": "mx4 prompt", "op": "mx4", "M": 4096, "K": 4096, "N": 11008, "type": "bf16",
         "bias": True},
        # decoding through the experts
        {"name": "mx4 experts decode", "op": "mx4_experts", "rows": 16, "experts": 16, "K": 4096,
         "N": 11008, "type": "bf16", "bias": False},
        # a prompt through the experts
        {"name": "mx4 experts prompt", "op": "mx4_experts", "rows": 8200, "experts": 16, "K": 1536,
         "N": 6912, "type": "bf16", "bias": True},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "exchange", "mx4_quantize", "mx4", "mx4_experts"])
    if op == "route":
        T = _spread(rng, 1, 16384)
        groups = rng.choice([1, 1, 4, 8])
        E = groups * max(2, _spread(rng, 8, 256) // groups)
        kept = 1 if groups == 1 else rng.randint(1, groups)
        k = min(_spread(rng, 1, 16), kept * (E // groups))
        return {"op": op, "T": T, "E": E, "k": k, "type": rng.choice(["fp32", "bf16", "fp16"]),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "groups": groups, "kept": kept, "group_top": rng.choice([1, 2]),
                "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]),
                "train": rng.random() < 0.4}
    if op == "exchange":
        T, k = _spread(rng, 1, 8192), _spread(rng, 1, 8)
        D = min(_spread(rng, 64, 8192), (1 << 27) // (T * k))
        D = max(1, D if rng.random() < 0.3 else D // 8 * 8)
        return {"op": op, "T": T, "E": _spread(rng, 8, 256), "k": k, "D": D,
                "type": rng.choice(["bf16", "fp16", "fp32"]) if D < 4096 else "bf16",
                "train": rng.random() < 0.5}
    K, N = _spread(rng, 64, 11008), _spread(rng, 64, 11008)
    if rng.random() < 0.7:  # most layers' sizes are multiples of 32
        K, N = max(32, K // 32 * 32), max(32, N // 32 * 32)
    if op == "mx4_quantize":
        return {"op": op, "rows": min(_spread(rng, 1, 65536), 45_000_000 // K), "K": K,
                "type": rng.choice(["bf16", "fp16", "fp32"])}
    most = 180_000_000_000 // (K * N)  # rows: no more products than the listed cases have
    case = {"op": op, "K": K, "N": N, "type": rng.choice(["bf16", "fp16"]),
            "bias": rng.random() < 0.5}
    if op == "mx4":
        return {**case, "M": _spread(rng, 1, min(8192, most))}
    rows = _spread(rng, 1, min(12000, most))
    return {**case, "rows": rows,
            "experts": max(1, min(_spread(rng, 2, 128), (1 << 29) // (K * N)))}


# ---------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_MX4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes; code 8 + i is minus the i-th


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ceil(a, b):
    return -(-a // b)


def _mx4_rows(x):
    """x [R, K] (32 bits) in blocks of 32: magnitudes' codes [R, blocks, 32]
    with the sign in bit 3, and the blocks' exponents, biased by 127."""
    R, K = x.shape
    x = torch.nn.functional.pad(x, (0, _ceil(K, 32) * 32 - K)).view(R, -1, 32)
    # the exponent field of the largest magnitude, less the largest element's exponent 2
    e = ((x.abs().amax(2).view(torch.int32) >> 23) - 2).clamp(min=0)
    inv = ((254 - e) << 23).view(torch.float32)  # 2^(127 - e)
    v = x.abs() * inv[..., None]
    v = torch.where(v < 2, torch.round(v * 2), torch.where(v < 4, torch.round(v) + 2,
                                                             torch.round(v * 0.5) + 4))
    return v.clamp(max=7).to(torch.int32) + torch.where(torch.signbit(x), 8, 0), e


def _mx4_values(code, e):
    """The 32-bit values of codes [.., blocks, 32] with exponents [.., blocks]."""
    table = torch.tensor(_MX4 + tuple(-v for v in _MX4), device="cuda")
    # 2^(e - 127) as a product of two powers that are both normal numbers
    half = e // 2
    two = lambda n: ((n + 127) << 23).view(torch.float32)
    return table[code] * (two(half - 63) * two(e - half - 64))[..., None]


def _mx4_pack(code, e):
    """Bytes as the library keeps them: two codes a byte, the even element
    low, and four blocks' exponents a 32-bit word, words [K / 128][row]."""
    R, B, _ = code.shape
    codes = (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8).view(R, B * 16)
    e = torch.nn.functional.pad(e, (0, _ceil(B, 4) * 4 - B)).to(torch.uint8)
    return codes, e.view(R, -1, 4).permute(1, 0, 2).contiguous()


def _mx4_unpack(codes, scales):
    """The reverse, over any leading dimensions: codes [.., R, blocks, 32] and
    exponents [.., R, blocks] in 32-bit integers."""
    B = codes.shape[-1] // 16
    c = codes.to(torch.int32)
    code = torch.stack([c & 15, c >> 4], -1).view(*c.shape[:-1], B, 32)
    e = scales.to(torch.int32).transpose(-3, -2).flatten(-2)[..., :B]
    return code, e


def _mx4_matrix(g, N, K):
    return _mx4_pack(*_mx4_rows(_randn(g, N, K) * 0.02))


def _shares(case):
    """Rows of each expert, largest first: a multinomial draw over unequal
    shares, the same for every seed of a case."""
    E = case["experts"]
    p = 1.0 / (4.0 + np.arange(E))
    r = np.random.RandomState(case["rows"] * 131 + E)
    return np.sort(r.multinomial(case["rows"], p / p.sum()))[::-1]


def _padding(T):
    """Rows at the end of a batch that hold no token."""
    return T // 50


def prepare(case, seed):
    g, dt, op, dev = _gen(seed), _TYPES[case["type"]], case["op"], "cuda"
    st = {"case": case}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # experts differ in how often they are liked
        z = (_randn(g, T, E) + 0.5 * _randn(g, E)).to(dt)
        if _padding(T):
            z[T - _padding(T):] = float("-inf")
        st["z"] = z
        st["b"] = 0.05 * _randn(g, E) if case["bias"] else None
        st["idx"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        st["w"] = torch.empty(T, k, dtype=torch.float32, device=dev)
        st["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
        st["pos"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        if case["train"]:
            st["dw"] = _randn(g, T, k)
            st["dz"] = torch.empty(T, E, dtype=dt, device=dev)
        return st
    if op == "exchange":
        T, E, k, D = case["T"], case["E"], case["k"], case["D"]
        like = _randn(g, T, E) + 0.5 * _randn(g, E)
        idx = like.argsort(dim=1, descending=True, stable=True)[:, :k].to(torch.int32)
        if _padding(T):
            idx[T - _padding(T):] = -1
        st["pos"], _ = _places(idx, E)
        st["w"] = torch.softmax(_randn(g, T, k), 1)
        st["x"], st["y"] = _randn(g, T, D).to(dt), _randn(g, T * k, D).to(dt)
        # rows that no slot fills keep what they held
        st["xs"] = torch.zeros(T * k, D, dtype=dt, device=dev)
        st["out"] = torch.empty(T, D, dtype=dt, device=dev)
        if case["train"]:
            st["dout"], st["dxs"] = _randn(g, T, D).to(dt), _randn(g, T * k, D).to(dt)
            st["dy"] = torch.zeros(T * k, D, dtype=dt, device=dev)
            st["dw"] = torch.empty(T, k, dtype=torch.float32, device=dev)
            st["dx"] = torch.empty(T, D, dtype=dt, device=dev)
        return st
    K = case["K"]
    B = _ceil(K, 32)
    M = case[{"mx4": "M"}.get(op, "rows")]
    x = _randn(g, M, K)
    # a few large channels, as activations have them
    st["x"] = (x * (1.0 + 20.0 * (torch.rand(K, generator=g, device=dev) < 0.002))).to(dt)
    st["xc"] = torch.empty(M, B * 16, dtype=torch.uint8, device=dev)
    st["xe"] = torch.empty(_ceil(K, 128), M, 4, dtype=torch.uint8, device=dev)
    if op == "mx4_quantize":
        st["values"] = torch.empty(M, K, dtype=dt, device=dev)
        return st
    N, E = case["N"], case.get("experts")
    w = [_mx4_matrix(g, N, K) for _ in range(E or 1)]
    st["wc"], st["we"] = (torch.stack([m[i] for m in w]) for i in range(2))
    if not E:
        st["wc"], st["we"] = st["wc"][0], st["we"][0]
    else:
        sizes = torch.from_numpy(_shares(case).copy())
        cpu = torch.Generator()
        cpu.manual_seed(seed)
        sizes = sizes[torch.randperm(E, generator=cpu)]
        st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(
            torch.int32).to(dev)
        st["sizes"] = sizes.tolist()
    st["b"] = (_randn(g, *((E, N) if E else (N,))) * 0.1).to(dt) if case["bias"] else None
    st["y"] = torch.empty(M, N, dtype=dt, device=dev)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    import scaled_quantize_fp8_amd as F

    case = st["case"]
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        how = dict(score=F.FP8_ROUTE_SOFTMAX if case["score"] == "softmax" else F.FP8_ROUTE_SIGMOID,
                   renorm=case["renorm"], scale=case["scale"])
        ws = torch.empty(F.fp8_route_workspace_bytes(T, E, k), dtype=torch.uint8, device="cuda")
        F.fp8_route_fwd(st["z"], st["idx"], st["w"], bias=st["b"], groups=case["groups"],
                        groups_kept=case["kept"], group_top=case["group_top"],
                        offsets=st["offsets"], pos=st["pos"], ws=ws, **how)
        out = {"idx": st["idx"], "w": st["w"], "offsets": st["offsets"], "pos": st["pos"]}
        if case["train"]:
            F.fp8_route_bwd(st["z"], st["idx"], st["dw"], st["dz"], **how)
            out["dz"] = st["dz"]
        return out
    if op == "exchange":
        F.fp8_route_gather(st["x"], st["pos"], st["xs"])
        F.fp8_route_combine(st["y"], st["pos"], st["w"], st["out"])
        if not case["train"]:
            return {"xs": st["xs"], "out": st["out"]}
        F.fp8_route_combine_bwd(st["dout"], st["y"], st["pos"], st["w"], st["dy"], st["dw"])
        F.fp8_route_combine(st["dxs"], st["pos"], None, st["dx"])
        return {n: st[n] for n in ("xs", "out", "dy", "dw", "dx")}
    if op == "mx4_quantize":
        F.fp8_mx4_quantize(st["x"], st["xc"], st["xe"])
        F.fp8_mx4_dequantize(F.QuantizedMx4(st["xc"], st["xe"], case["K"]), st["values"])
        return st["values"]
    w = F.QuantizedMx4(st["wc"], st["we"], case["K"])
    if op == "mx4":
        F.fp8_mx4_linear_fwd(st["x"], w, st["b"], st["y"], st["xc"], st["xe"])
    else:
        F.fp8_mx4_grouped_linear_fwd(st["x"], w, st["b"], st["offsets"], st["y"], st["xc"],
                                     st["xe"])
    return st["y"]


def _places(idx, E):
    """Where each slot's row lies when the rows are sorted by expert, in the
    order of the slots (-1: no expert), and the experts' first rows."""
    key = torch.where(idx < 0, E, idx).flatten().long()
    order = key.argsort(stable=True)
    pos = torch.empty_like(key)
    pos[order] = torch.arange(key.numel(), device=key.device)
    pos = torch.where(key < E, pos, -1).view(idx.shape).to(torch.int32)
    bounds = torch.arange(E + 1, device=key.device)
    return pos, torch.searchsorted(key[order], bounds).to(torch.int32)


def _chosen(case, z, b):
    """The k experts of each row, -1 where no more may be chosen."""
    T, E, G = case["T"], case["E"], case["groups"]
    z = z.double()
    none = z == float("-inf")
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-z))
    else:
        p = torch.exp(z - z.amax(1, keepdim=True).clamp(min=-1e300))
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    c = p if b is None else p + b.double()
    by = (z if b is None else c).masked_fill(none, float("-inf"))  # z: the order of the scores
    if G > 1:
        grouped = (by if case["group_top"] == 1 else c.masked_fill(none, float("-inf"))).view(T, G, -1)
        top = grouped.sort(dim=2, descending=True).values[:, :, :case["group_top"]]
        some = (top > float("-inf"))
        score = torch.where(some, top, 0.0).sum(2).masked_fill(~some[:, :, 0], float("-inf"))
        order = score.argsort(dim=1, descending=True, stable=True)[:, :case["kept"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order, True)
        by = by.masked_fill(~keep[:, :, None].expand(T, G, E // G).reshape(T, E), float("-inf"))
    best, idx = by.sort(dim=1, descending=True, stable=True)
    k = case["k"]
    return torch.where(best[:, :k] > float("-inf"), idx[:, :k], -1).to(torch.int32)


def _plain_route(st):
    case = st["case"]
    z = st["z"].float()
    idx = _chosen(case, st["z"], st["b"])
    there = idx >= 0
    at = idx.clamp(min=0).long()
    if case["score"] == "sigmoid":
        p = torch.sigmoid(z)
        slope = 1.0 - p
    else:
        p = torch.exp(z - z.amax(1, keepdim=True).clamp(min=-3e38))
        p = p / p.sum(1, keepdim=True).clamp(min=1e-30)
    q = p.gather(1, at) * there
    if case["renorm"]:
        q = q / q.sum(1, keepdim=True).clamp(min=1e-30)
    pos, offsets = _places(idx, case["E"])
    out = {"idx": idx, "w": q * case["scale"], "offsets": offsets, "pos": pos}
    if case["train"]:
        d = st["dw"] * there * case["scale"]
        if case["renorm"]:
            d = q * (d - (q * d).sum(1, keepdim=True))
        else:
            d = q * d
        if case["score"] == "sigmoid":
            d = d * slope.gather(1, at)
        dz = torch.zeros_like(z).scatter_add_(1, at, d)
        if case["score"] == "softmax" and not case["renorm"]:
            dz = dz - p * d.sum(1, keepdim=True)
        out["dz"] = dz.to(st["z"].dtype)
    return out


def _plain_exchange(st):
    case, pos, dt = st["case"], st["pos"], st["x"].dtype
    T, k, D = case["T"], case["k"], case["D"]
    there = pos >= 0
    at = pos.clamp(min=0).long()
    rows = pos[there].long()
    take = lambda m: m[at].float() * there[..., None]
    spread = lambda m: torch.zeros(T * k, D, dtype=dt, device="cuda").index_copy_(0, rows, m[there])
    w = st["w"][..., None]
    y = take(st["y"])
    out = {"xs": spread(st["x"][:, None].expand(T, k, D)), "out": (w * y).sum(1).to(dt)}
    if case["train"]:
        g = st["dout"].float()[:, None]
        out["dy"] = spread((w * g).to(dt))
        out["dw"] = (g * y).sum(2)
        out["dx"] = take(st["dxs"]).sum(1).to(dt)
    return out


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
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        return _plain_route(st)
    if op == "exchange":
        return _plain_exchange(st)
    dt = st["x"].dtype
    x = _mx4_values(*_mx4_rows(st["x"].float())).flatten(1)
    if op == "mx4_quantize":
        return x[:, :case["K"]].to(dt)
    if op == "mx4":
        y = x @ _mx4_values(*_mx4_unpack(st["wc"], st["we"])).flatten(1).T
        return (y if st["b"] is None else y + st["b"].float()).to(dt)
    r = _Rows(st)
    w = _mx4_values(*_mx4_unpack(st["wc"][r.live], st["we"][r.live])).flatten(2)
    y = torch.bmm(r.gather(x), w.transpose(1, 2).contiguous())
    if st["b"] is not None:
        y = y + st["b"][r.live].float()[:, None]
    return r.scatter(y).to(dt)


# ---------------------------------------------------------------- what it takes

def work(case):
    op, size = case["op"], {"fp32": 4}.get(case["type"], 2)
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        n = T * E * size + (4 * E if case["bias"] else 0) + 12 * T * k + 4 * (E + 1)
        f = 8 * T * E
        if case["train"]:  # dw read, dz written
            n, f = n + 4 * T * k + T * E * size, 2 * f
        return {"bytes": n, "flops": f}
    if op == "exchange":
        T, k, D = case["T"], case["k"], case["D"]
        slots = (T - _padding(T)) * k
        n = 2 * slots * D * size + 2 * T * D * size + 8 * T * k
        f = 2 * slots * D
        if case["train"]:  # dout, y, dxs read; dy, dw, dx written
            n, f = n + 3 * slots * D * size + 2 * T * D * size + 4 * T * k, 6 * slots * D
        return {"bytes": n, "flops": f}
    K = case["K"]
    row = 17 * _ceil(K, 32)  # one row's codes and exponents
    if op == "mx4_quantize":
        return {"bytes": 2 * case["rows"] * K * size, "flops": 2 * case["rows"] * K}
    N, E = case["N"], case.get("experts")
    M = case["rows"] if E else case["M"]
    live = int((_shares(case) > 0).sum()) if E else 1
    return {"bytes": M * K * size + live * N * (row + (size if case["bias"] else 0))
            + M * N * size + (4 * (E + 1) if E else 0), "flops": 2 * M * N * K}


# ---------------------------------------------------------------- exact results

def _exact_choice(case, z, b):
    """The choice by sorting (score, index) pairs on the host."""
    T, E, G, m = case["T"], case["E"], case["groups"], case["group_top"]
    z = z.double().cpu().numpy()
    out = np.isneginf(z)
    with np.errstate(over="ignore", invalid="ignore"):
        if case["score"] == "sigmoid":
            p = 1.0 / (1.0 + np.exp(-z))
        else:
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
    c = p if b is None else p + b.double().cpu().numpy()
    c = np.where(out, -np.inf, c)
    by = c if b is not None else z
    if G > 1:
        n = E // G
        high = np.sort((by if m == 1 else c).reshape(T, G, n), 2)[:, :, ::-1][:, :, :m]
        score = np.where(np.isneginf(high), 0.0, high).sum(2)
        score[np.isneginf(high[:, :, 0])] = -np.inf
        first = np.lexsort((np.broadcast_to(np.arange(G), (T, G)), -score))
        lost = first[:, case["kept"]:]
        by = by.reshape(T, G, n).copy()
        np.put_along_axis(by, lost[:, :, None], -np.inf, 1)
        by = by.reshape(T, E)
    first = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -by))[:, :case["k"]]
    none = np.isneginf(np.take_along_axis(by, first, 1))
    return np.where(none, -1, first).astype(np.int32)


def _exact_places(idx, E):
    """Counting: a slot's row follows those of lower experts and of earlier
    slots of its own."""
    flat = idx.reshape(-1)
    live = np.nonzero(flat >= 0)[0]
    slots = live[np.lexsort((live, flat[live]))]
    pos = np.full(flat.size, -1, np.int32)
    pos[slots] = np.arange(slots.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[live], minlength=E))])
    return pos.reshape(idx.shape), offsets.astype(np.int32)


def _exact_route(case, st):
    """The choice, the places, and weights and gradient in logarithms."""
    z, inf = st["z"].double(), float("inf")
    chosen_by = _exact_choice(case, st["z"], st["b"])
    pos, offsets = (torch.from_numpy(v).cuda() for v in _exact_places(chosen_by, case["E"]))
    idx = torch.from_numpy(chosen_by).cuda()
    chosen = idx >= 0
    zs = z.gather(1, idx.clamp(min=0).long()).masked_fill(~chosen, -inf)
    # log of the scores
    if case["score"] == "sigmoid":
        ls = torch.nn.functional.logsigmoid(zs)
    else:
        ls = zs - torch.logsumexp(z, 1, keepdim=True)
    ls = ls.masked_fill(~chosen, -inf)
    norm = torch.logsumexp(ls, 1, keepdim=True) if case["renorm"] else torch.zeros_like(ls[:, :1])
    q = torch.exp(ls - norm).masked_fill(~chosen, 0.0)
    out = {"idx": idx, "w": q * case["scale"], "offsets": offsets, "pos": pos}
    if case["train"]:
        d = (st["dw"].double() * case["scale"]).masked_fill(~chosen, 0.0)
        dl = q * d  # with respect to the logs of the scores
        if case["renorm"]:
            dl = dl - q * dl.sum(1, keepdim=True)
        hot = torch.nn.functional.one_hot(idx.clamp(min=0).long(), case["E"]).double()
        hot = hot * chosen[..., None]
        if case["score"] == "sigmoid":
            dl = (dl * torch.sigmoid(-zs)).masked_fill(~chosen, 0.0)
            dz = (dl[..., None] * hot).sum(1)
        else:
            p = torch.softmax(z, 1).nan_to_num(0.0)
            dz = (dl[..., None] * hot).sum(1) - dl.sum(1, keepdim=True) * p
        out["dz"] = dz
    return out


def _exact_exchange(case, st):
    T, k, D = case["T"], case["k"], case["D"]
    pos = st["pos"].tolist()
    slot = torch.full((T * k,), -1, dtype=torch.int64)
    flat = torch.tensor(pos).flatten()
    slot[flat[flat >= 0].long()] = torch.arange(T * k)[flat >= 0]
    slot = slot.to("cuda")  # the slot whose row each sorted row is
    live = (slot >= 0).nonzero()[:, 0]
    token, w = slot[live] // k, st["w"].double().flatten()[slot[live]]
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")
    y = st["y"][live].double()
    out = {"xs": zeros(T * k, D).index_copy_(0, live, st["x"].double()[token]),
           "out": zeros(T, D).index_add_(0, token, w[:, None] * y)}
    if case["train"]:
        g = st["dout"].double()[token]
        out["dy"] = zeros(T * k, D).index_copy_(0, live, w[:, None] * g)
        out["dw"] = zeros(T * k).index_copy_(0, slot[live], (g * y).sum(1)).view(T, k)
        out["dx"] = zeros(T, D).index_add_(0, token, st["dxs"].double()[live])
    return out


def _nearest_exact(x):
    """x [R, K] in 64 bits: each value's nearest of the block's sixteen, by
    comparing distances (ties to the even code), and the block's power."""
    R, K = x.shape
    x = torch.nn.functional.pad(x, (0, _ceil(K, 32) * 32 - K)).view(R, -1, 32)
    _, e = torch.frexp(x.abs().amax(2))  # 2^(e - 1) <= amax < 2^e
    e = (e - 3).clamp(min=-127).masked_fill(x.abs().amax(2) == 0, -127)
    s = ((e.long() + 1023) << 52).view(torch.float64)[..., None]
    v = x.abs() / s
    best, far = torch.zeros_like(v), v.clone()
    for code, m in enumerate(_MX4[1:], 1):
        d = (v - m).abs()
        take = (d < far) | ((d == far) & (code % 2 == 0))
        best, far = torch.where(take, m, best), torch.where(take, d, far)
    return (torch.copysign(best, x) * s).flatten(1)


def _decoded_exact(codes, scales):
    """Matrix of the codes' values in 64 bits, from the fields: sign, two
    exponent bits with bias 1, one bit of significand."""
    B = codes.shape[1] // 16
    c = torch.stack([codes.long() & 15, codes.long() >> 4], -1).view(codes.shape[0], B, 32)
    ex, man = (c >> 1) & 3, c & 1
    mag = torch.where(ex == 0, man * 0.5, (2 + man) * 0.5 * (1 << ex).double() * 0.5)
    s = ((scales.permute(1, 0, 2).reshape(codes.shape[0], -1)[:, :B].long() - 127 + 1023)
         << 52).view(torch.float64)
    return (torch.where(c >= 8, -mag, mag) * s[..., None]).flatten(1)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "exchange":
        return _exact_exchange(case, st)
    x = _nearest_exact(st["x"].double())
    if op == "mx4_quantize":
        return x[:, :case["K"]]
    b = st["b"]
    if op == "mx4":
        y = x @ _decoded_exact(st["wc"], st["we"]).T
        return y if b is None else y + b.double()
    off = st["offsets"].tolist()
    y = torch.empty(case["rows"], case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        i, j = off[e], off[e + 1]
        if j > i:
            y[i:j] = x[i:j] @ _decoded_exact(st["wc"][e], st["we"][e]).T
            if b is not None:
                y[i:j] += b[e].double()
    return y
