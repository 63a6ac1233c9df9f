"""Measured cases of the gated feed-forward block and of the products with 4-bit weights.

Gated block:   G = X Ag + bg,  U = X Au + bu,  H = act(G) * U,  Y = H B,  with X [T x d], Ag, Au [d x F], B [F x d];
act is SiLU, x / (1 + exp(-x)), or the exact GeLU, x Phi(x).

4-bit weights: a matrix W [K x N] stands for (q - z) s with codes q in 0..15, one bf16 scale s and one zero point z (8
where there are none) for each group of 32, 64 or 128 rows of a column: scales and zeros [ceil(K / group) x N].  Codes
are kept in tiles of 16 columns x 64 rows, 512 bytes each, tile (n / 16, k / 64): with n % 16 = 8 (i % 2) + g and
k % 64 = 16 j + 8 (i / 2) + 2 t + h, the code is in 32-bit word 4 (4 g + t) + j of the tile, at bit 4 i + 16 h.
Columns and rows past N and K hold 8.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TINY = 2.0 ** -100                     # least range a scale is made from
BIG = torch.finfo(torch.bfloat16).max  # and the largest


def _ceil(n, m):
    return (n + m - 1) // m


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through the whole block: the weights are read once
        {"name": "ffn_token", "op": "ffn", "T": 1, "d": 4096, "F": 16384, "shards": 8, "act": "silu", "bias": False,
         "save": False},
        # a prompt of odd length through a small model whose layers have biases
        {"name": "ffn_prompt_odd", "op": "ffn", "T": 1037, "d": 1024, "F": 4096, "shards": 8, "act": "gelu",
         "bias": True, "save": False},
        # the forward of a training step, which keeps both pre-activations
        {"name": "ffn_train", "op": "ffn", "T": 8192, "d": 4096, "F": 16384, "shards": 8, "act": "silu", "bias": False,
         "save": True},
        # gradients of a small batch, biases among them
        {"name": "ffn_bwd_small", "op": "ffn_bwd", "T": 320, "d": 1024, "F": 4096, "shards": 4, "act": "gelu",
         "bias": True},
        # the backward of the training step
        {"name": "ffn_bwd_train", "op": "ffn_bwd", "T": 8192, "d": 4096, "F": 16384, "shards": 8, "act": "silu",
         "bias": False},
        # one decoded token: the column-parallel product, and the row-parallel one with zero points and a bias
        {"name": "w4_token", "op": "w4", "M": 1, "K": 4096, "N": 16384, "group": 128, "zeros": False, "bias": False},
        {"name": "w4_token_zeros", "op": "w4", "M": 1, "K": 16384, "N": 4096, "group": 64, "zeros": True, "bias": True},
        # a batch of decoded tokens
        {"name": "w4_batch", "op": "w4", "M": 37, "K": 4096, "N": 16384, "group": 128, "zeros": True, "bias": False},
        # gate and up projections of one decoded token, and of a few in a small model with the finest groups
        {"name": "w4_gated_token", "op": "w4_gated", "M": 1, "K": 4096, "N": 16384, "group": 128, "zeros": False,
         "act": "silu", "bias": False},
        {"name": "w4_gated_batch", "op": "w4_gated", "M": 5, "K": 1024, "N": 4096, "group": 32, "zeros": True,
         "act": "gelu", "bias": True},
        # a layer's weights brought to 4 bits and read back for a prompt's bf16 product
        {"name": "w4_pack", "op": "w4_pack", "K": 4096, "N": 16384, "group": 128, "zeros": False},
        # the same with zero points, a ragged last group, last tile and last column
        {"name": "w4_pack_odd", "op": "w4_pack", "K": 1048, "N": 4104, "group": 32, "zeros": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    return max(step, min(hi, _log(rng, lo, hi) // step * step))


def draw(rng):
    op = rng.choice(["ffn", "ffn_bwd", "w4", "w4", "w4_gated", "w4_pack"])
    act, bias = rng.choice(["silu", "gelu"]), rng.random() < 0.5
    if op in ("ffn", "ffn_bwd"):
        shards = rng.choice([1, 2, 4, 8])
        d, F = _size(rng, 64, 8192, 8), _size(rng, 64, 16384, 8 * shards)
        T = _log(rng, 1, max(1, min(8192, 8192 * 4096 * 16384 // (d * F))))
        c = {"op": op, "T": T, "d": d, "F": F, "shards": shards, "act": act, "bias": bias}
        if op == "ffn":
            c["save"] = rng.random() < 0.5
        return c
    K, N = _size(rng, 64, 16384, 8), _size(rng, 64, 16384, 8)
    if K * N > 4096 * 16384:
        K = 4096 * 16384 // N // 8 * 8
    c = {"op": op, "K": K, "N": N, "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5}
    if op != "w4_pack":
        c.update(M=_log(rng, 1, 256), bias=bias)
        if op == "w4_gated":
            c["act"] = act
    return c


def work(case):
    op = case["op"]
    if op == "ffn":
        T, d, F = case["T"], case["d"], case["F"]
        values = 2 * T * d + 3 * d * F + (2 * T * F if case["save"] else 0) + (2 * F if case["bias"] else 0)
        return {"bytes": 2 * values, "flops": 6 * T * d * F}
    if op == "ffn_bwd":
        T, d, F = case["T"], case["d"], case["F"]
        # X, dY, both pre-activations and the weights; dX and the weights' gradients
        values = 3 * T * d + 2 * T * F + 6 * d * F + (2 * F if case["bias"] else 0)
        return {"bytes": 2 * values, "flops": 12 * T * d * F}
    K, N = case["K"], case["N"]
    packed = K * N / 2 + _ceil(K, case["group"]) * N * (3 if case["zeros"] else 2)
    if op == "w4_pack":
        return {"bytes": 2 * K * N + packed + packed + 2 * K * N, "flops": 6 * K * N}
    n = 2 if op == "w4_gated" else 1
    M = case["M"]
    return {"bytes": n * packed + 2 * M * (K + N) + (2 * n * N if case["bias"] else 0), "flops": 2 * n * M * K * N}


# ----------------------------------------------------------------------------- inputs

def _codes(W, group, with_zeros):
    """(codes 0..15, scales, zero points or None) of W [K x N]: the definition, in 32 bits."""
    K, N = W.shape
    G = _ceil(K, group)
    full = torch.zeros(G * group, N, dtype=F32, device=W.device)
    full[:K] = torch.nan_to_num(W.to(F32), nan=0.0, posinf=math.inf, neginf=-math.inf)
    b = full.view(G, group, N)
    if with_zeros:
        lo, hi = b.amin(dim=1).clamp_max(0), b.amax(dim=1).clamp_min(0)
        span, steps = hi - lo, 15.0
    else:
        span, steps = b.abs().amax(dim=1), 7.0
    span = span.clamp(TINY, BIG)
    s = (span / torch.full_like(span, steps)).to(BF16)
    zero = (-lo / s.to(F32)).round().clamp(0, 15) if with_zeros else torch.full_like(span, 8)
    q = ((b / s.to(F32)[:, None]).clamp(-16, 16).round() + zero[:, None]).clamp(0, 15)
    return q.view(G * group, N)[:K].to(torch.uint8), s, zero.to(torch.uint8) if with_zeros else None


def _packed(q):
    """Codes [K x N] in tiles."""
    K, N = q.shape
    nt, kc = _ceil(N, 16), _ceil(K, 64)
    full = torch.full((kc * 64, nt * 16), 8, dtype=torch.int32, device=q.device)
    full[:K, :N] = q
    v = full.view(kc, 4, 2, 4, 2, nt, 2, 8)                  # k: j, i / 2, t, h; n: i % 2, g
    v = v.permute(5, 0, 7, 3, 1, 4, 2, 6).reshape(nt, kc, 8, 4, 4, 8)  # tile, g, t, j, then bits 4 i + 16 h
    shift = 4 * torch.arange(8, dtype=torch.int32, device=q.device)
    words = torch.zeros(v.shape[:-1], dtype=torch.int32, device=q.device)
    for b in range(8):
        words |= v[..., b] << shift[b]
    return words.view(nt, kc, 128).view(torch.uint8)


def _unpacked(Q, K, N):
    """Codes [K x N] as fp32 of a packed matrix."""
    nt, kc = Q.shape[:2]
    words = Q.view(torch.int32).view(nt, kc, 8, 4, 4, 1)
    v = (words >> (4 * torch.arange(8, dtype=torch.int32, device=Q.device))) & 15
    v = v.view(nt, kc, 8, 4, 4, 2, 2, 2).permute(1, 4, 6, 3, 5, 0, 7, 2)
    return v.reshape(kc * 64, nt * 16)[:K, :N].to(F32)


def _activations(g, rows, cols):
    """Normal values of unit scale, some channels up to eight times the others."""
    x = torch.randn(rows, cols, generator=g, device=g.device)
    return (x * torch.exp2(3 * torch.rand(cols, generator=g, device=g.device) ** 4)).to(BF16)


def _weights(g, rows, cols):
    """Normal values that keep a product's size; columns differ by up to a factor of four."""
    w = torch.randn(rows, cols, generator=g, device=g.device) * rows ** -0.5
    return (w * torch.exp2(2 * torch.rand(cols, generator=g, device=g.device) - 1)).to(BF16)


def _bias(g, n):
    return (0.1 * torch.randn(n, generator=g, device=g.device)).to(BF16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, op = g.device, case["op"]
    s = {"case": case}

    def empty(*shape, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device=dev)

    if op in ("ffn", "ffn_bwd"):
        T, d, F = case["T"], case["d"], case["F"]
        s["X"], s["Ag"], s["Au"], s["B"] = _activations(g, T, d), _weights(g, d, F), _weights(g, d, F), _weights(g, F, d)
        s["bg"], s["bu"] = (_bias(g, F), _bias(g, F)) if case["bias"] else (None, None)
        if op == "ffn":
            s["Y"] = empty(T, d)
            s["G"], s["U"] = (empty(T, F), empty(T, F)) if case["save"] else (None, None)
            return s
        # what the forward kept: pre-activations of unit size
        s["G"], s["U"] = (torch.randn(T, F, generator=g, device=dev).to(BF16) for _ in range(2))
        dy = 1e-3 * torch.randn(T, d, generator=g, device=dev)
        s["dY"] = (dy * torch.exp2(-6 * torch.rand(T, 1, generator=g, device=dev))).to(BF16)
        s["dX"], s["dAg"], s["dAu"], s["dB"] = empty(T, d), empty(d, F), empty(d, F), empty(F, d)
        s["dbg"], s["dbu"] = (empty(F), empty(F)) if case["bias"] else (None, None)
        return s
    K, N, group = case["K"], case["N"], case["group"]
    if op == "w4_pack":
        s["W"] = _weights(g, K, N)
        s["Q"] = empty(_ceil(N, 16), _ceil(K, 64), 512, dtype=torch.uint8)
        s["scales"] = empty(_ceil(K, group), N)
        s["zeros"] = empty(_ceil(K, group), N, dtype=torch.uint8) if case["zeros"] else None
        s["back"] = empty(K, N)
        return s
    s["X"] = _activations(g, case["M"], K)
    s["mats"] = []
    for _ in range(2 if op == "w4_gated" else 1):
        q, scales, zeros = _codes(_weights(g, K, N), group, case["zeros"])
        s["mats"].append({"Q": _packed(q), "scales": scales, "zeros": zeros,
                          "bias": _bias(g, N) if case["bias"] else None})
    s["Y"] = empty(case["M"], N)
    return s


# ----------------------------------------------------------------------------- plain forms

def _act(x, act):
    return x / (1 + torch.exp(-x)) if act == "silu" else 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))


def _act_grad(x, act):
    if act == "silu":
        sig = 1 / (1 + torch.exp(-x))
        return sig * (1 + x * (1 - sig))
    return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)


def _matrix(m, K, N, group):
    """fp32 values of a 4-bit matrix."""
    q = _unpacked(m["Q"], K, N)
    if m["zeros"] is None:
        q = q - 8
    else:
        q = q - m["zeros"].to(F32).repeat_interleave(group, 0)[:K]
    return q * m["scales"].to(F32).repeat_interleave(group, 0)[:K]


def _product(x, m, K, N, group):
    y = x @ _matrix(m, K, N, group)
    return y if m["bias"] is None else y + m["bias"].to(F32)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "ffn":
        x = s["X"].to(F32)
        G, U = x @ s["Ag"].to(F32), x @ s["Au"].to(F32)
        if case["bias"]:
            G, U = G + s["bg"].to(F32), U + s["bu"].to(F32)
        out = {"Y": ((_act(G, case["act"]) * U) @ s["B"].to(F32)).to(BF16)}
        if case["save"]:
            out["G"], out["U"] = G.to(BF16), U.to(BF16)
        return out
    if op == "ffn_bwd":
        x, dy, G, U = (s[k].to(F32) for k in ("X", "dY", "G", "U"))
        Ag, Au, B = (s[k].to(F32) for k in ("Ag", "Au", "B"))
        a = _act(G, case["act"])
        dH = dy @ B.t()
        dG, dU = dH * U * _act_grad(G, case["act"]), dH * a
        out = {"dX": dG @ Ag.t() + dU @ Au.t(), "dAg": x.t() @ dG, "dAu": x.t() @ dU, "dB": (a * U).t() @ dy}
        if case["bias"]:
            out["dbg"], out["dbu"] = dG.sum(dim=0), dU.sum(dim=0)
        return {k: v.to(BF16) for k, v in out.items()}
    K, N, group = case["K"], case["N"], case["group"]
    if op == "w4_pack":
        q, scales, zeros = _codes(s["W"], group, case["zeros"])
        m = {"Q": _packed(q), "scales": scales, "zeros": zeros}
        out = {"scales": scales, "values": _matrix(m, K, N, group).to(BF16)}
        if case["zeros"]:
            out["zeros"] = zeros
        return out
    x = s["X"].to(F32)
    y = _product(x, s["mats"][0], K, N, group)
    if op == "w4_gated":
        y = _act(y, case["act"]) * _product(x, s["mats"][1], K, N, group)
    return {"Y": y.to(BF16)}


# ----------------------------------------------------------------------------- the framework's calls

def _own(s):
    from tensor_transformer_mlp_tp_gb300 import binding

    case = s["case"]
    op = case["op"]
    act = (binding.ACT_SILU if case["act"] == "silu" else binding.ACT_GELU) if "act" in case else None
    if op == "ffn":
        binding.tpmlp_gated_forward(s["X"], s["Ag"], s["Au"], s["B"], case["shards"], s["Y"], act=act, bg=s["bg"],
                                    bu=s["bu"], Gpre_out=s["G"], Upre_out=s["U"])
        out = {"Y": s["Y"]}
        if case["save"]:
            out["G"], out["U"] = s["G"], s["U"]
        return out
    if op == "ffn_bwd":
        binding.tpmlp_gated_backward(s["X"], s["Ag"], s["Au"], s["B"], s["G"], s["U"], s["dY"], case["shards"],
                                     s["dX"], s["dAg"], s["dAu"], s["dB"], act=act, dbg=s["dbg"], dbu=s["dbu"])
        return {k: s[k] for k in ("dX", "dAg", "dAu", "dB") + (("dbg", "dbu") if case["bias"] else ())}
    group = case["group"]
    if op == "w4_pack":
        binding.tpmlp_quantize_w4(s["W"], group, s["Q"], s["scales"], zeros=s["zeros"])
        binding.tpmlp_dequantize_w4(s["Q"], s["scales"], group, s["back"], zeros=s["zeros"])
        out = {"scales": s["scales"], "values": s["back"]}
        if case["zeros"]:
            out["zeros"] = s["zeros"]
        return out
    m = s["mats"][0]
    if op == "w4":
        binding.tpmlp_gemm_w4(s["X"], m["Q"], m["scales"], group, s["Y"], zeros=m["zeros"], bias=m["bias"])
    else:
        u = s["mats"][1]
        binding.tpmlp_gemm1_gated_w4(s["X"], m["Q"], m["scales"], u["Q"], u["scales"], group, s["Y"], act=act,
                                     g_zeros=m["zeros"], u_zeros=u["zeros"], bg=m["bias"], bu=u["bias"])
    return {"Y": s["Y"]}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- 64-bit values

def _gate64(x, act):
    """(act(x), act'(x)) in 64 bits."""
    if act == "silu":
        sig = torch.sigmoid(x)
        return x * sig, sig + x * sig * torch.sigmoid(-x)
    cdf = torch.special.ndtr(x)
    return x * cdf, cdf + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)


def _code_at(Q, k, n):
    """Codes at rows k and columns n (broadcast), from the place the layout gives each of them."""
    i = (n % 16) // 8 + 2 * ((k % 16) // 8)
    word = 4 * (4 * (n % 8) + (k % 8) // 2) + (k % 64) // 16
    at = ((n // 16) * Q.shape[1] + k // 64) * 128 + word
    return (Q.view(torch.int32).flatten()[at] >> (4 * i + 16 * (k % 2))) & 15


def _matrix64(m, K, N, group):
    dev = m["Q"].device
    out = torch.empty(K, N, dtype=F64, device=dev)
    n = torch.arange(N, device=dev)
    for k0 in range(0, K, group):
        k = torch.arange(k0, min(K, k0 + group), device=dev)
        zero = 8.0 if m["zeros"] is None else m["zeros"][k0 // group].to(F64)
        out[k] = (_code_at(m["Q"], k[:, None], n[None, :]).to(F64) - zero) * m["scales"][k0 // group].to(F64)
    return out


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "ffn":
        x = s["X"].to(F64)
        G, U = torch.matmul(x, s["Ag"].to(F64)), torch.matmul(x, s["Au"].to(F64))
        if case["bias"]:
            G += s["bg"].to(F64)
            U += s["bu"].to(F64)
        out = {"Y": torch.matmul(_gate64(G, case["act"])[0] * U, s["B"].to(F64))}
        if case["save"]:
            out["G"], out["U"] = G, U
        return out
    if op == "ffn_bwd":
        x, dy, G, U, Ag, Au, B = (s[k].to(F64) for k in ("X", "dY", "G", "U", "Ag", "Au", "B"))
        a, slope = _gate64(G, case["act"])
        dH = torch.einsum("td,fd->tf", dy, B)
        dU = dH * a
        dG = dH * U * slope
        out = {"dX": torch.einsum("tf,df->td", dG, Ag) + torch.einsum("tf,df->td", dU, Au),
               "dAg": torch.einsum("td,tf->df", x, dG), "dAu": torch.einsum("td,tf->df", x, dU),
               "dB": torch.einsum("tf,td->fd", a * U, dy)}
        if case["bias"]:
            out["dbg"], out["dbu"] = dG.sum(dim=0), dU.sum(dim=0)
        return out
    K, N, group = case["K"], case["N"], case["group"]
    if op == "w4_pack":
        W = s["W"].to(F64)
        scales, zeros, values = [], [], torch.empty_like(W)
        for k0 in range(0, K, group):
            part = W[k0:k0 + group]
            low = torch.minimum(part.min(dim=0).values, torch.zeros(N, dtype=F64, device=W.device))
            high = torch.maximum(part.max(dim=0).values, torch.zeros(N, dtype=F64, device=W.device))
            span = (high - low) / 15 if case["zeros"] else torch.maximum(high, -low) / 7
            span = torch.clamp(span, min=TINY / (15 if case["zeros"] else 7))
            step = span.to(BF16).to(F64)  # codes are taken with the scale that is kept
            z = torch.clamp(torch.round(-low / step), 0, 15) if case["zeros"] else torch.full_like(step, 8)
            q = torch.clamp(torch.round(part / step) + z, 0, 15)
            values[k0:k0 + group] = (q - z) * step
            scales.append(span)
            zeros.append(z)
        out = {"scales": torch.stack(scales), "values": values}
        if case["zeros"]:
            out["zeros"] = torch.stack(zeros).to(torch.uint8)
        return out
    x, y = s["X"].to(F64), []
    for m in s["mats"]:
        y.append(torch.matmul(x, _matrix64(m, K, N, group)))
        if m["bias"] is not None:
            y[-1] += m["bias"].to(F64)
    return {"Y": y[0] if op == "w4" else _gate64(y[0], case["act"])[0] * y[1]}
