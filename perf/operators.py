"""Measured cases of the block-scaled FP8 operators: the residual RMS norm with an 8-bit output and its backward, the
block quantiser, and the matrix products of 8-bit operands that carry one scale for each block of 128.

Conventions shared by all of them:
  - an 8-bit operand Q [R x K] (row-major bytes, E4M3 or E5M2) stands for Q * scale, one fp32 scale for each block of
    128 along K: either for every row (scales [ceil(K / 128) x R_pad], k-block major, R_pad = 128 ceil(R / 128)) or for
    tiles of 128 rows x 128 columns (scales [ceil(R / 128) x ceil(K / 128)]);
  - scale = max(amax, 2^-100) / 448 (E4M3) or / 57344 (E5M2), amax the block's largest magnitude.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
FMAX = {E4M3: 448.0, E5M2: 57344.0}
BLOCK = 128
TINY = 2.0 ** -100  # least amax a scale is made from
EPS = 1e-5


def _up(n, m):
    return (n + m - 1) // m * m


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through the norm before the MLP: latency alone
        {"name": "norm_token", "op": "norm", "T": 1, "d": 4096, "chunks": 1, "bf16": False, "q": True},
        # a prompt of odd length through a small model, bf16 kept beside the 8-bit output
        {"name": "norm_prompt_odd", "op": "norm", "T": 1037, "d": 1024, "chunks": 1, "bf16": True, "q": True},
        # the sequence-parallel region's norm over eight chunks, as a training step runs it
        {"name": "norm_seqpar", "op": "norm", "T": 8192, "d": 4096, "chunks": 8, "bf16": False, "q": True},
        # the norm's backward on a small batch, and on the training step's
        {"name": "norm_bwd_small", "op": "norm_bwd", "T": 320, "d": 1024, "chunks": 4},
        {"name": "norm_bwd_seqpar", "op": "norm_bwd", "T": 8192, "d": 4096, "chunks": 8},
        # a weight matrix to 128 x 128 tiles in both orientations, once an optimizer step
        {"name": "quant_weight", "op": "quant", "rows": 4096, "cols": 16384, "tile": True, "fmt": "e4m3"},
        # gradients of an odd number of tokens to E5M2: rows for the input gradient, transposed for the weights'
        {"name": "quant_grad_odd", "op": "quant", "rows": 1037, "cols": 4096, "tile": False, "fmt": "e5m2"},
        # one decoded token through the row-parallel layer
        {"name": "gemm_token", "op": "gemm", "M": 1, "N": 4096, "K": 16384, "b_tile": True, "bias": True,
         "a_fmt": "e4m3", "b_fmt": "e4m3", "f32": False},
        # the row-parallel layer of the training step
        {"name": "gemm_forward", "op": "gemm", "M": 8192, "N": 4096, "K": 16384, "b_tile": True, "bias": False,
         "a_fmt": "e4m3", "b_fmt": "e4m3", "f32": False},
        # the column-parallel layer's weight gradient: K runs over the tokens, both operands scaled by rows
        {"name": "gemm_wgrad", "op": "gemm", "M": 4096, "N": 16384, "K": 8192, "b_tile": False, "bias": False,
         "a_fmt": "e4m3", "b_fmt": "e5m2", "f32": True},
        # the column-parallel layer with bias, GeLU and its 8-bit output: a batch of decoded tokens, and a prompt
        {"name": "gemm1_batch", "op": "gemm1", "T": 37, "d": 4096, "F": 16384, "pre": False},
        {"name": "gemm1_prompt", "op": "gemm1", "T": 4096, "d": 4096, "F": 16384, "pre": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    return max(lo, min(hi, _log(rng, lo, hi) // step * step))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quant", "gemm", "gemm1"])
    if op in ("norm", "norm_bwd"):
        d = _size(rng, 64, 8192, 16)
        chunks = rng.choice([1, 1, 2, 4, 8])
        T = _log(rng, 1, max(1, 8192 * 4096 // d // chunks // 2)) * chunks
        c = {"op": op, "T": T, "d": d, "chunks": chunks}
        if op == "norm":
            c["bf16"] = rng.random() < 0.5
            c["q"] = not c["bf16"] or rng.random() < 0.5
        return c
    if op == "quant":
        cols = _size(rng, 64, 16384, 16)
        rows = _log(rng, 1, 8192 * 8192 // cols // 2 if cols > 4096 else 8192)
        return {"op": op, "rows": rows, "cols": cols, "tile": rng.random() < 0.4, "fmt": rng.choice(["e4m3", "e5m2"])}
    if op == "gemm":
        a, b = rng.choice([("e4m3", "e4m3"), ("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")])
        return {"op": op, "M": _log(rng, 1, 8192), "N": _size(rng, 64, 8192, 8), "K": _size(rng, 64, 8192, 16),
                "b_tile": rng.random() < 0.6, "bias": rng.random() < 0.5, "a_fmt": a, "b_fmt": b,
                "f32": rng.random() < 0.4}
    return {"op": op, "T": _log(rng, 1, 4096), "d": _size(rng, 64, 8192, 16), "F": _size(rng, 64, 16384, 16),
            "pre": rng.random() < 0.5}


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["d"]  # x, the residual and the sum in bf16, then the outputs
        out = (2 if case["bf16"] else 0) + (1 + 4 / BLOCK if case["q"] else 0)
        return {"bytes": n * (6 + out) + 2 * case["d"], "flops": 8 * n}
    if op == "norm_bwd":
        n = case["T"] * case["d"]  # the sum, dXg, the residual's gradient; dX
        return {"bytes": 8 * n + 6 * case["d"], "flops": 12 * n}
    if op == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 + 2 + (8 / BLOCK ** 2 if case["tile"] else 8 / BLOCK)), "flops": 4 * n}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        scales = 4 * -(-K // BLOCK) * (M + (-(-N // BLOCK) if case["b_tile"] else N))
        return {"bytes": M * K + N * K + M * N * (4 if case["f32"] else 2) + scales, "flops": 2 * M * N * K}
    T, d, F = case["T"], case["d"], case["F"]
    return {"bytes": T * d + d * F + T * F * (3 if case["pre"] else 1) + 4 * T * (d + F) / BLOCK,
            "flops": 2 * T * d * F}


# ----------------------------------------------------------------------------- inputs

def _fmt(name):
    return E4M3 if name == "e4m3" else E5M2


def _quantized(x, tile, fmt):
    """(codes, scales) of a bf16 matrix, in the layouts described at the top."""
    R, K = x.shape
    Rp, Kp = _up(R, BLOCK), _up(K, BLOCK)
    full = torch.zeros(Rp, Kp, dtype=F32, device=x.device)
    full[:R, :K] = x
    b = full.view(Rp // BLOCK, BLOCK, Kp // BLOCK, BLOCK)
    if tile:
        scale = b.abs().amax(dim=(1, 3), keepdim=True).clamp_min(TINY) / FMAX[fmt]
        scales = scale.reshape(Rp // BLOCK, Kp // BLOCK)
    else:
        scale = b.abs().amax(dim=3, keepdim=True).clamp_min(TINY) / FMAX[fmt]
        scales = scale.reshape(Rp, Kp // BLOCK).t().contiguous()
    q = (b / scale).clamp(-FMAX[fmt], FMAX[fmt]).reshape(Rp, Kp)[:R, :K].contiguous().to(fmt)
    return q, scales


def _activations(g, rows, cols):
    """Normal values of unit scale, some channels up to eight times the others."""
    dev = g.device
    x = torch.randn(rows, cols, generator=g, device=dev)
    x *= torch.exp2(3 * torch.rand(cols, generator=g, device=dev) ** 4)
    return x.to(BF16)


def _weights(g, rows, cols):
    return (0.02 * torch.randn(rows, cols, generator=g, device=g.device)).to(BF16)


def _gradients(g, rows, cols):
    """Small values whose size varies from token to token over three decades."""
    dev = g.device
    x = 1e-4 * torch.randn(rows, cols, generator=g, device=dev)
    return (x * torch.exp2(-10 * torch.rand(rows, 1, generator=g, device=dev))).to(BF16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, op = g.device, case["op"]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        T, d, n = case["T"], case["d"], case["chunks"]
        rows = T // n
        s["weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(BF16)
        s["x"] = list(_activations(g, T, d).split(rows))
        if op == "norm":
            s["r"] = list((2 * torch.randn(T, d, generator=g, device=dev)).to(BF16).split(rows))
            s["sum"] = torch.empty(T, d, dtype=BF16, device=dev)
            s["sums"] = list(s["sum"].split(rows))
            s["xg"] = torch.empty(T, d, dtype=BF16, device=dev) if case["bf16"] else None
            s["xq"] = torch.empty(T, d, dtype=torch.uint8, device=dev).view(E4M3) if case["q"] else None
            s["scales"] = torch.empty(-(-d // BLOCK), _up(T, BLOCK), dtype=F32, device=dev) if case["q"] else None
        else:
            s["dy"] = _gradients(g, T, d)
            s["ds"] = list(_gradients(g, T, d).split(rows))
            s["dx"] = torch.empty(T, d, dtype=BF16, device=dev)
            s["dxs"] = list(s["dx"].split(rows))
            s["dw"] = torch.empty(d, dtype=F32, device=dev)
        return s
    if op == "quant":
        R, C, f = case["rows"], case["cols"], _fmt(case["fmt"])
        s["src"] = _weights(g, R, C) if case["tile"] else _gradients(g, R, C) if f == E5M2 else _activations(g, R, C)
        s["q"] = torch.empty(R, C, dtype=torch.uint8, device=dev).view(f)
        s["qt"] = torch.empty(C, _up(R, 16), dtype=torch.uint8, device=dev).view(f)
        shape = (lambda r, c: (-(-r // BLOCK), -(-c // BLOCK))) if case["tile"] else \
            (lambda r, c: (-(-c // BLOCK), _up(r, BLOCK)))
        s["scales"] = torch.empty(shape(R, C), dtype=F32, device=dev)
        s["scales_t"] = torch.empty(shape(C, R), dtype=F32, device=dev)
        return s
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        make = {"e4m3": _activations, "e5m2": _gradients}
        s["a"], s["a_scales"] = _quantized(make[case["a_fmt"]](g, M, K), False, _fmt(case["a_fmt"]))
        b = _weights(g, N, K) if case["b_tile"] else make[case["b_fmt"]](g, N, K)
        s["b"], s["b_scales"] = _quantized(b, case["b_tile"], _fmt(case["b_fmt"]))
        s["bias"] = _weights(g, 1, N).view(N) if case["bias"] else None
        s["c"] = torch.empty(M, N, dtype=F32 if case["f32"] else BF16, device=dev)
        return s
    T, d, F = case["T"], case["d"], case["F"]
    s["x"], s["x_scales"] = _quantized(_activations(g, T, d), False, E4M3)
    s["a"], s["a_scales"] = _quantized(_weights(g, F, d), True, E4M3)
    s["bias"] = _weights(g, 1, F).view(F)
    s["hq"] = torch.empty(T, F, dtype=torch.uint8, device=dev).view(E4M3)
    s["h_scales"] = torch.empty(-(-F // BLOCK), _up(T, BLOCK), dtype=F32, device=dev)
    s["pre"] = torch.empty(T, F, dtype=BF16, device=dev) if case["pre"] else None
    return s


# ----------------------------------------------------------------------------- plain forms

def _blocks(y, fmt):
    """8-bit codes of the rows of y (fp32) and their scales [blocks x rows]."""
    R, K = y.shape
    b = torch.nn.functional.pad(y, (0, _up(K, BLOCK) - K)).view(R, -1, BLOCK)
    scale = b.abs().amax(dim=2, keepdim=True).clamp_min(TINY) / FMAX[fmt]
    q = (b / scale).clamp(-FMAX[fmt], FMAX[fmt]).view(R, -1)[:, :K].to(fmt)
    return q, scale.squeeze(2).t()


def _dequantized(q, scales, tile):
    """fp32 values of 8-bit codes."""
    R, K = q.shape
    v = q.to(F32)
    if tile:
        s = scales.repeat_interleave(BLOCK, 0)[:R]
    else:
        s = scales[:, :R].t()
    return v * s.repeat_interleave(BLOCK, 1)[:, :K]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        total = (torch.cat(s["x"]).to(F32) + torch.cat(s["r"]).to(F32)).to(BF16)
        t = total.to(F32)
        y = t * torch.rsqrt((t * t).mean(dim=1, keepdim=True) + EPS) * s["weight"].to(F32)
        out = {"sum": total}
        if case["bf16"]:
            out["xg"] = y.to(BF16)
        if case["q"]:
            out["xq"], out["scales"] = _blocks(y, E4M3)
        return out
    if op == "norm_bwd":
        x, dy = torch.cat(s["x"]).to(F32), s["dy"].to(F32)
        rstd = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)
        xhat, g = x * rstd, dy * s["weight"].to(F32)
        dx = rstd * (g - xhat * (g * xhat).mean(dim=1, keepdim=True)) + torch.cat(s["ds"]).to(F32)
        return {"dx": dx.to(BF16), "dweight": (dy * xhat).sum(dim=0)}
    if op == "quant":
        R, C, f = case["rows"], case["cols"], _fmt(case["fmt"])
        x = s["src"].to(F32)
        xt = torch.nn.functional.pad(x.t(), (0, _up(R, 16) - R))
        if not case["tile"]:
            q, scales = _blocks(x, f)
            qt, scales_t = _blocks(xt, f)
            return {"q": q, "scales": scales, "qt": qt, "scales_t": scales_t}
        b = torch.nn.functional.pad(x, (0, _up(C, BLOCK) - C, 0, _up(R, BLOCK) - R)).abs()
        scales = b.view(-1, BLOCK, b.shape[1] // BLOCK, BLOCK).amax(dim=(1, 3)).clamp_min(TINY) / FMAX[f]
        each = scales.repeat_interleave(BLOCK, 0)[:R].repeat_interleave(BLOCK, 1)[:, :C]
        q = (x / each).clamp(-FMAX[f], FMAX[f])
        qt = torch.nn.functional.pad(q.t(), (0, _up(R, 16) - R)).to(f)
        return {"q": q.to(f), "scales": scales, "qt": qt, "scales_t": scales.t()}
    if op == "gemm":
        c = _dequantized(s["a"], s["a_scales"], False) @ _dequantized(s["b"], s["b_scales"], case["b_tile"]).t()
        if s["bias"] is not None:
            c = c + s["bias"].to(F32)
        return {"c": c if case["f32"] else c.to(BF16)}
    p = _dequantized(s["x"], s["x_scales"], False) @ _dequantized(s["a"], s["a_scales"], True).t() + s["bias"].to(F32)
    hq, scales = _blocks(0.5 * p * (1 + torch.erf(p * math.sqrt(0.5))), E4M3)
    out = {"hq": hq, "scales": scales}
    if case["pre"]:
        out["pre"] = p.to(BF16)
    return out


# ----------------------------------------------------------------------------- the framework's calls

def _own(s):
    from tensor_transformer_mlp_tp_gb300 import binding

    case = s["case"]
    op = case["op"]
    if op == "norm":
        T = case["T"]
        binding.tpmlp_rmsnorm_add_gather(s["x"], s["weight"], case["chunks"], R_chunks=s["r"], S_chunks=s["sums"],
                                         Xg=s["xg"], Xq=s["xq"], x_scales=s["scales"], eps=EPS)
        out = {"sum": s["sum"]}
        if case["bf16"]:
            out["xg"] = s["xg"]
        if case["q"]:
            out["xq"], out["scales"] = s["xq"], s["scales"][:, :T]
        return out
    if op == "norm_bwd":
        binding.tpmlp_rmsnorm_add_backward(s["x"], s["weight"], s["dy"], case["chunks"], s["dxs"], s["dw"],
                                           dS_chunks=s["ds"], eps=EPS)
        return {"dx": s["dx"], "dweight": s["dw"]}
    if op == "quant":
        fmt = binding.E4M3 if case["fmt"] == "e4m3" else binding.E5M2
        binding.tpmlp_quantize_block(s["src"], BLOCK if case["tile"] else 1, fmt, q=s["q"], scales=s["scales"],
                                     qT=s["qt"], scalesT=s["scales_t"])
        if case["tile"]:
            return {"q": s["q"], "scales": s["scales"], "qt": s["qt"], "scales_t": s["scales_t"]}
        return {"q": s["q"], "scales": s["scales"][:, :case["rows"]], "qt": s["qt"],
                "scales_t": s["scales_t"][:, :case["cols"]]}
    if op == "gemm":
        a_fmt = binding.E4M3 if case["a_fmt"] == "e4m3" else binding.E5M2
        b_fmt = binding.E4M3 if case["b_fmt"] == "e4m3" else binding.E5M2
        binding.tpmlp_gemm_fp8_block(s["a"], s["a_scales"], s["b"], s["b_scales"], s["c"], bias=s["bias"],
                                     b_block_rows=BLOCK if case["b_tile"] else 1, a_fmt=a_fmt, b_fmt=b_fmt)
        return {"c": s["c"]}
    binding.tpmlp_gemm1_fp8_block(s["x"], s["x_scales"], s["a"], s["a_scales"], s["bias"], 1, s["hq"], s["h_scales"],
                                  Hpre=s["pre"])
    out = {"hq": s["hq"], "scales": s["h_scales"][:, :case["T"]]}
    if case["pre"]:
        out["pre"] = s["pre"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- 64-bit values

def _scaled64(y, fmt):
    """The rows of y (fp64) divided by their blocks' scales, before any rounding, and the scales [blocks x rows]."""
    R, K = y.shape
    out, scales = torch.empty_like(y), []
    for k in range(0, K, BLOCK):
        part = y[:, k:k + BLOCK]
        sc = torch.clamp(part.abs().max(dim=1).values, min=TINY) / FMAX[fmt]
        out[:, k:k + BLOCK] = part / sc[:, None]
        scales.append(sc)
    return out, torch.stack(scales)


def _codes64(out, fmt):
    """Two mantissa bits put an E5M2 code five per cent from the number it stands for, as far as a wrong one may be:
    such codes have no 64-bit value that would tell one from the other, and are compared with the plain form's alone."""
    if fmt == E5M2:
        out["q"] = out["qt"] = None
    return out


def _value64(q, scales, tile):
    v = q.to(F64)
    for j in range(-(-q.shape[1] // BLOCK)):
        cut = slice(j * BLOCK, (j + 1) * BLOCK)
        if tile:
            for i in range(-(-q.shape[0] // BLOCK)):
                v[i * BLOCK:(i + 1) * BLOCK, cut] *= scales[i, j].to(F64)
        else:
            v[:, cut] *= scales[j, :q.shape[0], None].to(F64)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        total = torch.cat([a.to(F64) + b.to(F64) for a, b in zip(s["x"], s["r"])])
        t = total.to(BF16).to(F64)  # the norm reads the stored sum
        y = t / torch.sqrt(t.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS) * s["weight"].to(F64)
        out = {"sum": total}
        if case["bf16"]:
            out["xg"] = y
        if case["q"]:
            out["xq"], out["scales"] = _scaled64(y, E4M3)
        return out
    if op == "norm_bwd":
        x, dy, w = torch.cat(s["x"]).to(F64), s["dy"].to(F64), s["weight"].to(F64)
        root = torch.sqrt(x.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS)
        inner = (dy * w * x).sum(dim=1, keepdim=True)
        dx = dy * w / root - x * inner / (case["d"] * root.pow(3)) + torch.cat(s["ds"]).to(F64)
        return {"dx": dx, "dweight": (dy * x / root).sum(dim=0)}
    if op == "quant":
        R, C, f = case["rows"], case["cols"], _fmt(case["fmt"])
        x = s["src"].to(F64)
        padded = torch.zeros(C, _up(R, 16), dtype=F64, device=x.device)
        padded[:, :R] = x.t()
        if not case["tile"]:
            q, scales = _scaled64(x, f)
            qt, scales_t = _scaled64(padded, f)
            return _codes64({"q": q, "scales": scales, "qt": qt, "scales_t": scales_t}, f)
        q, scales = x.clone(), torch.empty(-(-R // BLOCK), -(-C // BLOCK), dtype=F64, device=x.device)
        for i in range(scales.shape[0]):
            for j in range(scales.shape[1]):
                part = q[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
                scales[i, j] = part.abs().max().clamp(min=TINY) / FMAX[f]
                part /= scales[i, j]
        padded[:, :R] = q.t()
        return _codes64({"q": q, "scales": scales, "qt": padded, "scales_t": scales.t()}, f)
    if op == "gemm":
        a, b = _value64(s["a"], s["a_scales"], False), _value64(s["b"], s["b_scales"], case["b_tile"])
        c = a @ b.t()
        return {"c": c if s["bias"] is None else c + s["bias"].to(F64)}
    p = _value64(s["x"], s["x_scales"], False) @ _value64(s["a"], s["a_scales"], True).t() + s["bias"].to(F64)
    hq, scales = _scaled64(p * torch.special.ndtr(p), E4M3)
    out = {"hq": hq, "scales": scales}
    if case["pre"]:
        out["pre"] = p
    return out
