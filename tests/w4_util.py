"""4-bit weights in torch, from the definition: the quantiser, the layout of the codes, 64-bit values, and the largest
error of a product."""
import torch

F64, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
TINY, BIG = 2.0 ** -100, torch.finfo(torch.bfloat16).max


def quantize(W, group, with_zeros):
    """(codes [K x N] uint8, scales [G x N] bf16, zeros [G x N] uint8 or None)."""
    K, N = W.shape
    codes = torch.empty(K, N, dtype=torch.uint8, device=W.device)
    scales, zeros = [], []
    for k in range(0, K, group):
        w = W[k:k + group].to(F32)
        w = torch.where(w.isnan(), torch.zeros_like(w), w)
        lo, hi = w.min(0).values.clamp(max=0), w.max(0).values.clamp(min=0)
        span = (hi - lo if with_zeros else torch.maximum(hi, -lo)).clamp(TINY, BIG)
        # divisors as tensors: torch on CUDA multiplies by the reciprocal of a scalar one
        s = (span / torch.full_like(span, 15 if with_zeros else 7)).to(BF16)
        z = (-lo / s.to(F32)).round().clamp(0, 15) if with_zeros else torch.full_like(span, 8)
        codes[k:k + group] = ((w / s.to(F32)).clamp(-32, 32).round() + z).clamp(0, 15).to(torch.uint8)
        scales.append(s)
        zeros.append(z)
    return codes, torch.stack(scales), torch.stack(zeros).to(torch.uint8) if with_zeros else None


def _places(K, N, device):
    """(word, shift) of every place of the padded matrix, as the layout is documented."""
    k = torch.arange((K + 63) // 64 * 64, device=device)[:, None]
    n = torch.arange((N + 15) // 16 * 16, device=device)[None, :]
    tile = (n // 16) * ((K + 63) // 64) + k // 64
    j, r, t, h = k % 64 // 16, k % 16 // 8, k % 8 // 2, k % 2
    c, g = n % 16 // 8, n % 8
    return tile * 128 + 4 * (4 * g + t) + j, (4 * (c + 2 * r) + 16 * h).expand(k.numel(), n.numel())


def pack(codes):
    """Codes [K x N] in the documented layout, uint8 [tiles x tiles x 512]."""
    K, N = codes.shape
    word, shift = _places(K, N, codes.device)
    full = torch.full(word.shape, 8, dtype=torch.int64, device=codes.device)
    full[:K, :N] = codes.long()
    out = torch.zeros(word.max().item() + 1, dtype=torch.int64, device=codes.device)
    out.index_add_(0, word.flatten(), (full << shift).flatten())  # every code has bits of its own
    out = torch.where(out >= 2 ** 31, out - 2 ** 32, out).to(torch.int32)
    return out.view((N + 15) // 16, (K + 63) // 64, 128).view(torch.uint8)


def unpack(Q, K, N):
    """All codes of the padded matrix."""
    word, shift = _places(K, N, Q.device)
    return (Q.contiguous().view(torch.int32).flatten()[word].long() >> shift) & 15


def values(codes, scales, zeros, group):
    """64-bit values [K x N]."""
    K = codes.shape[0]
    z = 8.0 if zeros is None else zeros.to(F64).repeat_interleave(group, 0)[:K]
    return (codes.to(F64) - z) * scales.to(F64).repeat_interleave(group, 0)[:K]


def product_error(x, w, group):
    """Largest error of x @ w before the output's rounding: a group's sum of exact products in fp32 (a unit 2^-23 for each
    addition, as the tensor core's adder may truncate), one product with the scale, the sum over groups and its joins."""
    K = x.shape[1]
    return (min(K, group) + 3 + (K + group - 1) // group + 16) * 2.0 ** -23 * (x.abs() @ w.abs())
