"""64-bit references of the block-scaled FP8 operators, and the codes and scales their definition gives."""
import torch

F64, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
FMAX = {0: 448.0, 1: 57344.0}
TORCH_FMT = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}
HALF_STEP = {0: 2.0 ** -4, 1: 2.0 ** -3}         # relative, normal codes
HALF_SUBNORMAL = {0: 2.0 ** -10, 1: 2.0 ** -17}  # absolute, in units of the scale


def up(n, m):
    return (n + m - 1) // m * m


def block_amax(x, block_rows):
    """Largest finite-or-infinite magnitude of each block (NaN not counted), one entry per element of x."""
    R, K = x.shape
    a = torch.nan_to_num(x.abs(), nan=0.0, posinf=float("inf"))
    p = torch.zeros(up(R, block_rows), up(K, 128), dtype=a.dtype, device=a.device)
    p[:R, :K] = a
    return p.view(p.shape[0] // block_rows, block_rows, p.shape[1] // 128, 128).amax(dim=(1, 3))


def quantize(x, block_rows, fmt):
    """(codes as uint8, scales [blocks of rows x blocks of columns] fp32) of x (bf16 or fp32), from the definition."""
    x = x.to(F32)
    a = block_amax(x, block_rows).clamp(2.0 ** -100, torch.finfo(F32).max)
    top = torch.full_like(a, FMAX[fmt])  # a tensor: torch on CUDA multiplies by the reciprocal of a scalar divisor
    scale, inv = a / top, top / a
    each = inv.repeat_interleave(block_rows, 0)[:x.shape[0]].repeat_interleave(128, 1)[:, :x.shape[1]]
    v = x * each
    # saturating cast: the infinities become the largest finite value, NaN stays
    v = torch.where(v.isnan(), v, v.clamp(-FMAX[fmt], FMAX[fmt]))
    return v.to(TORCH_FMT[fmt]).view(torch.uint8), scale


def scales_layout(scale, rows, block_rows):
    """The ABI's layout of scales [rows or row tiles x k blocks]."""
    if block_rows == 128:
        return scale.contiguous()
    out = torch.full((scale.shape[1], up(rows, 128)), float("nan"), dtype=F32, device=scale.device)
    out[:, :rows] = scale.t()
    return out


def scales_from_layout(s, rows, block_rows):
    return s if block_rows == 128 else s[:, :rows].t()


def values(codes, scale, block_rows, fmt):
    """fp64 values of codes with scales [rows or row tiles x k blocks]."""
    R, K = codes.shape
    each = scale.to(F64).repeat_interleave(block_rows, 0)[:R].repeat_interleave(128, 1)[:, :K]
    return codes.view(TORCH_FMT[fmt]).to(F32).to(F64) * each


def gelu64(x):
    return x * torch.special.ndtr(x)


def operand(gen, rows, K, block_rows, fmt, sigma=1.0):
    """(codes, scales in the ABI's layout, fp64 values) of a random operand with channels of different size."""
    x = sigma * torch.randn(rows, K, generator=gen, device=gen.device) * torch.exp2(
        4 * torch.rand(K, generator=gen, device=gen.device))
    q, sc = quantize(x.to(BF16), block_rows, fmt)
    return q, scales_layout(sc, rows, block_rows), values(q, sc, block_rows, fmt)


def gemm_bound(a, b, K):
    """Largest error of the block-scaled product in fp32 before the output's rounding: 128 additions of exact products
    per block (alignment of the tensor core's adder may truncate: a whole unit 2^-23 each), then per block the two
    scales' product and one fused multiply-add."""
    l1 = a.abs() @ b.abs().t()
    return (128 + 3 + up(K, 128) // 128) * 2.0 ** -23 * l1


def norm_grad(s, w, dy, ds, eps=1e-5):
    """(dX, dweight) of the residual RMS norm's backward, formulas as they stand."""
    rstd = torch.rsqrt((s * s).mean(1, keepdim=True) + eps)
    xhat, g = s * rstd, dy * w
    return rstd * (g - xhat * (g * xhat).mean(1, keepdim=True)) + ds, (dy * xhat).sum(0)
