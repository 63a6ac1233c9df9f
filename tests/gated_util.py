"""64-bit references of the gated feed-forward block and the error its kernels may make."""
import math

import torch

F64, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
HALF = torch.finfo(BF16).eps / 2  # a rounding to bf16, relative
TINY = 2.0 ** -133                # half the step of bf16's subnormal numbers, and what flushing to zero adds in fp32 chains


def act64(x, act):
    """(act(x), act'(x)) in 64 bits; act 0 = SiLU, 1 = the exact GeLU."""
    if act == 0:
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    cdf = torch.special.ndtr(x)
    return x * cdf, cdf + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)


def sum_error(a, b, terms):
    """Largest error of the fp32 sum of `terms` exact products a @ b: alignment in the tensor core's adder may truncate a
    whole unit 2^-23 each, and a few more for the bias and the joins of partial sums."""
    return (terms + 16) * 2.0 ** -23 * (a.abs() @ b.abs())


# The kernels' activations: erf's approximation is off by 1.5e-7, Phi by half of that and three units 2^-24 of the chain
# behind it, so act is off by 3e-7 |x|; SiLU's by the units of 2^x, the sum, 1/x and the product (6 * 2^-24 act, and the
# exponent's own rounding, |x| 2^-23 relative): inside 3e-7 |x| (1 + |x| sigmoid(-|x|)), which is below 4e-7 |x|.
# The slopes are sums of two such terms: 1e-6 (1 + |x|).
def act_error(x):
    return 4e-7 * x.abs()


def slope_error(x):
    return 1e-6 * (1 + x.abs())


SLOPE_MAX = 1.13  # the largest slope of either activation


def forward(X, Ag, Au, bg, bu, act):
    """G, U, H and the errors the stored ones may have."""
    d = X.shape[1]
    G, U = X @ Ag, X @ Au
    if bg is not None:
        G = G + bg
    if bu is not None:
        U = U + bu
    eg = sum_error(X, Ag, d) + 2.0 ** -23 * G.abs()
    eu = sum_error(X, Au, d) + 2.0 ** -23 * U.abs()
    a = act64(G, act)[0]
    H = a * U
    ea = SLOPE_MAX * eg + act_error(G)
    eh = ea * U.abs() + a.abs() * eu + ea * eu
    return {"G": (G, eg + HALF * (G.abs() + eg) + TINY), "U": (U, eu + HALF * (U.abs() + eu) + TINY),
            "H": (H, eh + HALF * (H.abs() + eh) + TINY)}


def derivatives(dY, B, G, U, act):
    """dG, dU, H from the stored factors, the column sums, and their errors."""
    d, T = dY.shape[1], dY.shape[0]
    dH = dY @ B.t()
    e = sum_error(dY, B.t(), d)
    a, slope = act64(G, act)
    dU, dG, H = dH * a, dH * U * slope, a * U
    eu = e * (a.abs() + act_error(G)) + dH.abs() * act_error(G) + 2.0 ** -22 * dU.abs()
    eg = U.abs() * (e * (slope.abs() + slope_error(G)) + dH.abs() * slope_error(G)) + 2.0 ** -22 * dG.abs()
    eh = U.abs() * act_error(G) + 2.0 ** -23 * H.abs()

    def sums(v, err):  # of values before their rounding; at most T additions in fp32
        s = v.sum(0)
        es = err.sum(0) + T * 2.0 ** -24 * v.abs().sum(0)
        return s, es + HALF * (s.abs() + es) + TINY

    out = {"dbg": sums(dG, eg), "dbu": sums(dU, eu)}
    for name, v, err in (("dG", dG, eg), ("dU", dU, eu), ("H", H, eh)):
        out[name] = (v, err + HALF * (v.abs() + err) + TINY)
    return out


def product(*pairs):
    """Sum of the products a @ b, and the error of its bf16 form."""
    v = sum(a @ b for a, b in pairs)
    e = sum(sum_error(a, b, sum(p[0].shape[1] for p in pairs)) for a, b in pairs)
    return v, e + HALF * (v.abs() + e) + TINY


def check(name, got, want):
    ref, bound = want
    got = got.to(F64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - ref).abs() - bound
    worst = over.argmax()
    assert (over <= 0).all(), (f"{name}: {got.flatten()[worst].item()} for {ref.flatten()[worst].item()}, "
                               f"bound {bound.flatten()[worst].item()}")
