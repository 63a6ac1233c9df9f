"""4-bit products near the ends of the number range: a result that is finite comes out finite, whatever the number of tokens."""
import pytest
import torch

import gated_util as gated
import w4_util as ref
from gpu_util import Guarded
from tensor_transformer_mlp_tp_gb300 import binding

pytestmark = pytest.mark.gpu
BF16, F64, U8 = torch.bfloat16, torch.float64, torch.uint8


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    st, site = binding.tpmlp_get_device_status()
    assert st == binding.OK, f"device status {binding.status_string(st)} (wait site {site})"


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def pack(W, group, zeros):
    K, N = W.shape
    Q = torch.empty(binding.w4_codes_shape(K, N), dtype=U8, device="cuda")
    s = torch.empty(binding.w4_groups(K, group), N, dtype=BF16, device="cuda")
    z = torch.empty(binding.w4_groups(K, group), N, dtype=U8, device="cuda") if zeros else None
    binding.tpmlp_quantize_w4(W, group, Q, s, zeros=z)
    return Q, s, z


def values(m, K, N, group):
    return ref.values(ref.unpack(m[0], K, N)[:K, :N], m[1], m[2], group)


def error(x, w, group):
    """The sums' error, and up to eight tokens what is lost of values far below the largest of their token."""
    return ref.product_error(x, w, group) + 2.0 ** -39 * x.abs().amax(1, keepdim=True) * w.abs().sum(0)


def check_product(X, m, K, N, group):
    Y = Guarded((X.shape[0], N))
    binding.tpmlp_gemm_w4(X, m[0], m[1], group, Y.t, zeros=m[2])
    w, x = values(m, K, N, group), X.to(F64)
    y, e = x @ w, error(x, w, group)
    assert y.abs().max() < torch.finfo(BF16).max
    gated.check("Y", Y.t, (y, e + gated.HALF * (y.abs() + e) + gated.TINY))
    assert Y.intact()


def check_gated(X, mats, K, N, group, act):
    (Qg, sg, zg), (Qu, su, zu) = mats
    H = Guarded((X.shape[0], N))
    binding.tpmlp_gemm1_gated_w4(X, Qg, sg, Qu, su, group, H.t, act=act, g_zeros=zg, u_zeros=zu)
    x = X.to(F64)
    wg, wu = (values(m, K, N, group) for m in mats)
    G, U, eg, eu = x @ wg, x @ wu, error(x, wg, group), error(x, wu, group)
    a = gated.act64(G, act)[0]
    ea = gated.SLOPE_MAX * eg + gated.act_error(G)
    h, err = a * U, ea * U.abs() + a.abs() * eu + ea * eu
    assert h.abs().max() < torch.finfo(BF16).max
    gated.check("H", H.t, (h, err + gated.HALF * (h.abs() + err) + gated.TINY))
    assert H.intact()


@pytest.mark.parametrize("M", [1, 3, 8, 9, 40, 70])
@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("power", [-5, -20, -60, -110])
def test_small_tokens_on_the_largest_scales(M, group, zeros, power):
    """Columns that the quantiser made of infinities: eight weights at the ends of the codes, each the largest number's size,
    times tokens far below one."""
    K, N = 384, 72
    g = torch.Generator(device="cuda").manual_seed(M + group)
    W = normal(g, K, N)
    W[:8, 0], W[:8, 9] = float("-inf"), float("inf")
    W[300:308, 17], W[300:308, 30] = float("inf"), float("-inf")
    m = pack(W.to(BF16), group, zeros)
    X = normal(g, M, K) * 2.0 ** power
    X[:, :8] = X[:, 300:308] = 0.75 * 2.0 ** power
    check_product(X.to(BF16), m, K, N, group)


@pytest.mark.parametrize("M", [2, 8, 16, 65])
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
def test_gated_small_tokens_on_the_largest_scales(M, group, zeros):
    K, N = 384, 72
    g = torch.Generator(device="cuda").manual_seed(M + group)
    Wg, Wu = normal(g, K, N), normal(g, K, N)
    Wu[:8, 0], Wu[:8, 9] = float("-inf"), float("inf")
    X = normal(g, M, K) * 2.0 ** -20
    X[:, :8] = 0.75 * 2.0 ** -20
    mats = [pack(W.to(BF16), group, zeros) for W in (Wg, Wu)]
    check_gated(X.to(BF16), mats, K, N, group, binding.ACT_GELU)


@pytest.mark.parametrize("M", [1, 8, 9, 24, 40, 100, 150])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False), (128, True)])
def test_large_tokens_on_small_scales(M, group, zeros):
    """Tokens near the largest number on weights far below one: a group's sum before its scale is past the largest number."""
    K, N = 392, 136
    g = torch.Generator(device="cuda").manual_seed(M + group + 1)
    m = pack((normal(g, K, N) * 2.0 ** -90).to(BF16), group, zeros)
    check_product((normal(g, M, K) * 2.0 ** 124).to(BF16), m, K, N, group)


@pytest.mark.parametrize("M", [2, 12, 70])
@pytest.mark.parametrize("group,zeros", [(32, False), (128, True)])
@pytest.mark.parametrize("act", [binding.ACT_SILU, binding.ACT_GELU])
def test_gated_large_tokens_on_small_scales(M, group, zeros, act):
    K, N = 392, 136
    g = torch.Generator(device="cuda").manual_seed(M + group + 2)
    mats = [pack((normal(g, K, N) * 2.0 ** -95).to(BF16), group, zeros) for _ in range(2)]
    check_gated((normal(g, M, K) * 2.0 ** 124).to(BF16), mats, K, N, group, act)


@pytest.mark.parametrize("M", [1, 8, 16, 64, 128])
@pytest.mark.parametrize("power", [-116, -124, -128])
def test_tokens_near_the_smallest_numbers(M, power):
    """Beside the usual errors, an addition in fp32 is off by up to its smallest step, 2^-149, of sums that are kept 2^-11 times
    their size."""
    K, N, group = 1024, 256, 128
    g = torch.Generator(device="cuda").manual_seed(M)
    m = pack(normal(g, K, N).to(BF16), group, False)
    X = (normal(g, M, K).to(F64) * 2.0 ** power).to(BF16)
    Y = Guarded((M, N))
    binding.tpmlp_gemm_w4(X, m[0], m[1], group, Y.t)
    w, x = values(m, K, N, group), X.to(F64)
    y, e = x @ w, error(x, w, group) + (K + 32) * 2.0 ** -138 * m[1].to(F64).abs().amax(0).clamp(min=1)
    gated.check("Y", Y.t, (y, e + gated.HALF * (y.abs() + e) + gated.TINY))
    assert bool((Y.t != 0).any()) and Y.intact()
