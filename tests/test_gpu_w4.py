"""4-bit weights on the GPU: the quantiser and its inverse bit by bit against the definition, the products against 64-bit
values of the same codes."""
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


def weights(K, N, seed=0, sigma=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(K, N, generator=g, device="cuda") * (K ** -0.5 if sigma is None else sigma)
    return (w * torch.exp2(3 * torch.rand(N, generator=g, device="cuda"))).to(BF16)


def bits(t):
    return t.view(torch.int16)


def quantized(W, group, zeros):
    K, N = W.shape
    Q, s = Guarded(binding.w4_codes_shape(K, N), U8), Guarded((binding.w4_groups(K, group), N))
    z = Guarded((binding.w4_groups(K, group), N), U8) if zeros else None
    binding.tpmlp_quantize_w4(W, group, Q.t, s.t, zeros=z.t if zeros else None)
    assert Q.intact() and s.intact() and (z is None or z.intact())
    return Q.t, s.t, z.t if zeros else None


def check_pack(W, group, zeros):
    K, N = W.shape
    Q, s, z = quantized(W, group, zeros)
    codes, s_ref, z_ref = ref.quantize(W, group, zeros)
    assert torch.equal(bits(s), bits(s_ref))
    if zeros:
        assert torch.equal(z, z_ref)
    assert torch.equal(Q.reshape(-1), ref.pack(codes).reshape(-1))
    back = Guarded((K, N))
    binding.tpmlp_dequantize_w4(Q, s, group, back.t, zeros=z)
    assert torch.equal(back.t, ref.values(codes, s_ref, z_ref, group).to(BF16))
    assert back.intact()


@pytest.mark.parametrize("K,N", [(8, 8), (64, 16), (64, 64), (72, 40), (128, 136), (200, 264), (520, 72), (1032, 520)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_and_back(K, N, group, zeros):
    check_pack(weights(K, N, seed=K + N), group, zeros)


@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_halves_and_extremes(zeros):
    """Quotients that lie on a half (to even), all equal values, zeros, one sign, subnormal and the largest numbers,
    infinities and NaN."""
    K, N, group = 128, 64, 64
    W = torch.zeros(K, N, dtype=torch.float32, device="cuda")
    k = torch.arange(K, device="cuda")
    W[:, 0] = (k % 32 - 16) * 0.25          # halves of a scale of 0.5 (symmetric: a = 3.5 below)
    W[:, 0] = W[:, 0].clamp(-3.5, 3.5)
    W[:, 1] = 1.25
    W[:, 2] = -0.75
    W[:, 4] = (k + 1) * 2.0 ** -130
    W[:, 5] = 3.3e38 * (1 - 2 * (k % 2))
    W[:, 6] = torch.where(k == 5, float("inf"), 1.0 * k)
    W[:, 7] = torch.where(k == 70, float("-inf"), 1.0 * k)
    W[:, 8] = torch.where(k % 3 == 0, float("nan"), 0.01 * k)
    W[:, 9] = float("nan")
    W[:, 10] = 2.0 ** -110
    W[:, 11] = (k % 31 - 15) * 0.5          # every half between the codes of a scale of 1 (zero points)
    W[:, 12:] = torch.randint(-30, 31, (K, N - 12), device="cuda") * 0.5
    check_pack(W.to(BF16), group, zeros)


# one token to several tiles of tokens; K and N that end inside tiles and groups
PRODUCTS = [(1, 8, 8), (1, 64, 16), (1, 4096, 1024), (2, 72, 40), (3, 200, 264), (5, 1024, 4096), (8, 136, 128),
            (9, 520, 72), (16, 2048, 512), (17, 328, 520), (31, 128, 2048), (32, 1032, 264), (33, 64, 8), (48, 4096, 136),
            (64, 512, 1000), (65, 256, 392), (100, 1000, 200), (128, 384, 640), (129, 640, 384), (200, 72, 2056),
            (256, 1024, 1024),
            # as many column blocks as leave room for clusters of 7 to 3 blocks
            (24, 2048, 4096), (40, 1928, 5000), (12, 1544, 6152), (9, 1024, 9000),
            # more of X than a block's shared memory holds beside the codes in flight
            (8, 65544, 24), (1, 524296, 8)]


@pytest.mark.parametrize("M,K,N", PRODUCTS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_product(M, K, N, group, zeros):
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    Q, s, z = quantized(weights(K, N, seed=M), group, zeros)
    w = ref.values(ref.unpack(Q, K, N)[:K, :N], s, z, group)
    X = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    bias = torch.randn(N, generator=g, device="cuda").to(BF16)
    x = X.to(F64)
    e = ref.product_error(x, w, group)
    for b in (None, bias):
        Y = Guarded((M, N))
        binding.tpmlp_gemm_w4(X, Q, s, group, Y.t, zeros=z, bias=b)
        y = x @ w
        if b is not None:
            y = y + b.to(F64)
        err = e + 2.0 ** -23 * y.abs()
        gated.check("Y", Y.t, (y, err + gated.HALF * (y.abs() + err) + gated.TINY))
        assert Y.intact()


@pytest.mark.parametrize("M,K,N", [(1, 8, 8), (1, 4096, 1024), (3, 200, 264), (5, 1024, 4096), (8, 72, 16), (16, 520, 136),
                                   (17, 1032, 72), (37, 256, 1000), (64, 512, 264), (100, 136, 520), (128, 64, 128),
                                   (130, 328, 200)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("act", [binding.ACT_SILU, binding.ACT_GELU])
def test_gated_product(M, K, N, group, zeros, act):
    g = torch.Generator(device="cuda").manual_seed(M + K + N + 1)
    mats = [quantized(weights(K, N, seed=M + i), group, zeros) for i in range(2)]
    w = [ref.values(ref.unpack(Q, K, N)[:K, :N], s, z, group) for Q, s, z in mats]
    X = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    for bias in (False, True):
        b = [(0.3 * torch.randn(N, generator=g, device="cuda")).to(BF16) if bias else None for _ in range(2)]
        H = Guarded((M, N))
        (Qg, sg, zg), (Qu, su, zu) = mats
        binding.tpmlp_gemm1_gated_w4(X, Qg, sg, Qu, su, group, H.t, act=act, g_zeros=zg, u_zeros=zu, bg=b[0], bu=b[1])
        x = X.to(F64)
        v, e = [], []
        for wi, bi in zip(w, b):
            v.append(x @ wi + (0 if bi is None else bi.to(F64)))
            e.append(ref.product_error(x, wi, group) + 2.0 ** -23 * v[-1].abs())
        a = gated.act64(v[0], act)[0]
        ea = gated.SLOPE_MAX * e[0] + gated.act_error(v[0])
        err = ea * v[1].abs() + a.abs() * e[1] + ea * e[1]
        h = a * v[1]
        gated.check("H", H.t, (h, err + gated.HALF * (h.abs() + err) + gated.TINY))
        assert H.intact()


def test_exact_products():
    """Small integers and scales of powers of two: every product and sum is exact, and so is the output."""
    M, K, N, group = 7, 256, 80, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 16, (K, N), generator=g, device="cuda").to(U8)
    zeros = torch.randint(0, 16, (K // group, N), generator=g, device="cuda").to(U8)
    s = torch.exp2(torch.randint(-2, 3, (K // group, N), generator=g, device="cuda").float()).to(BF16)
    X = torch.zeros(M, K, dtype=BF16, device="cuda")
    for m in range(M):  # one row of W each, doubled
        X[m, (m * 37) % K] = 2
    Y = torch.empty(M, N, dtype=BF16, device="cuda")
    binding.tpmlp_gemm_w4(X, ref.pack(codes), s, group, Y, zeros=zeros)
    assert torch.equal(Y.to(F64), X.to(F64) @ ref.values(codes, s, zeros, group))
