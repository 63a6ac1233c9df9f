"""4-bit products at sizes where a bound on sums says little or a block takes its column tiles in several rounds."""
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


def exact_case(M, K, N, group, zeros, seed):
    """Small whole codes, scales of powers of two, and tokens with one 2 in each group, the last row among them: every product
    and sum is exact in fp32 (at most K / 32 terms, multiples of 1/2 below 120, in all below 2^22 of them)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    G = binding.w4_groups(K, group)
    codes = torch.randint(0, 16, (K, N), generator=g, device="cuda").to(U8)
    z = torch.randint(0, 16, (G, N), generator=g, device="cuda").to(U8) if zeros else None
    s = torch.exp2(torch.randint(-2, 3, (G, N), generator=g, device="cuda").float()).to(BF16)
    at = torch.arange(G, device="cuda") * group + torch.randint(0, group, (M, G), generator=g, device="cuda")
    X = torch.zeros(M, K, dtype=BF16, device="cuda")
    X.scatter_(1, at.clamp(max=K - 1), 2.0)
    return X, codes, s, z


@pytest.mark.parametrize("M,K", [(1, 524296), (3, 210024), (8, 65544), (8, 4104), (9, 524296), (40, 65544), (70, 16392)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_every_group_of_long_rows_counts(M, K, group, zeros):
    assert K // 32 * 2 * 15 * 4 * 2 < 2 ** 23
    N = 24
    X, codes, s, z = exact_case(M, K, N, group, zeros, M + K + group)
    Y = Guarded((M, N))
    binding.tpmlp_gemm_w4(X, ref.pack(codes), s, group, Y.t, zeros=z)
    want = X.to(F64) @ ref.values(codes, s, z, group)
    assert torch.equal(Y.t, want.to(BF16))  # one rounding
    assert Y.intact()


@pytest.mark.parametrize("M,K,N", [(3, 72, 44008), (8, 200, 30024), (5, 1032, 24584), (8, 4104, 22536)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_gated_product_in_several_rounds(M, K, N, group, zeros):
    """More column tiles of both matrices than a block joins at once."""
    g = torch.Generator(device="cuda").manual_seed(M + N + group)
    mats, w = [], []
    for _ in range(2):
        W = (torch.randn(K, N, generator=g, device="cuda") * K ** -0.5).to(BF16)
        Q = torch.empty(binding.w4_codes_shape(K, N), dtype=U8, device="cuda")
        s = torch.empty(binding.w4_groups(K, group), N, dtype=BF16, device="cuda")
        z = torch.empty(binding.w4_groups(K, group), N, dtype=U8, device="cuda") if zeros else None
        binding.tpmlp_quantize_w4(W, group, Q, s, zeros=z)
        codes, s_ref, z_ref = ref.quantize(W, group, zeros)
        assert torch.equal(s, s_ref) and (z is None or torch.equal(z, z_ref))
        mats.append((Q, s, z))
        w.append(ref.values(codes, s, z, group))
    X = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    b = [(0.3 * torch.randn(N, generator=g, device="cuda")).to(BF16) for _ in range(2)]
    H = Guarded((M, N))
    binding.tpmlp_gemm1_gated_w4(X, mats[0][0], mats[0][1], mats[1][0], mats[1][1], group, H.t, act=binding.ACT_SILU,
                                 g_zeros=mats[0][2], u_zeros=mats[1][2], bg=b[0], bu=b[1])
    x = X.to(F64)
    v = [x @ wi + bi.to(F64) for wi, bi in zip(w, b)]
    e = [ref.product_error(x, wi, group) + 2.0 ** -23 * vi.abs() for wi, vi in zip(w, v)]
    a = gated.act64(v[0], binding.ACT_SILU)[0]
    ea = gated.SLOPE_MAX * e[0] + gated.act_error(v[0])
    h, err = a * v[1], ea * v[1].abs() + a.abs() * e[1] + ea * e[1]
    gated.check("H", H.t, (h, err + gated.HALF * (h.abs() + err) + gated.TINY))
    assert H.intact()


def test_the_most_tokens_of_a_call():
    """Up to as many as the header states, and an error past them."""
    K, N, group = 8, 8, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    for most, gated_form in ((8388480, False), (4194240, True)):
        Q = ref.pack(torch.randint(0, 16, (K, N), generator=g, device="cuda").to(U8))
        s = torch.ones(1, N, dtype=BF16, device="cuda")
        w = ref.values(ref.unpack(Q, K, N)[:K, :N], s, None, group)
        X = torch.zeros(most + 1, K, dtype=BF16, device="cuda")
        X[torch.arange(most + 1, device="cuda"), torch.arange(most + 1, device="cuda") % K] = 1

        def call(M, Y):
            if gated_form:
                binding.tpmlp_gemm1_gated_w4(X[:M], Q, s, Q, s, group, Y, act=binding.ACT_GELU)
            else:
                binding.tpmlp_gemm_w4(X[:M], Q, s, group, Y)

        Y = Guarded((most, N))
        call(most, Y.t)
        rows = torch.tensor([0, 1, 127, 128, most // 2, most - 129, most - 1], device="cuda")
        y = w[rows % K]
        if gated_form:
            y = gated.act64(y, binding.ACT_GELU)[0] * y
            gated.check("H", Y.t[rows], (y, 1e-6 * (1 + y.abs() ** 2) + gated.HALF * y.abs() + gated.TINY))
        else:
            assert torch.equal(Y.t[rows].to(F64), y)
        assert Y.intact()
        with pytest.raises(binding.TpMlpError, match="unsupported"):
            call(most + 1, torch.empty(most + 1, N, dtype=BF16, device="cuda"))
