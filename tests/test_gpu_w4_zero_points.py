"""Zero points are the low four bits of their bytes, in every call that reads them."""
import pytest
import torch

import w4_util as ref
from tensor_transformer_mlp_tp_gb300 import binding

pytestmark = pytest.mark.gpu
BF16, U8 = torch.bfloat16, torch.uint8


@pytest.mark.parametrize("M", [1, 8, 9, 40, 70])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_high_bits_are_not_read(M, group):
    K, N = 520, 136
    g = torch.Generator(device="cuda").manual_seed(M + group)
    G = binding.w4_groups(K, group)
    Q = ref.pack(torch.randint(0, 16, (K, N), generator=g, device="cuda").to(U8))
    s = torch.rand(G, N, generator=g, device="cuda").to(BF16)
    z = torch.randint(0, 256, (G, N), generator=g, device="cuda").to(U8)
    X = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    out = []
    for zeros in (z, z & 15):
        Y, H, W = torch.empty(M, N, dtype=BF16, device="cuda"), torch.empty(M, N, dtype=BF16, device="cuda"), torch.empty(K, N, dtype=BF16, device="cuda")
        binding.tpmlp_gemm_w4(X, Q, s, group, Y, zeros=zeros)
        binding.tpmlp_gemm1_gated_w4(X, Q, s, Q, s, group, H, g_zeros=zeros, u_zeros=zeros)
        binding.tpmlp_dequantize_w4(Q, s, group, W, zeros=zeros)
        out.append((Y, H, W))
    for name, a, b in zip(("product", "gated product", "inverse"), *out):
        assert torch.equal(a, b), name
    st, site = binding.tpmlp_get_device_status()
    assert st == binding.OK, (st, site)
