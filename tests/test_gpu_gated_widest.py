"""The derivatives of the gated block at the widest F that a shape may have."""
import pytest
import torch

import gated_util as ref
from tensor_transformer_mlp_tp_gb300 import binding

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


def test_both_bias_gradients_of_the_widest_block():
    T, d, F = 1, 8, (2 ** 31 - 1) // 2 // 8 * 8
    if torch.cuda.mem_get_info()[0] < 80e9:
        pytest.skip("needs 80 GB")
    g = torch.Generator(device="cuda").manual_seed(1)
    dY, B, G, U = (torch.randn(*s, generator=g, dtype=BF16, device="cuda") for s in ((T, d), (F, d), (T, F), (T, F)))
    dG, dU, dbg, dbu = (torch.empty(*s, dtype=BF16, device="cuda") for s in ((T, F), (T, F), (F,), (F,)))
    binding.tpmlp_gemm_dh_gated(dY, B, G, U, 1, dG, dU, act=binding.ACT_SILU, dbg=dbg, dbu=dbu)
    cols = torch.cat([torch.arange(0, F, F // 1000, device="cuda"), torch.arange(F - 40, F, device="cuda")])
    want = ref.derivatives(dY.to(F64), B[cols].to(F64), G[:, cols].to(F64), U[:, cols].to(F64), binding.ACT_SILU)
    for name, t in (("dG", dG[:, cols]), ("dU", dU[:, cols]), ("dbg", dbg[cols]), ("dbu", dbu[cols])):
        ref.check(name, t, want[name])
    one = torch.full((F,), 7.0, dtype=BF16, device="cuda")  # a sum alone: the same bits
    for name, both in (("dbg", dbg), ("dbu", dbu)):
        binding.tpmlp_gemm_dh_gated(dY, B, G, U, 1, dG, dU, act=binding.ACT_SILU, **{name: one})
        assert torch.equal(one, both), name
    st, site = binding.tpmlp_get_device_status()
    assert st == binding.OK, (st, site)
