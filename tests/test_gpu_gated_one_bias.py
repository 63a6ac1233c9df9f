"""The derivatives of the gated block with one bias gradient asked for, against both."""
import pytest
import torch

from gpu_util import Guarded
from tensor_transformer_mlp_tp_gb300 import binding

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("T,d,F,N", [(1, 64, 64, 8), (63, 72, 392, 1), (129, 136, 264, 1), (320, 256, 1024, 4), (1000, 72, 136, 1)])
@pytest.mark.parametrize("act", [binding.ACT_SILU, binding.ACT_GELU])
def test_one_bias_gradient_has_the_bits_of_both(T, d, F, N, act):
    g = torch.Generator(device="cuda").manual_seed(T + d + F)

    def normal(*shape, sigma=1.0):
        return (sigma * torch.randn(*shape, generator=g, device="cuda")).to(BF16)

    X, dY, Ag, Au, B = normal(T, d), normal(T, d), normal(d, F, sigma=0.1), normal(d, F, sigma=0.1), normal(F, d, sigma=0.1)
    G, U = normal(T, F), normal(T, F)

    def step(**biases):
        dG, dU = Guarded((T, F)), Guarded((T, F))
        out = {k: Guarded((F,)) for k, wanted in biases.items() if wanted}
        binding.tpmlp_gemm_dh_gated(dY, B, G, U, N, dG.t, dU.t, act=act, **{k: v.t for k, v in out.items()})
        assert dG.intact() and dU.intact() and all(v.intact() for v in out.values())
        return {"dG": dG.t, "dU": dU.t, **{k: v.t for k, v in out.items()}}

    def block(**biases):
        out = {k: Guarded(s) for k, s in (("dX", (T, d)), ("dAg", (d, F)), ("dAu", (d, F)), ("dB", (F, d)))}
        out.update({k: Guarded((F,)) for k, wanted in biases.items() if wanted})
        binding.tpmlp_gated_backward(X, Ag, Au, B, G, U, dY, N, act=act, **{k: v.t for k, v in out.items()})
        assert all(v.intact() for v in out.values())
        return {k: v.t for k, v in out.items()}

    for call in (step, block):
        both = call(dbg=True, dbu=True)
        for one in (call(dbg=True, dbu=False), call(dbg=False, dbu=True), call()):
            for k, v in one.items():
                assert torch.equal(v, both[k]), (call.__name__, k)
    st, site = binding.tpmlp_get_device_status()
    assert st == binding.OK, (st, site)
