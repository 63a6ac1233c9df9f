"""The gated feed-forward block on the GPU against 64-bit formulas, step by step from the bf16 values that each step reads."""
import pytest
import torch

import gated_util as ref
from gpu_util import Guarded
from tensor_transformer_mlp_tp_gb300 import binding

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
SILU, GELU = binding.ACT_SILU, binding.ACT_GELU


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    st, site = binding.tpmlp_get_device_status()
    assert st == binding.OK, f"device status {binding.status_string(st)} (wait site {site})"


def make(T, d, F, seed=0, bias=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma=1.0):
        return (sigma * torch.randn(*shape, generator=g, device="cuda")).to(BF16)

    s = {"X": normal(T, d), "Ag": normal(d, F, sigma=1.5 * d ** -0.5), "Au": normal(d, F, sigma=d ** -0.5),
         "B": normal(F, d, sigma=F ** -0.5), "dY": normal(T, d, sigma=0.1),
         "bg": normal(F, sigma=0.2) if bias else None, "bu": normal(F, sigma=0.2) if bias else None}
    return s, {k: None if v is None else v.to(F64) for k, v in s.items()}


# one token to several row blocks; widths that end inside tiles of 64, 128 and 256; shards of eight columns
SHAPES = [(1, 8, 8, 1), (1, 64, 64, 8), (1, 1024, 4096, 4), (2, 136, 72, 1), (5, 200, 1024, 64), (16, 512, 264, 1),
          (17, 64, 128, 2), (37, 1024, 512, 4), (63, 72, 392, 1), (64, 256, 256, 2), (100, 328, 640, 8), (128, 128, 384, 1),
          (129, 136, 264, 1), (256, 64, 512, 8), (257, 200, 392, 1), (320, 1024, 1024, 4), (1000, 248, 1032, 1),
          (48, 512, 1280, 2), (9, 72, 1032, 1)]


@pytest.mark.parametrize("T,d,F,N", SHAPES)
@pytest.mark.parametrize("act", [SILU, GELU])
def test_forward(T, d, F, N, act):
    for bias in (True, False):
        s, v = make(T, d, F, seed=T + d + F, bias=bias)
        H, G, U, Y = Guarded((T, F)), Guarded((T, F)), Guarded((T, F)), Guarded((T, d))
        binding.tpmlp_gated_forward(s["X"], s["Ag"], s["Au"], s["B"], N, Y.t, act=act, bg=s["bg"], bu=s["bu"],
                                    Gpre_out=G.t, Upre_out=U.t, H_out=H.t)
        want = ref.forward(v["X"], v["Ag"], v["Au"], v["bg"], v["bu"], act)
        for name, t in (("G", G), ("U", U), ("H", H)):
            ref.check(name, t.t, want[name])
            assert t.intact(), name
        ref.check("Y", Y.t, ref.product((H.t.to(F64), v["B"])))
        assert Y.intact()
        # without the outputs that are optional, and the projections alone
        Y2, H2 = torch.empty_like(Y.t), torch.empty_like(H.t)
        binding.tpmlp_gated_forward(s["X"], s["Ag"], s["Au"], s["B"], N, Y2, act=act, bg=s["bg"], bu=s["bu"])
        binding.tpmlp_gemm1_gated(s["X"], s["Ag"], s["Au"], N, H2, act=act, bg=s["bg"], bu=s["bu"])
        assert torch.equal(Y2, Y.t) and torch.equal(H2, H.t)


@pytest.mark.parametrize("T,d,F,N", SHAPES)
@pytest.mark.parametrize("act", [SILU, GELU])
def test_backward(T, d, F, N, act):
    s, v = make(T, d, F, seed=T + d + F + 1)
    G, U, H, Y = (torch.empty(T, n, dtype=BF16, device="cuda") for n in (F, F, F, d))
    binding.tpmlp_gated_forward(s["X"], s["Ag"], s["Au"], s["B"], N, Y, act=act, bg=s["bg"], bu=s["bu"], Gpre_out=G,
                                Upre_out=U, H_out=H)
    out = {k: Guarded(sh) for k, sh in (("dG", (T, F)), ("dU", (T, F)), ("H", (T, F)), ("dbg", (F,)), ("dbu", (F,)))}
    binding.tpmlp_gemm_dh_gated(s["dY"], s["B"], G, U, N, out["dG"].t, out["dU"].t, act=act, H=out["H"].t,
                                dbg=out["dbg"].t, dbu=out["dbu"].t)
    want = ref.derivatives(v["dY"], v["B"], G.to(F64), U.to(F64), act)
    for name, t in out.items():
        ref.check(name, t.t, want[name])
        assert t.intact(), name
    dG, dU = out["dG"].t.to(F64), out["dU"].t.to(F64)
    grads = {k: Guarded(sh) for k, sh in (("dX", (T, d)), ("dAg", (d, F)), ("dAu", (d, F)), ("dB", (F, d)), ("dbg", (F,)),
                                          ("dbu", (F,)))}
    binding.tpmlp_gated_backward(s["X"], s["Ag"], s["Au"], s["B"], G, U, s["dY"], N, act=act,
                                 **{k: t.t for k, t in grads.items()})
    full = {"dX": ref.product((dG, v["Ag"].t()), (dU, v["Au"].t())), "dAg": ref.product((v["X"].t(), dG)),
            "dAu": ref.product((v["X"].t(), dU)), "dB": ref.product((out["H"].t.to(F64).t(), v["dY"])),
            "dbg": want["dbg"], "dbu": want["dbu"]}
    for name, t in grads.items():
        ref.check(name, t.t, full[name])
        assert t.intact(), name
    # the forward's H instead of one formed from the rounded factors, no bias gradients
    again = {k: torch.empty_like(t.t) for k, t in grads.items() if k not in ("dbg", "dbu")}
    binding.tpmlp_gated_backward(s["X"], s["Ag"], s["Au"], s["B"], G, U, s["dY"], N, act=act, H=H, **again)
    ref.check("dB", again["dB"], ref.product((H.to(F64).t(), v["dY"])))
    # both factors recomputed: the same bits as from the forward's
    anew = {k: torch.empty_like(t) for k, t in again.items()}
    binding.tpmlp_gated_backward(s["X"], s["Ag"], s["Au"], s["B"], None, None, s["dY"], N, act=act, bg=s["bg"],
                                 bu=s["bu"], **anew)
    for name, t in anew.items():
        assert torch.equal(t, again[name]), name
    for name in ("dX", "dAg", "dAu"):
        assert torch.equal(again[name], grads[name].t), name


@pytest.mark.parametrize("act", [SILU, GELU])
def test_gradients_of_the_whole_block(act):
    """Every gradient of Y = (act(G) U) B against 64-bit autograd, without the roundings between the steps: each of G, U,
    dG, dU and H is rounded once, half a step relative, and the products average over many of them."""
    T, d, F, N = 300, 256, 512, 4
    s, v = make(T, d, F, seed=9)
    G, U, Y = (torch.empty(T, n, dtype=BF16, device="cuda") for n in (F, F, d))
    binding.tpmlp_gated_forward(s["X"], s["Ag"], s["Au"], s["B"], N, Y, act=act, bg=s["bg"], bu=s["bu"], Gpre_out=G,
                                Upre_out=U)
    got = {"X": torch.empty(T, d, dtype=BF16, device="cuda"), "Ag": torch.empty(d, F, dtype=BF16, device="cuda"),
           "Au": torch.empty(d, F, dtype=BF16, device="cuda"), "B": torch.empty(F, d, dtype=BF16, device="cuda"),
           "bg": torch.empty(F, dtype=BF16, device="cuda"), "bu": torch.empty(F, dtype=BF16, device="cuda")}
    binding.tpmlp_gated_backward(s["X"], s["Ag"], s["Au"], s["B"], G, U, s["dY"], N, got["X"], got["Ag"], got["Au"],
                                 got["B"], act=act, dbg=got["bg"], dbu=got["bu"])
    leaves = {k: v[k].requires_grad_() for k in got}
    g = leaves["X"] @ leaves["Ag"] + leaves["bg"]
    a = torch.nn.functional.silu(g) if act == SILU else torch.nn.functional.gelu(g)
    y = (a * (leaves["X"] @ leaves["Au"] + leaves["bu"])) @ leaves["B"]
    y.backward(v["dY"])
    # two roundings of a factor (one of them through a slope up to 1.13) and the output's own: 2^-8 (1 + 1.13 + 1) at most
    # of the terms' size, which the norms keep
    assert torch.linalg.norm(Y.to(F64) - y) <= 3.2 * ref.HALF * torch.linalg.norm(y)
    for k, t in got.items():
        want = leaves[k].grad
        assert torch.linalg.norm(t.to(F64) - want) <= 4 * ref.HALF * torch.linalg.norm(want), k


@pytest.mark.parametrize("act", [SILU, GELU])
def test_activations_over_the_whole_range(act):
    """Gates from -200 to 200 one by one (a product with a single term, so that G is the weight itself), U = 1."""
    g = torch.cat([torch.linspace(-200, 200, 2048), torch.logspace(-30, 0, 1024), -torch.logspace(-30, 0, 1024)]).to(BF16)
    d, F = 8, g.numel()
    X = torch.zeros(3, d, dtype=BF16, device="cuda")
    X[:, 0] = 1
    Ag, Au = torch.zeros(d, F, dtype=BF16, device="cuda"), torch.zeros(d, F, dtype=BF16, device="cuda")
    Ag[0], Au[0] = g.cuda(), 1
    H = torch.empty(3, F, dtype=BF16, device="cuda")
    binding.tpmlp_gemm1_gated(X, Ag, Au, 1, H, act=act)
    a, slope = ref.act64(g.cuda().to(F64), act)
    x = g.cuda().to(F64)
    for row in H:
        ref.check("act", row, (a, ref.act_error(x) + ref.HALF * a.abs() + ref.TINY))
    # the slopes: dH = 1
    B = torch.zeros(F, d, dtype=BF16, device="cuda")
    B[:, 0] = 1
    G, U = g.cuda().expand(3, F).contiguous(), torch.ones(3, F, dtype=BF16, device="cuda")
    dG, dU = torch.empty_like(G), torch.empty_like(G)
    binding.tpmlp_gemm_dh_gated(X, B, G, U, 1, dG, dU, act=act)
    for row, col in zip(dG, dU):
        ref.check("slope", row, (slope, ref.slope_error(x) + ref.HALF * slope.abs() + ref.TINY))
        ref.check("act", col, (a, ref.act_error(x) + ref.HALF * a.abs() + ref.TINY))
