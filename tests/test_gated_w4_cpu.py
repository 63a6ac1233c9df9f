"""The gated block and the 4-bit weights without a GPU: the references' own checks, refusals of the library (which come
before anything reaches CUDA) and of its Python side, workspace sizes."""
import ctypes
import glob
import math
import os
import re

import pytest
import torch

import gated_util
import w4_util
from tensor_transformer_mlp_tp_gb300 import binding, build
from test_block_fp8_binding_cpu import Fake, fake, library  # noqa: F401  (a fixture)

BF16, F64, U8 = torch.bfloat16, torch.float64, torch.uint8
GOOD, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4)
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_transformer_mlp_tp_gb300", "csrc")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


# ----------------------------------------------------------------------------- the references

@pytest.mark.parametrize("act", [binding.ACT_SILU, binding.ACT_GELU])
def test_gradient_formulas_against_differences(act):
    """dG, dU and the products of them, as the GPU tests take them, against central differences of sum(Y dY)."""
    g = torch.Generator().manual_seed(5)
    T, d, F = 4, 6, 5
    v = {k: torch.randn(*s, generator=g, dtype=F64) for k, s in
         dict(X=(T, d), Ag=(d, F), Au=(d, F), B=(F, d), bg=(F,), bu=(F,), dY=(T, d)).items()}

    def loss(v):
        G, U = v["X"] @ v["Ag"] + v["bg"], v["X"] @ v["Au"] + v["bu"]
        return float(((gated_util.act64(G, act)[0] * U) @ v["B"] * v["dY"]).sum())

    G, U = v["X"] @ v["Ag"] + v["bg"], v["X"] @ v["Au"] + v["bu"]
    r = gated_util.derivatives(v["dY"], v["B"], G, U, act)
    dG, dU, H = r["dG"][0], r["dU"][0], r["H"][0]
    grads = {"X": gated_util.product((dG, v["Ag"].t()), (dU, v["Au"].t()))[0], "Ag": v["X"].t() @ dG, "Au": v["X"].t() @ dU,
             "B": H.t() @ v["dY"], "bg": r["dbg"][0], "bu": r["dbu"][0]}
    h = 1e-5
    for name, want in grads.items():
        for i in range(want.numel()):
            at = {}
            for sign in (1, -1):
                w = dict(v)
                w[name] = v[name].clone()
                w[name].view(-1)[i] += sign * h
                at[sign] = loss(w)
            assert (at[1] - at[-1]) / (2 * h) == pytest.approx(float(want.reshape(-1)[i]), rel=1e-6, abs=1e-7), (name, i)


def test_activations_against_torch():
    x = torch.linspace(-30, 30, 4001, dtype=F64, requires_grad=True)
    for act, f in ((binding.ACT_SILU, torch.nn.functional.silu), (binding.ACT_GELU, torch.nn.functional.gelu)):
        y = f(x)
        slope, = torch.autograd.grad(y.sum(), x)
        a, s = gated_util.act64(x.detach(), act)
        assert torch.allclose(a, y.detach(), rtol=1e-12, atol=1e-14) and torch.allclose(s, slope, rtol=1e-12, atol=1e-14)
        assert float(s.max()) <= gated_util.SLOPE_MAX


@pytest.mark.parametrize("K,N", [(8, 8), (64, 16), (72, 40), (200, 24)])
def test_layout_of_the_codes(K, N):
    """Place by place, as the header describes it; and back."""
    g = torch.Generator().manual_seed(K)
    codes = torch.randint(0, 16, (K, N), generator=g).to(U8)
    Q = w4_util.pack(codes)
    assert tuple(Q.shape) == binding.w4_codes_shape(K, N)
    words = Q.view(torch.int32).flatten().tolist()
    kts = (K + 63) // 64
    for n in range(Q.shape[0] * 16):
        for k in range(kts * 64):
            j, r, t, h, c, col = k % 64 // 16, k % 16 // 8, k % 8 // 2, k % 2, n % 16 // 8, n % 8
            word = words[((n // 16) * kts + k // 64) * 128 + 4 * (4 * col + t) + j] & 0xFFFFFFFF
            assert (word >> (4 * (c + 2 * r) + 16 * h)) & 15 == (int(codes[k, n]) if k < K and n < N else 8)
    assert torch.equal(w4_util.unpack(Q, K, N)[:K, :N], codes.long())


@pytest.mark.parametrize("zeros", [False, True])
def test_quantiser_of_the_references(zeros):
    """Half a step off at most, the ends of the range kept, and the code that is nearest."""
    g = torch.Generator().manual_seed(1)
    W = torch.randn(130, 24, generator=g).to(BF16)
    codes, s, z = w4_util.quantize(W, 32, zeros)
    v = w4_util.values(codes, s, z, 32)
    step = s.to(F64).repeat_interleave(32, 0)[:130]
    # the scale is rounded (half a step of bf16, over 15 or 7 steps) and so is the zero point (half of a code)
    assert float(((v - W.to(F64)).abs() / step).max()) <= (1 + 15 * 2 ** -8 if zeros else 0.5 + 7 * 2 ** -8)
    for k in range(0, 130, 32):
        part = slice(k, min(130, k + 32))
        zero = z[k // 32].to(F64) if zeros else torch.full((24,), 8.0, dtype=F64)
        q = W[part].to(F64) / s[k // 32].to(F64)
        assert torch.equal(codes[part].to(F64), (q.round() + zero).clamp(0, 15))


# ----------------------------------------------------------------------------- the library's refusals

def shape(T=256, d=64, F=256, N=2, dtype=binding.BF16):
    return ctypes.byref(binding.make_shape(T, d, F, N, dtype))


def gated_forward(lib, X=GOOD, Ag=GOOD, Au=GOOD, B=GOOD, bg=None, bu=None, act=0, s=None, Y=GOOD, G=None, U=None, H=None,
                  ws=GOOD, n=1 << 40):
    return lib.tpmlp_gated_forward(X, Ag, Au, B, bg, bu, act, s or shape(), Y, G, U, H, ws, n, None)


def gated_backward(lib, X=GOOD, Ag=GOOD, Au=GOOD, B=GOOD, bg=None, bu=None, act=0, G=GOOD, U=GOOD, H=None, dY=GOOD, s=None,
                   dX=GOOD, dAg=GOOD, dAu=GOOD, dB=GOOD, dbg=None, dbu=None, ws=GOOD, n=1 << 40):
    return lib.tpmlp_gated_backward(X, Ag, Au, B, bg, bu, act, G, U, H, dY, s or shape(), dX, dAg, dAu, dB, dbg, dbu, ws, n,
                                    None)


def gemm1_gated(lib, X=GOOD, Ag=GOOD, Au=GOOD, bg=None, bu=None, act=0, s=None, H=GOOD, G=None, U=None):
    return lib.tpmlp_gemm1_gated(X, Ag, Au, bg, bu, act, s or shape(), H, G, U, None)


def dh_gated(lib, dY=GOOD, B=GOOD, G=GOOD, U=GOOD, act=0, s=None, dG=GOOD, dU=GOOD, H=None, dbg=None, dbu=None, ws=None, n=0):
    return lib.tpmlp_gemm_dh_gated(dY, B, G, U, act, s or shape(), dG, dU, H, dbg, dbu, ws, n, None)


def dx_gated(lib, dG=GOOD, dU=GOOD, Ag=GOOD, Au=GOOD, s=None, dX=GOOD):
    return lib.tpmlp_gemm_dx_gated(dG, dU, Ag, Au, s or shape(), dX, None)


def gemm_w4(lib, X=GOOD, Q=GOOD, sc=GOOD, z=None, bias=None, M=4, N=64, K=64, group=64, Y=GOOD):
    return lib.tpmlp_gemm_w4(X, Q, sc, z, bias, M, N, K, group, Y, None)


def gated_w4(lib, X=GOOD, Qg=GOOD, sg=GOOD, zg=None, bg=None, Qu=GOOD, su=GOOD, zu=None, bu=None, act=0, group=32, s=None, H=GOOD):
    return lib.tpmlp_gemm1_gated_w4(X, Qg, sg, zg, bg, Qu, su, zu, bu, act, group, s or shape(), H, None)


def quantize_w4(lib, W=GOOD, K=64, N=64, group=32, Q=GOOD, sc=GOOD, z=None):
    return lib.tpmlp_quantize_w4(W, K, N, group, Q, sc, z, None)


def dequantize_w4(lib, Q=GOOD, sc=GOOD, z=None, K=64, N=64, group=32, W=GOOD):
    return lib.tpmlp_dequantize_w4(Q, sc, z, K, N, group, W, None)


BAD = binding.ERR_INVALID_ARG
REFUSED = (
    [(gated_forward, {k: None}) for k in ("X", "Ag", "Au", "B", "Y")] +
    [(gated_forward, {k: ODD}) for k in ("X", "Ag", "Au", "B", "Y", "bg", "bu", "G", "U", "H")] +
    [(gated_forward, kw) for kw in (dict(act=2), dict(act=-1), dict(G=GOOD), dict(U=GOOD), dict(s=shape(d=60)),
                                    dict(s=shape(F=264, N=5)), dict(s=shape(T=-1)), dict(s=shape(N=65)))] +
    [(gated_backward, {k: None}) for k in ("X", "Ag", "Au", "B", "dY", "dX", "dAg", "dAu", "dB", "G", "U")] +
    [(gated_backward, {k: ODD}) for k in ("bg", "bu", "G", "U", "H", "dbg", "dbu", "dX")] + [(gated_backward, dict(act=7))] +
    [(gemm1_gated, {k: None}) for k in ("X", "Ag", "Au", "H")] + [(gemm1_gated, kw) for kw in (dict(G=GOOD), dict(U=GOOD), dict(act=2))] +
    [(dh_gated, {k: None}) for k in ("dY", "B", "G", "U", "dG", "dU")] + [(dh_gated, kw) for kw in (dict(H=ODD), dict(act=3))] +
    [(dx_gated, {k: None}) for k in ("dG", "dU", "Ag", "Au", "dX")] + [(dx_gated, dict(dX=ODD))] +
    [(gemm_w4, {k: None}) for k in ("X", "Q", "sc", "Y")] + [(gemm_w4, {k: ODD}) for k in ("X", "Q", "sc", "z", "bias", "Y")] +
    [(gemm_w4, kw) for kw in (dict(K=0), dict(K=60), dict(N=60), dict(M=-1), dict(group=16), dict(group=0), dict(group=256))] +
    [(gated_w4, {k: None}) for k in ("X", "Qg", "sg", "Qu", "su", "H")] +
    [(gated_w4, kw) for kw in (dict(zg=GOOD), dict(zu=GOOD), dict(act=2), dict(group=96), dict(bg=ODD), dict(bu=ODD))] +
    [(quantize_w4, {k: None}) for k in ("W", "Q", "sc")] +
    [(quantize_w4, kw) for kw in (dict(z=ODD), dict(K=12), dict(N=12), dict(K=-8), dict(group=8))] +
    [(dequantize_w4, {k: None}) for k in ("W", "Q", "sc")] + [(dequantize_w4, kw) for kw in (dict(group=1), dict(N=4), dict(z=ODD))])


@pytest.mark.parametrize("call,kw", REFUSED, ids=lambda v: v.__name__ if callable(v) else "-".join(v))
def test_wrong_arguments_are_refused(lib, call, kw):
    assert call(lib, **kw) == BAD


def test_sizes_without_a_kernel_are_refused(lib):
    assert gemm_w4(lib, M=1 << 31) == binding.ERR_UNSUPPORTED
    assert gemm_w4(lib, K=1 << 31) == binding.ERR_UNSUPPORTED
    assert quantize_w4(lib, K=128 * 65536) == binding.ERR_UNSUPPORTED
    assert dequantize_w4(lib, K=128 * 65536) == binding.ERR_UNSUPPORTED
    assert gated_forward(lib, s=shape(dtype=binding.FP32)) == binding.ERR_UNSUPPORTED


def test_workspaces_that_are_too_small_are_refused(lib):
    n = ctypes.c_size_t(0)
    for op, call in ((binding.OP_GATED_FWD, gated_forward), (binding.OP_GATED_BWD, gated_backward)):
        assert lib.tpmlp_workspace_size(shape(), op, ctypes.byref(n)) == binding.OK
        for kw in (dict(n=n.value - 1), dict(ws=None), dict(ws=ODD)):
            assert call(lib, **kw) == binding.ERR_WORKSPACE
    assert lib.tpmlp_workspace_size(shape(), binding.OP_DH_GATED, ctypes.byref(n)) == binding.OK
    for kw in (dict(dbg=GOOD), dict(dbu=GOOD, ws=GOOD, n=n.value - 1), dict(dbg=GOOD, ws=ODD, n=n.value)):
        assert dh_gated(lib, **kw) == binding.ERR_WORKSPACE


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(0)

    def size(op, *a):
        assert lib.tpmlp_workspace_size(shape(*a), op, ctypes.byref(n)) == binding.OK
        return n.value

    T, d, F = 8192, 4096, 16384
    assert size(binding.OP_GATED_FWD, T, d, F, 8) == 2 * T * F             # H
    assert size(binding.OP_GATED_BWD, T, d, F, 8) == 10 * T * F + 2 * 4 * (4 * T // 128) * F  # dG, dU, H, G, U, column sums
    assert size(binding.OP_DH_GATED, T, d, F, 8) == 2 * 4 * (4 * T // 128) * F
    # K in parts where a few tiles leave most of the device idle: the parts' fp32 sums
    assert size(binding.OP_GATED_FWD, 1037, 1024, 4096, 8) == (2 * 1037 * 4096 + 255) // 256 * 256 + 3 * 4 * 1037 * 1024
    assert size(binding.OP_GATED_FWD, 128, 1024, 4096, 8) == 2 * 128 * 4096
    assert lib.tpmlp_workspace_size(shape(), 15, ctypes.byref(n)) == BAD
    assert lib.tpmlp_workspace_size(shape(), 19, ctypes.byref(n)) == BAD


def test_empty_calls(lib):
    """No tokens, or no columns: nothing is launched, and pointers may be NULL."""
    none = dict.fromkeys(("X", "Ag", "Au", "B", "Y", "ws"))
    assert gated_forward(lib, **none, s=shape(T=0)) == binding.OK
    assert gated_backward(lib, X=None, dX=None, ws=None, s=shape(T=0)) == binding.OK
    assert gemm1_gated(lib, X=None, H=None, s=shape(T=0)) == binding.OK
    assert dh_gated(lib, dY=None, s=shape(T=0)) == binding.OK
    assert dx_gated(lib, dX=None, s=shape(T=0)) == binding.OK
    assert gated_w4(lib, X=None, H=None, s=shape(T=0)) == binding.OK
    assert gemm_w4(lib, X=None, Y=None, M=0) == binding.OK and gemm_w4(lib, Q=None, N=0) == binding.OK
    assert quantize_w4(lib, W=None, N=0) == binding.OK and dequantize_w4(lib, W=None, K=0) == binding.OK


# ----------------------------------------------------------------------------- the Python side

T_, D_, F_ = 24, 64, 128


def py_forward(**kw):
    a = dict(X=Fake(T_, D_), Ag=Fake(D_, F_), Au=Fake(D_, F_), B=Fake(F_, D_), Y=Fake(T_, D_), bg=Fake(F_), bu=Fake(F_),
             G=Fake(T_, F_), U=Fake(T_, F_), H=Fake(T_, F_), ws=Fake(1 << 20, dtype=U8))
    a.update(kw)
    binding.tpmlp_gated_forward(a["X"], a["Ag"], a["Au"], a["B"], 2, a["Y"], bg=a["bg"], bu=a["bu"], Gpre_out=a["G"],
                                Upre_out=a["U"], H_out=a["H"], ws=a["ws"])


def py_backward(**kw):
    a = dict(X=Fake(T_, D_), Ag=Fake(D_, F_), Au=Fake(D_, F_), B=Fake(F_, D_), G=Fake(T_, F_), U=Fake(T_, F_), dY=Fake(T_, D_),
             dX=Fake(T_, D_), dAg=Fake(D_, F_), dAu=Fake(D_, F_), dB=Fake(F_, D_), bg=Fake(F_), bu=Fake(F_), dbg=Fake(F_),
             dbu=Fake(F_), H=Fake(T_, F_), ws=Fake(1 << 20, dtype=U8))
    a.update(kw)
    binding.tpmlp_gated_backward(a["X"], a["Ag"], a["Au"], a["B"], a["G"], a["U"], a["dY"], 2, a["dX"], a["dAg"], a["dAu"],
                                 a["dB"], bg=a["bg"], bu=a["bu"], dbg=a["dbg"], dbu=a["dbu"], H=a["H"], ws=a["ws"])


def py_gemm1(**kw):
    a = dict(X=Fake(T_, D_), Ag=Fake(D_, F_), Au=Fake(D_, F_), H=Fake(T_, F_), bg=Fake(F_), bu=Fake(F_), G=Fake(T_, F_), U=Fake(T_, F_))
    a.update(kw)
    binding.tpmlp_gemm1_gated(a["X"], a["Ag"], a["Au"], 2, a["H"], bg=a["bg"], bu=a["bu"], Gpre=a["G"], Upre=a["U"])


def py_dh(**kw):
    a = dict(dY=Fake(T_, D_), B=Fake(F_, D_), G=Fake(T_, F_), U=Fake(T_, F_), dG=Fake(T_, F_), dU=Fake(T_, F_), H=Fake(T_, F_),
             dbg=Fake(F_), dbu=Fake(F_), ws=Fake(1 << 20, dtype=U8))
    a.update(kw)
    binding.tpmlp_gemm_dh_gated(a["dY"], a["B"], a["G"], a["U"], 2, a["dG"], a["dU"], H=a["H"], dbg=a["dbg"], dbu=a["dbu"], ws=a["ws"])


def py_dx(**kw):
    a = dict(dG=Fake(T_, F_), dU=Fake(T_, F_), Ag=Fake(D_, F_), Au=Fake(D_, F_), dX=Fake(T_, D_))
    a.update(kw)
    binding.tpmlp_gemm_dx_gated(a["dG"], a["dU"], a["Ag"], a["Au"], 2, a["dX"])


CODES = binding.w4_codes_shape(D_, F_)


def py_quantize(**kw):
    a = dict(W=Fake(D_, F_), Q=Fake(*CODES, dtype=U8), s=Fake(2, F_), z=Fake(2, F_, dtype=U8), group=32)
    a.update(kw)
    binding.tpmlp_quantize_w4(a["W"], a["group"], a["Q"], a["s"], zeros=a["z"])


def py_dequantize(**kw):
    a = dict(W=Fake(D_, F_), Q=Fake(*CODES, dtype=U8), s=Fake(2, F_), z=Fake(2, F_, dtype=U8), group=32)
    a.update(kw)
    binding.tpmlp_dequantize_w4(a["Q"], a["s"], a["group"], a["W"], zeros=a["z"])


def py_gemm_w4(**kw):
    a = dict(X=Fake(3, D_), Q=Fake(*CODES, dtype=U8), s=Fake(2, F_), z=Fake(2, F_, dtype=U8), Y=Fake(3, F_), bias=Fake(F_), group=32)
    a.update(kw)
    binding.tpmlp_gemm_w4(a["X"], a["Q"], a["s"], a["group"], a["Y"], zeros=a["z"], bias=a["bias"])


def py_gated_w4(**kw):
    a = dict(X=Fake(3, D_), Qg=Fake(*CODES, dtype=U8), sg=Fake(2, F_), zg=Fake(2, F_, dtype=U8), Qu=Fake(*CODES, dtype=U8),
             su=Fake(2, F_), zu=Fake(2, F_, dtype=U8), H=Fake(3, F_), bg=Fake(F_), bu=Fake(F_), group=32)
    a.update(kw)
    binding.tpmlp_gemm1_gated_w4(a["X"], a["Qg"], a["sg"], a["Qu"], a["su"], a["group"], a["H"], g_zeros=a["zg"],
                                 u_zeros=a["zu"], bg=a["bg"], bu=a["bu"])


TD, TF, DF, FD, F1 = (T_, D_), (T_, F_), (D_, F_), (F_, D_), (F_,)
WS = (1 << 20, U8)
Q4, S4, Z4 = (*CODES, U8), (2, F_), (2, F_, U8)
OPERANDS = {
    py_forward: dict(X=TD, Ag=DF, Au=DF, B=FD, Y=TD, bg=F1, bu=F1, G=TF, U=TF, H=TF, ws=WS),
    py_backward: dict(X=TD, Ag=DF, Au=DF, B=FD, G=TF, U=TF, dY=TD, dX=TD, dAg=DF, dAu=DF, dB=FD, bg=F1, bu=F1, dbg=F1, dbu=F1,
                      H=TF, ws=WS),
    py_gemm1: dict(X=TD, Ag=DF, Au=DF, H=TF, bg=F1, bu=F1, G=TF, U=TF),
    py_dh: dict(dY=TD, B=FD, G=TF, U=TF, dG=TF, dU=TF, H=TF, dbg=F1, dbu=F1, ws=WS),
    py_dx: dict(dG=TF, dU=TF, Ag=DF, Au=DF, dX=TD),
    py_quantize: dict(W=DF, Q=Q4, s=S4, z=Z4), py_dequantize: dict(W=DF, Q=Q4, s=S4, z=Z4),
    py_gemm_w4: dict(X=(3, D_), Q=Q4, s=S4, z=Z4, Y=(3, F_), bias=F1),
    py_gated_w4: dict(X=(3, D_), Qg=Q4, sg=S4, zg=Z4, Qu=Q4, su=S4, zu=Z4, H=(3, F_), bg=F1, bu=F1)}


@pytest.mark.parametrize("call,name", [(c, n) for c in OPERANDS for n in OPERANDS[c]],
                         ids=lambda v: v if isinstance(v, str) else v.__name__)
def test_operands_that_do_not_fit_are_refused(library, call, name):  # noqa: F811
    """Of the host, of another device, of another type, too small, not contiguous: the library is not called."""
    spec = OPERANDS[call][name]
    call(**{name: fake(spec)})
    assert len(library.calls) == 1
    dims = [n for n in spec if isinstance(n, int)]
    dtype = spec[-1] if isinstance(spec[-1], torch.dtype) else BF16
    wrong = [fake(spec, dev=-1), fake(spec, dev=1), Fake(*dims, dtype=dtype, stride=tuple(2 * n for n in dims))]
    if name != "ws":
        wrong += [Fake(*dims, dtype=torch.float32), Fake(*dims, dtype=torch.float16)]
        if not (name == "X" and call in (py_gemm_w4, py_gated_w4)):
            wrong.append(Fake(*dims[:-1], dims[-1] - 8, dtype=dtype))
    for t in wrong:
        with pytest.raises(binding.TpMlpError) as e:
            call(**{name: t})
        assert e.value.status == BAD
    assert len(library.calls) == 1


@pytest.mark.parametrize("call", [py_quantize, py_dequantize, py_gemm_w4, py_gated_w4], ids=lambda c: c.__name__)
def test_groups_that_no_kernel_takes_are_refused(library, call):  # noqa: F811
    for group in (0, 16, 48, 256, -32):
        with pytest.raises(binding.TpMlpError):
            call(group=group)
    assert library.calls == []


def test_optional_operands_may_be_missing(library):  # noqa: F811
    py_forward(bg=None, bu=None, G=None, U=None, H=None)
    py_backward(bg=None, bu=None, dbg=None, dbu=None, H=None)
    py_backward(G=None, U=None)
    py_gemm1(bg=None, bu=None, G=None, U=None)
    py_dh(H=None, dbg=None, dbu=None, ws=None)
    py_quantize(z=None)
    py_gemm_w4(z=None, bias=None)
    py_gated_w4(zg=None, zu=None, bg=None, bu=None)
    assert len(library.calls) == 8


def test_large_workspaces_are_not_kept(library, monkeypatch):  # noqa: F811
    kept = {}
    monkeypatch.setattr(binding, "_WORKSPACES", kept)
    monkeypatch.setattr(binding.torch, "empty", lambda n, dtype=None, device=None: Fake(n, dtype=U8, ptr=1 << 24))
    binding._stream_workspace(binding._KEPT_BYTES, 0, None)
    assert [w.nbytes for w in kept.values()] == [binding._KEPT_BYTES]
    binding._stream_workspace(binding._KEPT_BYTES + 1, 0, None)
    assert [w.nbytes for w in kept.values()] == [binding._KEPT_BYTES]


# ----------------------------------------------------------------------------- the sources

def test_kernels_check_their_indices():
    """Every kernel of the new files that stores through hand-computed indices does so under the debug build's checks."""
    for name in ("w4.cu", "w4_tc.cuh", "gemm_few.cuh", "gated.cuh"):
        with open(os.path.join(CSRC, name)) as fh:
            text = re.sub(r"//.*", "", fh.read())
        assert "TPMLP_IN_BOUNDS(" in text, name
    with open(os.path.join(CSRC, "w4.cu")) as fh:
        kernels = re.split(r"__global__", re.sub(r"//.*", "", fh.read()))[1:]
    assert len(kernels) == 3
    for k in kernels:
        assert re.search(r"TPMLP_IN_BOUNDS\(|w4_finish", k), k[:120]


def test_scale_of_the_activation_errors():
    """The bounds that the GPU tests take for the kernels' activations cover erf's approximation (1.5e-7) and the roundings
    of the chain, at every x: SiLU's six units 2^-24 and its exponent's rounding."""
    x = torch.linspace(-90, 90, 5000, dtype=F64)
    s = torch.sigmoid(x)
    silu = x.abs() * s * (6 * 2.0 ** -24 + (x.abs() * math.log2(math.e)) * 2.0 ** -24 * math.log(2) * (1 - s))
    gelu = x.abs() * (0.75e-7 + 3 * 2.0 ** -24 * torch.special.ndtr(x))
    for e in (silu, gelu):
        assert bool((e <= gated_util.act_error(x) + 1e-30).all())
    assert len(glob.glob(os.path.join(CSRC, "w4*"))) == 4
