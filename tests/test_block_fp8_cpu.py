"""Block-scaled FP8 calls without a GPU: refusals and size arithmetic (no call here reaches the CUDA runtime), and the
references' own checks."""
import ctypes

import pytest
import torch

import block_fp8_util as u
from tensor_transformer_mlp_tp_gb300 import binding, build

GOOD, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4)
INV, UNS, WS, OK = binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED, binding.ERR_WORKSPACE, binding.OK


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def chunks(*p):
    return ctypes.cast((ctypes.c_void_p * len(p))(*p), binding._PP)


def shape(T=256, d=64, F=256, N=2, dtype=binding.BF16):
    return ctypes.byref(binding.make_shape(T, d, F, N, dtype))


C2 = chunks(1 << 20, 1 << 21)


@pytest.mark.parametrize("args,status", [
    (dict(x=None), INV), (dict(x=chunks(1 << 20, None)), INV), (dict(w=None), INV), (dict(w=ODD), INV),
    (dict(r=chunks(1 << 20, (1 << 20) + 2)), INV), (dict(r=None), INV),            # a sum kept without a residual
    (dict(s=chunks(None, 1 << 20)), INV), (dict(q=None), INV), (dict(sc=None), INV), (dict(sc=ODD), INV),
    (dict(q=None, sc=None, g=None), INV),                                          # nothing to write
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(sh=shape(d=72)), INV),  # d % 16 with an 8-bit output
    (dict(sh=shape(T=255)), INV), (dict(sh=shape(d=60)), INV), (dict(sh=shape(dtype=binding.FP32)), UNS),
    (dict(sh=shape(d=32784)), UNS), (dict(sh=shape(T=0), x=None, w=None), OK)])
def test_rmsnorm_add_gather_refusals(L, args, status):
    a = dict(x=C2, r=C2, w=GOOD, eps=1e-5, sh=shape(), s=C2, g=GOOD, q=GOOD, sc=GOOD)
    a.update(args)
    assert L.tpmlp_rmsnorm_add_gather(a["x"], a["r"], a["w"], a["eps"], a["sh"], a["s"], a["g"], a["q"], a["sc"],
                                      None) == status


@pytest.mark.parametrize("args,status", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(dy=None), INV), (dict(dy=ODD), INV), (dict(dx=None), INV),
    (dict(ds=chunks(1 << 20, None)), INV), (dict(dw=None), INV), (dict(eps=-1.0), INV), (dict(ws=None), WS),
    (dict(n=64), WS), (dict(ws=ODD), WS), (dict(sh=shape(d=32776)), UNS), (dict(sh=shape(T=255)), INV),
    (dict(sh=shape(T=0), x=None, ws=None), OK)])
def test_rmsnorm_add_backward_refusals(L, args, status):
    a = dict(x=C2, w=GOOD, eps=1e-5, dy=GOOD, ds=C2, sh=shape(), dx=C2, dw=GOOD, ws=GOOD, n=1 << 30)
    a.update(args)
    assert L.tpmlp_rmsnorm_add_backward(a["x"], a["w"], a["eps"], a["dy"], a["ds"], a["sh"], a["dx"], a["dw"], a["ws"],
                                        a["n"], None) == status


def test_rmsnorm_add_backward_workspace(L):
    n = ctypes.c_size_t(7)
    assert L.tpmlp_rmsnorm_add_backward_workspace_size(shape(T=0), ctypes.byref(n)) == OK and n.value == 0
    assert L.tpmlp_rmsnorm_add_backward_workspace_size(shape(T=2), ctypes.byref(n)) == OK
    assert n.value >= 64 * 4 and n.value % 256 == 0
    assert L.tpmlp_rmsnorm_add_backward_workspace_size(shape(), None) == INV
    assert L.tpmlp_rmsnorm_add_backward_workspace_size(shape(T=-2), ctypes.byref(n)) == INV
    assert L.tpmlp_rmsnorm_add_backward_workspace_size(shape(d=32776), ctypes.byref(n)) == UNS
    assert binding.tpmlp_rmsnorm_add_backward_workspace_size(2, 64, 2) >= 64 * 4


@pytest.mark.parametrize("args,status", [
    (dict(src=None), INV), (dict(src=ODD), INV), (dict(rows=-1), INV), (dict(cols=40), INV), (dict(ld=48), INV),
    (dict(ld=68), INV), (dict(br=64), INV), (dict(fmt=2), INV), (dict(q=None), INV), (dict(s=None), INV),
    (dict(qT=None), INV), (dict(sT=None), INV), (dict(sT=ODD), INV), (dict(q=None, s=None, qT=None, sT=None), INV),
    (dict(rows=128 * 65536), UNS), (dict(rows=1 << 31), UNS), (dict(rows=0, src=None), OK), (dict(cols=0, ld=0), OK)])
def test_quantize_block_refusals(L, args, status):
    a = dict(src=GOOD, ld=64, rows=100, cols=64, br=1, fmt=0, q=GOOD, s=GOOD, qT=GOOD, sT=GOOD)
    a.update(args)
    assert L.tpmlp_quantize_block(a["src"], a["ld"], a["rows"], a["cols"], a["br"], a["fmt"], a["q"], a["s"], a["qT"],
                                  a["sT"], None) == status


@pytest.mark.parametrize("args,status", [
    (dict(A=None), INV), (dict(B=ODD), INV), (dict(sa=None), INV), (dict(sb=ODD), INV), (dict(C=None), INV),
    (dict(bias=ODD), INV), (dict(af=2), INV), (dict(bf=-1), INV), (dict(br=2), INV), (dict(M=-1), INV),
    (dict(N=100), INV), (dict(K=24), INV), (dict(K=0), INV), (dict(ldc=56), INV), (dict(ldc=68), INV),
    (dict(dt=2), INV), (dict(M=1 << 31), UNS), (dict(M=0, A=None), OK), (dict(N=0, ldc=0, C=None), OK)])
def test_gemm_fp8_block_refusals(L, args, status):
    a = dict(A=GOOD, af=0, sa=GOOD, B=GOOD, bf=0, sb=GOOD, br=1, M=100, N=64, K=32, bias=None, C=GOOD, dt=0, ldc=64)
    a.update(args)
    assert L.tpmlp_gemm_fp8_block(a["A"], a["af"], a["sa"], a["B"], a["bf"], a["sb"], a["br"], a["M"], a["N"], a["K"],
                                  a["bias"], a["C"], a["dt"], a["ldc"], None) == status


@pytest.mark.parametrize("args,status", [
    (dict(X=None), INV), (dict(sx=None), INV), (dict(A=ODD), INV), (dict(sa=None), INV), (dict(bias=ODD), INV),
    (dict(H=None), INV), (dict(sh=None), INV), (dict(pre=ODD), INV), (dict(shape=shape(d=72)), INV),
    (dict(shape=shape(F=264, N=1)), INV), (dict(shape=shape(dtype=binding.FP32)), UNS),
    (dict(shape=shape(T=0), X=None, H=None), OK)])
def test_gemm1_fp8_block_refusals(L, args, status):
    a = dict(X=GOOD, sx=GOOD, A=GOOD, sa=GOOD, bias=GOOD, shape=shape(), H=GOOD, sh=GOOD, pre=None)
    a.update(args)
    assert L.tpmlp_gemm1_fp8_block(a["X"], a["sx"], a["A"], a["sa"], a["bias"], a["shape"], a["H"], a["sh"], a["pre"],
                                   None) == status


def test_binding_refuses_what_the_abi_cannot_express(L):
    """Strided or undersized tensors never reach the library (CPU tensors: a call that got through would fail)."""
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    x, w = torch.zeros(4, 64, dtype=bf), torch.ones(64, dtype=bf)
    xq, sc = torch.zeros(4, 64, dtype=u8), torch.zeros(1, 128)
    with pytest.raises(binding.TpMlpError):  # scales for fewer rows than a padded block
        binding.tpmlp_rmsnorm_add_gather([x], w, 1, Xq=xq, x_scales=torch.zeros(1, 4))
    with pytest.raises(binding.TpMlpError):  # a strided chunk
        binding.tpmlp_rmsnorm_add_gather([torch.zeros(4, 128, dtype=bf)[:, :64]], w, 1, Xq=xq, x_scales=sc)
    with pytest.raises(binding.TpMlpError):  # fp32 where bf16 is meant
        binding.tpmlp_rmsnorm_add_gather([x], w.to(f32), 1, Xq=xq, x_scales=sc)
    with pytest.raises(binding.TpMlpError):  # fewer chunks than N
        binding.tpmlp_rmsnorm_add_backward([x], w, torch.zeros(8, 64, dtype=bf), 2, [x], torch.zeros(64))
    with pytest.raises(binding.TpMlpError):  # qT without the padding of its rows
        binding.tpmlp_quantize_block(x, qT=torch.zeros(64, 4, dtype=u8), scalesT=torch.zeros(1, 128))
    with pytest.raises(binding.TpMlpError):  # columns, not rows, strided
        binding.tpmlp_quantize_block(torch.zeros(64, 4, dtype=bf).t(), q=xq, scales=sc)
    with pytest.raises(binding.TpMlpError):  # operands of different K
        binding.tpmlp_gemm_fp8_block(xq, sc, torch.zeros(8, 32, dtype=u8), sc, torch.zeros(4, 8))
    with pytest.raises(binding.TpMlpError):  # row scales where C's type is neither bf16 nor fp32
        binding.tpmlp_gemm_fp8_block(xq, sc, torch.zeros(8, 64, dtype=u8), sc, torch.zeros(4, 8, dtype=torch.float64))
    with pytest.raises(binding.TpMlpError):
        binding.tpmlp_gemm1_fp8_block(xq, sc, torch.zeros(128, 64, dtype=u8), torch.zeros(1, 1), None, 1,
                                      torch.zeros(4, 64, dtype=u8), sc)


def test_binding_refuses_host_tensors(L):
    """Well-formed tensors of the host: refused before the library sees their addresses."""
    bf, u8 = torch.bfloat16, torch.uint8
    x, w, xq, sc = torch.zeros(4, 64, dtype=bf), torch.ones(64, dtype=bf), torch.zeros(4, 64, dtype=u8), torch.zeros(1, 128)
    for call in (lambda: binding.tpmlp_rmsnorm_add_gather([x], w, 1, Xq=xq, x_scales=sc),
                 lambda: binding.tpmlp_rmsnorm_add_backward([x], w, x, 1, [x], torch.zeros(64)),
                 lambda: binding.tpmlp_quantize_block(x, q=xq, scales=sc),
                 lambda: binding.tpmlp_gemm_fp8_block(xq, sc, xq[:, :].repeat(2, 1), torch.zeros(1, 1), torch.zeros(4, 8)),
                 lambda: binding.tpmlp_gemm1_fp8_block(xq, sc, torch.zeros(16, 64, dtype=u8), torch.zeros(1, 1), None, 1,
                                                       torch.zeros(4, 16, dtype=u8), sc)):
        with pytest.raises(binding.TpMlpError):
            call()


def test_scale_shapes():
    assert binding.block_scales_shape(300, 144) == (2, 384)
    assert binding.block_scales_shape(300, 144, 128) == (3, 2)
    assert binding.block_scales_shape(1, 16) == (1, 128)


def test_reference_quantizer_on_known_values():
    x = torch.zeros(2, 130, dtype=torch.bfloat16)
    x[0, 0], x[0, 1], x[0, 129], x[1, 3], x[1, 4] = 2.0, -1.0, 3.0, float("inf"), float("nan")
    q, s = u.quantize(x, 1, 0)
    assert s.shape == (2, 2)
    assert s[0, 0] == 2.0 / 448 and s[0, 1] == 3.0 / 448 and s[1, 1] == 2.0 ** -100 / 448
    v = q.view(torch.float8_e4m3fn).float()
    assert v[0, 0] == 448 and v[0, 1] == -224 and v[0, 129] == 448 and v[0, 2] == 0
    assert v[1, 3] == 448 and v[1, 4].isnan() and v[1, 0] == 0
    t, st = u.quantize(x[:1], 128, 1)
    assert st.shape == (1, 2) and t.view(torch.float8_e5m2).float()[0, 0] == 57344


def test_reference_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(3)
    s, w, dy, ds = (torch.randn(n, generator=g, dtype=u.F64) for n in ((5, 24), (24,), (5, 24), (5, 24)))
    f = lambda s, w: ((s * torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-5) * w) * dy).sum() + (ds * s).sum()
    dx, dw = u.norm_grad(s, w, dy, ds)
    for name, t, grad in (("dx", s, dx), ("dw", w, dw)):
        v, h = torch.randn(t.shape, generator=g, dtype=u.F64), 1e-5
        a, b = ((t + h * v, w) if name == "dx" else (s, t + h * v)), ((t - h * v, w) if name == "dx" else (s, t - h * v))
        num = (f(*a) - f(*b)) / (2 * h)
        assert abs(num - (grad * v).sum()) <= 1e-8 * max(1.0, abs(num))
