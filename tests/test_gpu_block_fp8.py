"""Block-scaled FP8 operators on the GPU against 64-bit references.

Tolerances (derived, not fitted).  A rounding is off by at most half a step relative to the value: 2^-8 for bf16, 2^-24
for fp32, 2^-4 for E4M3 and 2^-3 for E5M2 (subnormal codes: 2^-10 and 2^-17 of the block's scale).  A norm's fp32
statistics add at most 32 terms in a thread, 5 shuffles and 32 warps, then a square root and three products: under 80
roundings, so under 80 * 2^-24 < 2^-17 relative.  The products' bound is block_fp8_util.gemm_bound.
"""
import pytest
import torch

import block_fp8_util as u
from gpu_util import Guarded
from tensor_transformer_mlp_tp_gb300 import binding

pytestmark = pytest.mark.gpu
F64, F32, BF16, U8 = torch.float64, torch.float32, torch.bfloat16, torch.uint8
STAT = 2.0 ** -17


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, ref, tol, name=""):
    err = (got.to(F64) - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - tol).max()):.3e} over"


def device_ok():
    assert binding.tpmlp_get_device_status() == (binding.OK, 0)


def norm_inputs(g, T, d, N):
    x = (torch.randn(T, d, generator=g, device="cuda") * torch.exp2(4 * torch.rand(T, 1, generator=g, device="cuda"))).to(BF16)
    r = torch.randn(T, d, generator=g, device="cuda").to(BF16)
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF16)
    return x, r, w, T // N


NORM_SHAPES = [(1, 8, 1), (1, 16, 1), (3, 136, 3), (7, 1024, 1), (320, 128, 64), (130, 264, 2), (37, 4096, 1),
               (9, 4104, 1), (5, 8192, 1), (4, 12288, 2), (3, 32768, 1), (2, 20008, 1), (1037, 256, 1)]


@pytest.mark.parametrize("T,d,N", NORM_SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_rmsnorm_add_gather(T, d, N, residual):
    x, r, w, rows = norm_inputs(gen(T + d), T, d, N)
    with_q = d % 16 == 0
    S, Xg = Guarded((T, d)), Guarded((T, d))
    Xq, sc = Guarded((T, d), U8), Guarded(binding.block_scales_shape(T, d), F32)
    binding.tpmlp_rmsnorm_add_gather(
        list(x.split(rows)), w, N, R_chunks=list(r.split(rows)) if residual else None,
        S_chunks=list(S.t.split(rows)) if residual else None, Xg=Xg.t, Xq=Xq.t if with_q else None,
        x_scales=sc.t if with_q else None, eps=1e-5)
    device_ok()
    assert S.intact() and Xg.intact() and Xq.intact() and sc.intact()
    if residual:
        total = x.to(F64) + r.to(F64)
        within(S.t, total, 2.0 ** -8 * (1 + 2.0 ** -15) * total.abs(), "sum")
        s = S.t.to(F64)  # the norm reads the stored sum
    else:
        s = x.to(F64)
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-5) * w.to(F64)
    within(Xg.t, y, (2.0 ** -8 + STAT) * y.abs(), "bf16")
    if not with_q:
        return
    scale = u.scales_from_layout(sc.t, T, 1)
    want = u.block_amax(y, 1).clamp_min(2.0 ** -100) / 448
    within(scale, want, STAT * want, "scales")
    each = scale.to(F64).repeat_interleave(128, 1)[:, :d]
    within(u.values(Xq.t, scale, 1, 0), y, (2.0 ** -4 + 2 * STAT) * y.abs() + 2.0 ** -10 * each, "e4m3")
    # rows of the scales behind the last token are left as they were
    assert (sc.t.view(torch.int32)[:, T:] == 0x7F3B).all()


def test_rmsnorm_add_gather_in_place_and_8bit_only():
    T, d, N = 64, 4096, 4
    x, r, w, rows = norm_inputs(gen(5), T, d, N)
    S, Xq, sc = torch.empty(T, d, dtype=BF16, device="cuda"), torch.empty(T, d, dtype=U8, device="cuda"), \
        torch.empty(32, 128, device="cuda")
    binding.tpmlp_rmsnorm_add_gather(list(x.split(rows)), w, N, R_chunks=list(r.split(rows)),
                                     S_chunks=list(S.split(rows)), Xq=Xq, x_scales=sc)
    for into in (0, 1):
        x2, r2, q2, s2 = x.clone(), r.clone(), torch.empty_like(Xq), torch.empty_like(sc)
        binding.tpmlp_rmsnorm_add_gather(list(x2.split(rows)), w, N, R_chunks=list(r2.split(rows)),
                                         S_chunks=list((x2, r2)[into].split(rows)), Xq=q2, x_scales=s2)
        assert torch.equal((x2, r2)[into], S) and torch.equal((r2, x2)[into], (r, x)[into])
        assert torch.equal(q2, Xq) and torch.equal(s2[:, :T], sc[:, :T])


def test_rmsnorm_add_gather_zero_infinite_and_nan_rows():
    T, d = 6, 256
    x, r, w = torch.randn(T, d, generator=gen(1), device="cuda").to(BF16), torch.zeros(T, d, dtype=BF16, device="cuda"), \
        torch.ones(d, dtype=BF16, device="cuda")
    x[0] = 0
    x[1, 5], x[2, 7], x[3] = float("nan"), float("inf"), 3e38
    Xg, Xq, sc = torch.empty(T, d, dtype=BF16, device="cuda"), torch.empty(T, d, dtype=U8, device="cuda"), \
        torch.empty(2, 128, device="cuda")
    binding.tpmlp_rmsnorm_add_gather([x], w, 1, R_chunks=[r], Xg=Xg, Xq=Xq, x_scales=sc)
    v = Xq.view(torch.float8_e4m3fn).float()
    assert (Xg[0] == 0).all() and (v[0] == 0).all() and (sc[:, 0] == torch.tensor(2.0 ** -100) / 448).all()
    assert Xg[1].isnan().all() and v[1].isnan().all()      # a NaN spoils its row's statistics, and no other row
    assert v[2, 7].isnan() and (v[2, :7] == 0).all()       # rstd 0: inf * 0, and zeros
    assert (v[3] == 0).all()                               # the squares overflow: rstd 0
    alone = torch.empty(2, d, dtype=U8, device="cuda")
    sc2 = torch.empty(2, 128, device="cuda")
    binding.tpmlp_rmsnorm_add_gather([x[4:]], w, 1, R_chunks=[r[4:]], Xq=alone, x_scales=sc2)
    assert torch.equal(alone, Xq[4:]) and torch.equal(sc2[:, :2], sc[:, 4:6])


@pytest.mark.parametrize("T,d,N", NORM_SHAPES + [(1500, 512, 4), (640, 1024, 1)])
@pytest.mark.parametrize("residual", [True, False])
def test_rmsnorm_add_backward(T, d, N, residual):
    g = gen(T * 3 + d)
    s, ds, w, rows = norm_inputs(g, T, d, N)
    dy = (1e-2 * torch.randn(T, d, generator=g, device="cuda")).to(BF16)
    dX, dw = Guarded((T, d)), Guarded((d,), F32)
    need = binding.tpmlp_rmsnorm_add_backward_workspace_size(T, d, N)
    ws = Guarded((need,), U8)
    binding.tpmlp_rmsnorm_add_backward(list(s.split(rows)), w, dy, N, list(dX.t.split(rows)), dw.t,
                                       dS_chunks=list(ds.split(rows)) if residual else None, ws=ws.t)
    device_ok()
    assert dX.intact() and dw.intact() and ws.intact()
    S, W, DY, DS = s.to(F64), w.to(F64), dy.to(F64), ds.to(F64) if residual else torch.zeros_like(s, dtype=F64)
    ref_dx, ref_dw = u.norm_grad(S, W, DY, DS)
    rstd = torch.rsqrt((S * S).mean(1, keepdim=True) + 1e-5)
    size = (rstd * DY * W).abs() + S.abs() * rstd ** 3 * (DY * W * S).abs().sum(1, keepdim=True) / d + DS.abs()
    within(dX.t, ref_dx, 2.0 ** -8 * ref_dx.abs() + 2 * STAT * size, "dx")
    # per column: T products added one after the other at worst, each with rstd's error
    within(dw.t, ref_dw, (2 * STAT + (T + 64) * 2.0 ** -24) * (DY * S * rstd).abs().sum(0), "dweight")
    # in place over the residual's gradient and over the sums
    for src in ([ds] if residual else []) + [s]:
        buf = src.clone()
        dw2 = torch.empty(d, device="cuda")
        args = dict(dS_chunks=list((buf if src is ds else ds).split(rows)) if residual else None)
        binding.tpmlp_rmsnorm_add_backward(list((buf if src is s else s).split(rows)), w, dy, N, list(buf.split(rows)),
                                           dw2, **args)
        assert torch.equal(buf, dX.t) and torch.equal(dw2, dw.t)


def test_rmsnorm_add_gradient_against_differences():
    """dX and dweight of the kernel against central differences of the 64-bit forward."""
    T, d = 6, 64
    g = gen(11)
    s, ds, w, _ = norm_inputs(g, T, d, 1)
    dy = torch.randn(T, d, generator=g, device="cuda").to(BF16)
    dX, dw = torch.empty_like(s), torch.empty(d, device="cuda")
    binding.tpmlp_rmsnorm_add_backward([s], w, dy, 1, [dX], dw, dS_chunks=[ds])
    S, W, DY, DS = (t.to(F64) for t in (s, w, dy, ds))
    f = lambda s, w: ((s * torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-5) * w) * DY).sum() + (DS * s).sum()
    v, h = torch.randn(T, d, generator=g, device="cuda", dtype=F64), 1e-5
    num = (f(S + h * v, W) - f(S - h * v, W)) / (2 * h)
    tol = ((2.0 ** -8 + 4 * STAT) * dX.to(F64) * v).abs().sum() + 1e-6 * num.abs()
    assert (num - (dX.to(F64) * v).sum()).abs() <= tol
    v = torch.randn(d, generator=g, device="cuda", dtype=F64)
    num = (f(S, W + h * v) - f(S, W - h * v)) / (2 * h)
    rstd = torch.rsqrt((S * S).mean(1, keepdim=True) + 1e-5)
    assert (num - (dw.to(F64) * v).sum()).abs() <= 4 * STAT * ((DY * S * rstd).abs().sum(0) * v.abs()).sum() + 1e-6 * num.abs()


@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 144), (16, 128), (127, 256), (128, 128), (129, 272), (300, 1040),
                                       (1037, 512), (17, 4096)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_block(rows, cols, block_rows, fmt):
    g = gen(rows + cols)
    full = (torch.randn(rows, cols + 8, generator=g, device="cuda") * torch.exp2(
        10 * torch.rand(rows, 1, generator=g, device="cuda"))).to(BF16)
    src = full[:, :cols]  # rows cols + 8 elements apart
    P = u.up(rows, 16)
    q, sc = Guarded((rows, cols), U8), Guarded(binding.block_scales_shape(rows, cols, block_rows), F32)
    qt, st = Guarded((cols, P), U8), Guarded(binding.block_scales_shape(cols, rows, block_rows), F32)
    binding.tpmlp_quantize_block(src, block_rows, fmt, q=q.t, scales=sc.t, qT=qt.t, scalesT=st.t)
    device_ok()
    assert q.intact() and sc.intact() and qt.intact() and st.intact()
    want, scale = u.quantize(src, block_rows, fmt)
    assert torch.equal(q.t, want) and torch.equal(u.scales_from_layout(sc.t, rows, block_rows), scale)
    want, scale = u.quantize(src.t(), block_rows, fmt)
    assert torch.equal(qt.t[:, :rows], want) and torch.equal(u.scales_from_layout(st.t, cols, block_rows), scale)
    assert (qt.t[:, rows:] == 0).all()
    if block_rows == 1:
        assert (sc.t.view(torch.int32)[:, rows:] == 0x7F3B).all() and (st.t.view(torch.int32)[:, cols:] == 0x7F3B).all()
    # each orientation alone gives the same
    q2, sc2, qt2, st2 = (torch.empty_like(t.t) for t in (q, sc, qt, st))
    binding.tpmlp_quantize_block(src.contiguous(), block_rows, fmt, q=q2, scales=sc2)
    binding.tpmlp_quantize_block(src, block_rows, fmt, qT=qt2, scalesT=st2)
    assert torch.equal(q2, q.t) and torch.equal(qt2, qt.t)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_block_special_values(block_rows, fmt):
    src = torch.randn(256, 256, generator=gen(2), device="cuda").to(BF16)
    src[0, :128] = 0
    src[1, 3], src[2, 4], src[3, 200], src[130, 5] = float("nan"), float("inf"), -float("inf"), 3.3e38
    src[200:, 128:] = 1e-40  # bf16 subnormals: below the least amax
    q, sc = torch.empty(256, 256, dtype=U8, device="cuda"), torch.empty(binding.block_scales_shape(256, 256, block_rows), device="cuda")
    qt, st = torch.empty_like(q), torch.empty_like(sc)
    binding.tpmlp_quantize_block(src, block_rows, fmt, q=q, scales=sc, qT=qt, scalesT=st)
    for got, gs, x in ((q, sc, src), (qt, st, src.t())):
        want, scale = u.quantize(x, block_rows, fmt)
        a, b = got.view(u.TORCH_FMT[fmt]).float(), want.view(u.TORCH_FMT[fmt]).float()
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(9), b.nan_to_num(9))
        assert torch.equal(u.scales_from_layout(gs, 256, block_rows), scale)


GEMM_SHAPES = [(1, 8, 16), (1, 4096, 1024), (3, 136, 144), (16, 128, 128), (17, 264, 272), (33, 1000, 400),
               (64, 512, 2064), (65, 128, 640), (127, 256, 256), (128, 640, 1280), (129, 264, 384), (255, 136, 528),
               (300, 1024, 1040), (513, 520, 912), (1037, 1024, 512), (700, 2304, 256)]


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
@pytest.mark.parametrize("b_block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gemm_fp8_block(M, N, K, b_block_rows, dtype):
    g = gen(M * 7 + N + K)
    a_fmt, b_fmt = [(0, 0), (0, 1), (1, 0)][(M + N // 8) % 3]
    a, sa, av = u.operand(g, M, K, 1, a_fmt)
    b, sb, bv = u.operand(g, N, K, b_block_rows, b_fmt, 0.02)
    bias = torch.randn(N, generator=g, device="cuda").to(BF16) if M % 2 else None
    C = Guarded((M, N + 24), dtype)  # rows N + 24 elements apart
    C.t.zero_()
    binding.tpmlp_gemm_fp8_block(a, sa, b, sb, C.t[:, :N], bias=bias, b_block_rows=b_block_rows, a_fmt=a_fmt,
                                 b_fmt=b_fmt)
    device_ok()
    assert C.intact() and (C.t[:, N:] == 0).all()
    ref = av @ bv.t()
    tol = u.gemm_bound(av, bv, K)
    if bias is not None:
        ref = ref + bias.to(F64)
    tol = tol + (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * (ref.abs() + tol)
    within(C.t[:, :N], ref, tol, "C")
    C2 = torch.empty(M, N, dtype=dtype, device="cuda")  # another row pitch, the same values, and run to run
    binding.tpmlp_gemm_fp8_block(a, sa, b, sb, C2, bias=bias, b_block_rows=b_block_rows, a_fmt=a_fmt, b_fmt=b_fmt)
    assert torch.equal(C2, C.t[:, :N])


# many tiles, of either kernel: rows, columns and k-blocks that end inside
PAIR_SHAPES = [(700, 2312, 272), (1030, 1160, 400), (4104, 264, 144), (300, 5000, 16), (2050, 4104, 1040)]


@pytest.mark.parametrize("M,N,K", PAIR_SHAPES)
@pytest.mark.parametrize("b_block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gemm_fp8_block_many_tiles(M, N, K, b_block_rows, dtype):
    test_gemm_fp8_block(M, N, K, b_block_rows, dtype)


@pytest.mark.parametrize("T,d,F", [(1030, 400, 1168), (700, 272, 2320), (4104, 144, 272), (2050, 1040, 4112)])
@pytest.mark.parametrize("pre", [True, False])
def test_gemm1_fp8_block_many_tiles(T, d, F, pre):
    test_gemm1_fp8_block(T, d, F, 1, pre)


# more than a wave of 128 x 128 tiles and no more waves of pairs: on pairs whatever a k-block takes in either kernel
@pytest.mark.parametrize("M,N,K", [(1300, 2312, 272), (2300, 1160, 400), (8200, 264, 144), (300, 7000, 16), (513, 4104, 528),
                                   (1300, 2312, 8464), (1285, 2568, 4112)])
@pytest.mark.parametrize("b_block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gemm_fp8_block_on_pairs(M, N, K, b_block_rows, dtype):
    test_gemm_fp8_block(M, N, K, b_block_rows, dtype)


@pytest.mark.parametrize("T,d,F", [(1300, 272, 2320), (2300, 400, 1168), (8200, 144, 272), (513, 4112, 4112)])
@pytest.mark.parametrize("pre", [True, False])
def test_gemm1_fp8_block_on_pairs(T, d, F, pre):
    test_gemm1_fp8_block(T, d, F, 1, pre)


@pytest.mark.parametrize("M,N,K", [(33, 16, 16), (41, 272, 912), (48, 4096, 1040), (47, 520, 16384), (49, 1000, 2048)])
@pytest.mark.parametrize("b_block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gemm_fp8_block_between_32_and_64_rows(M, N, K, b_block_rows, dtype):
    test_gemm_fp8_block(M, N, K, b_block_rows, dtype)


@pytest.mark.parametrize("M", [2, 200])
def test_gemm_fp8_block_infinities_and_nan_stay_in_their_rows(M):
    """A NaN code spoils its row of C alone; scales of rows behind the last are not used."""
    g = gen(8)
    a, sa, av = u.operand(g, M, 256, 1, 0)
    b, sb, bv = u.operand(g, 136, 256, 128, 0)
    clean = torch.empty(M, 136, device="cuda")
    binding.tpmlp_gemm_fp8_block(a, sa, b, sb, clean)
    a[1, 200] = 0x7F
    C = torch.empty(M, 136, device="cuda")
    binding.tpmlp_gemm_fp8_block(a, sa, b, sb, C)
    assert C[1].isnan().all() and torch.equal(C[0], clean[0]) and torch.equal(C[2:], clean[2:])


@pytest.mark.parametrize("rows", [1, 7, 17, 23, 33, 40, 57, 127])
def test_products_of_few_rows_after_a_product_of_nan(rows):
    """Nothing that an earlier call left on the device reaches the rows or scales of a call with fewer rows."""
    g = gen(rows)
    K, N = 2048, 2048
    a, sa, av = u.operand(g, rows, K, 1, 0)
    b, sb, bv = u.operand(g, N, K, 128, 0, 0.02)
    full = 16 if rows <= 16 else 32 if rows <= 32 else 48 if rows <= 48 else 64 if rows <= 64 else 128
    nan = torch.full((full, K), 0x7F, dtype=U8, device="cuda")
    s_nan = torch.full(binding.block_scales_shape(full, K), float("nan"), device="cuda")
    C = torch.empty(full, N, device="cuda")
    Hq, hs = torch.empty(full, N, dtype=U8, device="cuda"), torch.empty(binding.block_scales_shape(full, N), device="cuda")
    outs = []
    for spoil in (False, True):
        if spoil:
            binding.tpmlp_gemm_fp8_block(nan, s_nan, b, sb, C)
        binding.tpmlp_gemm_fp8_block(a, sa, b, sb, C[:rows])
        if spoil:
            binding.tpmlp_gemm1_fp8_block(nan, s_nan, b, sb, None, 1, Hq, hs)
        binding.tpmlp_gemm1_fp8_block(a, sa, b, sb, None, 1, Hq[:rows], hs)
        outs.append((C[:rows].clone(), Hq[:rows].clone(), hs[:, :rows].clone()))
    device_ok()
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    ref = av @ bv.t()
    tol = u.gemm_bound(av, bv, K)
    within(outs[1][0], ref, tol + 2.0 ** -23 * (ref.abs() + tol), "C")


@pytest.mark.parametrize("T,d,F,N", [(1, 16, 16, 1), (1, 4096, 1024, 8), (5, 144, 272, 1), (37, 512, 1040, 1),
                                     (64, 256, 128, 1), (130, 272, 400, 1), (257, 1024, 4096, 8), (520, 384, 656, 1)])
@pytest.mark.parametrize("pre", [True, False])
def test_gemm1_fp8_block(T, d, F, N, pre):
    g = gen(T + d + F)
    x, sx, xv = u.operand(g, T, d, 1, 0)
    a, sa, av = u.operand(g, F, d, 128, 0, 0.02)
    bias = (0.5 * torch.randn(F, generator=g, device="cuda")).to(BF16) if T != 5 else None
    Hq, hs, Hp = Guarded((T, F), U8), Guarded(binding.block_scales_shape(T, F), F32), Guarded((T, F))
    binding.tpmlp_gemm1_fp8_block(x, sx, a, sa, bias, N, Hq.t, hs.t, Hpre=Hp.t if pre else None)
    device_ok()
    assert Hq.intact() and hs.intact() and Hp.intact()
    P = xv @ av.t() + (bias.to(F64) if bias is not None else 0)
    tol = u.gemm_bound(xv, av, d) + 2.0 ** -23 * P.abs()
    if pre:
        within(Hp.t, P, tol + 2.0 ** -8 * (P.abs() + tol), "Hpre")
    H = u.gelu64(P)
    # |GeLU'| <= 1.13; the fp32 erf is off by 1.5e-7 at most, half of it times |P|, and a few roundings
    dev = 1.13 * tol + 2e-7 * P.abs() + 2.0 ** -21 * H.abs()
    scale = u.scales_from_layout(hs.t, T, 1)
    want = u.block_amax(H, 1).clamp_min(2.0 ** -100) / 448
    within(scale, want, u.block_amax(dev, 1) / 448 + 2.0 ** -23 * want, "scales")
    each = scale.to(F64).repeat_interleave(128, 1)[:, :F]
    within(u.values(Hq.t, scale, 1, 0), H, dev + (2.0 ** -4 + 2.0 ** -20) * (H.abs() + dev) + 2.0 ** -10 * each, "H")
    assert (hs.t.view(torch.int32)[:, T:] == 0x7F3B).all()


def mlp(T, d, F, N, seed):
    """Inputs and buffers of a block-scaled FP8 MLP step: residual norm, both layers, and their gradients."""
    g = gen(seed)
    x, r, w, rows = norm_inputs(g, T, d, N)
    A = (0.05 * torch.randn(d, F, generator=g, device="cuda")).to(BF16)
    B = (0.05 * torch.randn(F, d, generator=g, device="cuda")).to(BF16)
    bias = (0.1 * torch.randn(F, generator=g, device="cuda")).to(BF16)
    dY = (1e-2 * torch.randn(T, d, generator=g, device="cuda")).to(BF16)
    e = lambda *s, dt=U8: torch.empty(*s, dtype=dt, device="cuda")
    sc = lambda r, c, b=1: torch.empty(binding.block_scales_shape(r, c, b), device="cuda")
    P = u.up(T, 16)
    return dict(
        T=T, d=d, F=F, N=N, rows=rows, x=x, r=r, w=w, A=A, B=B, bias=bias, dY=dY, S=e(T, d, dt=BF16), Xg=e(T, d, dt=BF16),
        Xq=e(T, d), xs=sc(T, d), AqT=e(F, d), asT=sc(F, d, 128), BqT=e(d, F), bsT=sc(d, F, 128), Bq=e(F, d),
        bs=sc(F, d, 128), Aq=e(d, F), a_s=sc(d, F, 128), Hq=e(T, F), hs=sc(T, F), Hpre=e(T, F, dt=BF16), Y=e(T, d, dt=BF16),
        dYq=e(T, d), dys=sc(T, d), dYqT=e(d, P), dysT=sc(d, T), dH=e(T, F, dt=BF16), dHq=e(T, F), dhs=sc(T, F),
        dHqT=e(F, P), dhsT=sc(F, T), XqT=e(d, P), xsT=sc(d, T), dA=e(d, F, dt=F32), dXg=e(T, d, dt=BF16),
        dX=e(T, d, dt=BF16), dw=e(d, dt=F32), ws=e(max(256, binding.tpmlp_rmsnorm_add_backward_workspace_size(T, d, N))))


def mlp_step(m, stream=None):
    """Norm -> column layer -> row layer, then the column layer's gradients and the norm's."""
    b, s = binding, dict(stream=stream)
    b.tpmlp_quantize_block(m["A"], 128, 0, q=m["Aq"], scales=m["a_s"], qT=m["AqT"], scalesT=m["asT"], **s)
    b.tpmlp_quantize_block(m["B"], 128, 0, qT=m["BqT"], scalesT=m["bsT"], q=m["Bq"], scales=m["bs"], **s)
    b.tpmlp_rmsnorm_add_gather(list(m["x"].split(m["rows"])), m["w"], m["N"], R_chunks=list(m["r"].split(m["rows"])),
                               S_chunks=list(m["S"].split(m["rows"])), Xg=m["Xg"], Xq=m["Xq"], x_scales=m["xs"], **s)
    b.tpmlp_gemm1_fp8_block(m["Xq"], m["xs"], m["AqT"], m["asT"], m["bias"], m["N"], m["Hq"], m["hs"], Hpre=m["Hpre"], **s)
    b.tpmlp_gemm_fp8_block(m["Hq"], m["hs"], m["BqT"], m["bsT"], m["Y"], **s)
    # dH = dY B^T (E5M2 rows x weight tiles), taken as the column layer's gradient
    b.tpmlp_quantize_block(m["dY"], 1, 1, q=m["dYq"], scales=m["dys"], qT=m["dYqT"], scalesT=m["dysT"], **s)
    b.tpmlp_gemm_fp8_block(m["dYq"], m["dys"], m["Bq"], m["bs"], m["dH"], a_fmt=1, **s)
    b.tpmlp_quantize_block(m["dH"], 1, 1, q=m["dHq"], scales=m["dhs"], qT=m["dHqT"], scalesT=m["dhsT"], **s)
    b.tpmlp_quantize_block(m["Xg"], 1, 0, qT=m["XqT"], scalesT=m["xsT"], **s)
    # dA = Xg^T dH with K = the padded tokens, dXg = dH A^T, then the norm
    b.tpmlp_gemm_fp8_block(m["XqT"], m["xsT"], m["dHqT"], m["dhsT"], m["dA"], b_block_rows=1, b_fmt=1, **s)
    b.tpmlp_gemm_fp8_block(m["dHq"], m["dhs"], m["Aq"], m["a_s"], m["dXg"], a_fmt=1, **s)
    b.tpmlp_rmsnorm_add_backward(list(m["S"].split(m["rows"])), m["w"], m["dXg"], m["N"], list(m["dX"].split(m["rows"])),
                                 m["dw"], dS_chunks=list(m["dY"].split(m["rows"])), ws=m["ws"], **s)


OUTPUTS = ("S", "Xq", "Hq", "Hpre", "Y", "dH", "dA", "dXg", "dX", "dw")


@pytest.mark.parametrize("T,d,F,N", [(2, 64, 256, 2), (96, 256, 1024, 4), (333, 512, 1296, 3)])
def test_mlp_step_stage_by_stage(T, d, F, N):
    """The operators in a row; each stage against 64 bits on what the stage before it stored."""
    m = mlp(T, d, F, N, 17)
    mlp_step(m)
    device_ok()
    val = lambda q, s, R, br, f: u.values(q, u.scales_from_layout(s, R, br), br, f)
    x, a = val(m["Xq"], m["xs"], T, 1, 0), val(m["AqT"], m["asT"], F, 128, 0)
    h, b = val(m["Hq"], m["hs"], T, 1, 0), val(m["BqT"], m["bsT"], d, 128, 0)
    dy, dh = val(m["dYq"], m["dys"], T, 1, 1), val(m["dHq"], m["dhs"], T, 1, 1)
    xt, dht = val(m["XqT"], m["xsT"], d, 1, 0), val(m["dHqT"], m["dhsT"], F, 1, 1)
    assert torch.equal(m["Aq"].t(), m["AqT"]) and torch.equal(m["a_s"].t(), m["asT"])
    for name, got, l, r, K, add in (("Hpre", m["Hpre"], x, a, d, m["bias"].to(F64)), ("Y", m["Y"], h, b, F, 0),
                                    ("dH", m["dH"], dy, b.t(), d, 0), ("dA", m["dA"], xt, dht, T, 0),
                                    ("dXg", m["dXg"], dh, a.t(), F, 0)):
        ref, tol = l @ r.t() + add, u.gemm_bound(l, r, K)
        within(got, ref, tol + (2.0 ** -8 if got.dtype == BF16 else 2.0 ** -23) * (ref.abs() + tol), name)
    # against the unquantised chain: the 8-bit roundings of E4M3 (2^-4 each on both sides) leave C's direction
    full = u.gelu64(m["Xg"].to(F64) @ m["A"].to(F64) + m["bias"].to(F64)) @ m["B"].to(F64)
    # each operand's error is at most 2^-4 an element and independent of the others': 4 roundings, the sum at most
    # 4 * 2^-4 of the norm
    assert (m["Y"].to(F64) - full).norm() <= 4 * 2.0 ** -4 * full.norm()


def test_mlp_step_in_a_captured_graph_and_on_two_streams():
    """Eager, replayed from a graph with changed inputs, and two steps at once on two streams: the same bits."""
    m, n = mlp(96, 256, 1024, 4, 21), mlp(160, 512, 768, 2, 22)
    mlp_step(m)
    mlp_step(n)
    torch.cuda.synchronize()
    want = [{k: t[k].clone() for k in OUTPUTS} for t in (m, n)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for t in (m, n):
        for k in OUTPUTS:
            t[k].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        mlp_step(m, s1)
        mlp_step(n, s2)
    torch.cuda.synchronize()
    for t, w in zip((m, n), want):
        assert all(torch.equal(t[k], w[k]) for k in OUTPUTS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlp_step(m)
    other = mlp(96, 256, 1024, 4, 23)
    mlp_step(other)
    torch.cuda.synchronize()
    for k in ("x", "r", "w", "A", "B", "bias", "dY"):
        m[k].copy_(other[k])
    for k in OUTPUTS:
        m[k].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(m[k], other[k]) for k in OUTPUTS)


def test_empty_batches_leave_outputs_alone():
    C = torch.full((0, 16), 7.0, device="cuda")
    binding.tpmlp_gemm_fp8_block(torch.empty(0, 32, dtype=U8, device="cuda"), torch.empty(1, 0, device="cuda"),
                                 torch.zeros(16, 32, dtype=U8, device="cuda"), torch.zeros(1, 128, device="cuda"), C)
    dw = torch.full((64,), 7.0, device="cuda")
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    binding.tpmlp_rmsnorm_add_backward([e], torch.ones(64, dtype=BF16, device="cuda"), e, 1, [e], dw)
    binding.tpmlp_rmsnorm_add_gather([e], torch.ones(64, dtype=BF16, device="cuda"), 1, Xg=e)
    binding.tpmlp_quantize_block(e, q=torch.empty(0, 64, dtype=U8, device="cuda"), scales=torch.empty(1, 0, device="cuda"))
    torch.cuda.synchronize()
    assert (dw == 7).all()


# ----------------------------------------------------------------------------- offsets past 2^31, threads, layouts

def _sample(n, k, seed):
    return torch.randint(0, n, (k,), generator=torch.Generator().manual_seed(seed)).tolist() + [0, n - 1]


def test_norm_and_backward_past_two_to_the_31():
    T, d, N = (1 << 19) + 256, 4096, 2
    g = gen(31)
    x = torch.empty(T, d, dtype=BF16, device="cuda").normal_(generator=g)
    r = torch.empty(T, d, dtype=BF16, device="cuda").normal_(generator=g)
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF16)
    S, q, sc = torch.empty_like(x), torch.empty(T, d, dtype=U8, device="cuda"), torch.empty(32, u.up(T, 128), device="cuda")
    rows = T // N
    binding.tpmlp_rmsnorm_add_gather(list(x.split(rows)), w, N, R_chunks=list(r.split(rows)),
                                     S_chunks=list(S.split(rows)), Xq=q, x_scales=sc)
    at = _sample(T, 40, 1)
    s = S[at].to(F64)
    total = x[at].to(F64) + r[at].to(F64)
    within(S[at], total, 2.0 ** -8 * (1 + 2.0 ** -15) * total.abs(), "sum")
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-5) * w.to(F64)
    scale = sc[:, at].t()
    each = scale.to(F64).repeat_interleave(128, 1)
    within(u.values(q[at], scale, 1, 0), y, (2.0 ** -4 + 2 * STAT) * y.abs() + 2.0 ** -10 * each, "e4m3")
    dX, dw = x, torch.empty(d, device="cuda")
    binding.tpmlp_rmsnorm_add_backward(list(S.split(rows)), w, r, N, list(dX.split(rows)), dw)
    device_ok()
    ref, _ = u.norm_grad(s, w.to(F64), r[at].to(F64), torch.zeros_like(s))
    rstd = torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-5)
    size = (rstd * r[at].to(F64) * w.to(F64)).abs() + s.abs() * rstd ** 3 * (r[at].to(F64) * w.to(F64) * s).abs().sum(1, keepdim=True) / d
    within(dX[at], ref, 2.0 ** -8 * ref.abs() + 2 * STAT * size, "dx")


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_block_past_two_to_the_31(block_rows):
    rows, cols = 131328, 16400
    src = torch.empty(rows, cols, dtype=BF16, device="cuda").normal_(generator=gen(32))
    q, qt = torch.empty(rows, cols, dtype=U8, device="cuda"), torch.empty(cols, rows, dtype=U8, device="cuda")
    sc = torch.empty(binding.block_scales_shape(rows, cols, block_rows), device="cuda")
    st = torch.empty(binding.block_scales_shape(cols, rows, block_rows), device="cuda")
    binding.tpmlp_quantize_block(src, block_rows, 0, q=q, scales=sc, qT=qt, scalesT=st)
    device_ok()
    for i, j in ((0, 0), (rows // 128 - 1, cols // 128), (rows // 128 - 1, 0), (700, 100)):
        a, b = slice(128 * i, 128 * (i + 1)), slice(128 * j, min(cols, 128 * (j + 1)))
        want, scale = u.quantize(src[a, b], block_rows, 0)
        assert torch.equal(q[a, b], want)
        assert torch.equal(sc[i, j:j + 1] if block_rows == 128 else sc[j, a], scale.reshape(-1))
        want, scale = u.quantize(src[a, b].t(), block_rows, 0)
        assert torch.equal(qt[b, a], want)
        assert torch.equal(st[j, i:i + 1] if block_rows == 128 else st[i, b], scale.reshape(-1))


@pytest.mark.parametrize("gelu", [False, True])
def test_products_past_two_to_the_31(gelu):
    M, N, K = 131328, 16400, 144
    g = gen(33)
    a, sa, av = u.operand(g, M, K, 1, 0)
    b, sb, bv = u.operand(g, N, K, 128, 0, 0.02)
    at = _sample(M, 30, 2)
    ref, tol = av[at] @ bv.t(), u.gemm_bound(av[at], bv, K)
    if not gelu:
        C = torch.empty(M, N, dtype=BF16, device="cuda")
        binding.tpmlp_gemm_fp8_block(a, sa, b, sb, C)
        device_ok()
        within(C[at], ref, tol + 2.0 ** -8 * (ref.abs() + tol), "C")
        return
    hq, hs = torch.empty(M, N, dtype=U8, device="cuda"), torch.empty(binding.block_scales_shape(M, N), device="cuda")
    pre = torch.empty(M, N, dtype=BF16, device="cuda")
    binding.tpmlp_gemm1_fp8_block(a, sa, b, sb, None, 1, hq, hs, Hpre=pre)
    device_ok()
    within(pre[at], ref, tol + 2.0 ** -8 * (ref.abs() + tol), "Hpre")
    H, scale = u.gelu64(ref), hs[:, at].t()
    dev = 1.13 * tol + 2e-7 * ref.abs() + 2.0 ** -21 * H.abs()
    each = scale.to(F64).repeat_interleave(128, 1)[:, :N]
    within(u.values(hq[at], scale, 1, 0), H, dev + (2.0 ** -4 + 2.0 ** -20) * (H.abs() + dev) + 2.0 ** -10 * each, "H")


def test_calls_from_several_threads():
    """Each thread on its own stream with its own buffers, shapes that take both product kernels."""
    import threading

    sets = [mlp(T, d, F, N, 40 + i) for i, (T, d, F, N) in enumerate([(96, 256, 1024, 4), (300, 512, 768, 3), (2, 128, 512, 2)])]
    for m in sets:
        mlp_step(m)
    torch.cuda.synchronize()
    want = [{k: m[k].clone() for k in OUTPUTS} for m in sets]
    for m in sets:
        for k in OUTPUTS:
            m[k].zero_()
    torch.cuda.synchronize()
    errors = []

    def work(m):
        try:
            s = torch.cuda.Stream()
            for _ in range(10):
                mlp_step(m, s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(m,)) for m in sets]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for m, w in zip(sets, want):
        assert all(torch.equal(m[k], w[k]) for k in OUTPUTS)


def test_weight_gradient_over_padded_tokens_equals_the_unpadded_sum():
    """dA with K = tokens rounded up to 16: the zero bytes behind the last token add nothing, whatever their scale."""
    T, d, F = 37, 144, 272
    g = gen(50)
    X, dH = (torch.randn(T, n, generator=g, device="cuda").to(BF16) for n in (d, F))
    P = u.up(T, 16)
    xt, ht = torch.empty(d, P, dtype=U8, device="cuda"), torch.empty(F, P, dtype=U8, device="cuda")
    xs, hs = (torch.empty(binding.block_scales_shape(n, T), device="cuda") for n in (d, F))
    binding.tpmlp_quantize_block(X, 1, 0, qT=xt, scalesT=xs)
    binding.tpmlp_quantize_block(dH, 1, 1, qT=ht, scalesT=hs)
    dA = torch.empty(d, F, device="cuda")
    binding.tpmlp_gemm_fp8_block(xt, xs, ht, hs, dA, b_block_rows=1, b_fmt=1)
    l = u.values(xt[:, :T], u.scales_from_layout(xs, d, 1), 1, 0)
    r = u.values(ht[:, :T], u.scales_from_layout(hs, F, 1), 1, 1)
    ref, tol = l @ r.t(), u.gemm_bound(l, r, T)
    within(dA, ref, tol + 2.0 ** -23 * ref.abs(), "dA")


def test_workspaces_kept_for_a_stream():
    """Backward calls without a workspace: one kept for each of torch's streams, grown when needed, a fresh one for an
    explicit stream and in a capture."""
    def case(T, d, seed):
        s, ds, w, _ = norm_inputs(gen(seed), T, d, 1)
        dy = torch.randn(T, d, generator=gen(seed + 1), device="cuda").to(BF16)
        return s, ds, w, dy, torch.empty_like(s), torch.empty(d, device="cuda")

    def run(c, **kw):
        binding.tpmlp_rmsnorm_add_backward([c[0]], c[2], c[3], 1, [c[4]], c[5], dS_chunks=[c[1]], **kw)
        return c[4], c[5]

    small, big = case(40, 64, 1), case(200, 8192, 3)
    need = lambda c: torch.empty(binding.tpmlp_rmsnorm_add_backward_workspace_size(*c[0].shape, 1), dtype=U8, device="cuda")
    want = [[t.clone() for t in run(c, ws=need(c))] for c in (small, big)]
    check = lambda c, w: all(torch.equal(a, b) for a, b in zip((c[4], c[5]), w))
    streams = [torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    binding._WORKSPACES.clear()
    for st in streams:
        with torch.cuda.stream(st):
            for c, w in ((small, want[0]), (big, want[1]), (small, want[0])):
                for t in (c[4], c[5]):
                    t.zero_()
                run(c)
                st.synchronize()
                assert check(c, w)
    kept = {k: v.data_ptr() for k, v in binding._WORKSPACES.items()}
    assert len(kept) == 3 and len(set(kept.values())) == 3
    # two streams at once, many times over, each with its own
    a, b = case(300, 1024, 5), case(300, 1024, 7)
    wa, wb = [[t.clone() for t in run(c)] for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, st in ((a, streams[1]), (b, streams[2])):
            with torch.cuda.stream(st):
                run(c)
    torch.cuda.synchronize()
    assert check(a, wa) and check(b, wb)
    before = dict(binding._WORKSPACES)
    run(a, stream=streams[1])                       # an explicit stream, as an object and as a handle
    run(b, stream=streams[2].cuda_stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(small)
    assert {k: v.data_ptr() for k, v in binding._WORKSPACES.items()} == {k: v.data_ptr() for k, v in before.items()}
    torch.cuda.synchronize()
    assert check(a, wa) and check(b, wb)
    small[4].zero_()
    with torch.cuda.stream(streams[2]):             # the graph beside eager calls on the stream it was not captured on
        graph.replay()
    run(big)
    torch.cuda.synchronize()
    assert check(small, want[0]) and check(big, want[1])
