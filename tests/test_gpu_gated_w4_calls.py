"""The gated block and the 4-bit products beside other calls: one after the other as a layer runs them, on explicit
streams, in captured graphs, from several threads, with values that are not finite, past 2^31 elements."""
import threading

import pytest
import torch

import gated_util as gated
import oracle
import w4_util as w4
from gpu_util import Guarded
from tensor_transformer_mlp_tp_gb300 import binding

pytestmark = pytest.mark.gpu
BF16, F64, U8 = torch.bfloat16, torch.float64, torch.uint8
SILU, GELU = binding.ACT_SILU, binding.ACT_GELU


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    st, site = binding.tpmlp_get_device_status()
    assert st == binding.OK, f"device status {binding.status_string(st)} (wait site {site})"


def normal(g, *shape, sigma=1.0):
    return (sigma * torch.randn(*shape, generator=g, device="cuda")).to(BF16)


def pack(W, group, zeros=True):
    K, N = W.shape
    G = binding.w4_groups(K, group)
    Q = torch.empty(binding.w4_codes_shape(K, N), dtype=U8, device="cuda")
    s = torch.empty(G, N, dtype=BF16, device="cuda")
    z = torch.empty(G, N, dtype=U8, device="cuda") if zeros else None
    binding.tpmlp_quantize_w4(W, group, Q, s, zeros=z)
    return Q, s, z


def values(m, K, N, group):
    return w4.values(w4.unpack(m[0], K, N)[:K, :N], m[1], m[2], group)


class Layer:
    """A gated layer in bf16 and in 4 bits, its inputs and outputs."""

    def __init__(self, T, d, F, seed, group=64):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.d, self.F, self.group = T, d, F, group
        self.X, self.dY = normal(g, T, d), normal(g, T, d, sigma=0.1)
        self.Ag, self.Au, self.B = (normal(g, d, F, sigma=d ** -0.5), normal(g, d, F, sigma=d ** -0.5), normal(g, F, d, sigma=F ** -0.5))
        self.q = [pack(w, group) for w in (self.Ag, self.Au, self.B)]
        self.out = {k: torch.empty(s, dtype=BF16, device="cuda") for k, s in
                    dict(Y=(T, d), G=(T, F), U=(T, F), dX=(T, d), dAg=(d, F), dAu=(d, F), dB=(F, d), dbg=(F,), dbu=(F,), H4=(T, F),
                         Y4=(T, d), W4=(d, F)).items()}

    def run(self, stream=None):
        o, (g4, u4, b4) = self.out, self.q
        binding.tpmlp_gated_forward(self.X, self.Ag, self.Au, self.B, 1, o["Y"], act=SILU, Gpre_out=o["G"], Upre_out=o["U"], stream=stream)
        binding.tpmlp_gated_backward(self.X, self.Ag, self.Au, self.B, o["G"], o["U"], self.dY, 1, o["dX"], o["dAg"], o["dAu"],
                                     o["dB"], act=SILU, dbg=o["dbg"], dbu=o["dbu"], stream=stream)
        binding.tpmlp_gemm1_gated_w4(self.X, g4[0], g4[1], u4[0], u4[1], self.group, o["H4"], act=SILU, g_zeros=g4[2],
                                     u_zeros=u4[2], stream=stream)
        binding.tpmlp_gemm_w4(o["H4"], b4[0], b4[1], self.group, o["Y4"], zeros=b4[2], stream=stream)
        binding.tpmlp_dequantize_w4(g4[0], g4[1], self.group, o["W4"], zeros=g4[2], stream=stream)

    def bits(self):
        return {k: v.clone() for k, v in self.out.items()}


def same(a, b):
    return [k for k in a if not torch.equal(a[k].view(torch.int16), b[k].view(torch.int16))]


@pytest.mark.parametrize("T", [1, 7, 16, 40, 128])
def test_a_layers_weights_in_four_bits(T):
    """Quantise once; decoded tokens through the gate and up projections and the row-parallel product in 4 bits, as a model
    serves them, against 64-bit values of the same codes; a prompt through the bf16 block on the weights read back gives
    the same up to its own roundings."""
    d, F, group = 512, 1536, 128
    L = Layer(T, d, F, seed=T, group=group)
    L.run()
    wg, wu, wb = (values(m, *s, group) for m, s in zip(L.q, ((d, F), (d, F), (F, d))))
    x = L.X.to(F64)
    G, U = x @ wg, x @ wu
    eg, eu = w4.product_error(x, wg, group), w4.product_error(x, wu, group)
    a = gated.act64(G, SILU)[0]
    err = (gated.SLOPE_MAX * eg + gated.act_error(G)) * (U.abs() + eu) + a.abs() * eu
    gated.check("H", L.out["H4"], (a * U, err + gated.HALF * ((a * U).abs() + err) + gated.TINY))
    h = L.out["H4"].to(F64)
    y, e = h @ wb, w4.product_error(h, wb, group)
    gated.check("Y", L.out["Y4"], (y, e + gated.HALF * (y.abs() + e) + gated.TINY))
    back = []
    for (Q, s, z), shape in zip(L.q, ((d, F), (d, F), (F, d))):
        W = torch.empty(shape, dtype=BF16, device="cuda")
        binding.tpmlp_dequantize_w4(Q, s, group, W, zeros=z)
        back.append(W)
    Y = torch.empty(T, d, dtype=BF16, device="cuda")
    binding.tpmlp_gated_forward(L.X, *back, 1, Y, act=SILU)
    # weights read back are rounded once more, half a step each, in both products: norms keep sqrt(3) of it, and H and Y
    # are rounded on both sides
    want = (gated.act64(G, SILU)[0] * U) @ wb
    assert torch.linalg.norm(Y.to(F64) - want) <= 4 * gated.HALF * torch.linalg.norm(want)


def test_gated_region_over_sequence_chunks():
    """LayerNorm of the chunks, both projections, and the row-parallel product stored back into chunks: the sequence-parallel
    region with a gated MLP, made of the steps."""
    T, d, F, N = 256, 128, 512, 4
    g = torch.Generator(device="cuda").manual_seed(2)
    X, gamma, beta = normal(g, T, d), (1 + 0.1 * normal(g, d)), normal(g, d, sigma=0.1)
    Ag, Au, B = normal(g, d, F, sigma=d ** -0.5), normal(g, d, F, sigma=d ** -0.5), normal(g, F, d, sigma=F ** -0.5)
    Xg, H = torch.empty(T, d, dtype=BF16, device="cuda"), torch.empty(T, F, dtype=BF16, device="cuda")
    chunks = [torch.empty(T // N, d, dtype=BF16, device="cuda") for _ in range(N)]
    binding.tpmlp_layernorm_gather(list(X.split(T // N)), gamma, beta, N, Xg)
    binding.tpmlp_gemm1_gated(Xg, Ag, Au, N, H, act=GELU)
    binding.tpmlp_gemm2_shard_accum(H, B, N, Y_chunks=chunks)
    x = X.to(F64)
    ln = torch.as_tensor(oracle.layer_norm(x.cpu().numpy(), gamma.to(F64).cpu().numpy(), beta.to(F64).cpu().numpy(), 1e-5)).cuda()
    want = (gated.act64(ln @ Ag.to(F64), GELU)[0] * (ln @ Au.to(F64))) @ B.to(F64)
    # Xg is rounded (half a step, through both factors) and H, and Y itself
    assert torch.linalg.norm(torch.cat(chunks).to(F64) - want) <= 5 * gated.HALF * torch.linalg.norm(want)


@pytest.mark.parametrize("T", [1, 9, 17, 200])
def test_explicit_streams_and_captured_graphs(T):
    """The same bits on a stream given as an object and as a handle, and from a graph replayed twice, on another stream."""
    L = Layer(T, 256, 384, seed=30 + T)
    L.run()
    torch.cuda.synchronize()
    want = L.bits()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for v in L.out.values():
            v.zero_()
        torch.cuda.synchronize()
        L.run(stream=stream)
        side.synchronize()
        assert not same(L.bits(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run()
    for stream in (torch.cuda.current_stream(), side):
        for v in L.out.values():
            v.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert not same(L.bits(), want)


def test_two_graphs_replayed_at_once():
    """Their workspaces are their own."""
    layers = [Layer(300, 256, 1024, seed=40), Layer(37, 256, 1024, seed=41)]
    graphs, want = [], []
    for L in layers:
        L.run()
        torch.cuda.synchronize()
        want.append(L.bits())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.run()
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for L, w in zip(layers, want):
        assert not same(L.bits(), w)


def test_several_threads_on_one_stream():
    layers = [Layer(T, 128, 256, seed=50 + T) for T in (1, 20, 130, 300)]
    want = []
    for L in layers:
        L.run()
        torch.cuda.synchronize()
        want.append(L.bits())
    wrong, errors = [], []

    def work(L, w):
        try:
            for _ in range(30):
                L.run()
                wrong.extend(same(L.bits(), w))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(layers, want)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors and not wrong


@pytest.mark.parametrize("M", [3, 12, 40])
def test_values_that_are_not_finite_stay_in_their_token(M):
    K, N, group = 512, 272, 64
    g = torch.Generator(device="cuda").manual_seed(M)
    m = pack(normal(g, K, N), group)
    X = normal(g, M, K)
    Y, Z = (torch.empty(M, N, dtype=BF16, device="cuda") for _ in range(2))
    binding.tpmlp_gemm_w4(X, m[0], m[1], group, Y, zeros=m[2])
    X[1, 77], X[2, 400] = float("nan"), float("-inf")
    binding.tpmlp_gemm_w4(X, m[0], m[1], group, Z, zeros=m[2])
    rest = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(Z[rest], Y[rest]) and bool(Z[1].isnan().all())
    w = values(m, K, N, group)[400]
    want = torch.where(w == 0, float("nan"), -torch.sign(w) * float("inf"))
    assert torch.equal(Z[2].to(F64).nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


@pytest.mark.parametrize("M", [5, 16, 33])
@pytest.mark.parametrize("power", [-126, -110, -40, 40, 100])
def test_a_token_times_a_power_of_two(M, power):
    """Its outputs are those times the power, bit by bit; a token of zeros gives zeros."""
    K, N, group = 1032, 136, 128
    g = torch.Generator(device="cuda").manual_seed(M)
    m = pack(normal(g, K, N, sigma=1.0 if power < 0 else 2.0 ** -20), group, zeros=False)
    X = normal(g, M, K)
    X[0] = 0
    X = torch.where(X.abs() < 2.0 ** -4, torch.zeros_like(X), X)  # no value falls below the normal numbers
    Y, Z = (torch.empty(M, N, dtype=BF16, device="cuda") for _ in range(2))
    binding.tpmlp_gemm_w4(X, m[0], m[1], group, Y)
    scaled = (X.to(F64) * 2.0 ** max(power, -122)).to(BF16)
    binding.tpmlp_gemm_w4(scaled, m[0], m[1], group, Z)
    assert bool((Y[0] == 0).all()) and bool((Z[0] == 0).all())
    if M > 8 and power == -126:
        # On the UMMA X is multiplied as it is.  Its values are multiples of 2^-133 here, so sums of products can be subnormal
        # in fp32, where the tensor core may flush: up to 2^-126 for each of the K additions, times the scale.  (At 2^-110
        # every sum is a multiple of 2^-121, and the scaled one has the same bits.)
        w, x = values(m, K, N, group), scaled.to(F64)
        y, e = x @ w, w4.product_error(x, w, group) + K * 2.0 ** -126 * m[1].to(F64).abs().amax(0)
        gated.check("Z", Z, (y, e + gated.HALF * (y.abs() + e) + gated.TINY))
    else:
        assert torch.equal(Z.to(F64), Y.to(F64) * 2.0 ** max(power, -122))


@pytest.mark.parametrize("M", [2, 10])
def test_tokens_with_outlying_channels(M):
    """A value of 2^28 where the weights are zero, beside normal ones: those count as far as they lie within 2^-32 of it.  (Up
    to 8 tokens the values are brought below 2^15 and into fp16, whose least step is 2^-24: a half of it is 2^-39 of a
    largest value that becomes 2^14.)"""
    K, N, group = 256, 64, 32
    g = torch.Generator(device="cuda").manual_seed(4)
    W = normal(g, K, N)
    W[:32] = 0
    m = pack(W, group)
    X = normal(g, M, K)
    X[:, 5] = 2.0 ** 28
    Y = torch.empty(M, N, dtype=BF16, device="cuda")
    binding.tpmlp_gemm_w4(X, m[0], m[1], group, Y, zeros=m[2])
    w = values(m, K, N, group)
    assert bool((w[:32] == 0).all())
    x = X.to(F64)
    y, e = x @ w, w4.product_error(x, w, group) + 2.0 ** -39 * 2.0 ** 28 * w.abs().sum(0)
    gated.check("Y", Y, (y, e + gated.HALF * (y.abs() + e) + gated.TINY))


def test_empty_batches_leave_their_outputs():
    d, F = 64, 128
    L = Layer(1, d, F, seed=1)
    X, H = torch.empty(0, d, dtype=BF16, device="cuda"), torch.empty(0, F, dtype=BF16, device="cuda")
    dA, dB = torch.full((d, F), 7.0, dtype=BF16, device="cuda"), torch.full((F, d), 7.0, dtype=BF16, device="cuda")
    binding.tpmlp_gated_forward(X, L.Ag, L.Au, L.B, 1, X)
    binding.tpmlp_gated_backward(X, L.Ag, L.Au, L.B, H, H, X, 1, X, dA, dA, dB)
    binding.tpmlp_gemm1_gated_w4(X, L.q[0][0], L.q[0][1], L.q[1][0], L.q[1][1], L.group, H, g_zeros=L.q[0][2], u_zeros=L.q[1][2])
    binding.tpmlp_gemm_w4(X, L.q[0][0], L.q[0][1], L.group, H, zeros=L.q[0][2])
    torch.cuda.synchronize()
    assert bool((dA == 7).all()) and bool((dB == 7).all())


def test_results_do_not_change_from_run_to_run():
    for T in (1, 30, 320):
        L = Layer(T, 512, 1024, seed=T)
        L.run()
        first = L.bits()
        for _ in range(3):
            L.run()
            assert not same(L.bits(), first)


# ----------------------------------------------------------------------------- past 2^31 elements

def test_gated_block_past_2_31_elements():
    T, d, F = 131328, 64, 16448
    g = torch.Generator(device="cuda").manual_seed(6)
    X, dY = normal(g, T, d), normal(g, T, d, sigma=0.1)
    Ag, Au, B = normal(g, d, F, sigma=0.1), normal(g, d, F, sigma=0.1), normal(g, F, d, sigma=0.01)
    Y = Guarded((T, d))
    G, U, H = (torch.empty(T, F, dtype=BF16, device="cuda") for _ in range(3))
    binding.tpmlp_gated_forward(X, Ag, Au, B, 1, Y.t, Gpre_out=G, Upre_out=U, H_out=H)
    dG, dU = torch.empty_like(G), torch.empty_like(G)
    binding.tpmlp_gemm_dh_gated(dY, B, G, U, 1, dG, dU)
    dX = Guarded((T, d))
    binding.tpmlp_gemm_dx_gated(dG, dU, Ag, Au, 1, dX.t)
    rows = torch.tensor([0, 1, 65537, 130560, 130561, T - 129, T - 1], device="cuda")  # offsets on both sides of 2^31
    x, dy = X[rows].to(F64), dY[rows].to(F64)
    want = gated.forward(x, Ag.to(F64), Au.to(F64), None, None, SILU)
    for name, t in (("G", G), ("U", U), ("H", H)):
        gated.check(name, t[rows], want[name])
    gated.check("Y", Y.t[rows], gated.product((H[rows].to(F64), B.to(F64))))
    want = gated.derivatives(dy, B.to(F64), G[rows].to(F64), U[rows].to(F64), SILU)
    for name, t in (("dG", dG), ("dU", dU)):
        gated.check(name, t[rows], want[name])
    gated.check("dX", dX.t[rows], gated.product((dG[rows].to(F64), Ag.to(F64).t()), (dU[rows].to(F64), Au.to(F64).t())))
    assert Y.intact() and dX.intact()


def test_4_bit_weights_past_2_31_elements():
    K, N, group = 16384, 139272, 64
    g = torch.Generator(device="cuda").manual_seed(8)
    W = torch.empty(K, N, dtype=BF16, device="cuda")
    for k in range(0, K, 1024):
        W[k:k + 1024] = normal(g, 1024, N, sigma=0.01)
    m = pack(W, group)
    cols = torch.tensor([0, 9, 131071, 131072, 131080, N - 1], device="cuda")
    codes, s, z = w4.quantize(W[:, cols].contiguous(), group, True)
    assert torch.equal(m[1][:, cols], s) and torch.equal(m[2][:, cols], z)
    w = w4.values(codes, s, z, group)
    back = torch.empty_like(W)
    binding.tpmlp_dequantize_w4(m[0], m[1], group, back, zeros=m[2])
    assert torch.equal(back[:, cols], w.to(BF16))
    del back, W
    for M in (1, 3, 40):
        X = normal(g, M, K)
        Y = Guarded((M, N))
        binding.tpmlp_gemm_w4(X, m[0], m[1], group, Y.t, zeros=m[2])
        x = X.to(F64)
        y, e = x @ w, w4.product_error(x, w, group)
        gated.check(f"Y {M}", Y.t[:, cols], (y, e + gated.HALF * (y.abs() + e) + gated.TINY))
        assert Y.intact()


def test_products_wider_and_longer_than_a_staged_row():
    """X that the kernel for few tokens has no room for, a single group, and more tokens than a block of the grid holds."""
    for M, K, N, group in ((1, 210000, 16, 128), (8, 40000, 24, 32), (16, 20000, 40, 64), (3, 32, 16, 32), (700, 64, 8, 64)):
        g = torch.Generator(device="cuda").manual_seed(K)
        m = pack(normal(g, K, N, sigma=K ** -0.5), group)
        X, Y = normal(g, M, K), Guarded((M, N))
        binding.tpmlp_gemm_w4(X, m[0], m[1], group, Y.t, zeros=m[2])
        w, x = values(m, K, N, group), X.to(F64)
        y, e = x @ w, w4.product_error(x, w, group)
        gated.check(f"{M} {K}", Y.t, (y, e + gated.HALF * (y.abs() + e) + gated.TINY))
        assert Y.intact()
