"""How the block-scaled FP8 calls behave on the GPU beside other calls: several host threads on one stream, explicit
streams, operands in other places."""
import threading

import pytest
import torch

from tensor_transformer_mlp_tp_gb300 import binding

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def case(T, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s, ds, dy = (torch.randn(T, d, generator=g, device="cuda").to(BF16) for _ in range(3))
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF16)
    return s, ds, dy, w, torch.empty_like(s), torch.empty(d, device="cuda")


def run(c, **kw):
    binding.tpmlp_rmsnorm_add_backward([c[0]], c[3], c[2], 1, [c[4]], c[5], dS_chunks=[c[1]], **kw)


def own_workspace(c):
    return torch.empty(binding.tpmlp_rmsnorm_add_backward_workspace_size(*c[0].shape, 1), dtype=U8, device="cuda")


def test_norm_backwards_of_several_threads_on_one_stream():
    """No workspace given: each call's dweight is its own, bit for bit, however the threads' calls come in between."""
    cases = [case(T, d, 60 + i) for i, (T, d) in enumerate([(300, 1024), (320, 1024), (2, 1024), (64, 512)])]
    want = []
    for c in cases:
        run(c, ws=own_workspace(c))
        want.append((c[4].clone(), c[5].clone()))
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(c, w):
        try:
            for i in range(300):
                run(c)
                if i % 20 == 19:  # its own outputs, in the stream's order
                    if not (torch.equal(c[4], w[0]) and torch.equal(c[5], w[1])):
                        wrong.append(tuple(c[0].shape))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors and not wrong


def test_workspace_of_an_explicit_stream_is_that_streams_memory():
    """A block that the current stream has just freed, its work perhaps still queued, is not the workspace of a call on
    another stream; the stream given as an object, as a handle, and as the default stream's handle."""
    n = 5 << 20
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for cur, stream in ((torch.cuda.default_stream(), side), (torch.cuda.default_stream(), other.cuda_stream), (side, 0)):
        with torch.cuda.stream(cur):
            t = torch.empty(n, dtype=U8, device="cuda")
            freed = t.data_ptr()
            del t
            assert torch.empty(n, dtype=U8, device="cuda").data_ptr() == freed  # what the current stream would be given
            ws = binding._stream_workspace(n, torch.cuda.current_device(), stream)
            assert ws.data_ptr() != freed
            del ws
    torch.cuda.synchronize()


@pytest.mark.parametrize("form", ["object", "handle", "default", "legacy", "per-thread"])
def test_norm_backward_on_an_explicit_stream(form):
    c = case(300, 1024, 70)
    run(c, ws=own_workspace(c))
    want = c[4].clone(), c[5].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = {"object": side, "handle": side.cuda_stream, "default": 0, "legacy": 1, "per-thread": 2}[form]
    for t in c[4:]:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(20):
            run(c, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(c[4], want[0]) and torch.equal(c[5], want[1])


def test_norm_backward_captured_with_its_stream_given():
    """The graph keeps its workspace: replays beside eager calls on the captured stream and on another."""
    cases = [case(200, 2048, 71 + i) for i in range(3)]
    want = []
    for c in cases:
        run(c, ws=own_workspace(c))
        want.append((c[4].clone(), c[5].clone()))
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(cases[0], stream=side)
    for c in cases:
        c[4].zero_()
        c[5].zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        graph.replay()
        run(cases[1], stream=side)
        run(cases[2])
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c[4], w[0]) and torch.equal(c[5], w[1])


def test_a_step_over_no_tokens_leaves_the_gradients_alone():
    """Quantiser, products and norm backward of an empty batch in a row, as a step of a rank without tokens makes them."""
    d, F = 64, 128
    e = lambda *s, dt=U8: torch.empty(*s, dtype=dt, device="cuda")
    sc = lambda r, c, b=1: e(*binding.block_scales_shape(r, c, b), dt=F32)
    w, X, dH = torch.ones(d, dtype=BF16, device="cuda"), e(0, d, dt=BF16), e(0, F, dt=BF16)
    dA, dw = torch.full((d, F), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
    XT, xs, HT, hs = e(d, 0), sc(d, 0), e(F, 0), sc(F, 0)
    binding.tpmlp_rmsnorm_add_gather([X], w, 1, Xq=e(0, d), x_scales=sc(0, d))
    binding.tpmlp_quantize_block(X, 1, 0, qT=XT, scalesT=xs)
    binding.tpmlp_quantize_block(dH, 1, 1, qT=HT, scalesT=hs)
    binding.tpmlp_gemm_fp8_block(XT, xs, HT, hs, dA, b_block_rows=1, b_fmt=1)
    binding.tpmlp_rmsnorm_add_backward([X], w, X, 1, [X], dw)
    assert (dA == 7).all() and (dw == 7).all()
    assert binding.tpmlp_get_device_status() == (binding.OK, 0)


@pytest.mark.parametrize("form", ["object", "handle", "default", "legacy", "per-thread"])
def test_layernorm_backward_on_an_explicit_stream(form):
    """The other calls' workspaces: the same bits on a stream that is not the current one, whose memory it is."""
    T, d, N = 512, 1024, 4
    g = torch.Generator(device="cuda").manual_seed(80)
    x, dy = (torch.randn(T, d, generator=g, device="cuda").to(BF16) for _ in range(2))
    gamma = torch.ones(d, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()
    stream = {"object": side, "handle": side.cuda_stream, "default": 0, "legacy": 1, "per-thread": 2}[form]
    outs = []
    for s in (None, stream):
        dx, dg, db = torch.zeros_like(x), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            binding.tpmlp_layernorm_backward(list(x.split(T // N)), gamma, dy, N, list(dx.split(T // N)), dg, db, stream=s)
            assert s is None or torch.empty(1 << 22, dtype=U8, device="cuda").fill_(255).sum() > 0  # what it may be given
        torch.cuda.synchronize()
        outs.append((dx, dg, db))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
