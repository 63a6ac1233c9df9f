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
