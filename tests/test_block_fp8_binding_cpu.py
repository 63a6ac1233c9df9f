"""The Python side of the block-scaled FP8 calls without a GPU: stand-ins for device tensors and for the library, so that
nothing reaches CUDA whatever gets past the checks."""
import math
import threading
import time

import pytest
import torch

from tensor_transformer_mlp_tp_gb300 import binding

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
DEV = 0


class Fake:
    """What the binding asks of a tensor, for a tensor of device `dev` (-1: the host)."""

    def __init__(self, *shape, dtype=BF16, dev=DEV, ptr=1 << 20, stride=None):
        self.shape, self.dtype, self._dev, self._ptr = torch.Size(shape), dtype, dev, ptr
        self._stride = stride or tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))
        self._plain = stride is None

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def is_contiguous(self):
        return self._plain

    def stride(self):
        return self._stride

    def get_device(self):
        return self._dev

    def data_ptr(self):
        return self._ptr


class Library:
    """Records the calls of the five entry points."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith(("workspace_size", "status_string")):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return binding.OK
        return call


@pytest.fixture
def library(monkeypatch):
    from tensor_transformer_mlp_tp_gb300 import build

    build.build()
    fake = Library()
    fake.real = binding.lib()
    monkeypatch.setattr(binding, "_lib", fake)
    monkeypatch.setattr(binding, "_current_device", lambda: DEV)
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(binding, "_current_stream", lambda dev: (0, 0, 0))
    monkeypatch.setattr(binding, "_capturing", lambda: False)
    binding.tpmlp_rmsnorm_add_backward_workspace_size.cache_clear()
    return fake


def backward(**kw):
    a = dict(S=Fake(64, 256), w=Fake(256), dXg=Fake(64, 256), dX=Fake(64, 256), dw=Fake(256, dtype=F32), dS=Fake(64, 256),
             ws=Fake(1 << 20, dtype=U8))
    a.update(kw)
    binding.tpmlp_rmsnorm_add_backward([a["S"]], a["w"], a["dXg"], 1, [a["dX"]], a["dw"], dS_chunks=[a["dS"]], ws=a["ws"])


def test_calls_on_one_streams_kept_workspace_do_not_overlap(library, monkeypatch):
    """The backward is two launches; another thread's call on the same stream and workspace between them would have its
    partial sums added up."""
    monkeypatch.setattr(binding, "_WORKSPACES", {(DEV, 0): Fake(1 << 20, dtype=U8, ptr=1 << 24)})
    inside, most, used = [0], [0], set()

    def call(*args):
        inside[0] += 1
        most[0] = max(most[0], inside[0])
        used.add(args[8])
        time.sleep(0.002)  # as ctypes does, without the interpreter's lock
        inside[0] -= 1
        return binding.OK

    library.tpmlp_rmsnorm_add_backward = call
    threads = [threading.Thread(target=lambda: [backward(ws=None) for _ in range(5)]) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert used == {1 << 24} and most[0] == 1
    backward(ws=Fake(1 << 20, dtype=U8, ptr=1 << 25))  # a workspace of the caller's own
    assert used == {1 << 24, 1 << 25}


def test_a_failed_call_leaves_the_kept_workspace_free(library, monkeypatch):
    monkeypatch.setattr(binding, "_WORKSPACES", {(DEV, 0): Fake(1 << 20, dtype=U8, ptr=1 << 24)})
    library.tpmlp_rmsnorm_add_backward = lambda *a: binding.ERR_CUDA
    with pytest.raises(binding.TpMlpError):
        backward(ws=None)
    done = []
    library.tpmlp_rmsnorm_add_backward = lambda *a: done.append(1) or binding.OK
    t = threading.Thread(target=lambda: backward(ws=None))
    t.start()
    t.join(10)
    assert done == [1]


def test_a_fresh_workspace_comes_from_the_stream_that_runs_the_call(library, monkeypatch):
    """Which stream is current where the memory is taken (the allocator's blocks are ordered by their own stream)."""
    current, taken = [None], []

    class Stream:
        def __init__(self, name):
            self.name = name

    class Use:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.before, current[0] = current[0], self.s.name

        def __exit__(self, *a):
            current[0] = self.before

    def empty(n, dtype=None, device=None):
        taken.append((current[0], n))
        return Fake(n, dtype=U8, ptr=1 << 24)

    monkeypatch.setattr(binding.torch.cuda, "Stream", Stream)
    monkeypatch.setattr(binding.torch.cuda, "stream", Use)
    monkeypatch.setattr(binding.torch.cuda, "ExternalStream", lambda h, device: Stream(h))
    monkeypatch.setattr(binding.torch.cuda, "default_stream", lambda device: Stream("default"))
    monkeypatch.setattr(binding.torch, "empty", empty)
    monkeypatch.setattr(Fake, "record_stream", lambda self, s: None, raising=False)
    for stream, want in ((Stream("side"), "side"), (1 << 30, 1 << 30), (0, "default"), (1, "default"), (None, None)):
        taken.clear()
        assert binding._stream_workspace(4096, DEV, stream) is not None
        assert [t[0] for t in taken] == [want] and taken[0][1] >= 4096
    with pytest.raises(binding.TpMlpError):
        binding._stream_workspace(4096, DEV, 2)
