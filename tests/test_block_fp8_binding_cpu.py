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
    current, taken, waits, recorded = [None], [], [], []

    class Stream:
        def __init__(self, name):
            self.name = name

        def wait_stream(self, other):
            waits.append((self.name, other.name))

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
    monkeypatch.setattr(binding.torch.cuda, "current_stream", lambda device: Stream("current"))
    monkeypatch.setattr(Fake, "record_stream", lambda self, s: recorded.append(s.name), raising=False)
    for stream, want in ((Stream("side"), "side"), (1 << 30, 1 << 30), (0, "default"), (1, "default"), (None, None)):
        taken.clear()
        assert binding._stream_workspace(4096, DEV, stream) is not None
        assert [t[0] for t in taken] == [want] and taken[0][1] >= 4096
        taken.clear()  # the other calls' workspaces
        binding.workspace(binding.make_shape(256, 64, 256, 2), binding.OP_FWD, torch.device("cuda", DEV), stream)
        assert [t[0] for t in taken] == [want] and taken[0][1] >= 256 * 256 * 2
    # the per-thread default stream's handle has no pool of its own: the current stream's memory, ordered on both sides
    taken.clear()
    binding._stream_workspace(4096, DEV, 2)
    assert taken == [(None, 4096)] and waits == [(2, "current")] and recorded == [2]


def test_every_call_passes_its_stream_to_its_workspace():
    import inspect
    import re

    n = 0
    for name, f in inspect.getmembers(binding, inspect.isfunction):
        if {"ws", "stream"} <= set(inspect.signature(f).parameters):
            made = re.findall(r"ws = (?:_scratch|workspace|_stream_workspace|torch\.empty)\([^=]*?stream\)", inspect.getsource(f))
            assert len(made) == 1 and "torch.empty" not in made[0], name
            n += 1
    assert n >= 16


def gather(**kw):
    a = dict(X=Fake(4, 64), R=Fake(4, 64), S=Fake(4, 64), X2=Fake(4, 64), w=Fake(64), Xg=Fake(8, 64), Xq=Fake(8, 64, dtype=U8),
             xs=Fake(1, 128, dtype=F32))
    a.update(kw)
    binding.tpmlp_rmsnorm_add_gather([a["X"], a["X2"]], a["w"], 2, R_chunks=[a["R"], a["R"]], S_chunks=[a["S"], a["S"]],
                                     Xg=a["Xg"], Xq=a["Xq"], x_scales=a["xs"])


def quantize(**kw):
    a = dict(src=Fake(40, 64), q=Fake(40, 64, dtype=U8), s=Fake(1, 128, dtype=F32), qT=Fake(64, 48, dtype=U8),
             sT=Fake(1, 128, dtype=F32))
    a.update(kw)
    binding.tpmlp_quantize_block(a["src"], 1, 0, q=a["q"], scales=a["s"], qT=a["qT"], scalesT=a["sT"])


def gemm(**kw):
    a = dict(A=Fake(5, 64, dtype=U8), sa=Fake(1, 128, dtype=F32), B=Fake(16, 64, dtype=U8), sb=Fake(1, 1, dtype=F32),
             C=Fake(5, 16), bias=Fake(16), a_fmt=0, b_fmt=0)
    a.update(kw)
    binding.tpmlp_gemm_fp8_block(a["A"], a["sa"], a["B"], a["sb"], a["C"], bias=a["bias"], a_fmt=a["a_fmt"], b_fmt=a["b_fmt"])


def gemm1(**kw):
    a = dict(X=Fake(5, 64, dtype=U8), sx=Fake(1, 128, dtype=F32), A=Fake(16, 64, dtype=U8), sa=Fake(1, 1, dtype=F32),
             bias=Fake(16), H=Fake(5, 16, dtype=U8), sh=Fake(1, 128, dtype=F32), pre=Fake(5, 16))
    a.update(kw)
    binding.tpmlp_gemm1_fp8_block(a["X"], a["sx"], a["A"], a["sa"], a["bias"], 1, a["H"], a["sh"], Hpre=a["pre"])


OPERANDS = {gather: dict(X=(4, 64), X2=(4, 64), R=(4, 64), S=(4, 64), w=(64,), Xg=(8, 64), Xq=(8, 64, U8), xs=(1, 128, F32)),
            backward: dict(S=(64, 256), w=(256,), dXg=(64, 256), dX=(64, 256), dw=(256, F32), dS=(64, 256), ws=(1 << 20, U8)),
            quantize: dict(src=(40, 64), q=(40, 64, U8), s=(1, 128, F32), qT=(64, 48, U8), sT=(1, 128, F32)),
            gemm: dict(A=(5, 64, U8), sa=(1, 128, F32), B=(16, 64, U8), sb=(1, 1, F32), C=(5, 16), bias=(16,)),
            gemm1: dict(X=(5, 64, U8), sx=(1, 128, F32), A=(16, 64, U8), sa=(1, 1, F32), bias=(16,), H=(5, 16, U8),
                        sh=(1, 128, F32), pre=(5, 16))}


def fake(spec, **kw):
    dtype = spec[-1] if isinstance(spec[-1], torch.dtype) else BF16
    return Fake(*[n for n in spec if isinstance(n, int)], dtype=dtype, **kw)


@pytest.mark.parametrize("call,name", [(c, n) for c in OPERANDS for n in OPERANDS[c]],
                         ids=lambda v: v if isinstance(v, str) else v.__name__)
@pytest.mark.parametrize("dev", [-1, 1])
def test_each_operand_elsewhere_is_refused(library, call, name, dev):
    """One operand of the host or of another device among operands of this one: the library is not called."""
    call(**{name: fake(OPERANDS[call][name])})
    assert len(library.calls) == 1
    with pytest.raises(binding.TpMlpError) as e:
        call(**{name: fake(OPERANDS[call][name], dev=dev)})
    assert e.value.status == binding.ERR_INVALID_ARG and len(library.calls) == 1


E4M3T, E5M2T, OTHER = torch.float8_e4m3fn, torch.float8_e5m2, (torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.int8, torch.bool)
CODES = [(gather, "Xq", (8, 64)), (gemm, "A", (5, 64)), (gemm, "B", (16, 64)), (gemm1, "X", (5, 64)), (gemm1, "A", (16, 64)),
         (gemm1, "H", (5, 16)), (quantize, "q", (40, 64)), (quantize, "qT", (64, 48))]


@pytest.mark.parametrize("call,name,shape", CODES, ids=lambda v: getattr(v, "__name__", str(v)))
def test_codes_of_another_format_are_refused(library, call, name, shape):
    """Bytes pass as what the call's format says they are; a float8 type has to be that format's."""
    call(**{name: Fake(*shape, dtype=U8)})
    call(**{name: Fake(*shape, dtype=E4M3T)})
    assert len(library.calls) == 2
    for dtype in (E5M2T,) + OTHER:
        with pytest.raises(binding.TpMlpError) as e:
            call(**{name: Fake(*shape, dtype=dtype)})
        assert e.value.status == binding.ERR_INVALID_ARG
    assert len(library.calls) == 2


def test_products_take_the_format_that_they_are_told(library):
    gemm(A=Fake(5, 64, dtype=E5M2T), a_fmt=1)
    gemm(B=Fake(16, 64, dtype=E5M2T), b_fmt=1)
    assert len(library.calls) == 2
    for kw in (dict(A=Fake(5, 64, dtype=E4M3T), a_fmt=1), dict(B=Fake(16, 64, dtype=E4M3T), b_fmt=1)):
        with pytest.raises(binding.TpMlpError):
            gemm(**kw)
    assert len(library.calls) == 2


def test_a_weight_gradient_over_no_tokens_is_an_empty_call(library):
    """As every empty batch: nothing is launched and the output is left alone; what is wrong besides is still refused."""
    kw = dict(A=Fake(5, 0, dtype=U8), sa=Fake(0, 128, dtype=F32), B=Fake(16, 0, dtype=U8), sb=Fake(0, 1, dtype=F32), bias=None)
    gemm(**kw)
    assert library.calls == []
    for wrong in (dict(B=Fake(16, 32, dtype=U8)), dict(C=Fake(5, 24)), dict(A=Fake(5, 0, dtype=U8, dev=-1)), dict(sb=Fake(0, 1))):
        with pytest.raises(binding.TpMlpError):
            gemm(**{**kw, **wrong})
