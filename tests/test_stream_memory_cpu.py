"""Calls with stream=: what they allocate comes from that stream's memory (a
block of the current stream's may still be in use there by an earlier call that
freed it), and outputs are kept for the current stream, on which they are read.
Checked on the host: the library is replaced by one that launches nothing and
torch.cuda by a record of the streams."""
import contextlib
import types

import pytest
import torch

import weight_only_quantized_topk_amd as wq
from weight_only_quantized_topk_amd import ops

HERE, SIDE = 64, 128  # stream handles


class Tensor(torch.Tensor):
    def record_stream(self, s):
        Book.kept.append((self.data_ptr(), s.cuda_stream))


class Book:
    current = HERE
    made = {}   # address -> the stream whose memory it was taken from
    kept = []   # (address, stream it is kept for)


def make(fn):
    def f(*a, **k):
        t = fn(*a, **k).as_subclass(Tensor)
        Book.made[t.data_ptr()] = Book.current
        return t
    return f


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@contextlib.contextmanager
def on(s):
    was, Book.current = Book.current, s.cuda_stream
    try:
        yield
    finally:
        Book.current = was


def external(handle):
    """As torch's: for handle 0 (the default stream) it makes some other stream."""
    return Stream(handle or 999)


class FakeTorch:
    empty, empty_like = staticmethod(make(torch.empty)), staticmethod(make(torch.empty_like))
    cuda = types.SimpleNamespace(stream=on, ExternalStream=external, default_stream=lambda: Stream(0),
                                 current_stream=lambda: Stream(Book.current))
    _C = types.SimpleNamespace(_cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda d: Book.current)

    def __getattr__(self, name):
        return getattr(torch, name)


class FakeLib:
    """Sizes by the real library; calls are noted with the addresses they pass, and launch nothing."""
    def __init__(self, real, calls):
        self.real, self.calls = real, calls

    def __getattr__(self, name):
        fn = getattr(self.real, name)
        if name.endswith(("_bytes", "_capacity")):
            return fn

        def call(*a):
            self.calls.append((name, a))
            return wq.WQ_OK
        call.__name__ = name
        return call


@pytest.fixture
def calls(monkeypatch):
    real, noted = wq.load(), []
    fake = FakeTorch()
    Book.current, Book.made, Book.kept = HERE, {}, []
    monkeypatch.setattr(ops, "_torch", lambda: fake)
    monkeypatch.setattr(ops, "load", lambda: FakeLib(real, noted))
    return noted


BF, I32 = torch.bfloat16, torch.int32
X = torch.zeros((4, 64), dtype=BF)
LORA = wq.Lora(torch.zeros(4, dtype=I32), torch.zeros((2, 8, 64), dtype=BF), torch.zeros((2, 32, 8), dtype=BF), None)
LOGITS = torch.zeros((4, 8))
JOBS = {
    "rms_norm": lambda s: wq.rms_norm(X, residual=X, quant="row", stream=s),
    "moe_route_grouped": lambda s: wq.moe_route_grouped(LOGITS, 2, stream=s),
    "moe_route_grouped_align": lambda s: wq.moe_route_grouped_align(LOGITS, 2, 16, stream=s),
    "moe_route": lambda s: wq.moe_route(LOGITS, 2, stream=s),
    "moe_align": lambda s: wq.moe_align(torch.zeros((4, 2), dtype=I32), 8, 16, stream=s),
    "dense_lora_gemm": lambda s: wq.dense_lora_gemm(X, *LORA, torch.zeros((4, 32), dtype=BF), stream=s),
    "dense_w8a16_gemm": lambda s: wq.dense_w8a16_gemm(X, 32, X, X, lora=LORA, stream=s),
    "sparse24_w4a16_gemm": lambda s: wq.sparse24_w4a16_gemm(X.half(), X, X, X, 32, stream=s),
    "quantize_w8": lambda s: wq.quantize_w8(X, stream=s),
}


def flat(out):
    return [t for t in (out if isinstance(out, (tuple, list)) else [out]) if t is not None]


@pytest.mark.parametrize("name", JOBS)
def test_memory_of_the_calls_stream(calls, name):
    got = flat(JOBS[name](SIDE))
    assert Book.made and set(Book.made.values()) == {SIDE}
    assert all(a[-1] == SIDE for _, a in calls) and calls
    # every output allocated here is kept for the stream that reads it (views of one allocation by their first)
    for t in got:
        if t.data_ptr() in Book.made:
            assert (t.data_ptr(), HERE) in Book.kept
    assert all(s == HERE for _, s in Book.kept)


@pytest.mark.parametrize("name", JOBS)
def test_memory_of_the_default_stream(calls, name):
    """Handle 0, with another stream current."""
    JOBS[name](0)
    assert Book.made and set(Book.made.values()) == {0}
    assert all(a[-1] == 0 for _, a in calls)


@pytest.mark.parametrize("name", JOBS)
@pytest.mark.parametrize("stream", [None, HERE])
def test_current_stream(calls, name, stream):
    JOBS[name](stream)
    assert Book.made and set(Book.made.values()) == {HERE} and not Book.kept
    assert all(a[-1] == HERE for _, a in calls)


def test_a_copy_runs_on_the_calls_stream(calls, monkeypatch):
    """quantize_w8 of a strided weight: the contiguous copy is work of the call, too."""
    class Weight(Tensor):
        def contiguous(self):
            Book.made["copy"] = Book.current
            return torch.zeros(self.shape, dtype=self.dtype)
    wq.quantize_w8(torch.zeros((4, 64), dtype=BF).as_subclass(Weight), stream=SIDE)
    assert Book.made["copy"] == SIDE


def test_fused_layers(calls, monkeypatch):
    """A layer call's own runner is made on the call's stream; what is returned is kept for the current one."""
    p8 = types.SimpleNamespace(act=BF, k_perm1=None, bits=8, E=8, K=64, N=32)
    seen = []

    class Runner:
        def __init__(self, *a, **k):
            seen.append(Book.current)
            self.out, self.h = FakeTorch.empty(4), FakeTorch.empty(4)

        def __call__(self, x, logits, stream=None):
            seen.append(stream)
            return self.out

        def aux(self):
            return {"h": self.h, "block_size": 16, "y": None}

    from weight_only_quantized_topk_amd import layer
    monkeypatch.setattr(layer, "MoERunner", Runner)
    monkeypatch.setattr(layer, "Fp8MoERunner", Runner)
    for fn in (wq.fused_moe, wq.fused_moe_fp8):
        seen.clear(), Book.kept.clear()
        out, aux = fn(X, LOGITS, p8, 2, stream=SIDE, keep=True)
        assert seen == [SIDE, SIDE]
        assert set(Book.kept) == {(out.data_ptr(), HERE), (aux["h"].data_ptr(), HERE)}
        seen.clear(), Book.kept.clear()
        fn(X, LOGITS, p8, 2)
        assert seen == [HERE, None] and not Book.kept
