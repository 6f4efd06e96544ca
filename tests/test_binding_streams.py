"""The binding's own tensors on a caller's stream, without a GPU: the library, the allocator and the streams are stand-ins that
record what happens.

A call that is given `stream=` and no workspace or output makes them itself. They have to come from that stream's pool: memory of
the current stream's pool may be handed out again, to work that does not wait for the call's kernels, as soon as the binding
drops it."""

import contextlib

import pytest
import torch

from quantised_kv_cache_gb300 import tq


class Stream:
    def __init__(self, name):
        self.name, self.cuda_stream, self.device_index = name, 7, 0
        self.device = torch.device("cuda", 0)


CURRENT, OTHER = Stream("current"), Stream("other")


class Tensor:
    """What the binding asks of a tensor."""

    def __init__(self, shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.device, self.is_cuda = tuple(shape), dtype, torch.device("cuda", 0), True
        self.seen_by = []

    def stride(self):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x1000

    def is_contiguous(self):
        return True

    def record_stream(self, stream):
        self.seen_by.append(stream)


class Library:
    def __getattr__(self, name):
        def call(*args):
            if name.endswith(("workspace", "workspace_size")):
                args[-1]._obj.value = 4096
            return 0
        return call


class Cache:
    def __init__(self):
        self.batch, self.heads_kv, self.capacity, self.device_index, self.device = 2, 4, 128, 0, torch.device("cuda", 0)
        self.struct = tq.tq_cache()
        self.struct.batch, self.struct.heads_kv, self.struct.capacity = 2, 4, 128


@pytest.fixture()
def made(monkeypatch):
    """[(tensor, the stream it was made on)]"""
    on, out = [CURRENT], []

    @contextlib.contextmanager
    def enter(stream):
        on.append(stream)
        yield
        on.pop()

    def empty(*shape, dtype=torch.bfloat16, device=None):
        shape = shape[0] if len(shape) == 1 and isinstance(shape[0], (tuple, list)) else shape
        out.append((Tensor(shape, dtype), on[-1]))
        return out[-1][0]

    monkeypatch.setattr(tq, "_lib", Library())
    monkeypatch.setattr(torch, "empty_like", lambda x: empty(x.shape, dtype=x.dtype))
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: on[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: on[-1].cuda_stream, raising=False)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: real(*a, **kw) if a == ((),) else empty(*a, **kw))
    return out


F32, I32 = torch.float32, torch.int32
B, H, LENS = 2, 4, Tensor((2,), torch.int32)
Q3, KV = Tensor((B, 8, 128)), Tensor((B, H, 1, 128))
CALLS = {
    "rotary": (1, lambda s: tq.tq_rotary(1, Tensor((B, H, 3, 128)), Tensor((B, 3), I32), stream=s)),
    "attention": (2, lambda s: tq.tq_q8_attention(1, Cache(), Tensor((B, 8, 3, 128)), LENS, 128, stream=s)),
    "attention with weights": (2, lambda s: tq.tq_q8_attention(1, Cache(), Tensor((B, 8, 3, 128)), LENS, 128, weights=Tensor((B, H, 128), F32), stream=s)),
    "eviction": (4, lambda s: tq.tq_q8_evict(1, Cache(), Cache(), LENS, Tensor((B, H, 128), F32), 64, stream=s)),
    "decode": (2, lambda s: tq.tq_decode_attention(1, Cache(), Q3, LENS, 128, stream=s)),
    "decode without a workspace": (1, lambda s: tq.tq_decode_attention_static(1, Cache(), Q3, LENS, 128, stream=s)),
    "step": (2, lambda s: tq.tq_decode_step(1, Cache(), Q3, KV, KV, LENS, 128, stream=s)),
    "dequantise": (2, lambda s: tq.tq_dequantize(1, Cache(), 0, 128, stream=s)),
}


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_makes_belongs_to_its_stream(made, name):
    count, call = CALLS[name]
    got = call(OTHER)
    assert len(made) == count
    assert all(stream is OTHER for _, stream in made)
    # results are also the caller's: they are not handed out again before the current stream is done with them
    for t in got if isinstance(got, tuple) else (got,):
        assert CURRENT in t.seen_by


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_nothing_changes(made, name):
    count, call = CALLS[name]
    call(None)
    assert len(made) == count
    assert all(stream is CURRENT and not t.seen_by for t, stream in made)
