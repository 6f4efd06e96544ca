"""The binding's checks of where tensors lie, without a GPU (the library and the tensors are stand-ins): what would reach a kernel as
an address of another device, or as more memory than there is, is refused."""

import pytest
import torch

from quantised_kv_cache_gb300 import tq
from test_binding_streams import OTHER, Cache, Library, Stream, Tensor

F32, I32 = torch.float32, torch.int32
B, H = 2, 4


def lens():
    return Tensor((B,), I32)


@pytest.fixture(autouse=True)
def _no_gpu(monkeypatch):
    monkeypatch.setattr(tq, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 7, raising=False)


def on(tensor, index):
    tensor.get_device = lambda: index
    return tensor


def strided(tensor):
    tensor.is_contiguous = lambda: False
    return tensor


def attend(**kw):
    q = Tensor((B, 8, 3, 128))
    return tq.tq_q8_attention(1, Cache(), q, lens(), 128, out=Tensor(q.shape), **kw)


def test_a_workspace_elsewhere_or_with_gaps_is_refused():
    attend(workspace=Tensor((4096,), torch.uint8))
    for bad in (on(Tensor((4096,), torch.uint8), -1), on(Tensor((4096,), torch.uint8), 1), strided(Tensor((4096,), torch.uint8))):
        with pytest.raises(ValueError):
            attend(workspace=bad)


def calls(index):
    """The four calls with everything on device `index`."""
    def t(*a):
        return on(Tensor(*a), index)

    def cache():
        c = Cache()
        c.device_index = index
        return c

    x, at = (B, H, 3, 128), (B, H, 128)
    return [
        lambda s: tq.tq_rotary(1, t(x), t((B, 3), I32), out=t(x), stream=s),
        lambda s: tq.tq_q8_append(1, cache(), t(x), t(x), t((B,), I32), stream=s),
        lambda s: tq.tq_q8_attention(1, cache(), t((B, 8, 3, 128)), t((B,), I32), 128, out=t((B, 8, 3, 128)), workspace=t((4096,), torch.uint8), stream=s),
        lambda s: tq.tq_q8_evict(1, cache(), cache(), t((B,), I32), t(at, F32), 64, kept=t((B, H, 64), I32), dst_lens=t((B,), I32),
                                 dst_weights=t(at, F32), dst_positions=t(at, I32), stream=s),
    ]


@pytest.mark.parametrize("i", range(4))
def test_another_device_than_the_current_one_is_refused(i, monkeypatch):
    calls(0)[i](None)
    calls(0)[i](OTHER)
    with pytest.raises(ValueError):
        calls(1)[i](None)
    far = Stream("far")
    far.device_index = 1
    with pytest.raises(ValueError):
        calls(0)[i](far)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        calls(0)[i](None)
