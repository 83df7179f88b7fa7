"""What the dense layers do on the host around their C calls, on stand-ins for tensors and streams (CPU only)."""
import contextlib
import gc
import weakref

import pytest
import torch

from block_sparse_spherical_b200 import abi, api

DEV = torch.device("cuda", 0)
SHAPE, KV, STREAM = (1, 2, 8, 64), (1, 2, 16, 64), "the current stream"


class Stand:
    """Looks like a contiguous CUDA tensor to a layer; notes the streams it was recorded on."""

    def __init__(self, shape, address, dtype=torch.bfloat16):
        self.shape, self.address, self.dtype, self.device = torch.Size(shape), address, dtype, DEV
        self.streams = []

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.address

    def record_stream(self, stream):
        self.streams.append(stream)


@pytest.fixture
def trained(monkeypatch):
    """A training layer after a forward() on stream 0, its saved tensors, and the C calls it makes from now on."""
    layer = api.CrossAttentionTrain.__new__(api.CrossAttentionTrain)
    layer.cfg = abi.BsaCrossConfig(1, 2, 2, 8, 16, 64, abi.BSA_BF16, 0.0)
    layer.batch, layer.shape, layer.kv_shape, layer.dtype, layer.device = 1, SHAPE, KV, torch.bfloat16, DEV
    layer.bwd_workspace_bytes, layer._status_ptr = 0, 999
    saved = (Stand(SHAPE, 1), Stand(KV, 2), Stand(KV, 3), Stand((1,), 4, torch.int32), Stand(SHAPE, 5),
             Stand(SHAPE[:3], 6, torch.float32), Stand(SHAPE, 7))
    layer._saved, layer._stream, layer._captured, layer._replayed = saved, 0, False, []
    calls = []
    monkeypatch.setattr(abi, "bsa_cross_attention_backward", lambda *a: calls.append(a[1:]))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: STREAM)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(api, "_raw_stream", lambda index: 0)
    return layer, saved, calls


def grads():
    return [Stand(SHAPE, 11), Stand(KV, 12), Stand(KV, 13)]


def test_backward_passes_what_the_forward_saved(trained):
    layer, saved, calls = trained
    out = grads()
    assert layer.backward(Stand(SHAPE, 10), grads=out) == tuple(out)
    assert calls == [(1, 2, 3, 4, 5, 6, 7, 10, 11, 12, 13, None, 0, 999, 0)]
    assert not any(t.streams for t in saved)


def test_backward_on_another_stream_records_all_that_was_saved(trained, monkeypatch):
    """The layer may hold the last reference to q, k, v and key_len too, and drops it at the next forward()."""
    layer, saved, calls = trained
    monkeypatch.setattr(api, "_raw_stream", lambda index: 77)
    layer.backward(Stand(SHAPE, 10), grads=grads())
    assert calls[0][-1] == 77 and all(t.streams == [STREAM] for t in saved)


@pytest.mark.parametrize("count", [1, 2, 4])
def test_grads_of_another_number_are_refused(trained, count):
    """With two, every argument behind dk moved up by one: the workspace became dv, and its size an address."""
    layer, _, calls = trained
    with pytest.raises(ValueError, match="dq, dk and dv"):
        layer.backward(Stand(SHAPE, 10), grads=(grads() + grads())[:count])
    assert not calls


def test_grads_may_be_given_in_part(trained, monkeypatch):
    layer, _, calls = trained
    dq, dk, dv = grads()
    monkeypatch.setattr(torch, "empty_like", lambda like: dk)
    assert layer.backward(Stand(SHAPE, 10), grads=[dq, None, dv]) == (dq, dk, dv)
    assert calls[0][8:11] == (11, 12, 13)


@pytest.mark.parametrize("forward_captured", [False, True])
def test_a_captured_backward_keeps_what_an_eager_forward_saved(trained, monkeypatch, forward_captured):
    """A graph's replays read it, also after a later forward() took its place. What a captured forward saved lies in
    that graph's own memory and is not kept twice."""
    layer, saved, _ = trained
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    layer._captured = forward_captured
    layer.backward(Stand(SHAPE, 10), grads=grads())
    seen = [weakref.ref(t) for t in saved]
    saved = layer._saved = None
    trained = None
    gc.collect()
    assert len(layer._replayed) == (0 if forward_captured else 1)
    if not forward_captured:
        assert all(r() is not None for r in seen)


def test_check_status_waits_for_all_streams(trained, monkeypatch):
    layer, _, _ = trained
    order = []
    layer.status = "word"
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: order.append(device))
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(abi, "bsa_check_status", lambda word: order.append(word) or 7)
    assert layer.check_status() == 7 and order == [DEV, "word"]


@pytest.mark.parametrize("q", [None, [1.0], "q"])
def test_forward_refuses_what_is_no_tensor_as_serving_does(trained, monkeypatch, q):
    layer, _, _ = trained
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: empty(shape, dtype=dtype))
    for call in (layer.forward, super(type(layer), layer).__call__):
        with pytest.raises(ValueError, match="q must be a CUDA tensor"):
            call(q, Stand(KV, 2), Stand(KV, 3))
