"""The stream that a block-scaled call runs on, with torch's streams replaced by
records of what was asked for (no GPU is needed)."""

import contextlib

import pytest
import torch

from int8_int4_dequant_amd import qw


class Tensor(torch.Tensor):
    """A tensor that says it is on device 1."""

    def get_device(self):
        return 1


def on_device_1(*shape):
    return torch.zeros(*shape).as_subclass(Tensor)


class Stream:
    def __init__(self, handle, device):
        self.handle, self.device = handle, device


@pytest.fixture
def calls(monkeypatch):
    """What the decorated functions get, and the streams that were current meanwhile."""
    seen, current = [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0, device))
    monkeypatch.setattr(torch.cuda, "stream", stream)

    @qw._on_stream
    def call(x, rec=None, out=None, stream=None):
        seen.append((x, rec, out, stream, list(current)))
        return stream

    call.seen = seen
    return call


def test_no_stream(calls):
    assert calls(on_device_1(2)) is None and calls.seen[-1][4] == []


@pytest.mark.parametrize("place", ["keyword", "positional"])
def test_a_stream_is_current_for_the_whole_call(calls, place):
    s, x = Stream(5, 1), on_device_1(2)
    got = calls(x, None, None, s) if place == "positional" else calls(x, stream=s)
    assert got is s and calls.seen[-1][4] == [s]


@pytest.mark.parametrize("handle", [0, 77])
@pytest.mark.parametrize("call", [
    lambda f, h: f(on_device_1(2), stream=h),
    lambda f, h: f(on_device_1(2), None, None, h),
    lambda f, h: f(None, dict(codes=on_device_1(2)), stream=h),
    lambda f, h: f(None, rec=dict(pos=on_device_1(2)), stream=h),
])
def test_a_handle_is_of_the_tensors_device(calls, handle, call):
    """Whatever device is current."""
    s = call(calls, handle)
    assert (s.handle, s.device) == (handle, 1) and calls.seen[-1][4] == [s]


def test_every_call_takes_its_stream_last():
    import inspect
    for name in ("block_quantize", "block_quantize_swiglu", "block_unpack", "block_gemm", "block_matmul",
                 "block_gemm_grouped", "moe_sort", "moe_gather", "moe_gather_block", "moe_combine",
                 "moe_combine_backward", "moe_mlp"):
        f = getattr(qw, name)
        parameters = list(inspect.signature(f).parameters)
        assert parameters[-1] == "stream" and f.__wrapped__.__code__.co_varnames.index("stream") == len(parameters) - 1
