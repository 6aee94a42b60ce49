"""Whose memory the serving calls use, with streams and with graphs."""
import contextlib

import pytest
import torch

from verifiable_quantize_rows_gb300 import serving


class Made:
    """Stands for a tensor: where it was made, and the streams told of it."""

    def __init__(self, on):
        self.on, self.told = on, []

    def record_stream(self, stream):
        self.told.append(stream)


@pytest.fixture
def streams(monkeypatch):
    """The current stream of a machine without one, by name, and tensors that know theirs."""
    now = ["current"]

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch, "empty", lambda *shape, **kw: Made(now[-1]))


def test_results_are_of_the_given_streams_memory(streams):
    assert serving._made((3, 4), torch.float32, "cuda", None).on == "current"
    t = serving._made((3, 4), torch.float32, "cuda", "side")
    assert t.on == "side" and t.told == ["current"]


@pytest.mark.gpu
def test_a_result_does_not_take_memory_still_in_use():
    """The current stream has freed a tensor that its queued work still writes: a call on
    another stream, which does not wait for that, must not be given its memory."""
    import verifiable_quantize_rows_gb300 as bsg

    x = torch.randn(200, 50304, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    target = torch.zeros(200, dtype=torch.int64, device="cuda")
    r = bsg.logprobs(x, target)
    g = torch.ones(200, device="cuda")
    want = bsg.logprobs_backward(x, target, r.lse, r.entropy, g, g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = torch.empty_like(x)
    at = held.data_ptr()
    torch.cuda._sleep(50_000_000)
    held.fill_(7)
    del held
    got = bsg.logprobs_backward(x, target, r.lse, r.entropy, g, g, stream=side)
    assert got.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(got, want)
