"""Whose memory the serving calls use, with streams and with graphs."""
import contextlib
import weakref

import pytest
import torch

import verifiable_quantize_rows_gb300 as bsg
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


# ---------------------------------------------------------------------------
@pytest.fixture
def capture(monkeypatch):
    """Whether a capture is under way, as PyTorch is to say it."""
    on = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: on[0])
    monkeypatch.setattr(serving, "_capturing", lambda: on[0], raising=False)
    return on


def test_a_workspace_keeps_what_a_capture_has_taken(capture):
    ws = bsg.Workspace("cpu")
    plain = weakref.ref(ws.get(1000))
    ws.get(2000)
    assert plain() is None                      # no graph can hold it
    capture[0] = True
    taken = weakref.ref(ws.get(2000))           # made before the capture, taken in it
    capture[0] = False
    ws.get(100)
    ws.get(3000)
    assert taken() is not None
    capture[0] = True
    made = weakref.ref(ws.get(4000))            # made in a capture
    capture[0] = False
    ws.get(5000)
    ws.get(6000)
    assert taken() is not None and made() is not None and ws.buf.numel() == 6000


@pytest.mark.parametrize("stream", [None, "side"])
def test_a_call_in_a_capture_says_so_to_its_workspace(capture, monkeypatch, stream):
    """The calls' own way to a buffer, where that is large enough already."""
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    ws = bsg.Workspace("cpu")
    device = torch.device("cpu")
    serving._workspace(ws, 1000, device, stream, 0)
    capture[0] = True
    serving._workspace(ws, 500, device, stream, 0)
    capture[0] = False
    taken = weakref.ref(ws.buf)
    serving._workspace(ws, 2000, device, stream, 0)
    assert taken() is not None and ws.buf.numel() == 2000


def product(M, N, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    W = torch.randn((1024, N), generator=g, device="cuda") * 0.02
    X = torch.randn((M, 1024), generator=g, device="cuda")
    return (X, *bsg.wquant_groups(W, 64))


def strangers(n):
    """Tensors over whatever memory is free, with one value."""
    return [torch.full((1 << k,), 5.0, device="cuda") for k in range(8, 24) for _ in range(n)]


@pytest.mark.gpu
@pytest.mark.parametrize("side", [False, True], ids=["default capture stream", "its own"])
def test_a_graph_outlives_larger_calls_on_its_stream(side):
    """Captured with the default workspace; then a larger call makes that grow."""
    small, large = product(6, 3000, 1), product(16, 30000, 2)
    want_small, want_large = bsg.wgroups_matvec(*small), bsg.wgroups_matvec(*large)
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    if side:
        with torch.cuda.stream(stream):
            bsg.wgroups_matvec(*small)
        torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            out = bsg.wgroups_matvec(*small)
        graphs.append((g, out))
    del graphs[0]                # with the memory of its own that it may have had
    on = stream or torch.cuda.graph.default_capture_stream
    with torch.cuda.stream(on):
        got = bsg.wgroups_matvec(*large)
        theirs = strangers(4)
    torch.cuda.synchronize()
    theirs += strangers(4)
    assert torch.equal(got, want_large)
    for _ in range(3):
        graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want_small)
    assert all(bool((t == 5).all()) for t in theirs)
