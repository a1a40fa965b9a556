"""What the Python classes do around the library's calls: streams, outputs and
counts (no GPU: torch's stream functions and the calls are stood in for)."""

import contextlib

import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

POOL = "a stream of torch's pool"


@pytest.fixture
def streams(monkeypatch):
    """now[-1]: the handle of the stream that torch works on (0: the default one)."""
    now = [0]

    @contextlib.contextmanager
    def enter(handle):
        now.append(handle)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle or POOL)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: 0)
    return now


class Counter:
    """Stands in for the step tensor: its value, and where it was changed."""

    def __init__(self, now):
        self.now, self.value, self.on = now, 0, []

    def add_(self, n):
        self.value += n
        self.on.append(self.now[-1])


def trainable(now):
    mod = object.__new__(M.TrainableBf16MoE)
    mod.step, mod.tensors, mod.lr = Counter(now), None, None
    return mod


@pytest.mark.parametrize("stream,where", [(None, 7), (0, 0), (4096, 4096)])
def test_update_counts_on_the_stream_of_its_step(streams, monkeypatch, stream, where):
    """The count and the kernel that reads it run on one stream, also where that
    is the default one, whose handle is 0, and another stream is current."""
    calls = []
    monkeypatch.setattr(M, "moe_adamw", lambda *a: calls.append(a[-1]))
    mod = trainable(streams)
    streams.append(7)
    mod.update(stream=stream)
    assert calls == [stream] and mod.step.value == 1
    assert mod.step.on == [where]
