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
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    return now


class Counter:
    """Stands in for the step tensor: its value, and where it was changed."""

    def __init__(self, now):
        self.now, self.value, self.on = now, 0, []

    def add_(self, n):
        self.value += n
        self.on.append(self.now[-1])

    def sub_(self, n):
        self.add_(-n)


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


class Output:
    """Stands in for a tensor: the stream whose memory it has, and its users."""

    def __init__(self, on):
        self.on, self.users = on, [on]

    def record_stream(self, stream):
        self.users.append(stream)


class Tokens:
    device = "cuda"


@pytest.mark.parametrize("stream", [None, 0, 7, 4096])
@pytest.mark.parametrize("cls", [M.ExpandedMoE, M.StandardMoE, M.MaskedMoE, M.StandardBf16MoE,
                                 M.TrainableBf16MoE])
def test_outputs_are_of_the_stream_that_writes_them(streams, monkeypatch, cls, stream):
    """What a class allocates for a call on another stream is that stream's
    memory, and the current stream is a user of it."""
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: Output(streams[-1]))
    for name in dir(M):
        if name.startswith("moe_") and callable(getattr(M, name)):
            monkeypatch.setattr(M, name, lambda *a, **kw: None)
    mod = object.__new__(cls)
    mod.rows, mod.H, mod.topk, mod.fmt = 4, 128, 2, "f32"
    for step in ("layout", "experts", "gather"):
        monkeypatch.setattr(cls, step, lambda self, *a: None)
    streams.append(7)                                       # the current one
    args = (None,) * (3 if issubclass(cls, M.ExpandedMoE) and cls is not M.StandardMoE else 2)
    got = [mod(Tokens, *args, stream=stream)]
    if cls is M.TrainableBf16MoE:
        for name in ("psum status align src2dst down d_rows y dw2 wgrad_workspace w2 d_y gate_up "
                     "m_indices E d_gate_up ex dw13 w13 routed_scaling_factor").split():
            setattr(mod, name, None)
        got += mod.backward(Tokens, None, stream=stream)
    for t in got:
        assert t.on == (7 if stream is None else stream)
        assert 7 in t.users


class OnGpu:
    """Stands in for a contiguous tensor on a GPU."""

    def __init__(self, gpu, dtype, *shape):
        self.gpu, self.dtype, self.shape = gpu, dtype, torch.Size(shape)

    def get_device(self):
        return self.gpu

    device = property(lambda self: f"cuda:{self.gpu}")
    numel = lambda self: self.shape.numel()  # noqa: E731
    is_contiguous = lambda self: True  # noqa: E731
    data_ptr = lambda self: 0x1000  # noqa: E731


def test_adamw_refuses_a_list_of_another_gpu(monkeypatch):
    """Made while GPU 0 was current and used while GPU 1 is, with that one's step
    and rate: the kernel would run on GPU 1 on memory that is not its own."""
    current, calls = [0], []
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[-1], raising=False)

    class Library:
        moe_adamw = staticmethod(lambda *a: calls.append(a) or M.MOE_OK)

    monkeypatch.setattr(M, "lib", lambda: Library)
    f32 = lambda gpu, n: OnGpu(gpu, torch.float32, n)  # noqa: E731
    ts = M.AdamWTensors([(f32(0, 5), f32(0, 5), f32(0, 5), f32(0, 5), None, None, None)])
    scalars = lambda gpu: (OnGpu(gpu, torch.int64, 1), f32(gpu, 1))  # noqa: E731
    M.moe_adamw(ts, *scalars(0), stream=4096)
    assert len(calls) == 1
    current.append(1)
    with pytest.raises(ValueError, match="not on the current GPU"):
        M.moe_adamw(ts, *scalars(1), stream=4096)
    assert len(calls) == 1
    M.moe_adamw(M.AdamWTensors([]), *scalars(1), stream=4096)      # nothing to be elsewhere


@pytest.mark.parametrize("stream", [None, 0, 4096])
def test_a_refused_update_does_not_count(streams, monkeypatch, stream):
    def refuse(*a):
        raise M.MoeError("moe_adamw", M.MOE_ERR_SHAPE)

    monkeypatch.setattr(M, "moe_adamw", refuse)
    mod = trainable(streams)
    with pytest.raises(M.MoeError):
        mod.update(beta1=1.0, stream=stream)
    assert mod.step.value == 0
    assert set(mod.step.on) == {stream or 0}
