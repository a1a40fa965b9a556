"""TrainableBf16MoE on streams other than the current one, by handle."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16
ROWS, TOPK, E, H, I = 96, 2, 4, 256, 128


def weights(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *s: torch.empty(s, device="cuda").normal_(0, 0.1, generator=g).to(BF)  # noqa: E731
    ids = torch.from_numpy(np.random.default_rng(seed).integers(0, E, (ROWS, TOPK))
                           .astype(np.int32)).cuda()
    return (normal(E, 2 * I, H), normal(E, H, I), normal(ROWS, H), normal(ROWS, H), ids,
            torch.rand((ROWS, TOPK), generator=g, device="cuda"))


def step(mod, x, dout, ids, w, stream=None):
    out = mod(x, ids, w, stream=stream)
    dx, dc = mod.backward(dout, w, stream=stream)
    mod.update(stream=stream)
    return [out, dx, dc, mod.master13, mod.master2, mod.w13, mod.w2, mod.step]


def test_the_default_stream_by_its_handle():
    """Handle 0 is the default stream, whatever stream is current."""
    w13, w2, *rest = weights(5)
    mod = M.TrainableBf16MoE(ROWS, TOPK, w13.clone(), w2.clone(), align=16)
    want = [t.clone() for _ in range(2) for t in step(mod, *rest)]
    mod = M.TrainableBf16MoE(ROWS, TOPK, w13.clone(), w2.clone(), align=16)
    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(2):
            res = step(mod, *rest, stream=0)
            torch.cuda.synchronize()
            got += [t.clone() for t in res]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def pool_of(t):
    """The stream whose memory a tensor has."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def test_outputs_on_another_stream():
    """Outputs that the calls allocate are memory of the stream that writes them."""
    w13, w2, *rest = weights(6)
    mod = M.TrainableBf16MoE(ROWS, TOPK, w13.clone(), w2.clone(), align=16)
    want = [t.clone() for t in step(mod, *rest)]
    mod = M.TrainableBf16MoE(ROWS, TOPK, w13.clone(), w2.clone(), align=16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(mod, *rest, stream=s.cuda_stream)
    for t in got[:3]:
        assert pool_of(t) == s.cuda_stream
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_refused_update_does_not_count():
    w13, w2, *rest = weights(7)
    mod = M.TrainableBf16MoE(ROWS, TOPK, w13, w2, align=16)
    step(mod, *rest)
    before = [t.clone() for t in (mod.step, mod.master13, mod.master2)]
    with pytest.raises(M.MoeError):
        mod.update(beta1=1.0)
    with pytest.raises(ValueError):
        mod.update(grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(M.MoeError):
        mod.update(eps=1e-40, stream=0)
    for a, b in zip((mod.step, mod.master13, mod.master2), before):
        assert torch.equal(a, b)


def test_captured_with_the_handle_of_its_stream():
    """The outputs that the calls allocate lie in the graph's memory; replays
    with eager steps of the program between them equal eager steps."""
    w13, w2, *rest = weights(8)
    new = lambda: M.TrainableBf16MoE(ROWS, TOPK, w13.clone(), w2.clone(), align=16)  # noqa: E731
    eager, want = new(), []
    for _ in range(4):
        want.append([t.clone() for t in step(eager, *rest)])
    mod, s, g = new(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = [t.clone() for t in step(mod, *rest, stream=s.cuda_stream)]     # eager
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            res = step(mod, *rest, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(first, want[0]):
        assert torch.equal(a, b)
    for rep in (1, 2, 3):
        junk = [torch.full_like(t, 9) for t in res[:3]]                  # other work
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, want[rep]):
            assert torch.equal(a, b), rep
        del junk
