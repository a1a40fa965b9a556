"""MoEBlock around a StandardMoE (fp8 experts): the norm, gate and router in front of that
path, eager, with rows that were not received, and captured."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402
from oracle import block as B  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from tests.test_gpu_standard import to_gpu_std  # noqa: E402
from tests.test_oracle_standard import std_inputs  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def make(fmt):
    inp = std_inputs(fmt=fmt)
    g = to_gpu_std(inp)
    rows, topk = inp["ids"].shape
    moe = lambda: M.StandardMoE(rows, topk, g["w13"], g["w13_scale"], g["w2"],  # noqa: E731
                                g["w2_scale"], inp["align"], inp["fmt"], 2.5)
    experts = moe()
    E, H = experts.E, experts.H
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    gate, weight = (rand(E, H) * H ** -0.5).to(BF), 1 + 0.1 * rand(H)
    block = M.MoEBlock(experts, gate, weight, select_bias=0.1 * rand(E), score="sigmoid",
                       stream_dtype=F32)
    return block, moe(), rand


@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
@pytest.mark.parametrize("part", [1.0, 0.6])
def test_block_of_fp8_experts_is_its_calls(fmt, part):
    block, moe, rand = make(fmt)
    rows, n = block.rows, max(1, int(block.rows * part))
    prank = torch.tensor([n], dtype=torch.int32, device="cuda") if n < rows else None
    x, branch = rand(rows, block.H), rand(rows, block.H).to(BF)
    x[n:], branch[n:] = float("nan"), float("nan")
    out = torch.full((rows, block.H), 7.0, dtype=BF, device="cuda")
    got, h = block(x, branch, prank, out)
    assert got is out and h is block.sum
    assert torch.equal(h[:n], (x + branch.float())[:n])
    bias = block.select_bias.double().cpu().numpy()
    logits = block.logits[:n, :block.E].double().cpu().numpy()
    ids, w = B.router(logits, block.topk, bias, "sigmoid")
    assert np.array_equal(block.topk_ids[:n].cpu().numpy(), ids)
    want = torch.full_like(out, 7.0)
    moe(block.y[:rows], block.topk_ids, block.topk_weights, prank, want)
    assert torch.equal(out, want) and bool(torch.isfinite(out[:n]).all())
    assert bool((out[n:] == 7).all()) and bool(out[:n].abs().sum() > 0)
    with pytest.raises(TypeError):
        block.backward(out)


def test_captured():
    block, moe, rand = make("f32")
    rows = block.rows
    x, out = rand(rows, block.H), torch.zeros((rows, block.H), dtype=BF, device="cuda")
    prank = torch.tensor([rows], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, None, prank, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, None, prank, out)
    for n in (rows, 1, rows // 2, 0, rows):
        x.copy_(rand(rows, block.H))
        prank.fill_(n)
        out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.full_like(out, 3.0)
        moe(block.y[:rows], block.topk_ids, block.topk_weights, prank, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
