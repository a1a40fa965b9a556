"""MoEBlock and StandardW4MoE: the norm, the gate, the router and the experts run
together, forward and back, captured, on other streams.

Whole runs are compared with torch's float64 autograd on the CPU, the chosen
experts being those that the run chose.  Every stage that is rounded to bf16
puts a relative error of at most 2^-8 (half a step) on what it hands on, in the
2-norm; N such stages in a row put N * 2^-8 there (errors that a later stage
enlarges or shrinks count once: gains and weights here have norms near 1).
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402
from oracle import block as B  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF, F32 = torch.bfloat16, torch.float32
E, H, I, TOPK = 6, 256, 128, 2


def rand(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def make(rows, kind="rms", score="softmax", normalize=True, stream_dtype=BF, seed=1, grad="f32",
         bias=True, **kw):
    w13, w2 = rand(seed, E, 2 * I, H, scale=H ** -0.5), rand(seed + 1, E, H, I, scale=I ** -0.5)
    moe = M.TrainableBf16MoE(rows, TOPK, w13, w2, align=16, routed_scaling_factor=1.5)
    gate = rand(seed + 2, E, H, scale=H ** -0.5)
    weight = 1 + rand(seed + 3, H, scale=0.1, dtype=F32)
    b = rand(seed + 4, H, scale=0.1, dtype=F32) if bias else None
    return M.MoEBlock(moe, gate, weight, b, kind=kind, score=score, normalize=normalize,
                      stream_dtype=stream_dtype, grad=grad, **kw)


def reference(block, x, branch, dout, dsum, n):
    """float64 run over the first n rows with the run's own choice of experts."""
    d = lambda t: t.detach().double().cpu()  # noqa: E731
    leaf = lambda t: d(t).requires_grad_(True)  # noqa: E731
    h, gate = leaf(x[:n]), leaf(block.gate[0, :E])
    if branch is not None:
        h = (d(x[:n]) + d(branch[:n])).requires_grad_(True)
    weight, bias = leaf(block.weight), None if block.bias is None else leaf(block.bias)
    c = h - h.mean(1, keepdim=True) if block.kind == "layer" else h
    y = c / (c.pow(2).mean(1, keepdim=True) + block.eps).sqrt() * weight
    if bias is not None:
        y = y + bias
    logits = y @ gate.t()
    ids = block.topk_ids[:n].long().cpu()
    s = torch.softmax(logits, 1) if block.route["score"] == "softmax" else torch.sigmoid(logits)
    w = s.gather(1, ids)
    if block.route["normalize"]:
        w = w / w.sum(1, keepdim=True)
    w13, w2 = leaf(block.moe.w13), leaf(block.moe.w2)
    gu = torch.einsum("rh,ejh->rej", y, w13)
    z = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:]
    full = torch.einsum("rei,ehi->reh", z, w2)
    out = 1.5 * (full.gather(1, ids[..., None].expand(-1, -1, H)) * w[..., None]).sum(1)
    loss = (out * d(dout[:n])).sum()
    if dsum is not None:
        loss = loss + (h * d(dsum[:n])).sum()
    loss.backward()
    return dict(h=h, y=y, logits=logits, w=w, out=out, dx=h.grad, d_gate=gate.grad,
                d_weight=weight.grad, d_bias=None if bias is None else bias.grad,
                dw13=w13.grad, dw2=w2.grad)


def near(name, got, want, roundings):
    got, want = got.detach().double().cpu(), want.detach()
    off = float((got - want).norm() / want.norm())
    assert off <= roundings * 2.0 ** -8, (name, off * 256, roundings)


@pytest.mark.parametrize("rows,n,kind,score,normalize,dtype,with_branch", [
    (40, 40, "rms", "softmax", True, BF, False), (33, 20, "layer", "sigmoid", True, BF, True),
    (64, 50, "rms", "softmax", False, F32, True), (7, 7, "layer", "sigmoid", False, F32, False),
    (1, 1, "rms", "softmax", True, BF, True)])
def test_forward_and_backward(rows, n, kind, score, normalize, dtype, with_branch):
    block = make(rows, kind, score, normalize, dtype)
    x, dout = rand(20, rows, H, dtype=dtype), rand(21, rows, H)
    branch = rand(22, rows, H) if with_branch else None
    dsum = rand(23, rows, H, scale=0.5, dtype=dtype) if with_branch else None
    for t in (x, branch, dout, dsum):
        if t is not None:
            t[n:] = float("nan")
    prank = torch.tensor([n // 2, n], dtype=torch.int32, device="cuda") if n < rows else None
    out, h = block(x, branch, prank)
    dx = block.backward(dout, dsum, prank)
    ref = reference(block, x, branch, dout, dsum, n)
    near("stream", h[:n], ref["h"], 1)
    near("y", block.y[:n], ref["y"], 2)                       # stream, y
    near("logits", block.logits[:n, :E], ref["logits"], 3)
    # What a rounding of the logits (|x| about 1) does to the weights: as much.
    near("weights", block.topk_weights[:n], ref["w"], 4)
    near("out", out[:n], ref["out"], 9)          # and gate_up, its product, down, out
    # Back: the combine's, SiLU's and both products' gradients, d_logits and its
    # product, each rounded, from values that carry the errors above.
    near("dw2", block.moe.dw2, ref["dw2"], 10)
    near("dw13", block.moe.dw13, ref["dw13"], 14)
    near("d_weight", block.d_weight, ref["d_weight"], 16)
    if ref["d_bias"] is not None:
        near("d_bias", block.d_bias, ref["d_bias"], 16)
    near("dx", dx[:n], ref["dx"], 17)
    # The gate's gradient is a difference of near values (sum over a row: 0 but
    # for the sigmoid), small against its terms: measured against those.
    terms = torch.einsum("re,rh->eh", ref["logits"].abs() * 0 + 1, ref["y"].abs())
    scale = float((ref["out"].detach() * dout[:n].double().cpu()).abs().sum(1).mean())
    off = (block.d_gate[0, :E].double().cpu() - ref["d_gate"]).abs()
    assert bool((off <= 14 * 2.0 ** -8 * scale * terms).all())
    assert int(torch.count_nonzero(block.d_gate[0, E:])) == 0


def test_block_is_its_calls():
    """Bit for bit the calls in order; a second block takes the first one's stream
    and output."""
    rows = 48
    block = make(rows, select_bias=rand(9, E, scale=0.2, dtype=F32), num_groups=3, topk_groups=2)
    x, branch = rand(20, rows, H), rand(21, rows, H)
    out, h = block(x, branch)
    assert torch.equal(h, x + branch)
    y = torch.empty_like(x)
    rstd = torch.empty(rows, device="cuda")
    M.moe_layer_norm(h, block.weight, y, block.bias, rstd=rstd, kind="rms")
    assert torch.equal(y, block.y[:rows])
    logits = torch.empty((rows, 128), dtype=BF, device="cuda")
    M.moe_grouped_gemm_bf16(y, block.gate, block.all_rows, block.status, 16, logits)
    ids = torch.empty((rows, TOPK), dtype=torch.int32, device="cuda")
    w = torch.empty((rows, TOPK), device="cuda")
    M.moe_router(logits[:, :E], ids, w, block.select_bias, num_groups=3, topk_groups=2)
    want, _ = B.router(logits[:, :E].double().cpu().numpy(), TOPK,
                       block.select_bias.double().cpu().numpy(), "softmax", 3, 2)
    assert np.array_equal(ids.cpu().numpy(), want) and torch.equal(ids, block.topk_ids)
    moe = M.StandardBf16MoE(rows, TOPK, block.moe.w13, block.moe.w2, 16, 1.5)
    assert torch.equal(moe(y, ids, w), out)
    second = make(rows, seed=40)
    out2, h2 = second(h, out)
    assert torch.equal(h2, h + out) and bool(torch.isfinite(out2).all())


def test_accumulated_gradients_and_bf16_ones():
    rows = 32
    a, b = make(rows, grad="f32"), make(rows, grad="bf16")
    x, dout = rand(1, rows, H), rand(2, rows, H)
    for blk in (a, b):
        blk(x)
        blk.backward(dout)
    first = [t.clone() for t in (a.d_gate, a.d_weight, a.d_bias, a.moe.dw13)]
    a.backward(dout, accumulate=True)
    for t, f in zip((a.d_gate, a.d_weight, a.d_bias, a.moe.dw13), first):
        # a sum of two equal halves: one more fp32 rounding each
        assert bool(((t - 2 * f).abs() <= 2.0 ** -23 * t.abs() + 1e-12).all())
    for t, f in zip((b.d_gate, b.d_weight, b.d_bias), first):
        assert t.dtype == BF and torch.equal(t, f.to(BF))


def test_captured_block_follows_its_inputs():
    rows = 64
    block = make(rows, "layer", select_bias=torch.zeros(E, device="cuda"))
    twin = make(rows, "layer", select_bias=torch.zeros(E, device="cuda"))
    x, dout, dsum = rand(1, rows, H), rand(2, rows, H), rand(3, rows, H)
    prank = torch.tensor([rows], dtype=torch.int32, device="cuda")
    out, dx = torch.zeros_like(x), torch.zeros_like(x)

    def step(b):
        b(x, None, prank, out)
        b.backward(dout, dsum, prank, dx)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(block)
    side.synchronize()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(block)
    for n, seed in ((64, 5), (1, 6), (37, 7), (0, 8), (64, 9)):
        x.copy_(rand(seed, rows, H))
        prank.fill_(n)
        res = []
        for b, go in ((block, graph.replay), (twin, lambda: step(twin))):
            out.fill_(3)
            dx.fill_(3)
            go()
            torch.cuda.synchronize()
            res.append([t.clone() for t in (out, dx, b.d_gate, b.d_weight, b.d_bias, b.moe.dw13)])
        for p, q in zip(*res):
            assert torch.equal(p, q)
        assert bool((res[0][0][n:] == 3).all()) and bool((res[0][1][n:] == 3).all())


def test_two_blocks_on_two_streams():
    rows = 64
    blocks = [make(rows, seed=s) for s in (1, 30)]
    xs = [rand(50 + i, rows, H) for i in range(2)]
    dout = rand(60, rows, H)
    want = []
    for b, x in zip(blocks, xs):
        out, _ = b(x)
        dx = b.backward(dout)
        want.append([t.clone() for t in (out, dx, b.d_gate, b.d_weight)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for b, x, s in zip(blocks, xs, streams):
            out, _ = b(x, stream=s.cuda_stream)
            dx = b.backward(dout, stream=s.cuda_stream)
            got.append([out, dx, b.d_gate, b.d_weight])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for p, q in zip(g, w):
                assert torch.equal(p, q)


def test_refusals():
    block = make(16)
    with pytest.raises(RuntimeError):
        block.backward(rand(1, 16, H))
    with pytest.raises(ValueError):
        M.MoEBlock(block.moe, rand(1, E + 1, H), block.weight)
    with pytest.raises(ValueError):
        M.MoEBlock(block.moe, rand(1, E, H), block.weight, grad="fp8")
    plain = M.StandardBf16MoE(16, TOPK, block.moe.w13, block.moe.w2, 16)
    served = M.MoEBlock(plain, rand(1, E, H), block.weight)
    served(rand(2, 16, H))
    with pytest.raises(TypeError):
        served.backward(rand(1, 16, H))


def quantised(seed, n, k, fmt, group):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    if fmt == "mxfp4":  # weights of size k^-0.5
        sc = torch.full((E, n, k // group), 127 - int(np.log2(3 * k ** 0.5)), dtype=torch.uint8,
                        device="cuda")
    else:
        sc = torch.full((E, n, k // group), 1 / (4.6 * k ** 0.5), device="cuda").to(BF)
    v = B.w4_values(w.cpu().numpy(), sc.float().cpu().numpy() if fmt == "int4" else
                    sc.cpu().numpy(), fmt)
    return w, sc, torch.from_numpy(v)


@pytest.mark.parametrize("fmt,group", [("int4", 128), ("int4", 64), ("int4", 32), ("mxfp4", 32)])
@pytest.mark.parametrize("rows,align", [(1, 16), (37, 128), (400, 16)])
def test_w4_layer(fmt, group, rows, align):
    inter = 128
    w13, s13, v13 = quantised(1, 2 * inter, H, fmt, group)
    w2, s2, v2 = quantised(2, H, inter, fmt, group)
    moe = M.StandardW4MoE(rows, TOPK, w13, s13, w2, s2, fmt, align, 2.5)
    block = M.MoEBlock(moe, rand(3, E, H, scale=H ** -0.5), 1 + rand(4, H, scale=0.1, dtype=F32))
    x = rand(5, rows, H)
    out, _ = block(x)
    y, ids = block.y[:rows].double().cpu(), block.topk_ids.long().cpu()
    gu = torch.einsum("rh,ejh->rej", y, v13)
    z = torch.nn.functional.silu(gu[..., :inter]) * gu[..., inter:]
    full = torch.einsum("rei,ehi->reh", z, v2)
    w = block.topk_weights.double().cpu()
    want = 2.5 * (full.gather(1, ids[..., None].expand(-1, -1, H)) * w[..., None]).sum(1)
    near("out", out, want, 5)                    # gate_up (twice, as g and u), z, down, out
    # On the same values in bf16 (exact for MXFP4) the bf16 layer runs the same stages.
    if fmt == "mxfp4":
        bf = M.StandardBf16MoE(rows, TOPK, v13.to(BF).cuda(), v2.to(BF).cuda(), align, 2.5)
        near("bf16 layer", bf(block.y[:rows], block.topk_ids, block.topk_weights), want, 5)


def test_w4_layer_refuses_other_shapes():
    w13, s13, _ = quantised(1, 256, H, "int4", 128)
    w2, s2, _ = quantised(2, H, 128, "int4", 128)
    with pytest.raises(ValueError):
        M.StandardW4MoE(8, 2, w13, s13, w13, s2, "int4")
    with pytest.raises(KeyError):
        M.StandardW4MoE(8, 2, w13, s13, w2, s2, "int8")


def test_gradient_through_the_router_by_differences():
    """The whole block's gradient against differences of float64 runs of the same
    choice: one value of x moved by 1e-4 both ways."""
    rows = 4
    block = make(rows, "layer", stream_dtype=F32)
    x, dout = rand(20, rows, H, dtype=F32), rand(21, rows, H)
    block(x)
    dx = block.backward(dout)
    f = lambda v: float((reference(block, v, None, dout, None, rows)["out"].detach()  # noqa: E731
                         * dout.double().cpu()).sum())
    rng = np.random.default_rng(3)
    size = float(dx.double().norm()) / (rows * H) ** 0.5
    for _ in range(12):
        r, c = rng.integers(rows), rng.integers(H)
        hi, lo = x.double(), x.double()
        hi[r, c] += 1e-4
        lo[r, c] -= 1e-4
        d = (f(hi) - f(lo)) / 2e-4
        # 17 roundings (above) of values of the gradient's own size, of which a
        # single one may lie 4 deviations out
        assert abs(d - float(dx[r, c])) <= 17 * 2.0 ** -8 * max(abs(d), 4 * size)
