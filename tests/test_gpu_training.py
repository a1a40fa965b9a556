"""Training the bf16 path: TrainableBf16MoE's forward, backward and update,
run together as a training program runs them.

* the gradients of a whole layer against the oracle's float64 gradients.
  bf16 roundings (2^-8 each) of g, u, y, D and of their gradients separate
  the two; no more than eight lie on the way to any result, so their sum is
  below 8 * 2^-8 of the largest term and, independent, about sqrt(8) * 2^-9
  in the mean square: rms below 2% of the result's, as for the forward pass;
* the stage chain repeated through the plain functions, bit for bit;
* captured into a graph and replayed on new inputs and routings, on a stream
  of its own, against eager runs, bit for bit;
* two layers that share nothing, on two streams at once.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402
import workloads as W  # noqa: E402
from oracle import backward as B  # noqa: E402
from oracle import fp8  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16


def inputs(seed, name="std_bf16_tiny", **over):
    wl = W.workload(name, seed=seed, **over)
    d = W.generate(wl)
    g = np.random.default_rng(seed)
    dout = g.standard_normal(d["x"].shape).astype(np.float32) * np.float32(0.1)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    b = lambda a: t(a).to(BF)  # noqa: E731
    prank = None if d["psum_recv_per_rank"] is None else t(d["psum_recv_per_rank"])
    x = np.nan_to_num(d["x"])
    return wl, dict(x=b(x), ids=t(d["ids"]), w=t(np.nan_to_num(d["w"])), dout=b(dout),
                    prank=prank), b(d["w13"]), b(d["w2"]), d["num_valid"]


def layer(wl, w13, w2, **kw):
    return M.TrainableBf16MoE(wl.rows, wl.topk, w13, w2, wl.align, wl.routed_scale, **kw)


CASES = [{}, dict(rows=37, topk=3, align=16),
         dict(rows=120, hidden=384, inter=192, experts=6, global_experts=8, topk=3, align=16),
         dict(rows=90, valid_rows=41, src_ranks=4, experts=5, global_experts=8)]


@pytest.mark.parametrize("over", CASES, ids=["tiny", "37", "120", "padded"])
def test_layer_gradients(over):
    print(f"layer {over}", flush=True)
    wl, i, w13, w2, nv = inputs(41, **over)
    mod = layer(wl, w13, w2)
    mod(i["x"], i["ids"], i["w"], i["prank"])
    dx = torch.full((wl.rows, wl.hidden), 7.0, dtype=BF, device="cuda")
    dc = torch.full((wl.rows, wl.topk), 7.0, device="cuda")
    mod.backward(i["dout"], i["w"], i["prank"], dx, dc)
    h = {k: i[k].float().cpu().numpy().astype(np.float64) for k in ("x", "w", "dout")}
    h["dout"][nv:] = 0.0
    ids = i["ids"].cpu().numpy()
    f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    ref = B.layer_backward(h["x"], ids, h["w"], f(w13), f(w2), wl.routed_scale, nv, h["dout"])
    for name, got, want in (("dx", dx[:nv], ref[0][:nv]), ("dw", dc[:nv], ref[1][:nv]),
                            ("dw13", mod.dw13, ref[2]), ("dw2", mod.dw2, ref[3])):
        err = f(got) - want
        rms = np.sqrt(np.mean(want ** 2))
        assert np.sqrt(np.mean(err ** 2)) <= 0.02 * rms, name
        assert np.abs(err).max() <= 8 * 2.0 ** -8 * (np.abs(want).max() + rms), name
    assert torch.all(dx[nv:] == 7.0) and torch.all(dc[nv:] == 7.0)
    first = mod.dw13.clone(), mod.dw2.clone()
    mod.backward(i["dout"], i["w"], i["prank"], dx, dc, accumulate=True)
    for a, b in zip(first, (mod.dw13, mod.dw2)):
        assert torch.allclose(b, 2 * a, rtol=2.0 ** -20, atol=0)


@pytest.mark.parametrize("grad,state", [("f32", "f32"), ("bf16", "fp8")])
def test_update_is_the_oracles(grad, state):
    wl, i, w13, w2, _ = inputs(43)
    mod = layer(wl, w13, w2, grad=grad, state=state, lr=2e-3)
    for t in (1, 2):
        mod(i["x"], i["ids"], i["w"])
        mod.backward(i["dout"], i["w"])
        host = []
        for (m, v, ms, vs), master, dw in zip(mod.states, (mod.master13, mod.master2),
                                              (mod.dw13, mod.dw2)):
            n = lambda a: a.float().cpu().numpy().reshape(-1)  # noqa: E731
            if state == "fp8":
                c = lambda a: a.view(torch.uint8).cpu().numpy().reshape(-1)  # noqa: E731
                mm = B.decode_state(c(m), n(ms))
                vv = B.decode_state(c(v), n(vs)) ** 2
            else:
                mm, vv = n(m), n(v)
            host.append(B.adamw_f32(n(master), n(dw), mm, vv, t, 2e-3, 0.9, 0.95, 1e-8, 0.1,
                                    1.0)[0])
        mod.update(beta2=0.95, weight_decay=0.1)
        for ref, master, w in zip(host, (mod.master13, mod.master2), (mod.w13, mod.w2)):
            got = master.cpu().numpy().reshape(-1)
            assert np.all(np.abs(got - ref) <= 2.0 ** -22 * np.abs(ref) + 2.0 ** -19 * 2e-3 * 12)
            assert torch.equal(w, master.to(BF))
        assert mod.step.item() == t


def test_backward_does_not_need_the_pads():
    """The buffers' rows that hold no token may hold NaN."""
    wl, i, w13, w2, _ = inputs(44, rows=50, align=64)
    outs = []
    for fill in (0.0, float("nan")):
        mod = layer(wl, w13, w2)
        for b in (mod.ex, mod.gate_up, mod.y, mod.down, mod.d_rows, mod.d_y, mod.d_gate_up):
            b.fill_(fill)
        mod(i["x"], i["ids"], i["w"])
        dx, dc = mod.backward(i["dout"], i["w"])
        outs.append((dx, dc, mod.dw13, mod.dw2))
    for a, b in zip(*outs):
        assert torch.equal(a, b) and torch.all(torch.isfinite(a))


def _train_step(mod, bufs, out, dx, dc):
    mod(bufs["x"], bufs["ids"], bufs["w"], bufs["prank"], out=out)
    mod.backward(bufs["dout"], bufs["w"], bufs["prank"], dx, dc)
    mod.update(weight_decay=0.05)


def test_captured_training_steps():
    """Forward, backward and update captured once and replayed on other inputs
    and routings, with eager work and synchronisations between; every replay
    equals an eager step from the same weights and states."""
    over = dict(rows=90, valid_rows=60, src_ranks=4, topk=3, experts=6, global_experts=9,
                align=32)
    wl, a, w13, w2, _ = inputs(51, **over)
    _, b, _, _, _ = inputs(52, **dict(over, valid_rows=17))
    order = [a, b, a, b]

    def fresh():
        mod = layer(wl, w13.clone(), w2.clone(), grad="bf16", state="fp8")
        res = [torch.full((wl.rows, wl.hidden), -3.0, dtype=BF, device="cuda") for _ in range(2)]
        return mod, res + [torch.full((wl.rows, wl.topk), -3.0, device="cuda")]

    def snapshot(mod, res):
        st = [t for s in mod.states for t in s if t is not None]
        return [t.clone() for t in res + [mod.dw13, mod.dw2, mod.master13, mod.master2, mod.w13,
                                          mod.w2, mod.step] + st]

    def reset(res):
        for t in res:
            t.fill_(-3.0)

    eager, want = fresh(), []
    for i in order:
        reset(eager[1])
        _train_step(eager[0], i, *eager[1])
        torch.cuda.synchronize()
        want.append(snapshot(*eager))
    mod, res = fresh()
    bufs = {k: None if v is None else v.clone() for k, v in a.items()}
    keep = snapshot(mod, res)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _train_step(mod, bufs, *res)                    # warm-up
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            _train_step(mod, bufs, *res)
    torch.cuda.current_stream().wait_stream(s)
    now = res + [mod.dw13, mod.dw2, mod.master13, mod.master2, mod.w13, mod.w2, mod.step] + [
        t for st in mod.states for t in st if t is not None]
    for t, k in zip(now, keep):                         # as before the warm-up
        t.copy_(k)
    for rep, i in enumerate(order):
        for k, v in bufs.items():
            if v is not None:
                v.copy_(i[k])
        reset(res)
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(snapshot(mod, res), want[rep]):
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8)), rep


def test_two_layers_on_two_streams():
    wl, i, w13, w2, _ = inputs(61, rows=200, align=16)
    _, j, v13, v2, _ = inputs(62, rows=200, align=16)
    want, mods = [], []
    for inp, a, b in ((i, w13, w2), (j, v13, v2)):
        mod = layer(wl, a.clone(), b.clone())
        mod(inp["x"], inp["ids"], inp["w"])
        dx, dc = mod.backward(inp["dout"], inp["w"])
        mod.update()
        want.append([t.clone() for t in (dx, dc, mod.dw13, mod.dw2, mod.w13, mod.w2)])
        mods.append((layer(wl, a.clone(), b.clone()), inp, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for mod, inp, s in mods:      # the stream handed over explicitly
        h = s.cuda_stream
        out = torch.empty((wl.rows, wl.hidden), dtype=BF, device="cuda")
        dx, dc = torch.empty_like(out), torch.empty((wl.rows, wl.topk), device="cuda")
        mod(inp["x"], inp["ids"], inp["w"], out=out, stream=h)
        mod.backward(inp["dout"], inp["w"], None, dx, dc, stream=h)
        mod.update(stream=h)
        got.append([dx, dc, mod.dw13, mod.dw2, mod.w13, mod.w2, out])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)
