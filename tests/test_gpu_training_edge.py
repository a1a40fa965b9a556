"""TrainableBf16MoE at the ends of its range: no rows, none of them here, one
row, one expert for all slots, sizes far apart.  Gradients against the
oracle's float64 ones with the bars of test_gpu_training.py."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402
from oracle import backward as B  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16
f64 = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731


def run(ids, E, H, I, align, valid=None, factor=1.0, seed=0):
    g = np.random.default_rng(seed)
    rows, topk = ids.shape
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    normal = lambda *s: t(g.standard_normal(s).astype(np.float32))  # noqa: E731
    x, dout = normal(rows, H).to(BF), (normal(rows, H) * 0.1).to(BF)
    w13, w2 = (normal(E, 2 * I, H) * 0.1).to(BF), (normal(E, H, I) * 0.1).to(BF)
    w = t(g.random((rows, topk)).astype(np.float32) + np.float32(0.1))
    nv = rows if valid is None else valid
    prank = None if valid is None else t(np.array([nv // 2, nv], np.int32))
    mod = M.TrainableBf16MoE(rows, topk, w13.clone(), w2.clone(), align, factor)
    for b in (mod.ex, mod.gate_up, mod.y, mod.down, mod.d_rows, mod.d_y, mod.d_gate_up):
        b.fill_(float("nan"))
    mod(x, t(ids.astype(np.int32)), w, prank)
    dx = torch.full((rows, H), 7.0, dtype=BF, device="cuda")
    dc = torch.full((rows, topk), 7.0, device="cuda")
    mod.backward(dout, w, prank, dx, dc)
    ref = B.layer_backward(f64(x), ids, f64(w), f64(w13), f64(w2), factor, nv, f64(dout))
    for name, got, want in (("dx", dx[:nv], ref[0][:nv]), ("dw", dc[:nv], ref[1][:nv]),
                            ("dw13", mod.dw13, ref[2]), ("dw2", mod.dw2, ref[3])):
        if want.size == 0:
            continue
        err, rms = f64(got) - want, np.sqrt(np.mean(want ** 2))
        assert np.sqrt(np.mean(err ** 2)) <= 0.02 * rms, name
        assert np.abs(err).max() <= 8 * 2.0 ** -8 * (np.abs(want).max() + rms), name
        zero = want == 0
        assert np.all(f64(got)[zero] == 0), name
    assert torch.all(dx[nv:] == 7.0) and torch.all(dc[nv:] == 7.0)
    mod.update()
    assert torch.all(torch.isfinite(mod.master13)) and torch.all(torch.isfinite(mod.master2))
    assert torch.equal(mod.w13, mod.master13.to(BF)) and torch.equal(mod.w2, mod.master2.to(BF))


def ids_of(rows, topk, experts, seed=1):
    g = np.random.default_rng(seed)
    return np.stack([g.permutation(max(experts, topk))[:topk] for _ in range(rows)])


@pytest.mark.parametrize("what", ["none received", "none here", "one row", "one slot",
                                  "one expert", "one expert of many", "the same twice"])
@pytest.mark.parametrize("align", [16, 1024])
def test_ends(what, align):
    print(what, align, flush=True)
    if what == "none received":
        run(ids_of(40, 2, 4), 4, 256, 64, align, valid=0)
    elif what == "none here":
        run(np.full((40, 2), -1), 4, 256, 64, align)
    elif what == "one row":
        run(ids_of(1, 3, 4), 4, 256, 64, align, factor=2.5)
    elif what == "one slot":
        run(np.array([[-1, -1], [-1, 3]]), 4, 256, 64, align, valid=2)
    elif what == "one expert":
        run(np.zeros((300, 1), np.int64), 1, 128, 64, align)
    elif what == "one expert of many":
        run(np.full((300, 1), 130), 200, 128, 64, align)
    else:
        run(np.full((70, 4), 1), 3, 128, 128, align, factor=-0.5)


@pytest.mark.parametrize("H,I", [(128, 64), (8192, 64), (128, 2048)])
def test_sizes_far_apart(H, I):
    print(H, I, flush=True)
    ids = ids_of(33, 2, 5)
    ids[3:9] = -1
    run(ids, 5, H, I, 32, valid=31)
