"""GPU parity of moe_adamw with the oracle's step, in which every fp32
operation is rounded in the documented order.

Bars: states (fp32 values, codes and scales) are equal, bit for bit; the
update u = m^ / (sqrt(v^) + eps) + wd p may be a few fp32 steps off
(quotients and root), so |master| differs by at most 2^-23 |p| (the last
subtraction) plus 2^-20 lr |u|; the bf16 copy is the rounded master.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402
from oracle import backward as B  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

HYPER = dict(beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 8, 127, 128, 129, 1000, 2048, 8191, 8192, 8193, 40000]


def make(n, seed, fp8, grad_f32, copy):
    g = np.random.default_rng(seed)
    f = lambda s: (g.standard_normal(n) * s).astype(np.float32)  # noqa: E731
    p, grad = f(0.5), torch.from_numpy(f(1e-2) * np.exp(g.uniform(-8, 0, n)).astype(np.float32))
    if not grad_f32:
        grad = grad.to(torch.bfloat16)
    m, v = f(1e-3), f(1e-3) ** 2
    if n > 5:
        grad[3], m[3], v[3] = 0.0, 0.0, 0.0
    h = dict(p=p, grad=grad.float().numpy(), fp8=fp8)
    t = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    if fp8:
        (h["m"], h["ms"]), (h["v"], h["vs"]) = B.encode_state(m, False), B.encode_state(
            np.sqrt(v), True)
    else:
        h.update(m=m, v=v, ms=None, vs=None)
    d = [t(p), grad.cuda(), t(h["m"]), t(h["v"]),
         torch.full((n,), 7.0, dtype=torch.bfloat16, device="cuda") if copy else None,
         t(h["ms"]) if fp8 else None, t(h["vs"]) if fp8 else None]
    return h, d


def expect(h, t, lr, gs, hyper=HYPER):
    """The oracle's step on a host copy: (master, |bar|), and h's states updated."""
    m, v = h["m"], h["v"]
    if h["fp8"]:
        m = B.decode_state(h["m"], h["ms"])
        r = B.decode_state(h["v"], h["vs"])
        v = r * r
    p, m, v = B.adamw_f32(h["p"], h["grad"], m, v, t, lr, hyper["beta1"], hyper["beta2"],
                          hyper["eps"], hyper["weight_decay"], gs)
    step = np.abs(p.astype(np.float64) - h["p"])
    bar = 2.0 ** -23 * np.abs(p) + 2.0 ** -20 * (step + 2.0 ** -23 * np.abs(p)) + 2.0 ** -149
    if h["fp8"]:
        (h["m"], h["ms"]), (h["v"], h["vs"]) = B.encode_state(m, False), B.encode_state(
            np.sqrt(v), True)
    else:
        h["m"], h["v"] = m, v
    h["p"] = p
    return bar


def compare(h, d, bar, what):
    got = d[0].cpu().numpy()
    assert np.all(np.abs(got.astype(np.float64) - h["p"]) <= bar), what
    for i, key in ((2, "m"), (3, "v"), (5, "ms"), (6, "vs")):
        if d[i] is not None:
            assert np.array_equal(d[i].cpu().numpy().view(np.uint8),
                                  np.ascontiguousarray(h[key]).view(np.uint8)), (what, key)
    if d[4] is not None:
        assert torch.equal(d[4], d[0].to(torch.bfloat16)), what
    h["p"] = got          # the next step starts from the same master


def scalars(t, lr, gs=None):
    return (torch.tensor([t], dtype=torch.int64, device="cuda"),
            torch.tensor([lr], dtype=torch.float32, device="cuda"),
            None if gs is None else torch.tensor([gs], dtype=torch.float32, device="cuda"))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("grad_f32,copy", [(False, True), (True, False)])
def test_steps(fp8, grad_f32, copy):
    """Three steps over tensors of every size in one call each."""
    both = [make(n, i, fp8, grad_f32, copy) for i, n in enumerate(SIZES)]
    ts = M.AdamWTensors([d for _, d in both])
    for t in (1, 2, 3):
        print(f"adamw fp8 {fp8} step {t}", flush=True)
        step, lr, gs = scalars(t, 1e-3, 0.25)
        M.moe_adamw(ts, step, lr, grad_scale=gs, **HYPER)
        for (h, d), n in zip(both, SIZES):
            compare(h, d, expect(h, t, 1e-3, 0.25), f"size {n} step {t}")


def test_mixed_formats_and_more_tensors_than_a_launch_holds():
    both = [make(1 + 37 * i, i, i % 2 == 1, i % 3 == 1, i % 5 != 1) for i in range(75)]
    step, lr, _ = scalars(1000, 3e-4)
    M.moe_adamw(M.AdamWTensors([d for _, d in both]), step, lr, **HYPER)
    for i, (h, d) in enumerate(both):
        compare(h, d, expect(h, 1000, 3e-4, 1.0), f"tensor {i}")


@pytest.mark.parametrize("fp8", [False, True])
def test_neighbours_stay(fp8):
    """What lies behind a tensor of odd size in its allocation is not written."""
    n, pad = 1003, 64
    h, d = make(n, 5, fp8, False, True)
    big = [None if t is None else torch.cat([t, torch.full((pad,), 1, device="cuda").to(t.dtype)])
           for t in d]
    view = [None if t is None else t[:len(s)] for t, s in zip(big, d)]
    step, lr, _ = scalars(3, 1e-3)
    M.moe_adamw(M.AdamWTensors([view]), step, lr, **HYPER)
    compare(h, view, expect(h, 3, 1e-3, 1.0), "view")
    for t, s in zip(big, d):
        if t is not None:
            assert torch.all(t[len(s):].float() == 1.0)


def test_hyperparameters_at_their_ends():
    for hyper in (dict(beta1=0.0, beta2=0.0, eps=1e-8, weight_decay=0.0),
                  dict(beta1=0.99, beta2=0.999, eps=0.0, weight_decay=1.0)):
        h, d = make(500, 6, False, True, False)
        h["grad"] = np.where(h["grad"] == 0, np.float32(1e-3), h["grad"])
        d[1] = torch.from_numpy(h["grad"]).cuda()
        step, lr, _ = scalars(1, 1e-2)
        M.moe_adamw(M.AdamWTensors([d]), step, lr, **hyper)
        compare(h, d, expect(h, 1, 1e-2, 1.0, hyper), str(hyper))


def test_zero_gradients_and_states():
    """All zero: only the decay moves the master; codes stay 0."""
    for fp8 in (False, True):
        h, d = make(300, 7, fp8, False, True)
        for i in (1, 2, 3, 5, 6):
            if d[i] is not None:
                d[i].zero_()
        before = d[0].clone()
        step, lr, _ = scalars(1, 1e-2)
        M.moe_adamw(M.AdamWTensors([d]), step, lr, **HYPER)
        assert torch.allclose(d[0], before * (1 - 1e-3), rtol=2.0 ** -22, atol=0)
        assert not d[2].view(torch.uint8).any() and not d[3].view(torch.uint8).any()


def test_values_that_are_not_finite_stay_in_their_group():
    h, d = make(1000, 8, True, True, False)
    d[1][200] = float("inf")
    d[1][700] = float("nan")
    step, lr, _ = scalars(2, 1e-3)
    M.moe_adamw(M.AdamWTensors([d]), step, lr, **HYPER)
    fine = torch.isfinite(d[0])
    assert not fine[200] and not fine[700] and fine.sum() == 998
    scale = torch.isfinite(d[5])
    assert not scale[1] and scale.sum() == len(scale) - 1


def test_empty_list_and_empty_tensors():
    step, lr, _ = scalars(1, 1e-3)
    M.moe_adamw(M.AdamWTensors([]), step, lr)
    e = torch.empty(0, device="cuda")
    h, d = make(64, 9, False, False, True)
    M.moe_adamw(M.AdamWTensors([(e, e, e, e, None, None, None), d]), step, lr, **HYPER)
    compare(h, d, expect(h, 1, 1e-3, 1.0), "beside an empty one")


def test_binding_refusals():
    h, d = make(256, 10, True, False, True)
    for i, bad in ((0, d[0].half()), (1, d[1].half()), (2, d[2].float()), (5, d[5][:1]),
                   (4, d[4].float()), (3, d[3][::2])):
        e = list(d)
        e[i] = bad
        with pytest.raises(ValueError):
            M.AdamWTensors([e])
    step, lr, _ = scalars(1, 1e-3)
    ts = M.AdamWTensors([d])
    with pytest.raises(ValueError):
        M.moe_adamw(ts, step.int(), lr)
    with pytest.raises(ValueError):
        M.moe_adamw(ts, step, lr.double())
    with pytest.raises(M.MoeError) as err:
        M.moe_adamw(M.AdamWTensors([d, d]), step, lr)       # the same tensor twice
    assert err.value.code == M.MOE_ERR_UNSUPPORTED
    with pytest.raises(M.MoeError):
        M.moe_adamw(ts, step, lr, beta1=1.0)
