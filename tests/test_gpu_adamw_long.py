"""moe_adamw with 8-bit states whose betas are near 1: the codes against the
oracle's, bit for bit, and many steps against fp32 states."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402
from tests.test_gpu_adamw import compare, make, scalars  # noqa: E402
from oracle import backward as B  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

SIZES = [1, 127, 129, 1000, 2049, 40000]


def expect(h, t, hyper):
    """The oracle's step with the codes that both betas call for; the bar of the master."""
    m, r = B.decode_state(h["m"], h["ms"]), B.decode_state(h["v"], h["vs"])
    p, m, v = B.adamw_f32(h["p"], h["grad"], m, r * r, t, 1e-3, hyper["beta1"], hyper["beta2"],
                          hyper["eps"], hyper["weight_decay"], 0.25)
    step = np.abs(p.astype(np.float64) - h["p"])
    r = np.sqrt(v)
    bm, br = B.dither_bits(m, r, t)
    h["m"], h["ms"] = B.encode_state(m, False, bm if hyper["beta1"] > 31 / 32 else None)
    h["v"], h["vs"] = B.encode_state(r, True, br if hyper["beta2"] > 31 / 32 else None)
    h["p"] = p
    return 2.0 ** -23 * np.abs(p) + 2.0 ** -20 * (step + 2.0 ** -23 * np.abs(p)) + 2.0 ** -149


@pytest.mark.parametrize("beta1,beta2", [(0.9, 0.999), (0.99, 0.95), (0.99, 0.999),
                                         (31 / 32, 31 / 32), (0.96876, 0.96876)])
def test_codes(beta1, beta2):
    """Steps 1, 2 and ones past 32 bits."""
    hyper = dict(beta1=beta1, beta2=beta2, eps=1e-8, weight_decay=0.1)
    both = [make(n, i, True, i % 2 == 0, i % 3 != 0) for i, n in enumerate(SIZES)]
    ts = M.AdamWTensors([d for _, d in both])
    for t in (1, 2, (1 << 32) + 3):
        print(f"adamw beta {beta1} {beta2} step {t}", flush=True)
        step, lr, gs = scalars(t, 1e-3, 0.25)
        M.moe_adamw(ts, step, lr, grad_scale=gs, **hyper)
        for (h, d), n in zip(both, SIZES):
            compare(h, d, expect(h, t, hyper), f"size {n} step {t}")


def follow(beta1, beta2, drop, steps, mean, noise):
    """8-bit and fp32 states under the same gradients, normal ones around `mean`
    with deviation `noise` in units of each element's size; every other
    element's fall tenfold after `drop` steps.  Ratios of the states: m, root."""
    n = 64 * 128
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    normal = lambda: torch.empty(n, device="cuda").normal_(generator=g)  # noqa: E731
    size = torch.exp(normal()) * torch.sign(normal())
    falls = torch.arange(n, device="cuda") % 2 == 0
    z = lambda d=torch.float32, k=n: torch.zeros(k, dtype=d, device="cuda")  # noqa: E731
    grad, c = z(), torch.uint8
    coded = (z(), grad, z(c), z(c), None, z(k=64), z(k=64))
    plain = (z(), grad, z(), z(), None, None, None)
    ts = M.AdamWTensors([coded, plain])
    step, lr, _ = scalars(0, 1e-3)
    for t in range(1, steps + 1):
        now = size * torch.where(falls & (t > drop), 0.1, 1.0)
        grad.copy_(now * mean + now * noise * normal())
        step.add_(1)
        M.moe_adamw(ts, step, lr, beta1=beta1, beta2=beta2)
    value = lambda q, s: (q.view(torch.float8_e4m3fn).float().view(-1, 128)  # noqa: E731
                          * s[:, None]).view(-1)
    m = value(coded[2], coded[5]) / plain[2]
    r = value(coded[3], coded[6]) / plain[3].sqrt()
    return [x[k].median().item() for x in (m, r) for k in (falls, ~falls)]


@pytest.mark.parametrize("beta2,drop,steps", [(0.99, 500, 1500), (0.999, 2000, 10000)])
def test_second_moments_follow_their_gradients(beta2, drop, steps):
    """The bar is derived in test_state_coding.py: 15 % of the median root."""
    _, _, falling, others = follow(0.9, beta2, drop, steps, 0.0, 1.0)
    print(f"roots {falling:.3f} {others:.3f}", flush=True)
    assert abs(falling - 1) <= 0.15 and abs(others - 1) <= 0.15


def test_first_moments_follow_their_gradients():
    """Gradients around a mean of their own size.  A step adds at most gap * move
    to m's relative variance, gap 1/8, move (1 - beta1) * 0.8 for m and as much
    for its scale, and forgets 2 (1 - beta1) of it: s^2 <= 0.1, and m has no bias.
    The median of 4096 ratios is then within 4 * 1.25 s / 64 = 2.5 % of 1, but
    for what is left from before the fall (10 * 0.99^1000 < 0.1 %), and for the
    few m that noise brings near 0, whose ratios spread to both sides alike.
    10 % hold."""
    falling, others, _, _ = follow(0.99, 0.95, 500, 1500, 1.0, 1.0)
    print(f"first moments {falling:.3f} {others:.3f}", flush=True)
    assert abs(falling - 1) <= 0.1 and abs(others - 1) <= 0.1
