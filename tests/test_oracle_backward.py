"""Pins of the oracle's gradients and AdamW step (CPU only).

* the layer's gradients against central differences of the layer in float64;
* the stage gradients (combine, products, SiLU*up), chained over the expanded
  rows, against the per-token gradient of the layer;
* the AdamW step against torch.optim.AdamW in float64;
* the coded states against the rounding of E4M3.
Planted mistakes are caught.
"""

import numpy as np
import pytest

from oracle import backward as B
from oracle import layout

torch = pytest.importorskip("torch")


def small(seed=3, rows=5, hidden=6, inter=4, experts=3, topk=2):
    g = np.random.default_rng(seed)
    ids = np.stack([g.permutation(experts)[:topk] for _ in range(rows)]).astype(np.int32)
    ids[0, 0] = -1
    return dict(x=g.standard_normal((rows, hidden)), ids=ids, w=g.random((rows, topk)) + 0.1,
                w13=g.standard_normal((experts, 2 * inter, hidden)) * 0.5,
                w2=g.standard_normal((experts, hidden, inter)) * 0.5, f=2.5,
                num_valid=rows - 1), g.standard_normal((rows, hidden))


def _differences(a, dout, name, h=1e-5):
    d = np.zeros(a[name].shape)
    for i in np.ndindex(d.shape):
        v = []
        for sgn in (1, -1):
            b = dict(a)
            b[name] = a[name].copy()
            b[name][i] += sgn * h
            v.append((B.layer(**b) * dout).sum())
        d[i] = (v[0] - v[1]) / (2 * h)
    return d


def test_layer_gradient_against_differences():
    a, dout = small()
    dout[a["num_valid"]:] = 0.0
    got = dict(zip(("x", "w", "w13", "w2"), B.layer_backward(**a, dout=dout)))
    for name, d in got.items():
        # central differences: h^2 |f'''| / 6 plus 1e-16 |f| / h, both below 1e-8
        assert np.allclose(d, _differences(a, dout, name), rtol=1e-6, atol=1e-7), name
        assert np.abs(d).max() > 0.01


def test_planted_gate_up_swap_is_caught(monkeypatch):
    orig = B.silu_mul_backward
    monkeypatch.setattr(B, "silu_mul_backward", lambda g, u, dy: orig(g, u, dy)[::-1])
    with pytest.raises(AssertionError):
        test_layer_gradient_against_differences()


def test_stage_gradients_chain_to_the_layers():
    a, dout = small(seed=8, rows=9, hidden=10, inter=6)
    E, inter, align = 3, 6, 16
    cap = layout.capacity(9, 2, E, align)
    lay = layout.expand_layout(a["ids"], a["num_valid"], E, align, cap)
    lab = B.live_rows(lay["psum"], align, cap)
    src = lay["src2dst"]
    ex = np.zeros((cap, 10))
    for r, k in zip(*np.nonzero(src >= 0)):
        ex[src[r, k]] = a["x"][r]
    live = lab >= 0
    gu, D = np.zeros((cap, 2 * inter)), np.zeros((cap, 10))
    for m in np.nonzero(live)[0]:
        gu[m] = a["w13"][lab[m]] @ ex[m]
    y = gu[:, :inter] * B.sigmoid(gu[:, :inter]) * gu[:, inter:]
    for m in np.nonzero(live)[0]:
        D[m] = a["w2"][lab[m]] @ y[m]
    rows, dc = B.gather_backward(dout, D, src, a["w"], a["f"], a["num_valid"], cap)
    dD = np.zeros((cap, 10))
    for d, v in rows.items():
        dD[d] = v
    dw2, _ = B.wgrad(dD, y, lab, E)
    dy, _ = B.dgrad(dD, a["w2"], lab)
    dgu = np.concatenate(B.silu_mul_backward(gu[:, :inter], gu[:, inter:], dy), axis=1)
    dw13, _ = B.wgrad(dgu, ex, lab, E)
    dex, _ = B.dgrad(dgu, a["w13"], lab)
    dx = np.zeros((9, 10))
    for r, k in zip(*np.nonzero(src >= 0)):
        dx[r] += dex[src[r, k]]
    for got, want in zip((dx[:8], dc, dw13, dw2), B.layer_backward(**a, dout=dout)):
        assert np.allclose(got, want[:len(got)], rtol=1e-12, atol=1e-13)


def test_live_rows():
    assert B.live_rows([3, 16, 33], 16, 48).tolist() == (
        [0] * 3 + [-1] * 13 + [2] * 17 + [-1] * 15)  # expert 1 starts and ends at 16


@pytest.mark.parametrize("t,wd", [(1, 0.0), (7, 0.1)])
def test_adamw_against_torch(t, wd):
    g = np.random.default_rng(t)
    n, lr, b1, b2, eps = 257, 1e-2, 0.9, 0.95, 1e-8
    p = g.standard_normal(n).astype(np.float32)
    q = torch.nn.Parameter(torch.from_numpy(p).double())
    opt = torch.optim.AdamW([q], lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd)
    m, v = np.zeros(n, np.float32), np.zeros(n, np.float32)
    for i in range(1, t + 1):
        grad = g.standard_normal(n).astype(np.float32)
        q.grad = torch.from_numpy(grad).double()
        opt.step()
        p, m, v = B.adamw_f32(p, grad, m, v, i, lr, b1, b2, eps, wd, 1.0)
    # each step: at most half a step of p (2^-24 |p|, |p| < 8) twice, and a
    # dozen roundings of an update of about lr
    assert np.abs(p - q.detach().numpy()).max() <= t * (2 * 8 * 2 ** -24 + 12 * lr * 2 ** -22)


@pytest.mark.parametrize("n", [1, 127, 128, 129, 1000])
def test_coded_states(n):
    g = np.random.default_rng(n)
    x = (g.standard_normal(n) * np.exp(g.uniform(-12, 0, n))).astype(np.float32)
    for pos in (False, True):
        y = np.abs(x) if pos else x
        codes, scale = B.encode_state(y, pos)
        assert codes.shape == (n,) and scale.shape == (-(-n // 128),)
        s = np.repeat(scale, 128)[:n].astype(np.float64)
        # half a step: 2^-4 relative, 2^-10 in units of the scale below 2^-6; the
        # lifted positive values are at most 2^-9 off; plus three fp32 roundings
        err = np.abs(B.decode_state(codes, scale) - y.astype(np.float64))
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(y), (2.0 ** -9 if pos else 2.0 ** -10)
                                        * s) * (1 + 2.0 ** -20))
        if pos:
            assert np.all(B.decode_state(codes, scale) > 0)
    codes, scale = B.encode_state(np.zeros(n, np.float32), True)
    assert not codes.any() and np.all(scale > 0)


