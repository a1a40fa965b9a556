"""Pins of the oracle for the norm, the router and the 4-bit weights: against
torch in float64, and gradients against central differences."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import block as B  # noqa: E402

RNG = np.random.default_rng(11)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_against_torch_and_differences(rms):
    h, w, b = RNG.normal(2, 3, (5, 24)), RNG.normal(1, .2, 24), RNG.normal(0, 1, 24)
    y, mean, rstd = B.layer_norm(h, w, b, 1e-5, rms)
    if not rms:
        t = torch.nn.functional.layer_norm(*(torch.from_numpy(v) for v in (h,)), (24,),
                                           torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    else:
        t = torch.from_numpy(h)
        t = t / (t.pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * torch.from_numpy(w) + \
            torch.from_numpy(b)
    np.testing.assert_allclose(y, t.numpy(), rtol=1e-12, atol=1e-12)
    dy = RNG.normal(0, 1, h.shape)
    dx, dw, db = B.layer_norm_backward(dy, h, w, mean, rstd, rms)
    f = lambda h, w, b: (B.layer_norm(h, w, b, 1e-5, rms)[0] * dy).sum()  # noqa: E731
    step = 1e-5
    for got, args, k in ((dx, (h, w, b), 0), (dw, (h, w, b), 1), (db, (h, w, b), 2)):
        for at in list(np.ndindex(got.shape))[:60]:
            hi, lo = ([a.copy() for a in args] for _ in range(2))
            hi[k][at] += step
            lo[k][at] -= step
            d = (f(*hi) - f(*lo)) / (2 * step)
            assert abs(d - got[at]) < 1e-7 * (1 + abs(d))


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_gradient_against_differences(score, normalize):
    x = RNG.normal(0, 1.5, (4, 9))
    x[1, 3] = -np.inf
    x[2, 1:] = -np.inf
    ids, w = B.router(x, 3, None, score, 1, 1, normalize)
    g = RNG.normal(0, 1, w.shape)
    d = B.router_backward(x, ids, g, score, normalize)
    f = lambda v: (np.where(ids >= 0, B.router_weights(v, ids, score, normalize), 0) * g).sum()  # noqa: E731
    for at in np.ndindex(x.shape):
        if np.isneginf(x[at]):
            assert d[at] == 0
            continue
        hi, lo = x.copy(), x.copy()
        hi[at] += 1e-5
        lo[at] -= 1e-5
        assert abs((f(hi) - f(lo)) / 2e-5 - d[at]) < 1e-8


def test_router_by_hand():
    n, i = np.nan, np.inf
    x = np.array([[1, 3, 3, 2], [-i, n, 5, -i], [-i, -i, n, -i], [0, i, -3e38, 0]])
    ids, w = B.router(x, 2)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [1, 0]]
    np.testing.assert_allclose(w, [[.5, .5], [1, 0], [0, 0], [1, 0]], atol=1e-12)
    for score in ("softmax", "sigmoid"):             # equal lowest values share alike
        w = B.router(np.full((1, 5), -3e38), 4, None, score)[1]
        np.testing.assert_allclose(w, np.full((1, 4), 0.25))
    w = B.router(np.full((1, 5), -3e38), 4, normalize=False)[1]
    np.testing.assert_allclose(w, np.full((1, 4), 0.2))
    # Two groups: {0, 1} sums 4, {2, 3} sums 5; only the second is chosen from.
    s = lambda v: np.log(v / (1 - v))  # noqa: E731  a sigmoid's argument
    x = s(np.array([[.9, .1, .6, .7]]))
    assert B.router(x, 2, None, "sigmoid", 2, 1)[0].tolist() == [[3, 2]]
    ids, w = B.router(x, 3, np.array([0, -1, 0, 0.]), "sigmoid", 1, 1, False)
    assert ids.tolist() == [[0, 3, 2]]
    np.testing.assert_allclose(w, [[.9, .7, .6]])


def test_code_values():
    w = np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe] * 2], np.uint8)
    v = B.w4_values(w, np.array([[0.5, 2.0]]), "int4")[0]
    assert v[:16].tolist() == [x / 2 for x in [*range(8), *range(-8, 0)]]
    assert v[16:].tolist() == [x * 2 for x in [*range(8), *range(-8, 0)]]
    v = B.w4_values(w, np.array([[128]]), "mxfp4")[0]
    half = [0, 1, 2, 3, 4, 6, 8, 12]
    assert v[:16].tolist() == half + [-x for x in half]
