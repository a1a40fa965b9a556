"""8-bit optimiser states over many steps (oracle, CPU): a state whose beta is
near 1 has to follow its gradients although one step moves it by less than
its codes lie apart."""

import numpy as np
import pytest

from oracle import backward as B
from oracle import fp8

F = np.float32


def test_neighbours():
    """A code's own value stays; anything else goes to the two codes around it,
    up as often as it lies above the lower one."""
    grid = fp8.decode_e4m3(np.arange(0x7f, dtype=np.uint8)).astype(F)     # 0 .. 448, ascending
    assert np.all(np.diff(grid) > 0) and grid[-1] == 448
    ends = np.array([0, 1, 0x80000, 0xfffff], np.uint32)
    for s in (F(1), F(-1)):
        for b in ends:
            assert np.array_equal(B.to_neighbour(s * grid, b), s * grid)
    # Points at 1/8 .. 7/8 of each gap, exact in fp32 (and, lifted by 2^-6, too):
    # up for the bits from 2^20 (1 - part) on.
    for part in np.arange(1, 8) / F(8):
        q = (grid[:-1] + part * np.diff(grid)).astype(F)
        edge = np.uint32(2 ** 20 * (1 - part))
        assert np.array_equal(B.to_neighbour(q, edge), grid[1:])
        assert np.array_equal(B.to_neighbour(q, edge - np.uint32(1)), grid[:-1])
    over, nan = F(448.00003), F("nan")
    assert B.to_neighbour(over, ends[-1:])[0] == over and np.isnan(B.to_neighbour(nan, ends[-1:]))[0]


@pytest.mark.parametrize("which", ["m", "r"])
def test_the_expected_code_is_the_value(which):
    """Mean over T steps of states that stay: one step is at most a code's
    distance d off, so the mean's standard deviation is at most d / (2 sqrt T),
    and six of them hold for 2048 values (chance 4e-6); the state itself is
    decoded with three roundings."""
    g = np.random.default_rng(3)
    n, T = 2048, 4096
    m = (g.standard_normal(n) * np.exp(g.uniform(-6, 0, n))).astype(F)
    r = (np.abs(m) + F(1e-6)).astype(F)
    total, sum_scale = np.zeros(n), None
    for t in range(1, T + 1):
        bm, br = B.dither_bits(m, r, t)
        codes, scale = (B.encode_state(m, False, bm) if which == "m"
                        else B.encode_state(r, True, br))
        total += B.decode_state(codes, scale)
        sum_scale = scale
    x = (m if which == "m" else r).astype(np.float64)
    s = np.repeat(sum_scale, 128)[:n].astype(np.float64)
    q = np.abs(x) / s
    d = np.maximum(2.0 ** -9, 2.0 ** (np.floor(np.log2(np.maximum(q, 2.0 ** -6))) - 3)) * s
    if which == "r":   # a positive root gets the smallest code at least
        x = np.maximum(x, 2.0 ** -9 * s)
    assert np.all(np.abs(total / T - x) <= 6 * d / (2 * np.sqrt(T)) + 2.0 ** -21 * np.abs(x))


def second_moments(beta, drop, steps, dither):
    """Ratio of coded roots to fp32 ones; every other gradient falls tenfold."""
    g = np.random.default_rng(11)
    n = 16 * 128
    size = np.exp(g.normal(0, 1, n)).astype(F)
    falls = np.arange(n) % 2 == 0
    v = np.zeros(n, F)
    codes, scale = B.encode_state(v, True)
    m = np.zeros(n, F)
    for t in range(1, steps + 1):
        grad = (g.standard_normal(n) * size * np.where(falls & (t > drop), 0.1, 1.0)).astype(F)
        r = B.decode_state(codes, scale)
        new = np.sqrt(r * r * F(beta) + grad * grad * F(1 - beta)).astype(F)
        v = v * F(beta) + grad * grad * F(1 - beta)
        m = m * F(0.9) + grad * F(0.1)
        codes, scale = B.encode_state(new, True, B.dither_bits(m, new, t)[1] if dither else None)
    ratio = B.decode_state(codes, scale) / np.sqrt(v)
    return np.median(ratio[falls]), np.median(ratio[~falls])


@pytest.mark.parametrize("beta,drop,steps", [(0.99, 500, 1500), (0.999, 2000, 10000)])
def test_roots_follow_their_gradients(beta, drop, steps):
    """A root's relative spread s: each step adds at most gap * move to its
    variance, gap 1/8 and move |g^2/v - 1| (1 - beta)/2, 0.97 (1 - beta)/2 in the
    mean, for the root and as much for its group's scale; the average forgets
    (1 - beta) of it a step.  So s^2 <= 0.125 * 0.97 = 0.12.  The second moment
    is s^2 too large in the mean at most (a root is unbiased, its square is
    not), so the median root lies at most 6 % high, and the median of 1024 is
    within 4 * 1.25 s / 32 = 6 % more of that, for the falling ones 2 % of what
    was there before at most.  15 % hold."""
    for median in second_moments(beta, drop, steps, True):
        assert abs(median - 1) <= 0.15


def test_nearest_codes_would_not():
    """What the rule is for: far above what the falling gradients give."""
    assert second_moments(0.99, 500, 1500, False)[0] > 2
