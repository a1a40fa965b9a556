"""moe_router's choice where keys are hard to tell apart, exactly, against the float64
oracle, on every path: four rows to a wave (up to 256 experts and 14 choices), a wave
to a row, and groups that no path in fp32 takes."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402
from oracle import block as B  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF, F32 = torch.bfloat16, torch.float32


def choice(x, topk, bias=None, score="softmax", groups=1, topk_groups=1, dtype=F32):
    """Ids for the rows x as they are and for the same rows apart and off 16 bytes."""
    rows, E = x.shape
    held = torch.full((rows, E + 3), float("nan"), dtype=dtype, device="cuda")
    b = None if bias is None else torch.from_numpy(bias).float().cuda()
    got = []
    for view in (held[:, 1:1 + E], torch.empty((rows, E), dtype=dtype, device="cuda")):
        view.copy_(torch.from_numpy(x))
        ids = torch.full((rows, topk), -9, dtype=torch.int32, device="cuda")
        M.moe_router(view, ids, torch.empty((rows, topk), device="cuda"), b, score, groups,
                     topk_groups)
        got.append(ids.cpu().numpy())
    assert np.array_equal(*got)
    return got[0]


def keys(x, bias, score):
    return np.exp(B.log_scores(B.clean(x), score)) + bias.astype(np.float64)


# ------------------------------------------------------------- near keys

def pairs_on_edges(rng, rows, E, levels, score):
    """Logits and biases (as fp32) whose 2 * levels largest keys are pairs about
    multiples of 2^-13, a border of the numbers that are compared first for any number
    of experts: within some 2^-25 of it, on either side."""
    if score == "sigmoid":
        bias, lo, hi = rng.uniform(-0.25, 0.25, E), 0.45, 1.1
    else:                                            # scores of 0.01 to 0.04 beside biases
        bias, lo, hi = rng.uniform(0.5, 0.505, E), 0.515, 0.54
        bias[E - 1] = -1.0                           # takes what the others leave
    bias = bias.astype(np.float32)
    x = np.empty((rows, E))
    grid = np.arange(int(lo * 2 ** 13), int(hi * 2 ** 13))
    for r in range(rows):
        level = np.repeat(rng.choice(grid, levels, replace=False) / 2.0 ** 13, 2)
        at = rng.permutation(E - 1)[:2 * levels]
        s = level - bias[at].astype(np.float64)
        if score == "sigmoid":
            at, s = at[(s > 0.03) & (s < 0.97)], s[(s > 0.03) & (s < 0.97)]
            x[r] = -12.0                             # a key below 0.25 + 1e-5
            x[r, at] = np.log(s / (1 - s))
        else:
            x[r] = np.log(1e-9)
            x[r, at] = np.log(s)
            x[r, E - 1] = np.log(1 - s.sum() - 1e-9 * (E - 1 - len(at)))
    step = rng.integers(-1, 2, x.shape)
    x = x.astype(np.float32)
    return x + (step * np.spacing(np.abs(x))).astype(np.float32), bias


@pytest.mark.parametrize("E", [64, 100, 128, 200, 256, 300, 512, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_keys_on_both_sides_of_a_border(E, score):
    """The order of each pair, and which of a pair is the last one chosen.

    The oracle's score, exp of a logarithm l of size below 24, is off by 2^-53 (3 * 24 + 2)
    at most and a key near 1 by half a step more, the kernel's by less: keys that lie
    within 2 * (2^-46 + 2^-53) of each other may come in either order."""
    for topk in (1, 7, 8, 13, 14, 15, 16):
        print(f"[edges {E} {score} top {topk}]", flush=True)
        rng = np.random.default_rng(E + topk)
        x, bias = pairs_on_edges(rng, 301, E, topk // 2 + 1, score)
        got = choice(x, topk, bias, score)
        want, _ = B.router(x, topk, bias, score)
        key = keys(x, bias, score)
        d = np.take_along_axis(key, got, 1) - np.take_along_axis(key, want, 1)
        bad = np.nonzero((np.abs(d) > 2.0 ** -44).any(axis=1))[0]
        assert len(bad) == 0, (len(bad), bad[:3], got[bad[:3]], want[bad[:3]])
        assert all(len(set(row)) == topk and (row >= 0).all() for row in got)


# ---------------------------------------------------------- signed zeros

@pytest.mark.parametrize("E", [5, 8, 60, 64, 100, 128, 256, 300, 512, 1024])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_zeros_of_either_sign_are_equal(E, dtype):
    rng = np.random.default_rng(E)
    x = np.where(rng.random((203, E)) < 0.5, -0.0, 0.0)
    x[100:150][rng.random((50, E)) < 2 / E] = 1.0
    x[150:][rng.random((53, E)) < 0.5] = -2.0 ** -126    # the zeros lead
    for topk in sorted({1, 2, min(E, 8), min(E, 16), min(E, 32)}):
        print(f"[zeros {E} {dtype} top {topk}]", flush=True)
        for score in ("softmax", "sigmoid"):
            want, _ = B.router(x, topk, None, score)
            assert np.array_equal(choice(x, topk, None, score, dtype=dtype), want)
        zero = np.where(rng.random(E) < 0.5, -0.0, 0.0)
        assert np.array_equal(choice(x[:100], topk, zero, "sigmoid", dtype=dtype),
                              B.router(x[:100], topk, zero, "sigmoid")[0])
        if E % 4 == 0 and topk <= E // 2:
            assert np.array_equal(choice(x[:150], topk, None, "softmax", 4, 2, dtype),
                                  B.router(x[:150], topk, None, "softmax", 4, 2)[0])


# ------------------------------------------------------- sums that cancel

@pytest.mark.parametrize("E,groups", [(16, 4), (64, 8), (128, 4), (256, 8), (256, 4), (60, 5),
                                      (512, 8), (1024, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_that_cancel(E, groups, score):
    """Two keys of a group near +B and -B, the others below: their sum is known to
    their own errors, not to its own.  B is another one for each group, so that the
    keys are far apart.  fp64 holds one near 2^28 to 2^-25, two of two groups 2^-23
    together, and the sums here, of scores drawn at random, lie 2^-20 apart and more
    (looked at)."""
    rng = np.random.default_rng(E + groups)
    per = E // groups
    for size in (20.0, 1000.0, 2.0 ** 14, 2.0 ** 20, 2.0 ** 24):
        low = -4 * size * groups
        bias = np.full((groups, per), low)
        for g in range(groups):
            at = rng.permutation(per)[:2]
            bias[g, at] = size * (g + 1), -size * (g + 1)
        if size == 1000.0:
            bias[0] = low                            # one that does not cancel, and is last
        bias = bias.reshape(-1).astype(np.float32)
        x = np.round(rng.normal(0, 1.5, (151, E)) * 256) / 256
        if score == "softmax":
            x[:, bias < low / 2] -= 6              # leaves the pairs scores worth telling
        topk_groups = groups // 2
        s = np.exp(B.log_scores(x, score)).reshape(151, groups, per)
        two = np.where(bias.reshape(groups, per) > low / 2, s, 0).sum(axis=2)
        two[:, (bias.reshape(groups, per) < low / 2).all(axis=1)] = -1
        order = np.sort(two, axis=1)[:, ::-1]
        told = order[:, topk_groups - 1] - order[:, topk_groups] > 2.0 ** -20
        assert told.sum() > 120
        x = x[told]
        for topk in (topk_groups, min(2 * topk_groups, 32)):
            print(f"[cancel {E} {groups} {score} {size} top {topk}]", flush=True)
            got = choice(x, topk, bias, score, groups, topk_groups)
            want, _ = B.router(x, topk, bias, score, groups, topk_groups)
            of = lambda ids: np.sort(np.unique(ids // per))  # noqa: E731
            bad = [r for r in range(len(x)) if not np.array_equal(of(got[r]), of(want[r]))]
            assert not bad, (len(bad), got[bad[:3]], want[bad[:3]])


# ---------------------------------------------- scores that are one number

@pytest.mark.parametrize("E,groups", [(16, 4), (64, 4), (128, 8), (256, 8), (256, 2), (60, 4),
                                      (160, 8), (512, 8), (1024, 2), (7, 7)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_equal_scores_of_different_logits(E, groups, dtype):
    """With groups it is the scores that are compared: sigmoids of 40, 50 and 60 are 1,
    those of -800 and -900 are 0, and so are softmax's beside a 0; the lowest expert
    comes first.  Without groups and bias the logits are."""
    rng = np.random.default_rng(E)
    for score, some in (("sigmoid", [40.0, 50.0, 60.0, 2.0, 1.0, -1.0]),
                        ("sigmoid", [-800.0, -900.0, -1000.0, -2.0]),
                        ("softmax", [0.0, -800.0, -900.0, -1000.0]),
                        ("softmax", [1000.0, 20.0, 10.0, float("inf"), -float("inf")])):
        x = rng.choice(some, (101, E))
        x[:, 0] = some[0]
        if len(some) == 4 and score == "softmax":
            x[50:, 1:] = rng.choice(some[1:], (51, E - 1))
        for topk_groups in sorted({1, groups // 2, groups}):
            for topk in sorted({1, min(8, E // groups * topk_groups),
                                min(20, E // groups * topk_groups)}):
                print(f"[equal scores {E} {groups} {topk_groups} {score} {dtype} top {topk}]",
                      flush=True)
                got = choice(x, topk, None, score, groups, topk_groups, dtype)
                want, _ = B.router(x, topk, None, score, groups, topk_groups)
                assert np.array_equal(got, want)
        got = choice(x, min(8, E), None, score, dtype=dtype)
        assert np.array_equal(got, B.router(x, min(8, E), None, score)[0])
