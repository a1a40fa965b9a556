"""moe_router and its gradient against the float64 oracle: the choice exactly,
the weights within fp32.

Tolerances.  exp(v) of a rounded argument v is off by 2^-24 |v| and two half
steps of its own; a weight is a quotient of such terms and of a sum over at
most 16 values in a lane and 6 rounds of lanes.  With arguments below A in size
that makes 2^-24 (2 A + 40) of the weight; arguments beyond A = 90 give values
below 2^-126, which may be 0.
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
REL = 2.0 ** -24 * (2 * 90 + 40)
TINY = 2.0 ** -126
INF, NAN = float("inf"), float("nan")


def np64(t):
    return t.detach().double().cpu().numpy()


def recv(n):
    return torch.tensor([n], dtype=torch.int32, device="cuda")


def logits_of(seed, rows, E, dtype=F32, scale=1.5, masked=0.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, scale, (rows, E))
    x[rng.random((rows, E)) < masked] = -INF
    return torch.from_numpy(x).cuda().to(dtype)


def run(x, topk, bias=None, score="softmax", groups=1, topk_groups=1, normalize=True, nv=None):
    rows = x.shape[0]
    ids = torch.full((rows, topk), -9, dtype=torch.int32, device="cuda")
    w = torch.full((rows, topk), -9.0, device="cuda")
    M.moe_router(x, ids, w, bias, score, groups, topk_groups, normalize,
                 None if nv is None else recv(nv))
    n = rows if nv is None else max(0, min(nv, rows))
    want, ww = B.router(np64(x)[:n], topk, None if bias is None else np64(bias), score, groups,
                        topk_groups, normalize)
    got = ids.cpu().numpy()
    bad = np.nonzero((got[:n] != want).any(axis=1))[0]
    assert len(bad) == 0, (len(bad), bad[:3], got[bad[:3]], want[bad[:3]])
    err = np.abs(np64(w)[:n] - ww)
    assert (err <= REL * ww + TINY).all(), (err / np.maximum(ww, TINY)).max()
    assert (got[n:] == -9).all() and bool((w[n:] == -9).all())
    return ids, w


def run_backward(x, ids, score, normalize, nv=None, seed=0):
    rows, E = x.shape
    rng = np.random.default_rng(seed)
    dw = torch.from_numpy(rng.normal(0, 1, ids.shape)).cuda().float()
    dw[ids < 0] = NAN                               # of slots that chose nothing
    wide = torch.full((rows, E + 5), 7.0, dtype=x.dtype, device="cuda")
    dx = wide[:, :E]
    M.moe_router_backward(x, ids, dw, dx, score, normalize, None if nv is None else recv(nv))
    n = rows if nv is None else nv
    i = ids[:n].cpu().numpy().astype(np.int64)
    g = np.where(i >= 0, np64(dw)[:n], 0)
    want = B.router_backward(np64(x)[:n], i, g, score, normalize)
    w = B.router_weights(np64(x)[:n], i, score, normalize)
    # Terms: w_j g_j and s_j (or w_j) sum |w g|; the latter is at most
    # max(s_j, 1 of a named expert) times the sum.
    s = np.exp(B.log_scores(B.clean(np64(x)[:n]), score))
    if normalize:
        s = np.zeros_like(s)
    size = s * (np.abs(w * g)).sum(1, keepdims=True)
    for k in range(i.shape[1]):
        at = np.maximum(i[:, k], 0)
        add = np.abs(w[:, k]) * (np.abs(g[:, k]) + (np.abs(w * g)).sum(1)) * (i[:, k] >= 0)
        size[np.arange(n), at] += add
    half = 2.0 ** -8 if x.dtype == BF else 2.0 ** -24
    err = np.abs(np64(dx)[:n] - want)
    assert (err <= half * np.abs(want) + 2 * REL * size + TINY).all(), err.max()
    assert bool((dx[n:] == 7).all()) and bool((wide[:, E:] == 7).all())


@pytest.mark.parametrize("E", [1, 2, 5, 60, 64, 65, 128, 200, 256, 300, 512, 1000, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_plain_choice(E, score):
    for topk in sorted({1, min(E, 8), min(E, 32)}):
        for dtype, normalize, masked in ((F32, True, 0.0), (BF, False, 0.0), (F32, False, 0.4)):
            print(f"[router {E} top {topk} {score} {dtype} {normalize} {masked}]", flush=True)
            x = logits_of(E + topk, 67, E, dtype, masked=masked)
            ids, _ = run(x, topk, None, score, normalize=normalize, nv=61)
            run_backward(x, ids, score, normalize, nv=61, seed=E)


@pytest.mark.parametrize("E,groups,topk_groups", [(256, 8, 4), (256, 4, 1), (64, 8, 3), (60, 4, 2),
                                                  (160, 8, 3), (128, 64, 9), (7, 7, 3),
                                                  (1024, 2, 1), (1000, 40, 7), (512, 16, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(E, groups, topk_groups, score):
    topk = min(8, E // groups * topk_groups)
    for with_bias, masked in ((True, 0.0), (False, 0.0), (True, 0.6)):
        print(f"[router {E} {groups} {topk_groups} {score} {with_bias} {masked}]", flush=True)
        x = logits_of(E + groups, 131, E, masked=masked)
        bias = logits_of(3, 1, E, scale=0.2)[0] if with_bias else None
        run(x, topk, bias, score, groups, topk_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_bias(score):
    for E in (5, 64, 200, 256, 1024):
        bias = logits_of(7, 1, E, scale=0.3)[0]
        bias[E // 2] = -INF                          # never chosen, and still in the softmax
        bias[E - 1] = NAN
        bias[0] = INF if E > 64 else 0.0
        x = logits_of(E, 200, E)
        ids, _ = run(x, min(E, 6), bias, score, normalize=False)
        assert not bool(((ids == E // 2) | (ids == E - 1)).any())
        run_backward(x, ids, score, False)


def test_equal_scores_go_to_the_lowest():
    x = torch.zeros((3, 256), device="cuda")
    x[1, 100:] = 1
    x[2, ::2] = 2
    ids, w = run(x, 4)
    assert ids.tolist() == [[0, 1, 2, 3], [100, 101, 102, 103], [0, 2, 4, 6]]
    assert bool((w == 0.25).all())
    ids, _ = run(x, 4, torch.zeros(256, device="cuda"), "sigmoid", 8, 2)
    assert ids.tolist() == [[0, 1, 2, 3], [100, 101, 102, 103], [0, 2, 4, 6]]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for E in (33, 64, 256, 700):                     # whole numbers: equal ones everywhere
        x = torch.randint(-2, 3, (300, E), generator=g, device="cuda").float()
        run(x, 8)
        run(x.to(BF), 8, None, "sigmoid")
        run(x, 8, torch.zeros(E, device="cuda"), "sigmoid")
        if E % 4 == 0:
            run(x, 8, None, "softmax", 4, 2)


def test_scores_that_fp32_takes_for_equal():
    """Sigmoids of 17 and 17.25 are 1 - 4e-8 and 1 - 3e-8: one number in fp32."""
    x = torch.full((2, 64), -5.0, device="cuda")
    x[0, 3], x[0, 9] = 17.0, 17.25
    x[1, 9], x[1, 3] = 17.0, 17.25
    zero = torch.zeros(64, device="cuda")
    assert run(x, 2, zero, "sigmoid")[0].tolist() == [[9, 3], [3, 9]]
    assert run(x, 1, zero, "sigmoid", 2, 1)[0].tolist() == [[9], [3]]
    # A bias that makes up for all of the scores' difference but 2^-40.
    bias = torch.zeros(64, device="cuda")
    x = torch.full((1, 64), -5.0, device="cuda")
    x[0, 3], x[0, 9] = 0.0, 0.25
    s = 1 / (1 + np.exp(-0.25)) - 0.5
    bias[3] = float(np.float32(s))
    want = [3, 9] if float(np.float32(s)) > s else [9, 3]
    assert run(x, 2, bias, "sigmoid")[0].tolist() == [want]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_and_extreme_logits(dtype, score):
    low, top = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = logits_of(5, 12, 200, dtype)
    x[0] = -INF
    x[1] = -INF
    x[1, 77] = 3.0
    x[2] = NAN
    x[3, ::3] = NAN
    x[4, 150] = INF
    x[5] = low
    x[6, 5:] = low                                   # a mask of the type's lowest value
    x[7] = top
    x[8, 1:] = -INF
    x[8, 0] = low
    x[9] = -200.0                                    # sigmoids below fp32's range
    x[9, 4] = -190.0
    x[10] = 200.0
    x[11, 2:] = -INF
    for normalize in (True, False):
        for kw in (dict(), dict(bias=torch.zeros(200, device="cuda")),
                   dict(groups=8, topk_groups=3)):
            ids, w = run(x, 6, score=score, normalize=normalize, **kw)
            assert ids[0].tolist() == [-1] * 6 and ids[2].tolist() == [-1] * 6
            assert ids[1].tolist() == [77] + [-1] * 5
            assert bool(torch.isfinite(w).all())
            if not kw:
                run_backward(x, ids, score, normalize)


def test_rows_apart_and_received_rows():
    wide = logits_of(1, 20, 300, BF)
    for nv in (-1, 0, 1, 19, 50):
        run(wide[:, 7:199], 5, nv=nv)
    for rows in (0, 1):
        run(logits_of(2, rows, 64), 4)


def test_ids_that_name_nothing_and_the_same_twice():
    """Ids of other ranks' experts, of masked ones and -1 get no gradient; an
    expert that is named twice gets both."""
    x = logits_of(4, 6, 40)
    x[2, 5] = -INF
    ids = torch.tensor([[1, 1, 7], [-1, 40, 3], [5, 6, 6], [-7, -1, 99], [39, 0, 39], [2, 3, 4]],
                       dtype=torch.int32, device="cuda")
    clean = torch.where((ids < 40) & (ids >= 0), ids, torch.full_like(ids, -1))
    clean[2, 0] = -1
    dw = torch.randn((6, 3), device="cuda")
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            dx = torch.empty_like(x)
            M.moe_router_backward(x, ids, dw, dx, score, normalize)
            i = clean.cpu().numpy().astype(np.int64)
            want = B.router_backward(np64(x), i, np64(dw), score, normalize)
            # terms of size w g (w <= 1, |g| <= 4 here, three slots)
            assert np.abs(np64(dx) - want).max() <= 2 * REL * 16


def test_many_rows():
    """More rows than workgroups: each row's answer is its own."""
    x = logits_of(9, 64, 60)
    ids, w = run(x, 4)
    many = x.repeat(5000, 1)
    ids2 = torch.empty((len(many), 4), dtype=torch.int32, device="cuda")
    w2 = torch.empty((len(many), 4), device="cuda")
    M.moe_router(many, ids2, w2)
    assert torch.equal(ids2, ids.repeat(5000, 1)) and torch.equal(w2, w.repeat(5000, 1))
    dw = torch.randn((64, 4), device="cuda")
    dx, dx2 = torch.empty_like(x), torch.empty_like(many)
    M.moe_router_backward(x, ids, dw, dx)
    M.moe_router_backward(many, ids2, dw.repeat(5000, 1), dx2)
    assert torch.equal(dx2, dx.repeat(5000, 1))


def check_near(x, topk, bias, score, groups, topk_groups, normalize):
    """As run(); of keys that fp64 itself cannot tell, either order.  How many rows had
    such keys is returned.

    The oracle forms a score as exp(l), with l of a size below 8 here from a logarithm
    and a difference: l is off by at most 2^-53 (8 + 8 + 2), and exp adds a unit of
    2^-52: 2^-48 of the score at most.  The kernel's, an exp of a difference, a sum and
    a quotient, is nearer.  Adding the bias rounds by 2^-53 of a smaller number.  So two
    keys that are compared are off by 4 * 2^-48 of the row's largest score together, and
    sums of two by twice that.  (Logits 1 and 2 steps of 2^-20 apart and biases that make
    up for them do differ by less: 64 experts' scores lie about 2^-6, by a part of
    2^-20 to either side, and so the steps' products with them about 2^-26, the biases'
    own step: their keys differ by 1e-20 in more than one row.)"""
    rows, E = x.shape
    ids = torch.full((rows, topk), -9, dtype=torch.int32, device="cuda")
    w = torch.full((rows, topk), -9.0, device="cuda")
    M.moe_router(x, ids, w, bias, score, groups, topk_groups, normalize)
    want, _ = B.router(np64(x), topk, None if bias is None else np64(bias), score, groups,
                       topk_groups, normalize)
    got = ids.cpu().numpy().astype(np.int64)
    bad = np.nonzero((got != want).any(axis=1))[0]
    assert bias is not None or groups > 1 or len(bad) == 0
    s = np.exp(B.log_scores(B.clean(np64(x)), score))
    per = E // groups
    for r in bad:
        tol = 8 * 2.0 ** -48 * s[r].max()
        key = np.where(np.isneginf(np64(x)[r]), -np.inf,
                       s[r] + (0 if bias is None else np64(bias)))
        sums = np.sort(key.reshape(groups, per), axis=1)[:, -2:].sum(1)
        of = got[r] // per                           # the groups it chose, and the best others
        rest = [g for g in np.argsort(-sums, kind="stable") if g not in of]
        chosen = [*dict.fromkeys(of), *rest][:topk_groups]
        assert set(of) <= set(chosen), (r, got[r], want[r])
        out = [g for g in range(groups) if g not in chosen]
        if out:
            assert sums[chosen].min() >= sums[out].max() - tol, (r, got[r], want[r])
        best = np.sort(key[np.isin(np.arange(E) // per, chosen)])[::-1][:topk]
        assert len(set(got[r])) == topk and (got[r] >= 0).all(), (r, got[r])
        assert np.abs(key[got[r]] - best).max() <= tol, (r, got[r], want[r])
    ww = B.router_weights(np64(x), got, score, normalize)
    assert (np.abs(np64(w) - ww) <= REL * ww + TINY).all()
    return len(bad)


@pytest.mark.parametrize("E", [64, 100, 128, 200, 256, 512, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_keys_too_near_for_fp32(E, score):
    """Logits 2^-20 apart, with biases that take back their scores: every neighbour
    lies within fp32's errors."""
    rng = np.random.default_rng(E)
    for topk in (1, 8, 14, 15, 16):
        for groups, topk_groups in ((1, 1), (4, 2), (4, 3)):
            for taken_back in (True, False):
                if topk > E // groups * topk_groups:
                    continue
                print(f"[near keys {E} {score} top {topk} {groups} {topk_groups} "
                      f"{taken_back}]", flush=True)
                base = 0.5 + rng.integers(0, 3 if topk % 2 else 1 << 19, E) * 2.0 ** -20
                x = base + rng.integers(0, 4, (203, E)) * 2.0 ** -20
                x[7::9, ::3] = -INF
                bias = None
                if taken_back:
                    s = np.exp(B.log_scores(x[:1], score))[0]
                    b = -s.astype(np.float32) + np.float32(2.0 ** -26) * rng.integers(0, 4, E)
                    bias = torch.from_numpy(b.astype(np.float32)).cuda()
                held = torch.full((203, E + 4), -INF, device="cuda")
                for at in (0, 1):                    # 16-byte rows, and others
                    view = held[:, at:at + E]
                    view.copy_(torch.from_numpy(x))
                    print(f"  of 203 rows {check_near(view, topk, bias, score, groups, topk_groups, bool(at))}"
                          " in another order", flush=True)


@pytest.mark.parametrize("E,groups", [(256, 8), (64, 4), (128, 16), (60, 5), (512, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_whose_sums_leave_fp32(E, groups, score):
    """A bias of the lowest value is a key like others; two of a group's sum to less
    than fp32 holds, and the largest to more."""
    low = torch.finfo(F32).min
    x = logits_of(E, 37, E)
    for seed in range(3):
        rng = np.random.default_rng(seed)
        b = np.full(E, low)
        if seed:
            b[rng.random(E) < 0.1] = 0.0
        if seed == 2:
            b = rng.choice([low, low / 2, -low / 2, -low, 0.75 * -low], E)
        bias = torch.from_numpy(b).float().cuda()
        for topk in (3, 12):
            run(x, topk, bias, score, groups, 3)
            run(x, topk, bias, score)
