"""GPU parity of the bf16 path's gradients through the C ABI, against the
oracle's float64 gradients on the same inputs.

Bars (derived, per element):
* products: a product of two bf16 values is exact in fp32, and each of the
  L - 1 additions (and the joining ones) is off by at most one fp32 step of
  the running sum, so |err| <= L * 2^-23 * sum |a b|; then one rounding, bf16
  2^-8 or fp32 2^-24 of the value.
* SiLU*up: expf, the sum and the quotient leave s off by at most 2^-21 of
  itself (4 fp32 steps), so 1 + g (1 - s) is off by at most (1 + |g|) * 2^-20
  and d g by |dy u| s (1 + |g|) 2^-19; d u by |dy g s| 2^-20; then 2^-8.
* combine: rows are exact (two fp32 products, one rounding); the dots have
  H terms: H * 2^-23 * |f| sum |dout D|.
Rows and experts that are not live hold NaN in every input and sentinels in
every output.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402
from oracle import backward as B  # noqa: E402
from oracle import fp8, layout  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16
TINY = 2.0 ** -133   # half a step of the smallest bf16 values


def dev_layout(counts, align, spare=0, total=None):
    """psum, status, m_indices of expert blocks, on the GPU and on the host."""
    psum, end = [], 0
    for c in counts:
        psum.append(end + c)
        end = -(-psum[-1] // align) * align
    cap = end + spare * align
    labels = np.full(cap, -1, np.int32)
    start = 0
    for e, p in enumerate(psum):
        nxt = -(-p // align) * align
        labels[start:nxt] = e
        start = nxt
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    total = end if total is None else total
    lab = B.live_rows(psum, align, min(cap, total))
    lab = np.concatenate([lab, np.full(cap - len(lab), -1)])
    return dict(psum=t(psum), status=t([total, 0]), m_indices=t(labels), cap=cap, lab=lab,
                align=align, E=len(counts))


def bf16(gen, shape, scale=1.0):
    x = torch.from_numpy(gen.standard_normal(shape).astype(np.float32) * np.float32(scale))
    return x.to(BF)


def poisoned(x, lab):
    x = x.clone()
    x[torch.from_numpy(lab < 0)] = float("nan")
    return x.cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(got, ref, bar, what):
    bad = ~(np.abs(got - ref) <= bar)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - ref) / bar):.3g} of the bar")


# live rows per expert, n, k, align, spare blocks behind the total
PRODUCTS = [
    ([1], 128, 64, 16, 0),
    ([0, 0, 0], 128, 64, 16, 1),                       # nothing live at all
    ([5, 0, 16, 1], 128, 192, 16, 1),
    ([63, 64, 65], 256, 128, 64, 0),
    ([127, 0, 128, 129], 128, 320, 128, 1),
    ([31, 33, 2, 257, 0, 15, 17], 384, 256, 32, 2),
    ([255, 256, 257, 511, 513], 256, 384, 16, 0),
    ([1] * 70, 128, 128, 16, 3),                       # more experts than lanes
    ([300, 7], 512, 640, 256, 0),
    ([3000], 256, 256, 128, 0),                        # one long reduction, few tiles
    ([1500, 0, 700], 128, 64, 128, 4),
    ([20000, 1], 128, 128, 16, 0),
    ([40, 0, 1, 70] * 16, 384, 320, 16, 1),            # tiles enough for the wide kernels
    ([129, 300, 0, 513, 64, 1, 256, 33] * 2, 256, 1088, 64, 1),
    ([3000, 700, 0, 129], 128, 5056, 64, 1),           # ... and with a cut last round
    ([2, 0, 0, 17] * 50, 128, 64, 16, 0),
]
PIDS = [f"{'_'.join(map(str, c[0][:4]))}-n{c[1]}-k{c[2]}-a{c[3]}" for c in PRODUCTS]


@pytest.mark.parametrize("counts,n,k,align,spare", PRODUCTS, ids=PIDS)
def test_dgrad(counts, n, k, align, spare):
    print(f"dgrad {counts[:8]} n {n} k {k} align {align}", flush=True)
    g = np.random.default_rng(n + k)
    L = dev_layout(counts, align, spare)
    dy, w = bf16(g, (L["cap"], n), 0.1), bf16(g, (L["E"], n, k))
    dx = torch.full((L["cap"], k), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_dgrad_bf16(poisoned(dy, L["lab"]), w.cuda(), L["psum"], L["status"], align, dx)
    ref, mag = B.dgrad(dy.float().numpy(), w.float().numpy(), L["lab"])
    got, live = f64(dx), L["lab"] >= 0
    assert np.all(got[~live] == 7.0)
    check(got[live], ref[live],
          2.0 ** -8 * np.abs(ref[live]) + n * 2.0 ** -23 * mag[live] + TINY, "dx")


def workspace(L, n, k):
    need = M.moe_grouped_wgrad_workspace_bytes(L["cap"], n, k, L["E"])
    return None if need == 0 else torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("f32,accumulate", [(False, False), (True, False), (True, True),
                                            (False, True)])
@pytest.mark.parametrize("counts,n,k,align,spare", PRODUCTS, ids=PIDS)
def test_wgrad(counts, n, k, align, spare, f32, accumulate):
    print(f"wgrad {counts[:8]} n {n} k {k} align {align} f32 {f32} acc {accumulate}", flush=True)
    g = np.random.default_rng(n * k)
    L = dev_layout(counts, align, spare)
    dy, x = bf16(g, (L["cap"], n), 0.1), bf16(g, (L["cap"], k))
    dt = torch.float32 if f32 else BF
    old = torch.from_numpy(g.standard_normal((L["E"], n, k)).astype(np.float32)).to(dt)
    dw = (old if accumulate else torch.full_like(old, float("nan"))).cuda()
    a, b = poisoned(dy, L["lab"]), poisoned(x, L["lab"])
    M.moe_grouped_wgrad_bf16(a, b, L["psum"], L["status"], align, dw, workspace(L, n, k),
                             accumulate=accumulate)
    ref, mag = B.wgrad(dy.float().numpy(), x.float().numpy(), L["lab"], L["E"])
    if accumulate:
        base = old.float().numpy().astype(np.float64)
        ref, mag = ref + base, mag + np.abs(base)
    terms = np.array(counts, np.float64)[:, None, None] + 2
    eps = 2.0 ** -24 if f32 else 2.0 ** -8
    check(f64(dw), ref, eps * np.abs(ref) + terms * 2.0 ** -23 * mag + TINY, "dw")
    if not accumulate:      # equal calls give equal bits
        dw2 = torch.full_like(dw, float("nan"))
        M.moe_grouped_wgrad_bf16(a, b, L["psum"], L["status"], align, dw2, workspace(L, n, k))
        assert torch.equal(dw.view(torch.uint8), dw2.view(torch.uint8))


def test_products_on_random_layouts():
    g = np.random.default_rng(77)
    for case in range(12):
        E = int(g.integers(1, 12))
        align = int(2 ** g.integers(4, 9))
        counts = [int(c) for c in g.integers(0, 400, E) * (g.random(E) < 0.7)]
        n, k = 128 * int(g.integers(1, 6)), 64 * int(g.integers(1, 10))
        spare = int(g.integers(0, 3))
        print(f"random {case}", flush=True)
        test_dgrad(counts, n, k, align, spare)
        test_wgrad(counts, n, k, align, spare, bool(case & 1), bool(case & 2))


def test_products_past_the_capacity():
    """A layout that overflowed: the total and the ends lie past the capacity;
    rows from the capacity on are neither read nor written."""
    counts, n, k, align = [40, 100, 60], 128, 128, 16
    g = np.random.default_rng(5)
    L = dev_layout(counts, align)
    cap = 96                                            # inside expert 1
    lab = L["lab"][:cap]
    dy, x, w = bf16(g, (cap, n)), bf16(g, (cap, k)), bf16(g, (3, n, k))
    a, b = poisoned(dy, lab), poisoned(x, lab)
    dx = torch.full((cap + 16, k), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_dgrad_bf16(a, w.cuda(), L["psum"], L["status"], align, dx[:cap])
    ref, mag = B.dgrad(dy.float().numpy(), w.float().numpy(), lab)
    live = lab >= 0
    check(f64(dx)[:cap][live], ref[live],
          2.0 ** -8 * np.abs(ref[live]) + n * 2.0 ** -23 * mag[live], "dx")
    assert torch.all(dx[cap:] == 7.0)
    dw = torch.empty((3, n, k), dtype=torch.float32, device="cuda")
    M.moe_grouped_wgrad_bf16(a, b, L["psum"], L["status"], align, dw)
    ref, mag = B.wgrad(dy.float().numpy(), x.float().numpy(), lab, 3)
    check(f64(dw), ref, 2.0 ** -24 * np.abs(ref) + 100 * 2.0 ** -23 * mag, "dw")
    assert torch.count_nonzero(dw[2]) == 0


@pytest.mark.parametrize("experts,n,k", [(300, 1024, 1024), (70, 256, 4096), (129, 768, 2560)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad_few_experts_of_many(accumulate, experts, n, k):
    """Runs of experts without rows, shorter and longer than the wave that
    looks at them, at the start, in between and at the end."""
    print(f"wgrad {experts} experts n {n} k {k} acc {accumulate}", flush=True)
    g = np.random.default_rng(experts)
    counts = [0] * experts
    for e, c in ((1, 3), (2, 40), (4, 1), (experts // 2 + 1, 17), (experts - 3, 70)):
        counts[e] = c
    L = dev_layout(counts, 16, 1)
    dy, x = bf16(g, (L["cap"], n), 0.1), bf16(g, (L["cap"], k))
    a, b = poisoned(dy, L["lab"]), poisoned(x, L["lab"])
    dw = torch.full((experts, n, k), 3.0, dtype=BF, device="cuda")
    M.moe_grouped_wgrad_bf16(a, b, L["psum"], L["status"], 16, dw, workspace(L, n, k),
                             accumulate=accumulate)
    base = 3.0 if accumulate else 0.0
    dw = dw.cpu()
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.all(dw[e] == base), f"expert {e} without rows"
            continue
        mine = L["lab"] == e
        d, v = f64(dy[torch.from_numpy(mine)]), f64(x[torch.from_numpy(mine)])
        ref, mag = d.T @ v + base, np.abs(d.T) @ np.abs(v) + base
        check(f64(dw[e]), ref,
              2.0 ** -8 * np.abs(ref) + (c + 2) * 2.0 ** -23 * mag + TINY, f"dw[{e}]")


LONG_SUMS = [
    ([9000, 0, 4500, 8200], 256, 320, 16),   # each expert's sum in parts of uneven length
    ([12001, 11000], 384, 576, 64),
    ([70, 0, 16000, 1, 9000], 128, 64, 128),
]


@pytest.mark.parametrize("f32,accumulate", [(False, False), (True, False), (True, True),
                                            (False, True)])
@pytest.mark.parametrize("counts,n,k,align", LONG_SUMS)
def test_wgrad_long_sums(counts, n, k, align, f32, accumulate):
    cap = sum(-(-c // align) * align for c in counts) + align
    assert M.moe_grouped_wgrad_workspace_bytes(cap, n, k, len(counts)) > 0
    test_wgrad(counts, n, k, align, 1, f32, accumulate)


# Weight gradients too large for one round of 64 x 64 tiles, not of 128 x 128.
MIDDLE = [
    ([200, 0, 77, 1], 640, 832, 16),
    ([33], 2048, 1024, 64),
    ([1, 31, 32, 33, 63, 64, 65, 0, 700], 384, 704, 32),
    ([0, 900, 0, 2, 0, 129], 512, 960, 256),
]


@pytest.mark.parametrize("f32,accumulate", [(False, False), (True, False), (True, True),
                                            (False, True)])
@pytest.mark.parametrize("counts,n,k,align", MIDDLE)
def test_wgrad_middle(counts, n, k, align, f32, accumulate):
    test_wgrad(counts, n, k, align, 1, f32, accumulate)


# Numbers of 64 x 64, 128 x 128 and 256 x 256 tiles just below and above whole
# rounds of the CUs, and far fewer than the sizes allow.
ROUNDS = [
    ([65] * 8, 2048, 1024, 16),
    ([64] * 8, 1024, 2048, 16),
    ([1, 0, 0, 0, 0, 0, 0, 900], 1024, 1024, 16),
    ([256] * 7 + [257], 256, 2176, 16),
    ([300] * 9, 384, 4096, 16),
    ([2000, 0, 300, 2300], 256, 4160, 64),
    ([127, 128, 129, 0, 1, 255, 256, 257], 512, 1088, 128),   # 128 x 128 ones
    ([64, 1, 0, 65, 191, 192, 193, 700], 1152, 960, 32),
    ([1500], 128, 2048, 16),
]


@pytest.mark.parametrize("counts,n,k,align", ROUNDS)
def test_rounds_of_tiles(counts, n, k, align):
    test_dgrad(counts, n, k, align, 1)
    test_wgrad(counts, n, k, align, 1, False, False)
    test_wgrad(counts, n, k, align, 1, True, True)


def test_wgrad_without_rows():
    """Capacity 0: zeros, or unchanged when accumulating."""
    e = torch.empty((0, 128), dtype=BF, device="cuda")
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    for acc, want in ((False, 0.0), (True, 3.0)):
        dw = torch.full((2, 128, 64), 3.0, device="cuda")
        M.moe_grouped_wgrad_bf16(e, x, z, z, 16, dw, accumulate=acc)
        assert torch.all(dw == want)


def test_products_propagate_what_live_rows_hold():
    """An infinity in a live row reaches its own results and no others."""
    L = dev_layout([20, 20], 32)
    g = np.random.default_rng(9)
    dy, x, w = bf16(g, (L["cap"], 128)), bf16(g, (L["cap"], 64)), bf16(g, (2, 128, 64))
    dy[3, 5] = float("inf")
    dyg = poisoned(dy, L["lab"])
    dx = torch.zeros((L["cap"], 64), dtype=BF, device="cuda")
    M.moe_grouped_dgrad_bf16(dyg, w.cuda(), L["psum"], L["status"], 32, dx)
    bad = ~torch.isfinite(dx)
    assert torch.all(bad[3]) and bad.sum() == 64
    dw = torch.zeros((2, 128, 64), device="cuda")
    M.moe_grouped_wgrad_bf16(dyg, poisoned(x, L["lab"]), L["psum"], L["status"], 32, dw,
                             workspace(L, 128, 64))
    bad = ~torch.isfinite(dw)
    assert torch.all(bad[0, 5]) and bad.sum() == 64


@pytest.mark.parametrize("inter", [8, 64, 120, 128, 256, 2048, 2056, 4096])
def test_silu_backward(inter):
    print(f"silu backward I {inter}", flush=True)
    g = np.random.default_rng(inter)
    L = dev_layout([17, 0, 1, 40, 16], 16, 2)
    cap = L["cap"]
    gu, dy = bf16(g, (cap, 2 * inter), 2.0), bf16(g, (cap, inter), 0.1)
    edge = [0.0, -0.0, 1e-30, -1e-30, 88.0, -88.0, 200.0, -200.0, 3e38, -3e38, -1.2785, 17.0]
    gu[0, :8] = torch.tensor(edge[:8])
    gu[1, :4] = torch.tensor(edge[8:])
    gu[0, inter:inter + 8], gu[1, inter:inter + 4] = 1.5, 0.5
    d = torch.full((cap, 2 * inter), 7.0, dtype=BF, device="cuda")
    gug, dyg = poisoned(gu, L["lab"]), poisoned(dy, L["lab"])
    M.moe_silu_mul_bf16_backward(gug, dyg, L["m_indices"], L["psum"], L["status"], L["E"], 16, d)
    live = L["lab"] >= 0
    got = f64(d)
    assert np.all(got[~live] == 7.0)
    G, U, Y = (t.float().numpy().astype(np.float64)[live]
               for t in (gu[:, :inter], gu[:, inter:], dy))
    dg, du = B.silu_mul_backward(G, U, Y)
    s = B.sigmoid(G)
    check(got[live][:, :inter], dg,
          2.0 ** -8 * np.abs(dg) + np.abs(Y * U) * s * (1 + np.abs(G)) * 2.0 ** -19 + TINY, "dg")
    check(got[live][:, inter:], du, (2.0 ** -8 + 2.0 ** -19) * np.abs(du) + TINY, "du")
    M.moe_silu_mul_bf16_backward(gug, dyg, L["m_indices"], L["psum"], L["status"], L["E"], 16,
                                 gug)                    # in place
    assert torch.equal(gug[torch.from_numpy(live)], d[torch.from_numpy(live)])
    assert torch.all(torch.isnan(gug[torch.from_numpy(~live)]))


@pytest.mark.parametrize("rows,valid,hidden,topk,E,align,f,weighted,dots", [
    (1, 1, 128, 1, 1, 16, 1.0, True, True),
    (7, 7, 256, 3, 4, 16, 2.5, True, True),
    (50, 33, 384, 8, 6, 32, -0.5, True, True),
    (50, 0, 128, 2, 6, 32, 1.0, True, True),
    (40, 40, 1024, 2, 5, 64, 2.5, False, True),
    (40, 21, 640, 4, 5, 64, 2.5, True, False),
    (33, 33, 8192, 32, 40, 16, 1.0, True, True),
    (300, 299, 7168, 8, 16, 128, 2.5, True, True)])
def test_gather_backward(rows, valid, hidden, topk, E, align, f, weighted, dots):
    print(f"gather backward rows {rows} H {hidden} topk {topk}", flush=True)
    g = np.random.default_rng(rows + hidden)
    ids = np.stack([g.permutation(max(E, topk) * 2)[:topk] for _ in range(rows)])
    ids = np.where(ids < E, ids, -1).astype(np.int32)
    if topk > 1 and rows > 1:
        ids[1, :2] = 0                                   # the same expert twice
    cap = layout.capacity(rows, topk, E, align)
    src = layout.expand_layout(ids, valid, E, align, cap)["src2dst"]
    w = g.random((rows, topk)).astype(np.float32) + np.float32(0.01)
    dout, D = bf16(g, (rows, hidden), 0.1), bf16(g, (cap, hidden))
    used = np.zeros(cap, bool)
    used[src[src >= 0]] = True
    dog, Dg = dout.clone(), poisoned(D, np.where(used, 0, -1))
    dog[valid:] = float("nan")
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    srcg = t(src)
    if valid < rows:
        srcg[valid:] = 0                                 # never read as slots
    deo = torch.full((cap, hidden), 7.0, dtype=BF, device="cuda")
    dw = torch.full((rows, topk), 7.0, device="cuda") if dots else None
    prank = None if valid == rows else t(np.array([valid // 2, valid], np.int32))
    M.moe_gather_backward(dog.cuda(), Dg if dots else None, srcg, t(w) if weighted else None,
                          prank, deo, dw, routed_scaling_factor=f)
    d32 = dout.float().numpy()
    d_rows, dc = B.gather_backward(d32, D.float().numpy(), src, w if weighted else None, f,
                                   valid, cap)
    got = f64(deo)
    assert np.all(got[~used] == 7.0) and used.sum() == len(d_rows)
    for r, k in zip(*np.nonzero(src >= 0)):
        c = np.float32(f) * (w[r, k] if weighted else np.float32(1.0))
        assert np.array_equal(got[src[r, k]], fp8.round_bf16(c * d32[r]))
    if dots:
        mag = B.gather_backward(np.abs(d32), np.abs(D.float().numpy()), src, None, abs(f), valid,
                                cap)[1]
        gw = f64(dw)
        assert np.all(gw[valid:] == 7.0) and np.all(gw[:valid][src[:valid] < 0] == 0.0)
        check(gw[:valid], dc, hidden * 2.0 ** -23 * mag + 2.0 ** -149, "d_topk_weights")
