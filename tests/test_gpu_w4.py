"""moe_grouped_gemm_w4 against the float64 oracle, and exactly on whole numbers.

Tolerance: half a step of the bf16 result (2^-8 of it), and the fp32 sum: each
MFMA's result may be cut off (2^-23 of the sum so far), k / 32 times, with 32
terms inside.  Sizes of the terms: |a| s |q|, for int4 |a| s (2 * 8 + |q|),
since the codes enter as 8 + q and 8 a is taken off.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402
from oracle import block as B  # noqa: E402
from oracle.backward import live_rows  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16
FORMATS = [("int4", 128), ("int4", 64), ("int4", 32), ("mxfp4", 32)]


def layout(counts, align, spare=0):
    psum, end = [], 0
    for c in counts:
        psum.append(end + c)
        end = -(-psum[-1] // align) * align
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(psum), i32([end, 0]), end + spare * align


def weights(E, n, k, fmt, group, seed, whole=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    shape = (E, n, k // group)
    if fmt == "mxfp4":
        lo, hi = (126, 129) if whole else (110, 130)
        return w, torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda", generator=g)
    if whole:
        return w, (0.5 + torch.randint(0, 2, shape, device="cuda", generator=g) / 2).to(BF)
    return w, (torch.rand(shape, device="cuda", generator=g) * 0.02 - 0.005).to(BF)


def scale_values(sc):
    return sc.float().cpu().numpy() if sc.dtype == BF else sc.cpu().numpy()


def run(counts, n, k, fmt, group, align=16, spare=0, whole=False, seed=0):
    E = len(counts)
    psum, status, cap = layout(counts, align, spare)
    w, sc = weights(E, n, k, fmt, group, seed, whole)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    if whole:
        a = torch.randint(-3, 4, (cap, k), device="cuda", generator=g).to(BF)
    else:
        a = torch.randn((cap, k), device="cuda", generator=g).to(BF)
    lab = live_rows(psum.cpu().numpy(), align, cap)
    dead = torch.from_numpy(lab < 0).cuda()
    a[dead] = float("nan")
    out = torch.full((cap, n), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_gemm_w4(a, w, sc, fmt, psum, status, align, out)
    torch.cuda.synchronize()
    v = B.w4_values(w.cpu().numpy(), scale_values(sc), fmt)
    av = np.where(lab[:, None] >= 0, a.float().cpu().numpy(), 0)
    want, mag = B.grouped(av, v, lab)
    got = out.double().cpu().numpy()
    live = lab >= 0
    assert (got[~live] == 7).all()                   # rows that are not live stay
    if whole:  # every partial sum is exact: one rounding
        r = torch.from_numpy(want[live]).to(torch.float32).to(BF).double().numpy()
        assert np.array_equal(got[live], r)
        return
    if fmt == "int4":
        s = np.repeat(np.abs(scale_values(sc)).astype(np.float64), group, axis=-1)
        mag = mag + 16 * B.grouped(np.abs(av), s, lab)[0]
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -23 * (k / 32 + 32) * mag
    bad = ~(np.abs(got - want) <= tol)[live]
    assert not bad.any(), (bad.sum(), np.abs(got - want)[live][bad].max())


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("counts,n,k,align", [
    ([1], 128, 128, 16), ([1, 0, 3], 256, 384, 16), ([0, 0], 128, 128, 16),
    ([16, 17, 15, 1, 0, 33], 384, 640, 16), ([5, 0, 64, 65], 128, 1152, 64),
    ([129, 127, 128, 1], 256, 512, 128), ([300, 2], 640, 256, 32), ([257, 0, 511], 128, 896, 256),
    ([1] * 40, 128, 256, 16), ([700], 256, 128, 1024), ([90, 70, 40, 20, 100], 512, 2048, 16)])
def test_against_the_oracle(counts, n, k, align, fmt, group):
    print(f"[w4 {counts[:6]} {n} {k} {align} {fmt} {group}]", flush=True)
    run(counts, n, k, fmt, group, align)
    run(counts, n, k, fmt, group, align, spare=3, whole=True, seed=5)


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_every_length_exactly(fmt, group):
    """One expert of every length up to 150 rows and a few beyond, between two others."""
    for live in [*range(1, 150, 7), 63, 64, 128, 129, 191, 192, 193, 255, 256, 257, 384, 385, 520]:
        print(f"[w4 length {live} {fmt} {group}]", flush=True)
        run([3, live, 18], 128, 384, fmt, group, 16, whole=True, seed=live)


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_many_experts_and_long_rows(fmt, group):
    counts = [0] * 1024
    for e, c in ((0, 2), (63, 1), (64, 30), (700, 5), (1023, 1)):
        counts[e] = c
    run(counts, 128, 128, fmt, group, 16, whole=True)
    run([3, 20, 140], 128, 511 * 64 // 128 * 128, fmt, group, 16)
    run([2, 200], 511 * 64 // 128 * 128, 128, fmt, group, 16, whole=True)


@pytest.mark.parametrize("fmt,group,k", [("mxfp4", 32, 9472), ("mxfp4", 32, 9600),
                                         ("int4", 32, 4736), ("int4", 32, 4864),
                                         ("int4", 64, 9472), ("int4", 64, 9600),
                                         ("int4", 128, 18944), ("int4", 128, 19072)])
def test_where_the_scales_just_fit(fmt, group, k):
    """The longest reduction whose scales the items of few rows hold, and the next."""
    run([3, 0, 20, 33, 140], 256, k, fmt, group, 16, whole=True, seed=k)


@pytest.mark.parametrize("counts", [[500] * 8, [1000, 900, 1030, 129, 300, 33, 20, 640],
                                    [2300, 0, 1, 16, 1200, 700]])
@pytest.mark.parametrize("n", [2176, 2304])
def test_a_last_round_of_few_tiles(counts, n):
    """A little more than a round or two of wide items: the rest go in parts."""
    run(counts, n, 256, "mxfp4", 32, 128, whole=True, seed=n)


@pytest.mark.parametrize("counts", [[1024] * 8, [1270, 1300, 1000, 1400, 1281, 1153, 1500, 1300],
                                    [1600] * 7 + [1537, 33, 5, 0, 20]])
@pytest.mark.parametrize("n,k", [(2176, 128), (2304, 256), (2176, 640)])
def test_tiles_of_256_rows(counts, n, k):
    """A round and a few, and some more, and most of another one: the last round's
    tiles in quarters, in halves and whole."""
    run(counts, n, k, "mxfp4", 32, 128, whole=True, seed=k)
    run(counts, n, k, "mxfp4", 32, 128, whole=False, seed=k)


@pytest.mark.parametrize("fmt,group", [("mxfp4", 32), ("int4", 128)])
@pytest.mark.parametrize("rows", [1, 20])
def test_more_items_than_are_listed_at_once(fmt, group, rows):
    """1024 experts of 16384 columns: over 64 items for every workgroup."""
    E, n, k, align = 1024, 16384, 128, 32
    psum, status, cap = layout([rows] * E, align)
    w, sc = weights(E, n, k, fmt, group, 3, whole=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    a = torch.randint(-3, 4, (cap, k), device="cuda", generator=g).to(BF)
    out = torch.full((cap, n), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_gemm_w4(a, w, sc, fmt, psum, status, align, out)
    table = ([*range(8), *range(-8, 0)] if fmt == "int4" else
             [*B.E2M1.tolist(), *(-B.E2M1).tolist()])
    table = torch.tensor(table, device="cuda")
    for e in range(0, E, 61):
        q = torch.stack([w[e] & 15, w[e] >> 4], dim=-1).view(n, k)
        s = sc[e].float() if fmt == "int4" else torch.exp2(sc[e].float() - 127)
        v = table[q.long()].double() * s.double().repeat_interleave(group, dim=1)
        at = slice(e * align, e * align + rows)
        assert torch.equal(out[at], (a[at].double() @ v.t()).float().to(BF)), e
        assert bool((out[e * align + rows:(e + 1) * align] == 7).all())


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_one_code_at_a_time(fmt, group):
    """Row t of a is the unit vector of k = t: the output is the weights themselves,
    every code under every scale and place (rounded to bf16 once)."""
    E, n, k = 1, 128, 256
    w = torch.arange(n * k // 2, device="cuda").view(E, n, k // 2)
    w = ((w * 37 + w // 64 * 11) % 256).to(torch.uint8)
    shape = (E, n, k // group)
    i = torch.arange(n * (k // group), device="cuda").view(shape)
    if fmt == "mxfp4":
        sc = (2 + i % 251).to(torch.uint8)           # bytes 2..252: normal bf16 weights
    else:
        sc = ((i % 61 - 30) / 16.0).to(BF)
    a = torch.eye(k, device="cuda").to(BF)
    psum, status, cap = layout([k], 16)
    out = torch.empty((cap, n), dtype=BF, device="cuda")
    M.moe_grouped_gemm_w4(a, w, sc, fmt, psum, status, 16, out)
    v = B.w4_values(w.cpu().numpy(), scale_values(sc), fmt)[0].T
    want = torch.from_numpy(v).float().to(BF)
    assert torch.equal(out.cpu(), want)


def test_nan_scale_and_nan_rows_stay_where_they_are():
    psum, status, cap = layout([5, 40], 16)
    w, sc = weights(2, 128, 256, "mxfp4", 32, 1)
    a = torch.randn((cap, 256), device="cuda").to(BF)
    out, out2 = (torch.zeros((cap, 128), dtype=BF, device="cuda") for _ in range(2))
    M.moe_grouped_gemm_w4(a, w, sc, "mxfp4", psum, status, 16, out)
    w[0, 9, 0] = 0x22
    M.moe_grouped_gemm_w4(a, w, sc, "mxfp4", psum, status, 16, out)
    sc[0, 9, 0] = 255
    a[20, 3] = float("nan")
    M.moe_grouped_gemm_w4(a, w, sc, "mxfp4", psum, status, 16, out2)
    nan = torch.isnan(out2)
    want = torch.zeros_like(nan)
    want[:5, 9] = True
    want[20] = True
    assert torch.equal(nan, want)
    assert torch.equal(out2[~want], out[~want])


def test_malformed_layout_stays_inside():
    """A psum beyond the total and the capacity: rows are clamped to both."""
    w, sc = weights(2, 128, 128, "int4", 128, 1)
    a = torch.ones((64, 128), device="cuda").to(BF)
    for psum, total in (([30, 200], 48), ([30, 200], 1000), ([-4, 20], 64), ([90, 95], 64)):
        out = torch.full((80, 128), 7.0, dtype=BF, device="cuda")
        M.moe_grouped_gemm_w4(a, w, sc, "int4", torch.tensor(psum, dtype=torch.int32, device="cuda"),
                              torch.tensor([total, 0], dtype=torch.int32, device="cuda"), 16,
                              out[:64])
        torch.cuda.synchronize()
        assert bool((out[min(total, 64):] == 7).all())


def test_weights_past_32_bit_offsets():
    """The last of 200 experts lies 5 GB into the weights."""
    E, n, k = 200, 7168, 7168
    w = torch.zeros((E, n, k // 2), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((E, n, k // 32), dtype=torch.uint8, device="cuda")
    counts = [0] * (E - 1) + [20]
    counts[0] = 1
    w[E - 1, n - 1, -1] = 0x2f                        # codes 15 (-6) and 2 (1)
    w[E - 1, n - 1, 0] = 0x12
    sc[E - 1] = 127
    psum, status, cap = layout(counts, 16)
    a = torch.zeros((cap, k), dtype=BF, device="cuda")
    a[16:36, 0], a[16:36, 1] = 1, 2
    a[16:36, k - 2], a[16:36, k - 1] = 4, torch.arange(20, device="cuda").to(BF)
    out = torch.zeros((cap, n), dtype=BF, device="cuda")
    M.moe_grouped_gemm_w4(a, w, sc, "mxfp4", psum, status, 16, out)
    want = 1 + 1 - 24 + torch.arange(20, device="cuda").float()
    assert torch.equal(out[16:36, n - 1].float(), want)
    assert int(torch.count_nonzero(out[:, :n - 1])) == 0


def test_equal_calls_give_equal_bits():
    psum, status, cap = layout([3, 70, 200], 16)
    for fmt, group in FORMATS:
        w, sc = weights(3, 256, 1024, fmt, group, 3)
        a = torch.randn((cap, 1024), device="cuda").to(BF)
        outs = [torch.zeros((cap, 256), dtype=BF, device="cuda") for _ in range(3)]
        for o in outs:
            M.moe_grouped_gemm_w4(a, w, sc, fmt, psum, status, 16, o)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
