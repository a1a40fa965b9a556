"""moe_layer_norm and its gradient against the float64 oracle.

Tolerances.  A bf16 result is off by half a step of its own (2^-8 of it).  A
sum of n fp32 terms in a tree of depth d is off by at most d half steps (2^-24)
of the terms' sizes: a thread adds up to 32 values, the wave 6 times, the
workgroup up to 8, so d < 48 along a row; over the rows a thread adds at most
rows / 128 + 8 and the joins 48.  Every other fp32 operation adds a half step.
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
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24
DEPTH = 48


def np64(t):
    return t.detach().double().cpu().numpy()


def rand(seed, *shape, scale=1.0, dtype=BF, shift=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def recv(n):
    return torch.tensor([n // 3, n], dtype=torch.int32, device="cuda")


def check(name, got, want, tol):
    got = np64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), np.abs(got - want)[bad].max())


def forward(x, weight, bias, branch, kind, eps, nv, keep=True):
    rows, H = x.shape
    o = dict(y=torch.full((rows, H), 7.0, dtype=BF, device="cuda"),
             mean=torch.full((rows,), 7.0, device="cuda"),
             rstd=torch.full((rows,), 7.0, device="cuda"),
             sum=None if branch is None else torch.full((rows, H), 7.0, dtype=x.dtype,
                                                        device="cuda"))
    M.moe_layer_norm(x, weight, bias=bias, branch=branch, kind=kind, eps=eps,
                     psum_recv_per_rank=None if nv is None else recv(nv), **o)
    return o


def compare_forward(o, x, weight, bias, branch, kind, eps, nv):
    rows, H = x.shape
    nv = rows if nv is None else max(0, min(nv, rows))
    h = np64(x)[:nv]
    if branch is not None:
        want = h + np64(branch)[:nv]
        check("sum", o["sum"][:nv], want, (HALF[x.dtype] + 2 * U) * np.abs(want))
        h = np64(o["sum"])[:nv]
    rms = kind == "rms"
    y, mean, rstd = B.layer_norm(h, np64(weight), None if bias is None else np64(bias), eps, rms)
    size = np.abs(h).mean(axis=1)
    off = 0 if rms else DEPTH * U * size          # of the mean
    check("mean", o["mean"][:nv], mean, off)
    # A mean that is off by d adds d^2 to the variance; the rest is relative.
    rel = (DEPTH + 8) * U + (off * rstd) ** 2
    check("rstd", o["rstd"][:nv], rstd, rel * rstd)
    w = np.abs(np64(weight))
    part = np.abs(y - (0 if bias is None else np64(bias)))
    tol = HALF[BF] * np.abs(y) + part * (rel[:, None] + 8 * U) + 4 * U * np.abs(y)
    if not rms:
        tol += (off * rstd)[:, None] * w
    check("y", o["y"][:nv], y, tol)
    for name, t in o.items():                       # rows behind stay as they were
        assert t is None or bool((t[nv:] == 7).all()), name


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("hidden", [8, 64, 264, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 6144,
                                    6152, 7168, 8192])
def test_forward(hidden, kind):
    for rows, nv, dtype, with_branch in ((1, None, BF, True), (5, 3, F32, True),
                                         (37, 37, BF, False), (130, 129, F32, False)):
        print(f"[norm {hidden} {kind} rows {rows} {dtype}]", flush=True)
        x = rand(hidden + rows, rows, hidden, scale=2, dtype=dtype, shift=0.5)
        branch = rand(3, rows, hidden) if with_branch else None
        weight, bias = rand(4, hidden, dtype=F32, shift=1), rand(5, hidden, dtype=F32)
        if nv is not None:
            for t in (x, branch):
                if t is not None:
                    t[nv:] = float("nan")
        if rows == 37:
            weight, bias = weight.to(BF), None
        o = forward(x, weight, bias, branch, kind, 1e-5, nv)
        compare_forward(o, x, weight, bias, branch, kind, 1e-5, nv)


@pytest.mark.parametrize("nv", [-3, 0, 1, 99])
def test_received_rows_are_clamped(nv):
    x, w = rand(1, 6, 256), rand(2, 256, dtype=F32)
    compare_forward(forward(x, w, None, None, "layer", 1e-5, nv), x, w, None, None, "layer", 1e-5,
                    nv)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_apart_and_in_place(dtype):
    wide = rand(1, 9, 1056, dtype=dtype)
    x, w, b = wide[:, 16:528], rand(2, 512, dtype=F32), rand(3, 512, dtype=F32)
    compare_forward(forward(x, w, b, None, "layer", 1e-5, None), x, w, b, None, "layer", 1e-5, None)
    branch = rand(4, 9, 512)
    compare_forward(forward(x, w, b, branch, "rms", 1e-5, 7), x, w, b, branch, "rms", 1e-5, 7)
    y, y2 = (torch.empty((9, 512), dtype=BF, device="cuda") for _ in range(2))
    h, stream = torch.empty_like(branch, dtype=dtype), x.contiguous()
    M.moe_layer_norm(stream, w, y, b, branch, h)
    M.moe_layer_norm(stream, w, y2, b, branch, stream)
    assert torch.equal(stream, h) and torch.equal(y, y2)
    M.moe_layer_norm(x, w, y2, b, branch)            # the sum is not kept
    assert torch.equal(y, y2)


def test_hard_rows():
    """A mean of 3000 deviations in fp32, a constant row, an all-zero row without
    eps, the largest values, and infinities that stay in their rows."""
    x = rand(1, 8, 2048, dtype=F32, scale=0.01)
    x[1] += 30
    x[2] = 5.0
    x[3] = 0
    w = rand(2, 2048, dtype=F32, shift=1)
    o = forward(x, w, None, None, "layer", 1e-6, None)
    compare_forward(o, x, w, None, None, "layer", 1e-6, None)
    assert bool((o["y"][3] == 0).all())
    x[4, 7], x[5, 0], x[6, 9] = float("inf"), float("nan"), 1e30
    x[6, 1:9] = -1e30
    o2 = forward(x, w, None, None, "layer", 1e-6, None)
    for r in (0, 1, 2, 3, 7):
        assert torch.equal(o2["y"][r], o["y"][r])
    assert bool(torch.isnan(o2["y"][4]).all()) and bool(torch.isnan(o2["y"][5]).all())
    o = forward(x[3:4], w, None, None, "rms", 0.0, None)
    assert bool(torch.isinf(o["rstd"]).all())        # 1 / 0, as the formula has it


def test_infinities_under_rms():
    x, w, b = rand(1, 4, 2056, dtype=F32), rand(2, 2056, dtype=F32), rand(3, 2056, dtype=F32)
    x[0, 7], x[1, 7], x[2, 7] = float("inf"), float("nan"), 1e20
    o = forward(x, w, b, None, "rms", 1e-6, None)
    rest = torch.arange(2056, device="cuda") != 7
    assert bool(torch.isnan(o["y"][0, 7])) and bool(torch.isnan(o["y"][1]).all())
    assert o["rstd"][0] == 0 and o["rstd"][2] == 0
    assert torch.equal(o["y"][0, rest], b[rest].to(BF)) and torch.equal(o["y"][2], b.to(BF))
    compare_forward(forward(x[3:], w, b, None, "rms", 1e-6, None), x[3:], w, b, None, "rms",
                    1e-6, None)


def backward(case, x, dy, weight, mean, rstd, kind, nv, dy2=None, dsum=None, gdt=F32, bias=True,
             weight_grad=True, accumulate=False, in_place=False):
    rows, H = x.shape
    dx = dsum.clone() if in_place else torch.full((rows, H), 7.0, dtype=x.dtype, device="cuda")
    old = [rand(50 + i, H, dtype=gdt) for i in range(2)]
    dw = old[0].clone() if weight_grad else None
    db = old[1].clone() if bias else None
    need = M.moe_layer_norm_backward_workspace_bytes(rows, H)
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
    M.moe_layer_norm_backward(dy, x, weight, rstd, dx, mean=mean, dy2=dy2,
                              dsum=dx if in_place else dsum, dweight=dw, dbias=db,
                              accumulate=accumulate, kind=kind,
                              psum_recv_per_rank=None if nv is None else recv(nv), workspace=ws)
    n = rows if nv is None else nv
    d = np64(dy)[:n] + (0 if dy2 is None else np64(dy2)[:n])
    h, w, rs = np64(x)[:n], np64(weight), np64(rstd)[:n]
    mu = None if mean is None else np64(mean)[:n]
    rms = kind == "rms"
    want, gw, gb = B.layer_norm_backward(d, h, w, mu, rs, rms)
    xh = np.abs(h - (0 if rms else mu[:, None])) * rs[:, None]
    g = np.abs(d * w)
    size = rs[:, None] * (g + (0 if rms else g.mean(1, keepdims=True))
                          + xh * (g * xh).mean(1, keepdims=True))
    if dsum is not None:
        want = want + np64(dsum)[:n]
        size = size + np.abs(np64(dsum)[:n])
    check(case + " dx", dx[:n], want, HALF[x.dtype] * np.abs(want) + (DEPTH + 16) * U * size)
    if not in_place:
        assert bool((dx[n:] == 7).all())
    depth = rows / 128 + 8 + DEPTH + 4
    for name, got, new, mag, was in (("dw", dw, gw, (np.abs(d) * xh).sum(0), old[0]),
                                     ("db", db, gb, np.abs(d).sum(0), old[1])):
        if got is None:
            continue
        if accumulate:
            new, mag = new + np64(was), mag + np.abs(np64(was))
        check(case + name, got, new, HALF[gdt] * np.abs(new) + depth * U * mag)
    return dx, dw, db


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("hidden", [8, 264, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 6144,
                                    7168, 8192])
def test_backward(hidden, kind):
    for i, (rows, nv, dtype, opt) in enumerate((
            (1, None, BF, dict()),
            (7, 5, F32, dict(second=True, gdt=BF)),
            (67, 67, BF, dict(stream=True, accumulate=True)),
            (700, 613, BF, dict(second=True, stream=True, in_place=True, bias=False)),
            (300, 299, F32, dict(stream=True, weight_grad=False, gdt=BF, accumulate=True)))):
        print(f"[norm backward {hidden} {kind} rows {rows} {dtype} {opt}]", flush=True)
        opt = dict(opt)
        second, stream = opt.pop("second", False), opt.pop("stream", False)
        x = rand(hidden + i, rows, hidden, scale=2, dtype=dtype, shift=0.5)
        weight = rand(4, hidden, dtype=F32 if i % 2 else BF, shift=1)
        mean, rstd = (torch.from_numpy(v).cuda().float()
                      for v in B.layer_norm(np64(x), np64(weight), None, 1e-5, kind == "rms")[1:])
        dy = rand(9, rows, hidden, scale=0.1)
        dy2 = rand(10, rows, hidden, scale=0.1) if second else None
        dsum = rand(11, rows, hidden, scale=0.1, dtype=dtype) if stream else None
        if nv is not None:
            for t in (x, dy, dy2, mean, rstd):
                if t is not None:
                    t[nv:] = float("nan")
        args = ("", x, dy, weight, None if kind == "rms" else mean, rstd, kind, nv, dy2, dsum)
        first = backward(*args, **opt)
        again = backward(*args, **opt)               # equal calls give equal bits
        for a, b in zip(first, again):
            assert a is None or torch.equal(a[:nv], b[:nv]) if a is not None and a.dim() > 1 else \
                a is None or torch.equal(a, b)


@pytest.mark.parametrize("accumulate", [False, True])
def test_no_valid_row(accumulate):
    for rows in (0, 5):
        x, w = rand(1, rows, 512), rand(2, 512, dtype=F32)
        r = torch.full((rows,), float("nan"), device="cuda")
        backward("", x, torch.full_like(x, float("nan")), w, r, r, "layer", 0,
                 accumulate=accumulate)


def test_gradient_is_the_forward_calls():
    """dx, dweight and dbias against differences of the forward kernel's own
    mean-squared output: a step of 2^-6 in one value of x moves f by dx times it."""
    rows, H = 3, 64
    x, w, b = rand(1, rows, H, dtype=F32), rand(2, H, dtype=F32, shift=1), rand(3, H, dtype=F32)
    dy = rand(4, rows, H)
    o = forward(x, w, b, None, "layer", 1e-5, None)
    dx, dw, db = (torch.empty_like(t) for t in (x, w, b))
    ws = torch.empty(M.moe_layer_norm_backward_workspace_bytes(rows, H), dtype=torch.uint8,
                     device="cuda")
    M.moe_layer_norm_backward(dy, x, w, o["rstd"], dx, mean=o["mean"], dweight=dw, dbias=db,
                              workspace=ws)
    # f = sum(dy * y) with y rounded to bf16: off by 2^-8 sum |dy y|.  A step of
    # 1 in one weight moves f by dw exactly (f is linear in it); in x, where f
    # bends, the oracle's own difference is the measure.
    f = lambda x, w, b: float((np64(forward(x, w, b, None, "layer", 1e-5, None)["y"])  # noqa: E731
                               * np64(dy)).sum())
    noise = 2 * HALF[BF] * float((np.abs(np64(o["y"])) * np.abs(np64(dy))).sum())
    rng = np.random.default_rng(0)
    for got, k in ((dw, 1), (db, 2)):
        for i in rng.integers(0, H, 8):
            args = [x, w.clone(), b.clone()]
            args[k][i] += 64.0
            moved = f(*args) - f(x, w, b)
            big = noise + 2 * HALF[BF] * 64 * float(np.abs(np64(dy)[:, i]).sum()) * 4
            assert abs(moved / 64 - float(got[i])) <= big / 64
    y0 = B.layer_norm(np64(x), np64(w), np64(b), 1e-5, False)[0]
    for i in rng.integers(0, H, 8):
        x2 = np64(x).copy()
        x2[1, i] += 1e-4
        d = ((B.layer_norm(x2, np64(w), np64(b), 1e-5, False)[0] - y0) * np64(dy)).sum() / 1e-4
        # second order: |f''| step / 2 <= |dy| |w| rstd^2 * step, under 1e-2 here
        assert abs(d - float(dx[1, i])) <= 1e-2


def test_another_stream_and_capture():
    x, w, dy = rand(1, 64, 1024), rand(2, 1024, dtype=F32, shift=1), rand(3, 64, 1024)
    want = forward(x, w, None, None, "layer", 1e-5, None)
    y, mean, rstd = torch.zeros_like(x), torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros(1024, device="cuda")
    ws = torch.empty(M.moe_layer_norm_backward_workspace_bytes(64, 1024), dtype=torch.uint8,
                     device="cuda")
    nv = torch.tensor([64], dtype=torch.int32, device="cuda")

    def step():
        M.moe_layer_norm(x, w, y, mean=mean, rstd=rstd, psum_recv_per_rank=nv)
        M.moe_layer_norm_backward(dy, x, w, rstd, dx, mean=mean, dweight=dw, workspace=ws,
                                  psum_recv_per_rank=nv)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert torch.equal(y, want["y"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n, seed in ((64, 5), (17, 6), (0, 7), (63, 8)):
        x.copy_(rand(seed, 64, 1024))
        nv.fill_(n)
        for t in (y, dx):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw)]
        for t in (y, dx):
            t.fill_(3)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, dx, dw)):
            assert torch.equal(a, b)
        assert bool((got[0][n:] == 3).all()) and bool((got[1][n:] == 3).all())
