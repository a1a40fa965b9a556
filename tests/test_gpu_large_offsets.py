"""The training entry points where element offsets pass 2^31 (and byte offsets
2^32): the results at the far end against the same data in small buffers, bit
for bit."""

import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def normal(*shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(len(shape))
    return torch.empty(shape, dtype=BF, device="cuda").normal_(0, 1, generator=g)


def test_products():
    """2^31 + elements of dy and x: expert 1's rows lie behind 300001 of expert 0."""
    n, k, far, rows = 8192, 128, 300032, 77
    cap = far + 128
    dy, x, w = normal(cap, n), normal(cap, k), normal(2, n, k)
    assert dy.numel() > 1 << 31
    psum, status = ints(300001, far + rows), ints(cap, 0)  # far = align(300001)
    dx = torch.zeros((cap, k), dtype=BF, device="cuda")
    print("dgrad", flush=True)
    M.moe_grouped_dgrad_bf16(dy, w, psum, status, 32, dx)
    small = torch.zeros((128, k), dtype=BF, device="cuda")
    M.moe_grouped_dgrad_bf16(dy[far:], w[1:], ints(rows), ints(128, 0), 32, small)
    # (sums in another order: a bf16 step of the value, or of terms of size 1)
    assert torch.allclose(dx[far:far + rows].float(), small[:rows].float(), rtol=2.0 ** -7,
                          atol=n * 2.0 ** -20)
    print("wgrad", flush=True)
    dw = torch.empty((2, n, k), device="cuda")
    need = M.moe_grouped_wgrad_workspace_bytes(cap, n, k, 2)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    M.moe_grouped_wgrad_bf16(dy, x, psum, status, 32, dw, ws)
    ref = dy[far:far + rows].float().t() @ x[far:far + rows].float()
    assert torch.allclose(dw[1], ref, rtol=1e-5, atol=rows * 2.0 ** -18)


def test_many_weights():
    """2^31 + weights and gradients: only the last expert has rows."""
    E, n, k, rows = 70, 8192, 4096, 33
    w = torch.empty((E, n, k), dtype=BF, device="cuda")
    w[-1] = normal(n, k)
    dy, x = normal(64, n), normal(64, k)
    psum = torch.zeros(E, dtype=torch.int32, device="cuda")
    psum[-1] = rows
    dx = torch.zeros((64, k), dtype=BF, device="cuda")
    print("dgrad", flush=True)
    M.moe_grouped_dgrad_bf16(dy, w, psum, ints(64, 0), 32, dx)
    small = torch.zeros_like(dx)
    M.moe_grouped_dgrad_bf16(dy, w[-1:], ints(rows), ints(64, 0), 32, small)
    assert torch.allclose(dx[:rows].float(), small[:rows].float(), rtol=2.0 ** -7,
                          atol=n * 2.0 ** -20)
    print("wgrad", flush=True)
    M.moe_grouped_wgrad_bf16(dy, x, psum, ints(64, 0), 32, w)
    ref = dy[:rows].float().t() @ x[:rows].float()
    assert torch.allclose(w[-1].float(), ref, rtol=2.0 ** -7, atol=rows * 2.0 ** -18)
    assert torch.count_nonzero(w[-2]) == 0


def test_rows_of_the_combine_and_of_silu():
    H, I, cap = 8192, 4096, 300000
    D, dD = normal(cap, H), torch.zeros((cap, H), dtype=BF, device="cuda")
    dst = ints(cap - 1, -1, 5, cap - 3).view(2, 2)
    dout, wt = normal(2, H), torch.rand((2, 2), device="cuda")
    dc = torch.zeros((2, 2), device="cuda")
    print("gather", flush=True)
    M.moe_gather_backward(dout, D, dst, wt, None, dD, dc)
    few = torch.tensor([cap - 1, 5, cap - 3], device="cuda")
    sm, dc2 = torch.zeros((3, H), dtype=BF, device="cuda"), torch.zeros_like(dc)
    M.moe_gather_backward(dout, D[few], ints(0, -1, 1, 2).view(2, 2), wt, None, sm, dc2)
    assert torch.equal(dD[few], sm) and torch.equal(dc, dc2)
    print("silu", flush=True)
    cap = 300032
    gu = torch.cat([D, D[:32]])
    labels = torch.zeros(cap, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(gu)
    dy = normal(cap, I)
    M.moe_silu_mul_bf16_backward(gu, dy, labels, ints(cap), ints(cap, 0), 1, 32, out)
    small = torch.zeros((64, 2 * I), dtype=BF, device="cuda")
    M.moe_silu_mul_bf16_backward(gu[-64:], dy[-64:], labels[:64], ints(64), ints(64, 0), 1, 32,
                                 small)
    assert torch.equal(out[-64:], small)


@pytest.mark.parametrize("fp8", [False, True])
def test_adamw(fp8):
    n, tail = (1 << 31) + 1000, 1 << 12          # the tail starts inside a group
    start = (n - tail) // 128 * 128
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    master = torch.empty(n, device="cuda").normal_(0, 1, generator=g)
    grad = torch.empty(n, dtype=BF, device="cuda").normal_(0, 1e-2, generator=g)
    dt = torch.uint8 if fp8 else torch.float32
    m, v = torch.zeros(n, dtype=dt, device="cuda"), torch.zeros(n, dtype=dt, device="cuda")
    ms, vs = (torch.zeros(-(-n // 128), device="cuda") if fp8 else None for _ in range(2))
    full = (master, grad, m, v, None, ms, vs)
    part = tuple(None if t is None else
                 (t[start // 128:] if t is ms or t is vs else t[start:]).clone() for t in full)
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    lr = torch.full((1,), 1e-3, device="cuda")
    print(f"adamw fp8 {fp8}", flush=True)
    for e in (full, part):
        M.moe_adamw(M.AdamWTensors([e]), step, lr)
    for a, b, off in ((master, part[0], start), (m, part[2], start), (v, part[3], start)):
        assert torch.equal(a[off:], b)
    if fp8:
        assert torch.equal(ms[start // 128:], part[5]) and torch.equal(vs[start // 128:], part[6])
