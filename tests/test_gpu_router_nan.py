"""moe_router_backward beside gradients that are no numbers: experts that are not
available get 0 whatever the slots' gradients are, and other rows are untouched."""

import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E", [5, 64, 100, 256, 1024])
def test_unavailable_experts_get_nothing(E, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    x = torch.randn((12, E), device="cuda", generator=g)
    off = torch.rand((12, E), device="cuda", generator=g) < 0.4
    off[:, :2] = False
    x[off] = float("-inf")
    x[off.cumsum(1).eq(2) & off] = float("nan")
    x = x.to(dtype)
    ids = torch.empty((12, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((12, 2), device="cuda")
    M.moe_router(x, ids, w)
    dw = torch.randn((12, 2), device="cuda", generator=g)
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            clean, dx = torch.empty_like(x), torch.empty_like(x)
            M.moe_router_backward(x, ids, dw, clean, score, normalize)
            bad = dw.clone()
            bad[3, 0], bad[5, 1], bad[7] = float("inf"), float("nan"), float("-inf")
            M.moe_router_backward(x, ids, bad, dx, score, normalize)
            rows = [r for r in range(12) if r not in (3, 5, 7)]
            assert torch.equal(dx[rows], clean[rows])
            assert bool((dx[off] == 0).all())
            assert not bool(torch.isfinite(dx[[3, 5, 7]].float()).all(dim=1).any())
