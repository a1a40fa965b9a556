"""One token's row of a wider buffer, whose own pitch no call may depend on: equal bits
to the same row held by itself."""

import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF, F32 = torch.bfloat16, torch.float32


def view_of(row, pitch):
    held = torch.full((3, pitch), float("nan"), dtype=row.dtype, device="cuda")
    held[0, :row.shape[1]] = row[0]
    return held[:1, :row.shape[1]], held


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pitch", [265, 270, 301])
def test_norm_and_its_gradient(dtype, pitch):
    H = 264
    x, branch, dy = (torch.randn((1, H), device="cuda").to(t) for t in (dtype, BF, BF))
    weight = torch.randn(H, device="cuda")
    outs = []
    for x1 in (x.clone(), view_of(x, pitch)[0]):
        y = torch.zeros((1, H), dtype=BF, device="cuda")
        mean, rstd = (torch.zeros(1, device="cuda") for _ in range(2))
        M.moe_layer_norm(x1, weight, y, mean=mean, rstd=rstd)
        dx = torch.zeros((1, H), dtype=dtype, device="cuda")
        M.moe_layer_norm_backward(dy, x1, weight, rstd, dx, mean)
        M.moe_layer_norm(x1, weight, y2 := torch.zeros_like(y), branch=branch, sum=x1)
        outs.append([y, mean, rstd, dx, y2, x1.clone()])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(outs[0][5], (x.float() + branch.float()).to(dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,pitch", [(60, 61), (256, 257), (512, 1023)])
def test_router_and_its_gradient(dtype, E, pitch):
    x = torch.randn((1, E), device="cuda").to(dtype)
    dw = torch.randn((1, 4), device="cuda")
    outs = []
    for apart in (False, True):
        x1, held = view_of(x, pitch) if apart else (x, None)
        dx, held = (view_of(torch.zeros_like(x), pitch) if apart
                    else (torch.zeros_like(x), None))
        ids = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
        w = torch.zeros((1, 4), device="cuda")
        M.moe_router(x1, ids, w)
        M.moe_router_backward(x1, ids, dw, dx, normalize=False)
        outs.append([ids, w, dx.clone()])
        assert held is None or bool(torch.isnan(held.view(-1)[E:]).all())
    assert all(torch.equal(a, b) for a, b in zip(*outs))
