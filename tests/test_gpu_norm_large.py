"""moe_layer_norm_backward where dx is larger than the caches: bit for bit the same rows
in smaller calls, and the rows behind left as they were."""

import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,rows,H", [(BF, 16400, 4104), (BF, 9300, 7224), (BF, 270000, 256),
                                          (F32, 16400, 2056)])
@pytest.mark.parametrize("kind,second,in_place", [("layer", False, True), ("rms", True, False)])
def test_large_dx(dtype, rows, H, kind, second, in_place):
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    rand = lambda *s, t=BF: torch.randn(s, generator=g, device="cuda").to(t)  # noqa: E731
    x, dy, weight = rand(rows, H, t=dtype), rand(rows, H), rand(H, t=F32)
    dy2 = rand(rows, H) if second else None
    mean, rstd = rand(rows, t=F32), rand(rows, t=F32).abs() + 0.5
    dsum = rand(rows, H, t=dtype) if in_place else None
    dx = dsum.clone() if in_place else torch.full((rows, H), 7.0, dtype=dtype, device="cuda")
    kept = dx.clone()
    assert dx.numel() * dx.element_size() > 128 << 20
    nv = rows - 3
    prank = torch.tensor([nv], dtype=torch.int32, device="cuda")
    M.moe_layer_norm_backward(dy, x, weight, rstd, dx, mean if kind == "layer" else None, dy2,
                              dx if in_place else None, kind=kind, psum_recv_per_rank=prank)
    step = rows // 4 + 1
    for i in range(0, nv, step):
        at = slice(i, min(i + step, nv))
        part = torch.empty_like(dx[at])
        M.moe_layer_norm_backward(dy[at], x[at], weight, rstd[at].clone(), part,
                                  mean[at].clone() if kind == "layer" else None,
                                  None if dy2 is None else dy2[at],
                                  dsum[at] if in_place else None, kind=kind)
        assert torch.equal(dx[at], part)
    assert torch.equal(dx[nv:], kept[nv:])
