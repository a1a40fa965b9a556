"""What the binding and the Python classes around the experts check and hand on (no
GPU)."""

import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

CPU = -1                                             # what get_device() says of it


@pytest.mark.parametrize("pitch", [264, 265, 271, 1 << 31])
def test_a_single_row_has_no_distance_to_the_next(pitch):
    held = torch.empty(272, dtype=torch.bfloat16)
    for rows in (0, 1):
        view = held.as_strided((rows, 264), (pitch, 1))
        got = M._need_rows("f", "x", view, (torch.bfloat16,), (rows, 264), CPU)
        assert got == 264


def test_rows_apart_keep_their_distance():
    held = torch.empty((5, 272), dtype=torch.bfloat16)
    assert M._need_rows("f", "x", held[:, :264], (torch.bfloat16,), (5, 264), CPU) == 272
    for bad in (held[:, ::2][:, :100], held.t(), held[:1].expand(5, 272)):
        with pytest.raises(ValueError):
            M._need_rows("f", "x", bad, (torch.bfloat16,), bad.shape, CPU)


@pytest.mark.parametrize("H,inter", [(256, 64), (256, 192), (192, 128), (64, 256)])
def test_w4_layer_refuses_sizes_that_its_products_refuse(H, inter):
    """When it is built, not at the first call."""
    w13 = torch.zeros((2, 2 * inter, H // 2), dtype=torch.uint8)
    w2 = torch.zeros((2, H, inter // 2), dtype=torch.uint8)
    s13, s2 = (torch.zeros((2, w.shape[1], w.shape[2] // 16), dtype=torch.uint8) for w in (w13, w2))
    with pytest.raises(ValueError, match="multiples of 128"):
        M.StandardW4MoE(8, 2, w13, s13, w2, s2, "mxfp4", device="cpu")


def test_w4_layer_takes_multiples_of_128():
    w13 = torch.zeros((2, 768, 64), dtype=torch.uint8)
    w2 = torch.zeros((2, 128, 192), dtype=torch.uint8)
    s13, s2 = (torch.zeros((2, w.shape[1], w.shape[2] // 16), dtype=torch.uint8) for w in (w13, w2))
    moe = M.StandardW4MoE(8, 2, w13, s13, w2, s2, "mxfp4", device="cpu")
    assert (moe.H, moe.I, moe.E) == (128, 384, 2)


CALLS = ["moe_layer_norm", "moe_grouped_gemm_bf16", "moe_router", "moe_router_backward",
         "moe_grouped_wgrad_bf16", "moe_grouped_dgrad_bf16", "moe_layer_norm_backward"]


class Experts(M.TrainableBf16MoE):
    """Stands in for the experts: hands on what it gets."""

    def __init__(self, rows, topk, E, H):
        self.rows, self.topk, self.E, self.H = rows, topk, E, H

    def __call__(self, y, ids, weights, psum, out, stream):
        if getattr(self, "refuses", False):
            raise ValueError("refused")
        return y

    def backward(self, dout, weights, psum, accumulate, stream):
        return dout, weights


@pytest.mark.parametrize("refused", ["moe_layer_norm", "moe_grouped_gemm_bf16", "moe_router", None])
def test_no_gradient_of_a_forward_call_that_was_refused(monkeypatch, refused):
    """The buffers are then of two calls."""
    for name in CALLS:
        monkeypatch.setattr(M, name, lambda *a, **k: None)
    rows, E, H = 5, 6, 128
    x, branch = torch.zeros((rows, H), dtype=torch.bfloat16), torch.ones(1)
    block = M.MoEBlock(Experts(rows, 2, E, H), torch.zeros((E, H), dtype=torch.bfloat16),
                       torch.ones(H))
    with pytest.raises(RuntimeError):
        block.backward(x)
    for b, stream in ((None, x), (branch, block.sum)):
        out, h = block(x, b)
        assert h is stream and block.h is stream
        block.backward(x, dx=torch.empty_like(x))

    def no(*a, **k):
        raise ValueError("refused")

    with monkeypatch.context() as m:
        if refused:
            m.setattr(M, refused, no)
        else:
            block.moe.refuses = True
        with pytest.raises(ValueError, match="refused"):
            block(x)
        block.moe.refuses = False
    with pytest.raises(RuntimeError):
        block.backward(x, dx=torch.empty_like(x))
    block(x)
    block.backward(x, dx=torch.empty_like(x))
