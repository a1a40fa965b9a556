"""Argument checks of the norm, the router and the 4-bit products (no GPU: every
call fails a check before anything is launched, or has nothing to do)."""

import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

FAKE = 0x10000000        # 16-byte aligned, never dereferenced
APART = 0x10000000       # distance between the buffers of a call
MIS = 4


def at(i):
    return FAKE + i * APART


def _norm(**kw):
    a = dict(x=at(0), xs=256, xf=0, branch=at(1), w=at(2), b=at(3), wf=1, kind=0, eps=1e-5,
             prank=None, nsrc=0, rows=8, h=256, sum=at(4), y=at(5), mean=at(6), rstd=at(7))
    a.update(kw)
    return M.lib().moe_layer_norm(*a.values(), None)


def test_norm_rejects_bad_arguments():
    assert _norm(h=100) == M.MOE_ERR_SHAPE
    assert _norm(h=0) == M.MOE_ERR_SHAPE
    assert _norm(xs=248) == M.MOE_ERR_SHAPE
    assert _norm(rows=-1) == M.MOE_ERR_SHAPE
    assert _norm(rows=(1 << 30) + 1) == M.MOE_ERR_SHAPE
    assert _norm(prank=FAKE, nsrc=0) == M.MOE_ERR_SHAPE
    assert _norm(nsrc=-1) == M.MOE_ERR_SHAPE
    for eps in (-1e-5, float("nan"), float("inf")):
        assert _norm(eps=eps) == M.MOE_ERR_SHAPE
    assert _norm(h=8200, xs=8200) == M.MOE_ERR_UNSUPPORTED
    assert _norm(xf=2) == M.MOE_ERR_UNSUPPORTED
    assert _norm(wf=2) == M.MOE_ERR_UNSUPPORTED
    assert _norm(kind=2) == M.MOE_ERR_UNSUPPORTED
    assert _norm(branch=None) == M.MOE_ERR_UNSUPPORTED           # sum without a branch
    for name in ("x", "w", "y"):
        assert _norm(**{name: None}) == M.MOE_ERR_NULL
    for name in ("x", "branch", "w", "b", "sum", "y"):
        assert _norm(**{name: at(9) + MIS}) == M.MOE_ERR_ALIGNMENT
    assert _norm(xs=260) == M.MOE_ERR_ALIGNMENT
    assert _norm(mean=at(6) + 2) == M.MOE_ERR_ALIGNMENT
    assert _norm(rstd=at(6) + 2) == M.MOE_ERR_ALIGNMENT
    assert _norm(rows=0) == M.MOE_OK


def test_strides_past_the_limit():
    assert _norm(xs=(1 << 30) + 8) == M.MOE_ERR_SHAPE
    assert _norm(xs=1 << 62) == M.MOE_ERR_SHAPE
    assert _norm_back(xs=1 << 62) == M.MOE_ERR_SHAPE


def test_norm_refuses_shared_memory():
    for out in ("sum", "y", "mean", "rstd"):
        for other in ("x", "branch", "w", "b"):
            if (out, other) != ("sum", "x"):
                old = dict(x=at(0), branch=at(1), w=at(2), b=at(3))[other]
                assert _norm(**{out: old}) == M.MOE_ERR_UNSUPPORTED, (out, other)
    assert _norm(sum=at(0), xs=264) == M.MOE_ERR_UNSUPPORTED      # in place, rows apart
    assert _norm(sum=at(0) + 16) == M.MOE_ERR_UNSUPPORTED
    assert _norm(y=at(4)) == M.MOE_ERR_UNSUPPORTED                # two outputs
    assert _norm(rstd=at(6)) == M.MOE_ERR_UNSUPPORTED
    assert _norm(sum=at(0), rows=0) == M.MOE_OK


def _norm_back(**kw):
    a = dict(dy=at(0), dy2=at(1), x=at(2), xs=256, xf=0, w=at(3), wf=1, kind=0, mean=at(4),
             rstd=at(5), dsum=at(6), prank=None, nsrc=0, rows=8, h=256, dx=at(7), dw=at(8),
             db=at(9), gf=1, acc=0, ws=at(10), wsb=1 << 20)
    a.update(kw)
    return M.lib().moe_layer_norm_backward(*a.values(), None)


def test_norm_backward_rejects_bad_arguments():
    f = _norm_back
    assert f(h=100) == M.MOE_ERR_SHAPE
    assert f(xs=248) == M.MOE_ERR_SHAPE
    assert f(rows=-1) == M.MOE_ERR_SHAPE
    assert f(h=8200, xs=8200) == M.MOE_ERR_UNSUPPORTED
    assert f(gf=2) == M.MOE_ERR_UNSUPPORTED
    assert f(kind=2) == M.MOE_ERR_UNSUPPORTED
    for name in ("dy", "x", "w", "rstd", "mean", "dx"):
        assert f(**{name: None}) == M.MOE_ERR_NULL
    for name in ("dy", "dy2", "x", "w", "dsum", "dx", "dw", "db", "ws"):
        assert f(**{name: at(12) + MIS}) == M.MOE_ERR_ALIGNMENT
    assert f(ws=at(10) + 16) == M.MOE_ERR_ALIGNMENT
    need = M.moe_layer_norm_backward_workspace_bytes(8, 256)
    assert need > 0
    assert f(ws=None) == M.MOE_ERR_WORKSPACE
    assert f(wsb=need - 1) == M.MOE_ERR_WORKSPACE
    assert f(rows=0, acc=1) == M.MOE_OK
    assert f(rows=0, dw=None, db=None, ws=None) == M.MOE_OK


def test_norm_backward_refuses_shared_memory():
    places = dict(dy=at(0), dy2=at(1), x=at(2), w=at(3), mean=at(4), rstd=at(5), dsum=at(6))
    for out in ("dx", "dw", "db", "ws"):
        for other, p in places.items():
            if (out, other) != ("dx", "dsum"):
                assert _norm_back(**{out: p}) == M.MOE_ERR_UNSUPPORTED, (out, other)
    assert _norm_back(dx=at(6) + 16) == M.MOE_ERR_UNSUPPORTED
    assert _norm_back(db=at(8)) == M.MOE_ERR_UNSUPPORTED
    assert _norm_back(ws=at(7)) == M.MOE_ERR_UNSUPPORTED
    assert _norm_back(dw=at(6), dx=at(6)) == M.MOE_ERR_UNSUPPORTED


def test_norm_workspace_bytes():
    f = M.moe_layer_norm_backward_workspace_bytes
    assert f(-1, 256) == f(8, 100) == f(8, 8200) == f(0, 256) == 0
    assert f(1 << 30, 8192) < 64 << 20


def _router(**kw):
    a = dict(x=at(0), xs=64, fmt=1, bias=at(1), score=1, groups=4, tg=2, norm=1, prank=None,
             nsrc=0, rows=8, E=64, topk=4, ids=at(2), w=at(3))
    a.update(kw)
    return M.lib().moe_router(*a.values(), None)


def _router_back(**kw):
    a = dict(x=at(0), xs=64, fmt=1, score=1, norm=1, ids=at(2), dw=at(3), prank=None, nsrc=0,
             rows=8, E=64, topk=4, dx=at(4), dxs=64)
    a.update(kw)
    return M.lib().moe_router_backward(*a.values(), None)


@pytest.mark.parametrize("f", [_router, _router_back])
def test_router_rejects_bad_arguments(f):
    assert f(rows=-1) == M.MOE_ERR_SHAPE
    assert f(E=0) == M.MOE_ERR_SHAPE
    assert f(E=1025, xs=1025) == M.MOE_ERR_SHAPE
    assert f(topk=0) == M.MOE_ERR_SHAPE
    assert f(topk=33) == M.MOE_ERR_SHAPE
    assert f(E=4, topk=5) == M.MOE_ERR_SHAPE
    assert f(xs=63) == M.MOE_ERR_SHAPE
    assert f(prank=FAKE, nsrc=0) == M.MOE_ERR_SHAPE
    assert f(fmt=2) == M.MOE_ERR_UNSUPPORTED
    assert f(score=2) == M.MOE_ERR_UNSUPPORTED
    assert f(x=None) == M.MOE_ERR_NULL
    assert f(ids=None) == M.MOE_ERR_NULL
    assert f(x=at(0) + 2) == M.MOE_ERR_ALIGNMENT
    assert f(ids=at(2) + 2) == M.MOE_ERR_ALIGNMENT
    assert f(rows=0) == M.MOE_OK


def test_router_options():
    assert _router(groups=0) == M.MOE_ERR_SHAPE
    assert _router(groups=3) == M.MOE_ERR_SHAPE
    assert _router(groups=128, E=256, xs=256) == M.MOE_ERR_SHAPE
    assert _router(tg=0) == M.MOE_ERR_SHAPE
    assert _router(tg=5) == M.MOE_ERR_SHAPE
    assert _router(w=None) == M.MOE_ERR_NULL
    assert _router(bias=at(1) + 2) == M.MOE_ERR_ALIGNMENT
    for out in ("ids", "w"):
        for p in (at(0), at(0) + 8 * 64 * 4 - 4, at(1)):
            assert _router(**{out: p}) == M.MOE_ERR_UNSUPPORTED
    assert _router(w=at(2)) == M.MOE_ERR_UNSUPPORTED
    assert _router_back(dxs=63) == M.MOE_ERR_SHAPE
    assert _router_back(dx=None) == M.MOE_ERR_NULL
    assert _router_back(dw=None) == M.MOE_ERR_NULL
    assert _router_back(dx=at(4) + 2) == M.MOE_ERR_ALIGNMENT
    for p in (at(0), at(2), at(3)):
        assert _router_back(dx=p) == M.MOE_ERR_UNSUPPORTED


def _w4(**kw):
    a = dict(a=at(0), w=at(1), sc=at(2), fmt=0, group=128, psum=at(3), st=at(4), cap=320, n=256,
             k=256, E=4, align=64, out=at(5))
    a.update(kw)
    return M.lib().moe_grouped_gemm_w4(*a.values(), None)


def test_w4_rejects_bad_arguments():
    assert _w4(n=192) == M.MOE_ERR_SHAPE
    assert _w4(k=192) == M.MOE_ERR_SHAPE
    assert _w4(k=0) == M.MOE_ERR_SHAPE
    assert _w4(cap=-64) == M.MOE_ERR_SHAPE
    assert _w4(cap=100) == M.MOE_ERR_SHAPE
    assert _w4(E=0) == M.MOE_ERR_SHAPE
    assert _w4(E=1025) == M.MOE_ERR_SHAPE
    assert _w4(align=48) == M.MOE_ERR_UNSUPPORTED
    assert _w4(group=16) == M.MOE_ERR_UNSUPPORTED
    assert _w4(fmt=1) == M.MOE_ERR_UNSUPPORTED                    # MXFP4 with groups of 128
    assert _w4(fmt=2, group=32) == M.MOE_ERR_UNSUPPORTED
    assert _w4(k=512 * 64) == M.MOE_ERR_UNSUPPORTED
    assert _w4(n=512 * 64) == M.MOE_ERR_UNSUPPORTED
    for name in ("a", "w", "sc", "psum", "st", "out"):
        assert _w4(**{name: None}) == M.MOE_ERR_NULL
    for name in ("a", "w", "sc", "out"):
        assert _w4(**{name: at(9) + MIS}) == M.MOE_ERR_ALIGNMENT
    for i in range(5):
        assert _w4(out=at(i)) == M.MOE_ERR_UNSUPPORTED
    assert _w4(cap=0) == M.MOE_OK
    assert _w4(cap=0, fmt=1, group=32) == M.MOE_OK


class Tensor:
    """Stands in for a tensor of the current GPU."""

    def __init__(self, dtype, *shape, stride=None, gpu=0):
        self.dtype, self.shape, self.gpu = dtype, torch.Size(shape), gpu
        step, steps = 1, []
        for s in reversed(shape):
            steps.insert(0, step)
            step *= s
        self.steps, self.whole = tuple(stride or steps), stride is None

    get_device = lambda self: self.gpu  # noqa: E731
    device = property(lambda self: f"cuda:{self.gpu}")
    stride = lambda self: self.steps  # noqa: E731
    is_contiguous = lambda self: self.whole  # noqa: E731
    numel = lambda self: self.shape.numel()  # noqa: E731
    data_ptr = lambda self: FAKE  # noqa: E731


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, taken down."""
    got = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: got.append((name, a)) or M.MOE_OK

    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(M, "lib", lambda: Library())
    return got


BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def test_binding_refuses_what_the_library_cannot_see(calls):
    x, y, w = Tensor(BF, 8, 256), Tensor(BF, 8, 256), Tensor(F32, 256)
    M.moe_layer_norm(x, w, y, stream=1)
    M.moe_layer_norm(Tensor(F32, 8, 256, stride=(512, 1)), w, y, stream=1)
    assert [a[1] for _, a in calls] == [256, 512] and [a[2] for _, a in calls] == [False, True]
    for bad in (dict(x=Tensor(torch.float16, 8, 256)), dict(x=Tensor(BF, 8, 256, stride=(1, 8))),
                dict(x=Tensor(BF, 8, 256, stride=(0, 1))), dict(x=Tensor(BF, 8, 256, gpu=1)),
                dict(y=Tensor(F32, 8, 256)), dict(y=Tensor(BF, 7, 256)), dict(weight=Tensor(F32, 255)),
                dict(bias=Tensor(BF, 256)), dict(branch=Tensor(F32, 8, 256)),
                dict(branch=y, sum=Tensor(F32, 8, 256)), dict(mean=Tensor(F32, 9)),
                dict(rstd=Tensor(BF, 8)), dict(psum_recv_per_rank=Tensor(torch.int64, 1))):
        with pytest.raises(ValueError):
            M.moe_layer_norm(**{**dict(x=x, weight=w, y=y, stream=1), **bad})
    with pytest.raises(KeyError):
        M.moe_layer_norm(x, w, y, kind="batch", stream=1)
    r = Tensor(F32, 8)
    good = dict(dy=y, x=x, weight=w, rstd=r, dx=Tensor(BF, 8, 256), mean=r, stream=1)
    M.moe_layer_norm_backward(**good)
    for bad in (dict(dx=Tensor(F32, 8, 256)), dict(dsum=Tensor(F32, 8, 256)),
                dict(dweight=Tensor(torch.float16, 256)), dict(dy2=Tensor(BF, 8, 128)),
                dict(dweight=Tensor(F32, 256), dbias=Tensor(BF, 256)),
                dict(workspace=Tensor(F32, 256))):
        with pytest.raises(ValueError):
            M.moe_layer_norm_backward(**{**good, **bad})
    lg, ids, tw = Tensor(F32, 8, 64, stride=(128, 1)), Tensor(I32, 8, 4), Tensor(F32, 8, 4)
    M.moe_router(lg, ids, tw, stream=1)
    for bad in (dict(logits=Tensor(torch.float64, 8, 64)), dict(topk_ids=Tensor(torch.int64, 8, 4)),
                dict(topk_weights=Tensor(F32, 8, 5)), dict(bias=Tensor(BF, 64))):
        with pytest.raises(ValueError):
            M.moe_router(**{**dict(logits=lg, topk_ids=ids, topk_weights=tw, stream=1), **bad})
    M.moe_router_backward(lg, ids, tw, Tensor(F32, 8, 64), stream=1)
    with pytest.raises(ValueError):
        M.moe_router_backward(lg, ids, tw, Tensor(BF, 8, 64), stream=1)
    a, q = Tensor(BF, 64, 256), Tensor(torch.uint8, 4, 128, 128)
    rest = (Tensor(I32, 4), Tensor(I32, 2), 16, Tensor(BF, 64, 128))
    M.moe_grouped_gemm_w4(a, q, Tensor(BF, 4, 128, 4), "int4", *rest, stream=1)
    assert calls[-1][1][4] == 64
    M.moe_grouped_gemm_w4(a, q, Tensor(torch.uint8, 4, 128, 8), "mxfp4", *rest, stream=1)
    assert calls[-1][1][4] == 32
    for sc, fmt in ((Tensor(torch.uint8, 4, 128, 8), "int4"), (Tensor(BF, 4, 128, 8), "mxfp4"),
                    (Tensor(BF, 4, 127, 8), "int4"), (Tensor(BF, 4, 128, 3), "int4")):
        with pytest.raises(ValueError):
            M.moe_grouped_gemm_w4(a, q, sc, fmt, *rest, stream=1)
    with pytest.raises(ValueError):
        M.moe_grouped_gemm_w4(a, Tensor(torch.int8, 4, 128, 128), Tensor(BF, 4, 128, 2), "int4",
                              *rest, stream=1)
