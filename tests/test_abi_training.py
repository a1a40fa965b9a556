"""Argument checks of the training entry points (no GPU: every call fails a
host-side check before anything is launched, or has nothing to do)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

FAKE = 0x100000          # 16-byte aligned, never dereferenced
MIS = FAKE + 4


def _dgrad(**kw):
    a = dict(dy=FAKE, w=FAKE, psum=FAKE, st=FAKE, cap=320, n=256, k=256, E=4, align=64, dx=FAKE)
    a.update(kw)
    return M.lib().moe_grouped_dgrad_bf16(a["dy"], a["w"], a["psum"], a["st"], a["cap"], a["n"],
                                          a["k"], a["E"], a["align"], a["dx"], None)


def _wgrad(**kw):
    a = dict(dy=FAKE, x=FAKE, psum=FAKE, st=FAKE, cap=320, n=256, k=256, E=4, align=64, fmt=0,
             acc=0, dw=FAKE, ws=None, wsb=0)
    a.update(kw)
    return M.lib().moe_grouped_wgrad_bf16(
        a["dy"], a["x"], a["psum"], a["st"], a["cap"], a["n"], a["k"], a["E"], a["align"],
        a["fmt"], a["acc"], a["dw"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("f", [_dgrad, _wgrad])
def test_products_reject_bad_arguments(f):
    assert f(n=100) == M.MOE_ERR_SHAPE
    assert f(n=192) == M.MOE_ERR_SHAPE
    assert f(k=96) == M.MOE_ERR_SHAPE
    assert f(k=0) == M.MOE_ERR_SHAPE
    assert f(cap=-64) == M.MOE_ERR_SHAPE
    assert f(cap=100) == M.MOE_ERR_SHAPE
    assert f(E=0) == M.MOE_ERR_SHAPE
    assert f(E=1025) == M.MOE_ERR_SHAPE
    assert f(align=48) == M.MOE_ERR_UNSUPPORTED
    assert f(align=8) == M.MOE_ERR_UNSUPPORTED
    assert f(k=512 * 64) == M.MOE_ERR_UNSUPPORTED
    assert f(n=512 * 64) == M.MOE_ERR_UNSUPPORTED
    assert f(psum=None) == M.MOE_ERR_NULL
    assert f(st=None) == M.MOE_ERR_NULL
    assert f(dy=None) == M.MOE_ERR_NULL
    assert f(dy=MIS) == M.MOE_ERR_ALIGNMENT


def test_product_operands():
    assert _dgrad(w=None) == M.MOE_ERR_NULL
    assert _dgrad(dx=None) == M.MOE_ERR_NULL
    assert _dgrad(dx=MIS) == M.MOE_ERR_ALIGNMENT
    assert _dgrad(w=MIS) == M.MOE_ERR_ALIGNMENT
    assert _dgrad(cap=0) == M.MOE_OK                 # nothing to do, nothing launched
    assert _wgrad(x=None) == M.MOE_ERR_NULL
    assert _wgrad(dw=None) == M.MOE_ERR_NULL
    assert _wgrad(x=MIS) == M.MOE_ERR_ALIGNMENT
    assert _wgrad(dw=MIS) == M.MOE_ERR_ALIGNMENT
    assert _wgrad(fmt=2) == M.MOE_ERR_UNSUPPORTED


def test_silu_backward_rejects_bad_arguments():
    def f(**kw):
        a = dict(gu=FAKE, dy=FAKE, mi=FAKE, psum=FAKE, st=FAKE, cap=320, inter=128, E=4,
                 align=64, out=FAKE)
        a.update(kw)
        return M.lib().moe_silu_mul_bf16_backward(
            a["gu"], a["dy"], a["mi"], a["psum"], a["st"], a["cap"], a["inter"], a["E"],
            a["align"], a["out"], None)
    assert f(inter=100) == M.MOE_ERR_SHAPE
    assert f(cap=100) == M.MOE_ERR_SHAPE
    assert f(E=0) == M.MOE_ERR_SHAPE
    assert f(align=48) == M.MOE_ERR_UNSUPPORTED
    assert f(mi=None) == M.MOE_ERR_NULL
    assert f(st=None) == M.MOE_ERR_NULL
    assert f(dy=None) == M.MOE_ERR_NULL
    assert f(out=None) == M.MOE_ERR_NULL
    assert f(dy=MIS) == M.MOE_ERR_ALIGNMENT
    assert f(out=MIS) == M.MOE_ERR_ALIGNMENT
    assert f(cap=0) == M.MOE_OK


def test_gather_backward_rejects_bad_arguments():
    def f(**kw):
        a = dict(do=FAKE, eo=FAKE, s2d=FAKE, w=None, f=1.0, prank=None, nsrc=0, rows=64,
                 hidden=256, topk=2, cap=320, deo=FAKE, dw=FAKE)
        a.update(kw)
        return M.lib().moe_gather_backward(
            a["do"], a["eo"], a["s2d"], a["w"], a["f"], a["prank"], a["nsrc"], a["rows"],
            a["hidden"], a["topk"], a["cap"], a["deo"], a["dw"], None)
    assert f(f=float("nan")) == M.MOE_ERR_UNSUPPORTED
    assert f(f=float("-inf")) == M.MOE_ERR_UNSUPPORTED
    assert f(hidden=100) == M.MOE_ERR_SHAPE
    assert f(hidden=8320) == M.MOE_ERR_UNSUPPORTED
    assert f(topk=0) == M.MOE_ERR_SHAPE
    assert f(topk=33) == M.MOE_ERR_SHAPE
    assert f(rows=-1) == M.MOE_ERR_SHAPE
    assert f(prank=FAKE, nsrc=0) == M.MOE_ERR_SHAPE
    assert f(s2d=None) == M.MOE_ERR_NULL
    assert f(do=None) == M.MOE_ERR_NULL
    assert f(deo=None) == M.MOE_ERR_NULL
    assert f(eo=None) == M.MOE_ERR_NULL              # needed for d_topk_weights
    assert f(do=MIS) == M.MOE_ERR_ALIGNMENT
    assert f(deo=MIS) == M.MOE_ERR_ALIGNMENT
    assert f(dw=FAKE + 2) == M.MOE_ERR_ALIGNMENT
    assert f(rows=0) == M.MOE_OK


def _adamw(tensors=None, num=None, step=FAKE, lr=FAKE, gs=None, b1=0.9, b2=0.95, eps=1e-8,
           wd=0.1, **kw):
    if tensors is None:
        a = dict(master=FAKE, grad=FAKE, m=FAKE, v=FAKE, param=None, m_scale=None, v_scale=None,
                 numel=10, grad_fmt=0, state_fmt=0)
        a.update(kw)
        tensors = [a]
    arr = (M._AdamWTensor * max(len(tensors), 1))(*[M._AdamWTensor(**t) for t in tensors])
    return M.lib().moe_adamw(arr, len(tensors) if num is None else num, step, lr, gs, b1, b2,
                             eps, wd, None)


def test_adamw_rejects_bad_arguments():
    nan, inf = float("nan"), float("inf")
    assert _adamw(num=-1) == M.MOE_ERR_SHAPE
    for bad in (dict(b1=1.0), dict(b1=-0.1), dict(b2=nan), dict(b2=1.0), dict(eps=-1e-8),
                dict(eps=inf), dict(wd=nan), dict(wd=-1.0)):
        assert _adamw(**bad) == M.MOE_ERR_SHAPE, bad
    assert _adamw(step=None) == M.MOE_ERR_NULL
    assert _adamw(lr=None) == M.MOE_ERR_NULL
    assert _adamw(step=FAKE + 4) == M.MOE_ERR_ALIGNMENT
    assert _adamw(numel=-1) == M.MOE_ERR_SHAPE
    assert _adamw(numel=(1 << 33) + 1) == M.MOE_ERR_SHAPE
    assert _adamw(grad_fmt=2) == M.MOE_ERR_UNSUPPORTED
    assert _adamw(state_fmt=2) == M.MOE_ERR_UNSUPPORTED
    for name in ("master", "grad", "m", "v"):
        assert _adamw(**{name: None}) == M.MOE_ERR_NULL
        assert _adamw(**{name: MIS}) == M.MOE_ERR_ALIGNMENT
    assert _adamw(param=MIS) == M.MOE_ERR_ALIGNMENT
    assert _adamw(state_fmt=1) == M.MOE_ERR_NULL                    # no scales
    assert _adamw(state_fmt=1, m_scale=FAKE, v_scale=FAKE + 2) == M.MOE_ERR_ALIGNMENT
    assert _adamw(numel=0, master=None) == M.MOE_OK                 # skipped
    assert _adamw(tensors=[]) == M.MOE_OK
    two = [dict(master=FAKE + o, grad=FAKE, m=FAKE, v=FAKE, numel=10, grad_fmt=0, state_fmt=0)
           for o in (0, 32)]
    assert _adamw(tensors=two) == M.MOE_ERR_UNSUPPORTED             # masters overlap
    far = [dict(two[0], master=FAKE + 0x1000 * i) for i in (5, 9, 1, 7, 5)]
    assert _adamw(tensors=far) == M.MOE_ERR_UNSUPPORTED             # the first again, last
    assert _adamw(tensors=[dict(t, numel=0) for t in far]) == M.MOE_OK


# A list that passes every check is launched, and without a GPU the launch fails.
PASSES = M.MOE_ERR_LAUNCH


def _entry(i, **kw):
    """Tensor i of 1000 values, with arrays of its own."""
    at = lambda j: 0x10000000 * (i + 1) + 0x100000 * j  # noqa: E731
    a = dict(master=at(0), grad=at(1), m=at(2), v=at(3), param=None, m_scale=None, v_scale=None,
             numel=1000, grad_fmt=0, state_fmt=0)
    a.update(kw)
    return a


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: never launched")
def test_adamw_passes_over_empty_tensors():
    """An empty tensor overlaps nothing, wherever its pointer lies."""
    last = _entry(1)
    empty = _entry(7, master=last["master"] + 16, numel=0)
    far = [_entry(0), _entry(5)]
    assert _adamw(tensors=far + [empty, last]) == PASSES
    assert _adamw(tensors=far + [last, empty]) == PASSES
    assert _adamw(tensors=far + [last]) == PASSES


def _coded(i, **kw):
    """The same with a bf16 copy and 8-bit states: 1000 codes, 8 scales each."""
    base = 0x10000000 * (i + 1)
    a = dict(param=base + 0x400000, m_scale=base + 0x500000, v_scale=base + 0x600000, state_fmt=1)
    a.update(kw)
    return _entry(i, **a)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: never launched")
def test_adamw_keeps_written_arrays_apart():
    """Any two arrays of a call of which one is written, within a tensor and
    between two, by their last byte and by their first."""
    assert _adamw(tensors=[_coded(0), _entry(1), _coded(2)]) == PASSES
    size = dict(master=4000, grad=2000, m=1000, v=1000, param=2000, m_scale=32, v_scale=32)
    for a in size:
        for b in size:
            for other in (0, 1):
                if (a, 0) == (b, other):
                    continue
                one = _coded(0)
                # Arrays begin at multiples of 16.
                for at in (one[a], (one[a] + size[a] - 1) // 16 * 16):
                    two = [dict(one), _coded(1)]
                    two[other][b] = at
                    want = PASSES if a == b == "grad" else M.MOE_ERR_UNSUPPORTED
                    assert _adamw(tensors=two) == want, (a, b, other)
                two = [dict(one), _coded(1)]
                two[other][b] = -(-(one[a] + size[a]) // 16) * 16       # right behind it
                assert _adamw(tensors=two) == PASSES, (a, b, other)
    one = _entry(0)
    for scalar in ("step", "lr", "gs"):
        for a in ("master", "m", "v"):
            assert _adamw(tensors=[one], **{scalar: one[a] + 8}) == M.MOE_ERR_UNSUPPORTED
        assert _adamw(tensors=[one], **{scalar: one["grad"] + 8}) == PASSES
    many = [_coded(i) for i in range(90)]
    assert _adamw(tensors=many) == PASSES
    many[80]["v_scale"] = many[3]["param"] + 16
    assert _adamw(tensors=many) == M.MOE_ERR_UNSUPPORTED


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: never launched")
def test_adamw_takes_no_eps_below_the_normal_range():
    """The step divides by eps alone where v is 0: 0 gives what 0 gives, and any
    other eps is a normal fp32 number."""
    for eps in (5e-324, 1e-46, 1e-45, 1e-40, 2.0 ** -126 * (1 - 2.0 ** -20)):
        assert _adamw(tensors=[_entry(0)], eps=eps) == M.MOE_ERR_SHAPE, eps
    for eps in (0.0, 2.0 ** -126, 1e-30, 1.0):
        assert _adamw(tensors=[_entry(0)], eps=eps) == PASSES, eps


def _apart(call, size, outputs, allowed=()):
    """Every output on every other buffer, at its first 16 bytes and at its last."""
    base = {name: 0x10000000 * (i + 1) for i, name in enumerate(size)}
    assert call(base) == PASSES
    for out in outputs:
        for other in size:
            if other == out:
                continue
            for at in (base[other], base[other] + (size[other] - 1) // 256 * 256):
                same = at == base[other]
                want = PASSES if same and (out, other) in allowed else M.MOE_ERR_UNSUPPORTED
                assert call({**base, out: at}) == want, (out, other, same)
            behind = base[other] + -(-size[other] // 256) * 256
            assert call({**base, out: behind}) == PASSES, (out, other)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: never launched")
def test_outputs_share_no_memory_with_other_buffers():
    L, ints = M.lib(), FAKE
    cap, n, k, E, rows, topk = 320, 256, 256, 4, 64, 2
    _apart(lambda p: L.moe_grouped_dgrad_bf16(p["dy"], p["w"], ints, ints, cap, n, k, E, 64,
                                              p["dx"], None),
           dict(dy=cap * n * 2, w=E * n * k * 2, dx=cap * k * 2), ["dx"])
    cap, E = 20480, 1                                       # sums in parts: a workspace
    for fmt, bytes_ in ((0, 2), (1, 4)):
        need = M.moe_grouped_wgrad_workspace_bytes(cap, n, k, E)
        assert need > 0
        _apart(lambda p: L.moe_grouped_wgrad_bf16(p["dy"], p["x"], ints, ints, cap, n, k, E, 64,
                                                  fmt, 0, p["dw"], p["ws"], need, None),
               dict(dy=cap * n * 2, x=cap * k * 2, dw=E * n * k * bytes_, ws=need), ["dw", "ws"])
    cap, E = 320, 4
    _apart(lambda p: L.moe_silu_mul_bf16_backward(p["gu"], p["dy"], ints, ints, ints, cap, 128, E,
                                                  64, p["out"], None),
           dict(gu=cap * 512, dy=cap * 256, out=cap * 512), ["out"], [("out", "gu")])
    _apart(lambda p: L.moe_gather_backward(p["dout"], p["eo"], p["s2d"], p["w"], 1.0, None, 0,
                                           rows, n, topk, cap, p["deo"], p["dw"], None),
           dict(dout=rows * n * 2, eo=cap * n * 2, s2d=rows * topk * 4, w=rows * topk * 4,
                deo=cap * n * 2, dw=rows * topk * 4), ["deo", "dw"])
    # Without d_topk_weights expert_out is not read: its place may be written.
    assert L.moe_gather_backward(0x10000000, 0x20000000, 0x30000000, None, 1.0, None, 0, rows, n,
                                 topk, cap, 0x20000000, None, None) == PASSES


def test_header_matches_the_struct():
    assert ctypes.sizeof(M._AdamWTensor) == 72


def test_wgrad_workspace_bad_input():
    f = M.moe_grouped_wgrad_workspace_bytes
    assert f(-1, 256, 256, 4) == 0
    assert f(256, 100, 256, 4) == 0
    assert f(256, 256, 256, 0) == 0


def test_binding_refuses_what_the_library_cannot_see():
    """The binding raises on shapes, types, strides and devices before any call."""
    bf = torch.bfloat16
    z = lambda *s, d=bf: torch.zeros(s, dtype=d)  # noqa: E731
    psum, st = z(2, d=torch.int32), z(2, d=torch.int32)
    with pytest.raises(ValueError, match="not on the current GPU"):
        M.moe_grouped_dgrad_bf16(z(64, 128), z(2, 128, 64), psum, st, 32, z(64, 64))
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_grouped_dgrad_bf16(z(128, 64).t(), z(2, 128, 64), psum, st, 32, z(64, 64))
    with pytest.raises(ValueError, match="dy must be"):
        M.moe_grouped_wgrad_bf16(z(64, 128, d=torch.float16), z(64, 64), psum, st, 32,
                                 z(2, 128, 64))
    with pytest.raises(ValueError, match="master 0 must be"):
        f = z(5, d=torch.float32)
        M.AdamWTensors([(z(5), f, f, f, None, None, None)])
