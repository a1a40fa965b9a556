"""Measured cases of what stands around the experts in an MoE block: the norm
of the residual stream with its backward pass, the router with its backward
pass, and the grouped products with 4-bit expert weights.

`own` false: the plain forms, in elementary torch operations in fp32 (the
router's choice in fp64, so that near scores keep their order).  `own` true:
the framework's calls.  Both take the state that prepare() makes and write the
state's own output buffers: rows outside the result keep what was there.

Rows at or past the received ones, and expanded rows that hold no token, hold
NaN: no result may depend on them.
"""

import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
F32_MAX = torch.finfo(torch.float32).max


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One token of a decode step: the norm in front of the layer, with the
        # attention branch added to the residual stream on the way.
        dict(name="norm_token", op="norm", rows=1, valid=1, hidden=7168, kind="rms", f32=False,
             branch=True, bias=False),
        # A prefill chunk, residual stream in fp32, mean and deviation kept for
        # the backward pass.
        dict(name="norm_prefill", op="norm", rows=16384, valid=16384, hidden=6144, kind="layer",
             f32=True, branch=True, bias=True),
        # A padded buffer of a small layer.
        dict(name="norm_backward_small", op="norm_backward", rows=64, valid=37, hidden=264,
             kind="layer", f32=False, second=False, stream=False, bias=True, grad_f32=True,
             accumulate=False),
        # A training batch: the norm feeds the experts and the gate, so two
        # gradients come back, and the residual stream's own joins them.
        dict(name="norm_backward_train", op="norm_backward", rows=16384, valid=16384,
             hidden=7168, kind="rms", f32=False, second=True, stream=True, bias=False,
             grad_f32=True, accumulate=True),
        # One token over 256 experts in 8 groups, with a balancing bias.
        dict(name="router_token", op="router", rows=1, valid=1, experts=256, topk=8, f32=True,
             score="sigmoid", bias=True, groups=8, topk_groups=4, normalize=True, masked=0.0),
        # The same for a prefill chunk.
        dict(name="router_prefill", op="router", rows=16384, valid=16384, experts=256, topk=8,
             f32=True, score="sigmoid", bias=True, groups=8, topk_groups=4, normalize=True,
             masked=0.0),
        # bf16 logits (equal ones are common), experts that are switched off.
        dict(name="router_bf16_masked", op="router", rows=4096, valid=3001, experts=60, topk=4,
             f32=False, score="softmax", bias=False, groups=1, topk_groups=1, normalize=True,
             masked=0.3),
        dict(name="router_backward_small", op="router_backward", rows=50, valid=41, experts=60,
             topk=4, f32=False, score="sigmoid", normalize=True, masked=0.2),
        # A training batch: every expert's logit gets a gradient.
        dict(name="router_backward_train", op="router_backward", rows=16384, valid=16384,
             experts=256, topk=8, f32=True, score="softmax", normalize=False, masked=0.0),
        # One token's eight experts out of 32: products of one row each.
        dict(name="w4_token", op="w4", live=8, spread=8, experts=32, n=4096, k=7168, align=16,
             fmt="mxfp4", group=32),
        # A decode batch over one rank's share (8 experts), down projection.
        dict(name="w4_decode_int4", op="w4", live=200, spread=8, experts=8, n=7168, k=2048,
             align=128, fmt="int4", group=128),
        # Prefill over one rank's share: the matrix cores decide.
        dict(name="w4_prefill", op="w4", live=8192, spread=8, experts=8, n=4096, k=7168,
             align=128, fmt="mxfp4", group=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "router", "router_backward", "w4", "w4"])
    coin = lambda p=0.5: rng.random() < p  # noqa: E731
    rows = _log(rng, 1, 16384)
    valid = rows if coin(0.6) else rng.randint(1, rows)
    if op == "norm":
        return dict(op=op, rows=rows, valid=valid, hidden=8 * _log(rng, 4, 896),
                    kind=rng.choice(["layer", "rms"]), f32=coin(0.4), branch=coin(), bias=coin())
    if op == "norm_backward":
        return dict(op=op, rows=rows, valid=valid, hidden=8 * _log(rng, 4, 896),
                    kind=rng.choice(["layer", "rms"]), f32=coin(0.3), second=coin(),
                    stream=coin(), bias=coin(), grad_f32=coin(0.6), accumulate=coin())
    if op in ("router", "router_backward"):
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "router" else 1
        experts = groups * max(2, _log(rng, 4, 512) // groups)
        topk_groups = rng.randint(1, groups)
        c = dict(op=op, rows=rows, valid=valid, experts=experts,
                 topk=rng.randint(1, min(10, experts // groups * topk_groups)), f32=coin(),
                 score=rng.choice(["softmax", "sigmoid"]), normalize=coin(0.6),
                 masked=rng.choice([0.0, 0.0, 0.3]))
        if op == "router":
            c.update(bias=coin(), groups=groups, topk_groups=topk_groups)
        return c
    while True:
        fmt = rng.choice(["int4", "mxfp4"])
        experts = _log(rng, 1, 64)
        c = dict(op=op, live=_log(rng, 1, 8192), spread=rng.randint(1, experts), experts=experts,
                 n=128 * _log(rng, 1, 56), k=128 * _log(rng, 1, 56),
                 align=rng.choice([16, 32, 64, 128, 256]), fmt=fmt,
                 group=rng.choice([32, 64, 128]) if fmt == "int4" else 32)
        w = work(c)
        weights = c["n"] * c["k"]
        if (w["flops"] <= 4.8e11 and experts * weights <= 1.0e9
                and min(c["spread"], c["live"]) * weights <= 2.3e8):
            return c


def work(case):
    op = case["op"]
    if op == "norm":
        size = 4 if case["f32"] else 2
        per = size + 2 + (2 + size if case["branch"] else 0)
        return dict(bytes=float(case["valid"]) * case["hidden"] * per
                    + 4.0 * case["hidden"] * (1 + case["bias"]),
                    flops=8.0 * case["valid"] * case["hidden"])
    if op == "norm_backward":
        size = 4 if case["f32"] else 2
        per = 2 + 2 * size + (2 if case["second"] else 0) + (size if case["stream"] else 0)
        grads = (4 if case["grad_f32"] else 2) * (2 if case["accumulate"] else 1)
        return dict(bytes=float(case["valid"]) * case["hidden"] * per
                    + case["hidden"] * (4.0 + grads * (1 + case["bias"])),
                    flops=15.0 * case["valid"] * case["hidden"])
    if op in ("router", "router_backward"):
        size = 4 if case["f32"] else 2
        values = case["valid"] * case["experts"]
        slots = case["valid"] * case["topk"]
        return dict(bytes=float(values) * size * (1 if op == "router" else 2) + 8.0 * slots,
                    flops=6.0 * values)
    n, k = case["n"], case["k"]
    used = min(case["spread"], case["live"])
    scales = k // case["group"] * (2 if case["fmt"] == "int4" else 1)
    return dict(bytes=2.0 * case["live"] * (n + k) + float(used) * n * (k / 2 + scales),
                flops=2.0 * case["live"] * n * k)


# ----------------------------------------------------------------- inputs

def _normal(shape, scale, gen, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)


def _recv(valid):
    """Rows received from each of four source ranks, summed up."""
    return torch.tensor([valid // 4, valid // 2, valid // 2, valid], dtype=torch.int32,
                        device="cuda")


def _prepare_norm(s, c, gen):
    rows, H, nv = c["rows"], c["hidden"], c["valid"]
    dt = torch.float32 if c["f32"] else torch.bfloat16
    # A residual stream whose channels differ in size and are not centred.
    channel = _normal((H,), 0.5, gen, torch.float32).exp_()
    offset = _normal((H,), 0.3, gen, torch.float32)
    s["x"] = (_normal((rows, H), 1.0, gen, torch.float32) * channel + offset).to(dt)
    s["x"][nv:] = float("nan")
    s["weight"] = 1.0 + _normal((H,), 0.1, gen, torch.float32)
    s["bias"] = _normal((H,), 0.1, gen, torch.float32) if c["bias"] else None
    s["psum_recv"] = _recv(nv)
    s["eps"] = 1e-5
    if c["op"] == "norm":
        s["branch"] = s["sum"] = None
        if c["branch"]:
            s["branch"] = _normal((rows, H), 0.3, gen)
            s["branch"][nv:] = float("nan")
            s["sum"] = torch.zeros((rows, H), dtype=dt, device="cuda")
        s["y"] = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
        s["mean"] = torch.zeros(rows, device="cuda") if c["kind"] == "layer" else None
        s["rstd"] = torch.zeros(rows, device="cuda")
        return
    mean = torch.zeros(rows, dtype=torch.float64, device="cuda")
    square = torch.zeros_like(mean)
    for i in range(0, rows, 2048):
        x = s["x"][i:i + 2048].double()
        if c["kind"] == "layer":
            mean[i:i + 2048] = x.mean(dim=1)
            x -= mean[i:i + 2048, None]
        square[i:i + 2048] = x.square_().mean(dim=1)
    s["mean"] = mean.float() if c["kind"] == "layer" else None
    s["rstd"] = (square + s["eps"]).rsqrt().float()
    s["dy"] = _normal((rows, H), 0.01, gen)
    s["dy2"] = _normal((rows, H), 0.002, gen) if c["second"] else None
    s["dsum"] = _normal((rows, H), 0.01, gen, dt) if c["stream"] else None
    for name in ("dy", "dy2", "dsum"):
        if s[name] is not None:
            s[name][nv:] = float("nan")
    s["dx"] = torch.zeros((rows, H), dtype=dt, device="cuda")
    gdt = torch.float32 if c["grad_f32"] else torch.bfloat16
    for name in ("dweight", "dbias"):
        s[name] = _normal((H,), 0.05, gen, gdt)
    if not c["bias"]:
        s["dbias"] = None
    s["workspace"] = None


def _prepare_router(s, c, gen):
    rows, E, T, nv = c["rows"], c["experts"], c["topk"], c["valid"]
    dt = torch.float32 if c["f32"] else torch.bfloat16
    x = _normal((rows, E), 1.5, gen, torch.float32)
    if c["masked"]:
        off = torch.rand((rows, E), generator=gen, device="cuda") < c["masked"]
        off[3::16] = True               # every expert switched off
        off[5::16, 1:] = True           # one left
        x[off] = float("-inf")
        x[7::16, 0] = float("nan")
        x[9::16, E // 2] = torch.finfo(dt).min
        x[11::16, E - 1] = float("inf")
    s["logits"] = x.to(dt)
    s["logits"][nv:] = float("nan")
    s["psum_recv"] = _recv(nv)
    s["topk_ids"] = torch.full((rows, T), -9, dtype=torch.int32, device="cuda")
    s["topk_weights"] = torch.full((rows, T), -9.0, device="cuda")
    if c["op"] == "router":
        s["bias"] = _normal((E,), 0.1, gen, torch.float32) if c["bias"] else None
        return
    x = _clean(s["logits"].double())
    value, ids = torch.sort(x, dim=1, descending=True, stable=True)
    ids = torch.where(value[:, :T] > float("-inf"), ids[:, :T], -1)
    s["topk_ids"][:nv] = ids[:nv].int()
    s["d_topk_weights"] = _normal((rows, T), 0.1, gen, torch.float32)
    s["d_topk_weights"][ids < 0] = float("nan")
    s["d_topk_weights"][nv:] = float("nan")
    s["d_logits"] = torch.zeros((rows, E), dtype=dt, device="cuda")


def _prepare_w4(s, c, gen, seed):
    g = np.random.Generator(np.random.PCG64(seed * 7919 + 41))
    E, n, k, align = c["experts"], c["n"], c["k"], c["align"]
    used = min(c["spread"], c["live"])
    counts = np.zeros(E, np.int64)
    chosen = g.permutation(E)[:used]
    counts[chosen] = 1
    counts[chosen] += g.multinomial(c["live"] - used, np.full(used, 1.0 / used))
    psum, end = [], 0
    for x in counts:
        psum.append(end + int(x))
        end = (psum[-1] + align - 1) // align * align
    blocks = min(c["live"], E)
    cap = align * (blocks + (c["live"] - blocks) // align)
    s["counts"] = [int(x) for x in counts]      # the host's plan of the batch
    s["psum"] = torch.tensor(psum, dtype=torch.int32, device="cuda")
    s["status"] = torch.tensor([end, 0], dtype=torch.int32, device="cuda")
    s["a"] = _normal((cap, k), 1.0, gen)
    first = 0
    for last in psum:
        nxt = (last + align - 1) // align * align
        s["a"][last:nxt] = float("nan")
        first = nxt
    s["a"][first:] = float("nan")
    s["w"] = torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, device="cuda",
                           generator=gen)
    shape = (E, n, k // c["group"])
    if c["fmt"] == "int4":
        s["w_scale"] = (torch.rand(shape, generator=gen, device="cuda") * 0.008
                        + 0.001).to(torch.bfloat16)
    else:
        s["w_scale"] = torch.randint(117, 123, shape, dtype=torch.uint8, device="cuda",
                                     generator=gen)
    s["out"] = torch.zeros((cap, n), dtype=torch.bfloat16, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("norm", "norm_backward"):
        _prepare_norm(s, case, gen)
    elif op in ("router", "router_backward"):
        _prepare_router(s, case, gen)
    else:
        _prepare_w4(s, case, gen, seed)
    return s


# ------------------------------------------------------------ plain forms

def _valid(s, rows):
    return torch.arange(rows, device="cuda") < s["psum_recv"][-1]


def _keep(s, name, value, live):
    """Rows that are live take the new value, rounded to the buffer's type."""
    live = live.view(-1, *([1] * (value.dim() - 1)))
    s[name].copy_(torch.where(live, value.to(s[name].dtype), s[name]))


def _plain_norm(s):
    live = _valid(s, s["x"].shape[0])
    h = s["x"].float()
    if s["branch"] is not None:
        _keep(s, "sum", h + s["branch"].float(), live)
        h = s["sum"].float()            # the stream as it is kept
    mean = 0.0
    if s["mean"] is not None:
        mean = h.mean(dim=1, keepdim=True)
        _keep(s, "mean", mean[:, 0], live)
    d = h - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + s["eps"])
    _keep(s, "rstd", rstd[:, 0], live)
    y = d * rstd * s["weight"]
    _keep(s, "y", y if s["bias"] is None else y + s["bias"], live)
    return _outputs(s, "sum", "y", "mean", "rstd")


def _outputs(s, *names):
    return {n: s[n] for n in names if s[n] is not None}


def _plain_norm_backward(s):
    live = _valid(s, s["x"].shape[0])
    zero = torch.zeros((), device="cuda")
    dy = s["dy"].float()
    if s["dy2"] is not None:
        dy = dy + s["dy2"].float()
    dy = torch.where(live[:, None], dy, zero)
    x = torch.where(live[:, None], s["x"].float(), zero)
    rstd = torch.where(live, s["rstd"], zero)[:, None]
    g = dy * s["weight"]
    if s["mean"] is not None:
        xhat = (x - torch.where(live, s["mean"], zero)[:, None]) * rstd
        d = rstd * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
    else:
        xhat = x * rstd
        d = rstd * (g - xhat * (g * xhat).mean(dim=1, keepdim=True))
    if s["dsum"] is not None:
        d = d + s["dsum"].float()
    _keep(s, "dx", d, live)
    for name, new in (("dweight", (dy * xhat).sum(dim=0)), ("dbias", dy.sum(dim=0))):
        if s[name] is not None:
            s[name].copy_(new + s[name].float() if s["case"]["accumulate"] else new)
    return _outputs(s, "dx", "dweight", "dbias")


def _clean(x):
    """-inf and NaN: an expert that is not available; +inf: the largest value."""
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x)
    return x.clamp(max=F32_MAX)


def _scores(x, score):
    """Scores of cleaned logits; 0 where an expert is not available."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - torch.where(top > float("-inf"), top, torch.zeros_like(top)))
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _choose(x, c, bias):
    """Ids by falling score, the lowest first among equals; -1 where none is left."""
    minus = torch.full_like(x, float("-inf"))
    if bias is None and c["groups"] == 1:
        key = x                         # the scores' order
    else:
        key = _scores(x, c["score"])
        key = torch.where(x > float("-inf"), key if bias is None else key + bias.double(), minus)
    if c["groups"] > 1:
        per = key.view(key.shape[0], c["groups"], -1)
        two = torch.sort(per, dim=2, descending=True).values[:, :, :2]
        of = torch.where(two > float("-inf"), two, torch.zeros_like(two)).sum(dim=2)
        of = torch.where(two[:, :, 0] > float("-inf"), of, torch.full_like(of, float("-inf")))
        order = torch.sort(of, dim=1, descending=True, stable=True).indices
        chosen = torch.zeros_like(of, dtype=torch.bool)
        chosen.scatter_(1, order[:, :c["topk_groups"]], True)
        key = torch.where(chosen[:, :, None], per, minus.view_as(per)).view_as(key)
    value, ids = torch.sort(key, dim=1, descending=True, stable=True)
    T = c["topk"]
    return torch.where(value[:, :T] > float("-inf"), ids[:, :T], -1)


def _weights(x, ids, c):
    """Weights of the chosen experts, 0 in free slots."""
    here = ids >= 0
    if not c["normalize"]:
        w = _scores(x, c["score"]).gather(1, ids.clamp(min=0))
        return torch.where(here, w, torch.zeros_like(w))
    v = x.gather(1, ids.clamp(min=0))
    v = torch.where(here, v, torch.full_like(v, float("-inf")))
    low = v if c["score"] == "softmax" else v.clamp(max=0.0)
    top = low.amax(dim=1, keepdim=True)
    w = torch.exp(low - torch.where(top > float("-inf"), top, torch.zeros_like(top)))
    if c["score"] == "sigmoid":         # sigmoid(v) = exp(min(v, 0)) / (1 + exp(-|v|))
        w = w / (1.0 + torch.exp(-v.abs()))
    w = torch.where(here, w, torch.zeros_like(w))
    total = w.sum(dim=1, keepdim=True)
    return w / torch.where(total > 0, total, torch.ones_like(total))


def _plain_router(s):
    live = _valid(s, s["logits"].shape[0])
    x = _clean(s["logits"].float())
    ids = _choose(x.double(), s["case"], s["bias"])
    _keep(s, "topk_ids", ids, live)
    _keep(s, "topk_weights", _weights(x, ids, s["case"]), live)
    return _outputs(s, "topk_ids", "topk_weights")


def _router_gradient(x, ids, g, c):
    here = ids >= 0
    at = ids.clamp(min=0)
    g = torch.where(here, g, torch.zeros_like(g))
    w = _weights(x, ids, c)
    dot = (w * g).sum(dim=1, keepdim=True)
    d = torch.zeros_like(x)
    if c["score"] == "softmax":
        if c["normalize"]:
            return d.scatter_add_(1, at, w * (g - dot))
        return d.scatter_add_(1, at, w * g) - _scores(x, "softmax") * dot
    off = 1.0 / (1.0 + torch.exp(x.gather(1, at)))      # 1 - sigmoid
    if c["normalize"]:
        g = g - dot
    return d.scatter_add_(1, at, torch.where(here, w * off * g, torch.zeros_like(g)))


def _plain_router_backward(s):
    live = _valid(s, s["logits"].shape[0])
    x = _clean(torch.where(live[:, None], s["logits"].float(), torch.zeros((), device="cuda")))
    ids = torch.where(live[:, None], s["topk_ids"].long(), -1)
    _keep(s, "d_logits", _router_gradient(x, ids, s["d_topk_weights"], s["case"]), live)
    return s["d_logits"]


def _codes(w, fmt, dtype):
    """The values of one expert's 4-bit codes [n, k], the low half of a byte first."""
    q = torch.stack([w & 15, w >> 4], dim=-1).view(w.shape[0], -1).long()
    if fmt == "int4":
        table = torch.tensor([*range(8), *range(-8, 0)], dtype=dtype, device=w.device)
    else:
        table = torch.tensor([*E2M1, *(-v for v in E2M1)], dtype=dtype, device=w.device)
    return table[q]


def _dequantised(s, e, dtype):
    c = s["case"]
    q = _codes(s["w"][e], c["fmt"], dtype).view(c["n"], -1, c["group"])
    scale = s["w_scale"][e]
    scale = scale.to(dtype) if c["fmt"] == "int4" else torch.exp2(scale.to(dtype) - 127.0)
    return (q * scale[:, :, None]).view(c["n"], -1)


def _plain_w4(s):
    first, align = 0, s["case"]["align"]
    for e, live in enumerate(s["counts"]):
        if live:
            w = _dequantised(s, e, torch.float32)
            s["out"][first:first + live] = torch.mm(s["a"][first:first + live].float(),
                                                    w.t()).to(torch.bfloat16)
        first = (first + live + align - 1) // align * align
    return s["out"]


# ------------------------------------------------------- framework's calls

def _own(s):
    import expanded_dispatch_layout_amd as M
    c = s["case"]
    if c["op"] == "norm":
        M.moe_layer_norm(s["x"], s["weight"], s["y"], bias=s["bias"], branch=s["branch"],
                         sum=s["sum"], mean=s["mean"], rstd=s["rstd"], kind=c["kind"],
                         eps=s["eps"], psum_recv_per_rank=s["psum_recv"])
        return _outputs(s, "sum", "y", "mean", "rstd")
    if c["op"] == "norm_backward":
        if s["workspace"] is None:      # kept by the caller, as other workspaces are
            need = M.moe_layer_norm_backward_workspace_bytes(c["rows"], c["hidden"])
            s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        M.moe_layer_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], s["dx"],
                                  mean=s["mean"], dy2=s["dy2"], dsum=s["dsum"],
                                  dweight=s["dweight"], dbias=s["dbias"],
                                  accumulate=c["accumulate"], kind=c["kind"],
                                  psum_recv_per_rank=s["psum_recv"], workspace=s["workspace"])
        return _outputs(s, "dx", "dweight", "dbias")
    if c["op"] == "router":
        M.moe_router(s["logits"], s["topk_ids"], s["topk_weights"], bias=s["bias"],
                     score=c["score"], num_groups=c["groups"], topk_groups=c["topk_groups"],
                     normalize=c["normalize"], psum_recv_per_rank=s["psum_recv"])
        return _outputs(s, "topk_ids", "topk_weights")
    if c["op"] == "router_backward":
        M.moe_router_backward(s["logits"], s["topk_ids"], s["d_topk_weights"], s["d_logits"],
                              score=c["score"], normalize=c["normalize"],
                              psum_recv_per_rank=s["psum_recv"])
        return s["d_logits"]
    M.moe_grouped_gemm_w4(s["a"], s["w"], s["w_scale"], c["fmt"], s["psum"], s["status"],
                          c["align"], s["out"])
    return s["out"]


_PLAIN = dict(norm=_plain_norm, norm_backward=_plain_norm_backward, router=_plain_router,
              router_backward=_plain_router_backward, w4=_plain_w4)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------- 64-bit values

def _exact_norm(s):
    c, nv = s["case"], s["case"]["valid"]
    out = {n: s[n].double() for n in ("sum", "y", "mean", "rstd") if s[n] is not None}
    for i in range(0, nv, 2048):
        at = slice(i, min(i + 2048, nv))
        h = s["x"][at].double()
        if c["branch"]:
            h += s["branch"][at].double()
            out["sum"][at] = h
            h = h.to(s["sum"].dtype).double()   # the norm is of the stream as it is kept
        if c["kind"] == "layer":
            out["mean"][at] = h.mean(dim=1)
            h = h - out["mean"][at, None]
        out["rstd"][at] = (h.pow(2).mean(dim=1) + s["eps"]).pow(-0.5)
        y = h * out["rstd"][at, None] * s["weight"].double()
        out["y"][at] = y + s["bias"].double() if c["bias"] else y
    return out


def _exact_norm_backward(s):
    c, nv, H = s["case"], s["case"]["valid"], s["case"]["hidden"]
    dx = s["dx"].double()
    dw = torch.zeros(H, dtype=torch.float64, device="cuda")
    db = torch.zeros_like(dw)
    for i in range(0, nv, 2048):
        at = slice(i, min(i + 2048, nv))
        dy, xhat, r = s["dy"][at].double(), s["x"][at].double(), s["rstd"][at].double()
        if c["second"]:
            dy += s["dy2"][at].double()
        if c["kind"] == "layer":
            xhat -= s["mean"][at].double()[:, None]
        xhat *= r[:, None]
        db += dy.sum(dim=0)
        dw += (dy * xhat).sum(dim=0)
        dy *= s["weight"].double()
        along = torch.bmm(dy[:, None], xhat[:, :, None]).view(-1, 1) / H
        d = dy - xhat * along
        if c["kind"] == "layer":
            d -= dy.sum(dim=1, keepdim=True) / H
        d *= r[:, None]
        dx[at] = d + s["dsum"][at].double() if c["stream"] else d
    out = dict(dx=dx)
    for name, new in (("dweight", dw), ("dbias", db)):
        if s[name] is not None:
            out[name] = new + s[name].double() if c["accumulate"] else new
    return out


def _log_scores(x, score):
    """Logarithm of the scores of cleaned 64-bit logits."""
    if score == "sigmoid":
        return -torch.nn.functional.softplus(-x)
    return x - torch.logsumexp(x, dim=1, keepdim=True)


def _exact_weights(x, ids, c):
    """x 64-bit; rows without any chosen expert are zeros."""
    log_w = _log_scores(x, c["score"]).gather(1, ids.clamp(min=0))
    log_w = log_w.masked_fill(ids < 0, float("-inf"))
    if c["normalize"]:
        log_w = log_w - torch.logsumexp(log_w, dim=1, keepdim=True)
    return torch.where(ids < 0, torch.zeros_like(log_w), log_w.exp())


def _exact_router(s):
    c, nv = s["case"], s["case"]["valid"]
    x = _clean(s["logits"][:nv].double())
    key = x
    if s["bias"] is not None or c["groups"] > 1:
        key = torch.nan_to_num(_log_scores(x, c["score"]).exp(), nan=0.0)
        if s["bias"] is not None:
            key = key + s["bias"].double()
        key[x == float("-inf")] = float("-inf")
    if c["groups"] > 1:
        key = key.view(nv, c["groups"], -1)
        first, at = key.max(dim=2)
        rest = key.scatter(2, at[:, :, None], float("-inf")).amax(dim=2)
        total = first + torch.where(rest == float("-inf"), torch.zeros_like(rest), rest)
        rank = torch.argsort(total, dim=1, descending=True, stable=True).argsort(dim=1)
        key = key.masked_fill((rank >= c["topk_groups"])[:, :, None], float("-inf")).view(nv, -1)
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :c["topk"]]
    ids = ids.masked_fill(key.gather(1, ids) == float("-inf"), -1)
    out_ids, out_w = s["topk_ids"].clone(), s["topk_weights"].double()
    out_ids[:nv] = ids.int()
    out_w[:nv] = _exact_weights(x, ids, c)
    return dict(topk_ids=out_ids, topk_weights=out_w)


def _exact_router_backward(s):
    c, nv = s["case"], s["case"]["valid"]
    x, ids = _clean(s["logits"][:nv].double()), s["topk_ids"][:nv].long()
    g = s["d_topk_weights"][:nv].double().masked_fill(ids < 0, 0.0)
    w = _exact_weights(x, ids, c)
    out = s["d_logits"].double()
    dense = lambda v: torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), v)  # noqa: E731
    if c["score"] == "softmax":
        p = torch.nan_to_num(_log_scores(x, "softmax").exp(), nan=0.0)
        if c["normalize"]:
            p = dense(w)
        out[:nv] = dense(w * g) - p * (w * g).sum(dim=1, keepdim=True)
        return out
    if c["normalize"]:
        g = g - (w * g).sum(dim=1, keepdim=True)
    out[:nv] = dense(w * g * torch.sigmoid(-x.gather(1, ids.clamp(min=0)))
                     .masked_fill(ids < 0, 0.0))
    return out


def _exact_w4(s):
    c, out, first = s["case"], s["out"].double(), 0
    for e, live in enumerate(s["counts"]):
        if live:
            w = torch.empty((c["n"], c["k"]), dtype=torch.float64, device="cuda")
            for half, code in ((0, s["w"][e] % 16), (1, s["w"][e] // 16)):
                code = code.double()
                if c["fmt"] == "int4":
                    value = code - 16.0 * (code >= 8)
                else:
                    m = code % 8
                    power, odd = torch.floor(m / 2), m % 2
                    value = torch.where(power > 0, torch.exp2(power - 1) * (1 + odd / 2), odd / 2)
                    value = torch.where(code >= 8, -value, value)
                w[:, half::2] = value
            scale = s["w_scale"][e].double()
            if c["fmt"] == "mxfp4":
                scale = torch.exp2(scale - 127)
            w *= scale.repeat_interleave(c["group"], dim=1)
            out[first:first + live] = s["a"][first:first + live].double() @ w.t().contiguous()
        first = -(-(first + live) // c["align"]) * c["align"]
    return out


def exact(case, seed):
    return dict(norm=_exact_norm, norm_backward=_exact_norm_backward, router=_exact_router,
                router_backward=_exact_router_backward, w4=_exact_w4)[case["op"]](
                    prepare(case, seed))
