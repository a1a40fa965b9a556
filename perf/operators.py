"""Measured cases of the expert training operators: the gradients of the
grouped bf16 products (input and weight), of SiLU*up and of the combine, and
the AdamW step over many tensors.

`own` false: the plain forms, in elementary torch operations in fp32.  `own`
true: the framework's calls.  Both take the state that prepare() makes, and
write the state's own output buffers (rows and weights outside the result
keep what was there).

Expanded rows are laid out as the layout makes them: expert e owns rows
[align(psum[e-1]), align(psum[e])), its live rows end at psum[e], and
status[0] is the padded total.  Padding rows and rows past the total hold NaN:
no gradient may depend on them.
"""

import math

import numpy as np
import torch

own = False

GROUP = 128          # elements that share a scale of an 8-bit state
FP8_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
CODE_MIN = 2.0 ** -9  # smallest positive e4m3 value


# ------------------------------------------------------------------ cases

def listed():
    return [
        # A few rows over a tiny layer: what a call costs by itself.
        dict(name="dgrad_tiny", op="dgrad", live=32, experts=4, n=256, k=256, align=64,
             skew=False),
        # The down projection's input gradient of one rank's share (8 of 256
        # experts, about 128 rows each): the weights' stream decides.
        dict(name="dgrad_share", op="dgrad", live=1024, experts=8, n=4096, k=7168, align=128,
             skew=False),
        # Prefill-sized batch, uneven experts: the matrix cores decide.
        dict(name="dgrad_prefill", op="dgrad", live=18432, experts=8, n=6144, k=2048, align=128,
             skew=True),
        dict(name="wgrad_tiny", op="wgrad", live=37, experts=4, n=256, k=192, align=16,
             skew=False, f32=False, accumulate=False),
        # Micro-batch gradient accumulation in fp32 for one rank's share: the
        # gradients' read and write decide.
        dict(name="wgrad_share_accumulate", op="wgrad", live=1024, experts=8, n=4096, k=7168,
             align=128, skew=False, f32=True, accumulate=True),
        dict(name="wgrad_prefill", op="wgrad", live=18432, experts=8, n=4096, k=6144, align=128,
             skew=False, f32=False, accumulate=False),
        dict(name="silu_backward_small", op="silu", live=77, experts=8, inter=128, align=16),
        dict(name="silu_backward_prefill", op="silu", live=18432, experts=8, inter=2048,
             align=128),
        # A padded receive buffer: rows past the boundary are not touched.
        dict(name="gather_backward_small", op="gather", rows=64, valid=50, experts=4,
             hidden=256, topk=2, align=16, local=0.5, factor=1.0),
        # Every expert on this GPU: each token has topk rows.
        dict(name="gather_backward_standard", op="gather", rows=4096, valid=4096, experts=256,
             hidden=7168, topk=8, align=128, local=1.0, factor=2.5),
        # Norm gains, biases and a router beside each other: odd, small tensors.
        dict(name="adamw_small_f32", op="adamw", sizes="256,65536,33,7168,1000,1", state="f32",
             grad_f32=False, copy=True),
        # Both expert weights of one rank's share, a router and two odd tensors.
        dict(name="adamw_share_fp8", op="adamw",
             sizes="234881024,117440512,1835008,7168,255", state="fp8", grad_f32=False,
             copy=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dgrad", "wgrad", "silu", "gather", "adamw"])
    align = rng.choice([16, 32, 64, 128, 256])
    if op in ("dgrad", "wgrad"):
        while True:
            c = dict(op=op, live=_log(rng, 1, 20000), experts=_log(rng, 1, 32),
                     n=128 * _log(rng, 1, 56), k=64 * _log(rng, 1, 112), align=align,
                     skew=rng.random() < 0.4)
            if op == "wgrad":
                c.update(f32=rng.random() < 0.5, accumulate=rng.random() < 0.4)
            w = work(c)
            if w["flops"] <= 9.0e11 and w["bytes"] <= 2.0e9:
                return c
    if op == "silu":
        return dict(op=op, live=_log(rng, 1, 18432), experts=_log(rng, 1, 64),
                    inter=64 * _log(rng, 1, 32), align=align)
    if op == "gather":
        rows = _log(rng, 1, 4096)
        return dict(op=op, rows=rows, valid=rows if rng.random() < 0.5 else rng.randint(1, rows),
                    experts=_log(rng, 1, 256), hidden=128 * _log(rng, 1, 56),
                    topk=rng.randint(1, 8), align=align, local=rng.choice([0.1, 0.5, 1.0]),
                    factor=rng.choice([1.0, 2.5]))
    sizes = [_log(rng, 1, 30_000_000) for _ in range(rng.randint(1, 9))]
    return dict(op=op, sizes=",".join(map(str, sizes)), state=rng.choice(["f32", "fp8"]),
                grad_f32=rng.random() < 0.4, copy=rng.random() < 0.7)


def work(case):
    op = case["op"]
    if op in ("dgrad", "wgrad"):
        live, E, n, k = case["live"], case["experts"], case["n"], case["k"]
        flops = 2.0 * live * n * k
        if op == "dgrad":
            return dict(bytes=2.0 * (live * (n + k) + min(E, live) * n * k), flops=flops)
        size = (4 if case["f32"] else 2) * (2 if case["accumulate"] else 1)
        return dict(bytes=2.0 * live * (n + k) + float(E) * n * k * size, flops=flops)
    if op == "silu":
        return dict(bytes=10.0 * case["live"] * case["inter"],
                    flops=12.0 * case["live"] * case["inter"])
    if op == "gather":
        slots = case["valid"] * case["topk"] * case["local"]
        return dict(bytes=2.0 * case["hidden"] * (case["valid"] + 2 * slots)
                    + 12.0 * case["valid"] * case["topk"],
                    flops=3.0 * slots * case["hidden"])
    per = (4 if case["grad_f32"] else 2) + 8 + (2 if case["copy"] else 0)
    per += 16 if case["state"] == "f32" else 4 + 16 / GROUP
    total = sum(map(int, case["sizes"].split(",")))
    return dict(bytes=float(per) * total, flops=20.0 * total)


# ----------------------------------------------------------------- inputs

def _counts(case, seed):
    """Rows per expert, `live` in all."""
    g = np.random.Generator(np.random.PCG64(seed * 7919 + 17))
    E = case["experts"]
    p = np.full(E, 1.0 / E)
    if case.get("skew") and E > 1:
        # Zipf(1.2) over the experts in a random order, an eighth of them idle.
        p = np.arange(1, E + 1, dtype=np.float64) ** -1.2
        p[E - E // 8:] = 0.0
        p = g.permutation(p / p.sum())
    return g.multinomial(case["live"], p / p.sum())


def _capacity(slots, E, align):
    n = min(slots, E)
    return align * (n + (slots - n) // align) if slots else align


def _layout(counts, align, capacity):
    """psum, status and m_indices of expert blocks padded to `align` rows."""
    psum, labels, end = [], np.full(capacity, -1, np.int32), 0
    for e, c in enumerate(counts):
        psum.append(end + int(c))
        nxt = (psum[-1] + align - 1) // align * align
        labels[end:nxt] = e
        end = nxt
    dev = "cuda"
    return (torch.tensor(psum, dtype=torch.int32, device=dev),
            torch.tensor([end, 0], dtype=torch.int32, device=dev),
            torch.from_numpy(labels).to(dev))


def _live_rows(s):
    """Truth value of each expanded row: does it hold a token's row."""
    label = s["m_indices"].long()
    row = torch.arange(label.numel(), device=label.device)
    return (label >= 0) & (row < s["psum"].long()[label.clamp(min=0)]) & (row < s["status"][0])


def _normal(shape, scale, gen, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    bf = torch.bfloat16
    s = dict(case=case)
    if op in ("dgrad", "wgrad", "silu"):
        counts = _counts(case, seed)
        E, align = case["experts"], case["align"]
        cap = _capacity(case["live"], E, align)
        s["psum"], s["status"], s["m_indices"] = _layout(counts, align, cap)
        s["most"] = int(counts.max())   # the longest expert: a plan's size, known to the host
        dead = ~_live_rows(s)
    if op in ("dgrad", "wgrad"):
        n, k = case["n"], case["k"]
        s["dy"] = _normal((cap, n), 0.01, gen)
        s["dy"][dead] = float("nan")
        if op == "dgrad":
            s["w"] = _normal((E, n, k), 0.02, gen)
            s["dx"] = torch.zeros((cap, k), dtype=bf, device="cuda")
        else:
            s["x"] = _normal((cap, k), 1.0, gen)
            s["x"][dead] = float("nan")
            dt = torch.float32 if case["f32"] else bf
            s["dw"] = (_normal((E, n, k), 0.05, gen, dt) if case["accumulate"]
                       else torch.zeros((E, n, k), dtype=dt, device="cuda"))
            s["workspace"] = None
    elif op == "silu":
        I = case["inter"]
        s["gate_up"] = _normal((cap, 2 * I), 1.7, gen)
        s["dy"] = _normal((cap, I), 0.01, gen)
        s["gate_up"][dead] = float("nan")
        s["dy"][dead] = float("nan")
        s["d_gate_up"] = torch.zeros((cap, 2 * I), dtype=bf, device="cuda")
    elif op == "gather":
        rows, nv, E, T, H = (case[x] for x in ("rows", "valid", "experts", "topk", "hidden"))
        g = np.random.Generator(np.random.PCG64(seed * 7919 + 29))
        ids = g.integers(0, E, size=(rows, T))
        away = g.random((rows, T)) >= case["local"]
        away[0, 0] = False              # one row at least came here
        ids[away] = -1
        ids[nv:] = -1
        flat = ids.reshape(-1)
        counts = np.bincount(flat[flat >= 0], minlength=E)
        cap = _capacity(rows * T, E, case["align"])
        s["psum"], s["status"], s["m_indices"] = _layout(counts, case["align"], cap)
        start = np.concatenate([[0], (np.cumsum(-(-counts // case["align"])) * case["align"])])
        order = np.argsort(flat, kind="stable")
        order = order[flat[order] >= 0]
        rank = np.arange(len(order)) - np.concatenate([[0], np.cumsum(counts)])[flat[order]]
        dst = np.full(rows * T, -1, np.int32)
        dst[order] = start[flat[order]] + rank
        s["src2dst"] = torch.from_numpy(dst.reshape(rows, T)).cuda()
        # How many rows arrived from each of four source ranks, summed up.
        s["psum_recv"] = torch.tensor([nv // 4, nv // 2, nv // 2, nv], dtype=torch.int32,
                                      device="cuda")
        s["topk_weights"] = torch.rand((rows, T), generator=gen, device="cuda") + 0.01
        s["dout"] = _normal((rows, H), 0.01, gen)
        s["dout"][nv:] = float("nan")
        s["expert_out"] = _normal((cap, H), 1.0, gen)
        s["expert_out"][~_live_rows(s)] = float("nan")
        s["d_expert_out"] = torch.zeros((cap, H), dtype=bf, device="cuda")
        s["d_topk_weights"] = torch.zeros((rows, T), dtype=torch.float32, device="cuda")
    else:
        s["tensors"] = []
        for size in map(int, case["sizes"].split(",")):
            t = dict(master=_normal(size, 0.02, gen, torch.float32),
                     grad=_normal(size, 1e-3, gen, torch.float32 if case["grad_f32"] else bf))
            t["param"] = t["master"].to(bf) if case["copy"] else None
            m = _normal(size, 3e-4, gen, torch.float32)
            v = _normal(size, 1e-3, gen, torch.float32).square_()
            if case["state"] == "f32":
                t.update(m=m, v=v, m_scale=None, v_scale=None)
            else:
                t["m"], t["m_scale"] = _code(m, False)
                t["v"], t["v_scale"] = _code(v.sqrt_(), True)
            s["tensors"].append(t)
        s["step"] = torch.tensor([100 + seed % 50], dtype=torch.int64, device="cuda")
        s["lr"] = torch.tensor([3e-4], dtype=torch.float32, device="cuda")
        s["grad_scale"] = torch.tensor([0.5], dtype=torch.float32, device="cuda")
        s["hyper"] = dict(beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    return s


# ------------------------------------------------------------ plain forms

def _groups(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % GROUP)).view(-1, GROUP)


def _code(x, positive):
    """(e4m3 codes, fp32 scale of each group of 128): scale = amax / 448."""
    g = _groups(x)
    amax = g.abs().amax(dim=1, keepdim=True).clamp_(min=AMAX_FLOOR)
    q = g * (FP8_MAX / amax)
    if positive:  # a positive second moment never becomes zero
        q = torch.where(g > 0, q.clamp(min=CODE_MIN), q)
    q = q.to(torch.float8_e4m3fn).view(-1)[:x.numel()]
    return q, (amax / FP8_MAX).view(-1)


def _decode(codes, scale):
    return (_groups(codes.float()) * scale[:, None]).view(-1)[:codes.numel()]


def _by_expert(s, rows):
    """Each expert's live rows in fp32, [E, longest, columns], zeros behind
    them; and each expanded row's place in that."""
    align, psum = s["case"]["align"], s["psum"].long()
    ends = (psum + align - 1) // align * align
    start = torch.cat([torch.zeros_like(ends[:1]), ends[:-1]])
    pos = start[:, None] + torch.arange(s["most"], device=psum.device)
    live = pos < psum[:, None]
    got = rows[pos.clamp(max=rows.shape[0] - 1)].float()
    place = torch.arange(rows.shape[0], device=psum.device) - start[
        s["m_indices"].long().clamp(min=0)]
    place = place + s["m_indices"].long().clamp(min=0) * s["most"]
    return torch.where(live[..., None], got, got.new_zeros(())), place


def _plain_dgrad(s):
    a, place = _by_expert(s, s["dy"])
    d = torch.bmm(a, s["w"].float()).view(-1, s["dx"].shape[1])
    d = d[place.clamp(max=d.shape[0] - 1)].to(torch.bfloat16)
    s["dx"].copy_(torch.where(_live_rows(s)[:, None], d, s["dx"]))
    return s["dx"]


def _plain_wgrad(s):
    a, _ = _by_expert(s, s["dy"])
    b, _ = _by_expert(s, s["x"])
    d = torch.bmm(a.transpose(1, 2), b)
    s["dw"].copy_(s["dw"].float() + d if s["case"]["accumulate"] else d)
    return s["dw"]


def _plain_silu(s):
    gate, up = s["gate_up"].float().chunk(2, dim=1)
    dy = s["dy"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    d = torch.cat([dy * up * (sig * (1.0 + gate * (1.0 - sig))), dy * (gate * sig)], dim=1)
    s["d_gate_up"].copy_(torch.where(_live_rows(s)[:, None], d.to(torch.bfloat16),
                                     s["d_gate_up"]))
    return s["d_gate_up"]


def _plain_gather(s):
    dst, w, f = s["src2dst"].long(), s["topk_weights"], s["case"]["factor"]
    (rows, T), cap = dst.shape, s["d_expert_out"].shape[0]
    valid = (torch.arange(rows, device=dst.device) < s["psum_recv"][-1])[:, None]
    live = valid & (dst >= 0)
    dout = s["dout"].float()
    dots = (s["expert_out"][dst.clamp(min=0)].float() * dout[:, None]).sum(-1) * f
    dw = torch.where(live, dots, torch.zeros_like(dots))
    s["d_topk_weights"].copy_(torch.where(valid, dw, s["d_topk_weights"]))
    slot = torch.full((cap + 1,), -1, dtype=torch.int64, device=dst.device)
    slot.scatter_(0, torch.where(live, dst, cap).view(-1),
                  torch.arange(rows * T, device=dst.device))
    slot = slot[:cap]
    at = slot.clamp(min=0)
    d = (dout[at // T] * (f * w.view(-1)[at])[:, None]).to(torch.bfloat16)
    s["d_expert_out"].copy_(torch.where(slot[:, None] >= 0, d, s["d_expert_out"]))
    return dict(d_expert_out=s["d_expert_out"], d_topk_weights=s["d_topk_weights"])


def _plain_adamw(s):
    h, t = s["hyper"], s["step"].double()
    b1, b2 = h["beta1"], h["beta2"]
    c1, c2 = (1.0 - b1 ** t).float(), (1.0 - b2 ** t).float()
    for p in s["tensors"]:
        coded = p["m_scale"] is not None
        m = _decode(p["m"], p["m_scale"]) if coded else p["m"]
        r = _decode(p["v"], p["v_scale"]) if coded else None
        v = r * r if coded else p["v"]
        g = p["grad"].float() * s["grad_scale"]
        m = m * b1 + g * (1.0 - b1)
        v = v * b2 + (g * g) * (1.0 - b2)
        step = (m / c1) / (torch.sqrt(v / c2) + h["eps"]) + p["master"] * h["weight_decay"]
        p["master"].copy_(p["master"] - step * s["lr"])
        if p["param"] is not None:
            p["param"].copy_(p["master"])
        for name, x in (("m", m), ("v", torch.sqrt(v) if coded else v)):
            if coded:
                q, scale = _code(x, name == "v")
                p[name].view(torch.uint8).copy_(q.view(torch.uint8))
                p[name + "_scale"].copy_(scale)
            else:
                p[name].copy_(x)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return [{k: v for k, v in p.items() if k != "grad" and v is not None} for p in s["tensors"]]


# ------------------------------------------------------- framework's calls

def _own(s):
    import expanded_dispatch_layout_amd as M
    c = s["case"]
    if c["op"] == "dgrad":
        M.moe_grouped_dgrad_bf16(s["dy"], s["w"], s["psum"], s["status"], c["align"], s["dx"])
        return s["dx"]
    if c["op"] == "wgrad":
        if s["workspace"] is None:  # kept by the caller, as the layout's workspace is
            need = M.moe_grouped_wgrad_workspace_bytes(s["dy"].shape[0], c["n"], c["k"],
                                                       c["experts"])
            s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        M.moe_grouped_wgrad_bf16(s["dy"], s["x"], s["psum"], s["status"], c["align"], s["dw"],
                                 s["workspace"], accumulate=c["accumulate"])
        return s["dw"]
    if c["op"] == "silu":
        M.moe_silu_mul_bf16_backward(s["gate_up"], s["dy"], s["m_indices"], s["psum"],
                                     s["status"], c["experts"], c["align"], s["d_gate_up"])
        return s["d_gate_up"]
    if c["op"] == "gather":
        M.moe_gather_backward(s["dout"], s["expert_out"], s["src2dst"], s["topk_weights"],
                              s["psum_recv"], s["d_expert_out"], s["d_topk_weights"],
                              routed_scaling_factor=c["factor"])
        return dict(d_expert_out=s["d_expert_out"], d_topk_weights=s["d_topk_weights"])
    if "list" not in s:  # a training program makes its list of tensors once
        s["list"] = M.AdamWTensors([(p["master"], p["grad"], p["m"], p["v"], p["param"],
                                     p["m_scale"], p["v_scale"]) for p in s["tensors"]])
    M.moe_adamw(s["list"], s["step"], s["lr"], grad_scale=s["grad_scale"], **s["hyper"])
    return _adamw_outputs(s)


_PLAIN = dict(dgrad=_plain_dgrad, wgrad=_plain_wgrad, silu=_plain_silu, gather=_plain_gather,
              adamw=_plain_adamw)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------- 64-bit values

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("dgrad", "wgrad"):
        out = (s["dx"] if op == "dgrad" else s["dw"]).double()
        first = 0
        for e, last in enumerate(s["psum"].tolist()):
            dy = s["dy"][first:last].double()
            if op == "dgrad":
                out[first:last] = dy @ s["w"][e].double()
            else:
                d = dy.t().contiguous() @ s["x"][first:last].double()
                out[e] = out[e] + d if case["accumulate"] else d
            first = -(-last // case["align"]) * case["align"]
        return out
    if op == "silu":
        out = s["d_gate_up"].double()
        I, first = case["inter"], 0
        for last in s["psum"].tolist():
            g, u = (x.double() for x in s["gate_up"][first:last].split(I, dim=1))
            dy, sig = s["dy"][first:last].double(), torch.sigmoid(g)
            out[first:last, :I] = dy * u * (sig + g * sig * (1 - sig))
            out[first:last, I:] = dy * g * sig
            first = -(-last // case["align"]) * case["align"]
        return out
    if op == "gather":
        d_out, dw = s["d_expert_out"].double(), s["d_topk_weights"].double()
        nv, f = case["valid"], case["factor"]
        for k in range(case["topk"]):
            rows = torch.nonzero(s["src2dst"][:nv, k] >= 0).view(-1)
            dst = s["src2dst"][rows, k].long()
            dout = s["dout"][rows].double()
            d_out[dst] = dout * (f * s["topk_weights"][rows, k].double())[:, None]
            dw[rows, k] = f * (dout * s["expert_out"][dst].double()).sum(-1)
        return dict(d_expert_out=d_out, d_topk_weights=dw)
    h, t, outs = s["hyper"], s["step"].item(), []
    lr, gs = s["lr"].double().item(), s["grad_scale"].double().item()
    for p in s["tensors"]:
        per = lambda name: p[name + "_scale"].double().repeat_interleave(GROUP)[:p["m"].numel()]  # noqa: E731
        coded = p["m_scale"] is not None
        m, v = p["m"].double(), p["v"].double()
        if coded:
            m, v = m * per("m"), (v * per("v")) ** 2
        g = p["grad"].double() * gs
        m = h["beta1"] * m + (1 - h["beta1"]) * g
        v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
        up = (m / (1 - h["beta1"] ** t)) / ((v / (1 - h["beta2"] ** t)) ** 0.5 + h["eps"])
        master = p["master"].double() * (1 - lr * h["weight_decay"]) - lr * up
        o = dict(master=master)
        if p["param"] is not None:
            o["param"] = master
        if coded:
            for name, x in (("m", m), ("v", v ** 0.5)):
                n = x.numel()
                top = torch.nn.functional.pad(x.abs(), (0, -n % GROUP)).view(-1, GROUP)
                top = top.max(dim=1).values.clamp(min=AMAX_FLOOR)
                o[name + "_scale"] = top / FP8_MAX
                # A code is a rounded value; what it stands for is the state
                # itself in units of its group's scale.
                o[name] = x / (top / FP8_MAX).repeat_interleave(GROUP)[:n]
        else:
            o.update(m=m, v=v)
        outs.append(o)
    return outs
