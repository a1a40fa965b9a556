"""Gradients of the bf16 expert path and the AdamW step (oracle; test
infrastructure only).

The forward functions are those of ``layer``'s bf16 path: D = y w2^T,
y = silu(g) * u, [g u] = x w13^T per expert, out[r] = f * sum_k c[r,k] *
D[dst(r,k)].  The gradients here are those of the mathematics, in float64
and without the roundings between the stages; the AdamW step with coded
states repeats its fp32 operations one by one, since its codes are decided
by them.
"""

import numpy as np

from . import fp8

F32 = np.float32


def live_rows(psum, align, rows):
    """Label of each live row below `rows`, -1 elsewhere."""
    lab = np.full(rows, -1, np.int64)
    start = 0
    for e, end in enumerate(np.asarray(psum, np.int64)):
        lab[start:min(int(end), rows)] = e
        start = -(-int(end) // align) * align
    return lab


def dgrad(dy, w, lab):
    """dx[m] = dy[m] @ w[lab[m]]; 0 where lab < 0.  Also sum |dy w|."""
    dx = np.zeros((dy.shape[0], w.shape[2]))
    mag = np.zeros_like(dx)
    for e in np.unique(lab[lab >= 0]):
        r = lab == e
        dx[r] = dy[r].astype(np.float64) @ w[e].astype(np.float64)
        mag[r] = np.abs(dy[r]).astype(np.float64) @ np.abs(w[e]).astype(np.float64)
    return dx, mag


def wgrad(dy, x, lab, E):
    """dw[e] = dy[rows of e]^T @ x[rows of e], and sum |dy x|."""
    dw = np.zeros((E, dy.shape[1], x.shape[1]))
    mag = np.zeros_like(dw)
    for e in range(E):
        r = lab == e
        a, b = dy[r].astype(np.float64), x[r].astype(np.float64)
        dw[e], mag[e] = a.T @ b, np.abs(a).T @ np.abs(b)
    return dw, mag


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, e) / (1.0 + e)


def silu_mul_backward(g, u, dy):
    g, u, dy = (np.asarray(a, np.float64) for a in (g, u, dy))
    s = sigmoid(g)
    return dy * u * (s + g * s * sigmoid(-g)), dy * g * s


def gather_backward(dout, expert_out, src2dst, w, f, num_valid, capacity):
    """(rows written {dst: gradient row}, d_topk_weights of the valid rows)."""
    d_rows = {}
    dc = np.zeros((num_valid, src2dst.shape[1]))
    for r in range(num_valid):
        for k, d in enumerate(src2dst[r]):
            if 0 <= d < capacity:
                c = 1.0 if w is None else float(w[r, k])
                d_rows[int(d)] = f * c * dout[r].astype(np.float64)
                dc[r, k] = f * (dout[r].astype(np.float64) @ expert_out[d].astype(np.float64))
    return d_rows, dc


def layer(x, ids, w, w13, w2, f, num_valid):
    """The layer in float64 with no rounding: out [rows, H]."""
    out = np.zeros(x.shape)
    inter = w2.shape[2]
    for r in range(num_valid):
        for k, e in enumerate(ids[r]):
            if 0 <= e < len(w13):
                gu = w13[e] @ x[r]
                g, u = gu[:inter], gu[inter:]
                out[r] += f * w[r, k] * (w2[e] @ (g * sigmoid(g) * u))
    return out


def layer_backward(x, ids, w, w13, w2, f, num_valid, dout):
    """Gradients of <out, dout> of `layer`: dx, dw, dw13, dw2."""
    dx, dw = np.zeros(x.shape), np.zeros(w.shape)
    dw13, dw2 = np.zeros(w13.shape), np.zeros(w2.shape)
    inter = w2.shape[2]
    for r in range(num_valid):
        for k, e in enumerate(ids[r]):
            if not 0 <= e < len(w13):
                continue
            gu = w13[e] @ x[r]
            g, u = gu[:inter], gu[inter:]
            y = g * sigmoid(g) * u
            dd = f * w[r, k] * dout[r]
            dw[r, k] = f * (dout[r] @ (w2[e] @ y))
            dw2[e] += np.outer(dd, y)
            dgu = np.concatenate(silu_mul_backward(g, u, w2[e].T @ dd))
            dw13[e] += np.outer(dgu, x[r])
            dx[r] += w13[e].T @ dgu
    return dx, dw, dw13, dw2


def dither_bits(m, r, t):
    """(20 bits for m's codes, 20 bits for r's) of each element at step t."""
    u = lambda a: np.ascontiguousarray(a, F32).view(np.uint32)  # noqa: E731
    c = np.uint32
    step = np.array([t], np.int64).astype(np.uint32)
    h = (u(m) ^ (u(r) << c(11) | u(r) >> c(21))) * c(0x9e3779b9) + step * c(0xbb67ae85)
    h = (h ^ h >> c(16)) * c(0x9e3779b9)
    h = (h ^ h >> c(15)) * c(0x6a09e667)
    h = h ^ h >> c(16)
    return h >> c(12), h & c(0xfffff)


def to_neighbour(q, bits):
    """fp32 q to one of its two neighbouring e4m3 values, by 20 bits each."""
    a = np.abs(q)
    low = a < F32(2.0 ** -6)
    t = np.where(low, a + F32(2.0 ** -6), a).astype(F32)
    t = ((t.view(np.uint32) + bits) & np.uint32(0xfff00000)).view(F32)
    t = np.where(low, t - F32(2.0 ** -6), t)
    return np.where(a <= F32(448), np.copysign(t, q), q).astype(F32)


def encode_state(x, positive, bits=None):
    """Codes and scales of fp32 values x, in the order of the fp32 operations:
    scale = amax * fl(1/448), code = rne(x * (fl(1/amax) * 448)), or one of the
    neighbouring codes by `bits`."""
    n = x.size
    g = np.zeros(-(-n // 128) * 128, F32)
    g[:n] = x
    g = g.reshape(-1, 128)
    amax = np.maximum(np.abs(g).max(axis=1), F32(2.0 ** -100)).astype(F32)
    inv = (F32(1.0) / amax * F32(448.0)).astype(F32)
    q = g * inv[:, None]
    if positive:
        q = np.where(g > 0, np.maximum(q, F32(2.0 ** -9)), q)
    q = q.astype(F32).reshape(-1)[:n]
    codes = fp8.encode_e4m3(q if bits is None else to_neighbour(q, bits))
    return codes, (amax * (F32(1.0) / F32(448.0))).astype(F32)


def decode_state(codes, scale):
    return (fp8.decode_e4m3(codes).astype(F32) * np.repeat(scale, 128)[:codes.size]).astype(F32)


def adamw_f32(p, grad, m, v, t, lr, b1, b2, eps, wd, gs):
    """One step, each fp32 operation rounded in order."""
    b1f, ob1, b2f, ob2 = F32(b1), F32(1.0 - b1), F32(b2), F32(1.0 - b2)
    c1, c2 = F32(1.0 - b1 ** t), F32(1.0 - b2 ** t)
    g = (grad.astype(F32) * F32(gs)).astype(F32)
    m = m * b1f + g * ob1
    v = v * b2f + (g * g) * ob2
    up = (m / c1) / (np.sqrt(v / c2) + F32(eps)) + p * F32(wd)
    return (p - up * F32(lr)).astype(F32), m.astype(F32), v.astype(F32)
