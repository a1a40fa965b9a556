"""What stands around the experts in a block: the norm, the router, and 4-bit
expert weights (oracle; test infrastructure only).  The mathematics in float64,
without roundings between steps; products also return the sum of the terms'
sizes, which bounds what a sum in fewer bits may be off by.
"""

import numpy as np

F64 = np.float64
F32_MAX = np.finfo(np.float32).max
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def layer_norm(h, weight, bias, eps, rms):
    """(y, mean, rstd) of rows h."""
    h = h.astype(F64)
    mean = np.zeros(len(h)) if rms else h.mean(axis=1)
    d = h - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None] * weight.astype(F64)
    return (y if bias is None else y + bias.astype(F64)), mean, rstd


def layer_norm_backward(dy, h, weight, mean, rstd, rms):
    """(dx, dweight, dbias) with the forward call's mean and rstd."""
    dy, h = dy.astype(F64), h.astype(F64)
    xh = (h - (0 if rms else mean.astype(F64)[:, None])) * rstd.astype(F64)[:, None]
    g = dy * weight.astype(F64)
    dx = g - xh * (g * xh).mean(axis=1, keepdims=True)
    if not rms:
        dx -= g.mean(axis=1, keepdims=True)
    return dx * rstd.astype(F64)[:, None], (dy * xh).sum(axis=0), dy.sum(axis=0)


def clean(x):
    """Logits: NaN and -inf are experts that are not available (-inf)."""
    x = np.minimum(x.astype(F64), F32_MAX)
    return np.where(np.isnan(x), -np.inf, x)


def _log_share(v):
    """v - log sum exp(v) along the last axis; -inf where nothing is there.  The
    largest v is taken off first: beside 1e38 the logarithm would be lost."""
    top = v.max(axis=-1, keepdims=True)
    d = v - np.where(np.isfinite(top), top, 0)
    total = np.exp(d).sum(axis=-1, keepdims=True)
    return d - np.log(np.where(total > 0, total, 1))


def log_scores(x, score):
    if score == "sigmoid":
        return np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))
    return _log_share(x)


def router(logits, topk, bias=None, score="softmax", groups=1, topk_groups=1, normalize=True):
    """(ids [rows, topk], weights): row by row, expert by expert."""
    x = clean(logits)
    keys = x
    if bias is not None or groups > 1:
        keys = np.exp(log_scores(x, score))
        if bias is not None:
            b = np.minimum(bias.astype(F64), F32_MAX)
            keys = keys + np.where(np.isnan(b), -np.inf, b)
        keys = np.where(np.isneginf(x), -np.inf, keys)
    ids = np.full((len(x), topk), -1, np.int64)
    per = x.shape[1] // groups
    for r, key in enumerate(keys):
        free = [e for e in range(len(key)) if key[e] > -np.inf]
        if groups > 1:
            best = []
            for g in range(groups):
                mine = sorted((key[e] for e in free if e // per == g), reverse=True)
                if mine:
                    best.append((-sum(mine[:2]), g))
            keep = {g for _, g in sorted(best)[:topk_groups]}
            free = [e for e in free if e // per in keep]
        chosen = sorted(free, key=lambda e: (-key[e], e))[:topk]
        ids[r, :len(chosen)] = chosen
    return ids, router_weights(logits, ids, score, normalize)


def router_weights(logits, ids, score, normalize):
    x = clean(logits)
    lw = np.take_along_axis(log_scores(x, score), np.maximum(ids, 0), axis=1)
    lw = np.where(ids >= 0, lw, -np.inf)
    return np.exp(_log_share(lw) if normalize else lw)


def router_backward(logits, ids, dw, score, normalize):
    """d logits: slot by slot."""
    x = clean(logits)
    w = router_weights(logits, ids, score, normalize)
    s = np.exp(log_scores(x, score))
    d = np.zeros_like(x)
    for r in range(len(x)):
        slots = [k for k in range(ids.shape[1]) if ids[r, k] >= 0]
        dot = sum(w[r, k] * F64(dw[r, k]) for k in slots)
        for k in slots:
            e, g = ids[r, k], F64(dw[r, k])
            if normalize:
                g = g - dot
            with np.errstate(over="ignore"):
                d[r, e] += w[r, k] * g * (1 / (1 + np.exp(x[r, e])) if score == "sigmoid" else 1)
        if score == "softmax" and not normalize:
            d[r] -= s[r] * dot
    return d


def w4_values(w, scale, fmt):
    """The weights [..., k] that codes [..., k/2] and scales [..., k/group] stand
    for.  scale: bf16 values as floats (int4) or UE8M0 bytes (mxfp4)."""
    q = np.stack([w & 15, w >> 4], axis=-1).reshape(*w.shape[:-1], -1).astype(np.int64)
    if fmt == "int4":
        v = np.where(q < 8, q, q - 16).astype(F64)
        s = scale.astype(F64)
    else:
        v = np.where(q < 8, 1, -1) * E2M1[q & 7]
        s = np.exp2(scale.astype(F64) - 127)
    return v * np.repeat(s, v.shape[-1] // s.shape[-1], axis=-1)


def grouped(a, w, lab):
    """out[m] = a[m] @ w[lab[m]]^T for lab >= 0, and sum |a w|."""
    out = np.zeros((len(a), w.shape[1]))
    mag = np.zeros_like(out)
    for e in np.unique(lab[lab >= 0]):
        r = lab == e
        out[r] = a[r].astype(F64) @ w[e].T
        mag[r] = np.abs(a[r].astype(F64)) @ np.abs(w[e]).T
    return out, mag
