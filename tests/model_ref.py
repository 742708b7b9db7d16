"""Plain binary64 forms of the sequence-side operators (norm + rotation,
quantised cache, attention, sampling) in numpy, for the tests: nothing here
is shared with the library."""
import math

import numpy as np


def rms_rope(x, weight, offset, eps, table, positions, interleaved):
    """x [T, heads, D] float64; weight [D] or None; table [P, rot/2, 2]."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * (weight + offset)
    if table is None:
        return y
    half = table.shape[1]
    c, s = (table[positions][:, None, :, i].astype(np.float64) for i in (0, 1))
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if interleaved else (y[..., :half], y[..., half:2 * half])
    out = y.copy()
    ra, rb = a * c - b * s, b * c + a * s
    if interleaved:
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = ra, rb
    else:
        out[..., :half], out[..., half:2 * half] = ra, rb
    return out


def held(x, bits):
    """What the cache holds of x [..., D] (values representable in fp32): blocks of 32, fp16 scales."""
    top, low = (127, -127) if bits == 8 else (7, -8)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32).astype(np.float32)
    amax = np.abs(b).max(-1)
    with np.errstate(all="ignore"):
        d = (amax / np.float32(top)).astype(np.float16).astype(np.float32)
        d = np.where(amax <= 65024, d, np.nan)[..., None]
        q = np.where(d > 0, np.clip(np.rint(b / d), low, top), 0.0)
        q = np.where(np.isnan(q), 0.0, q)
    return (q.astype(np.float64) * d).reshape(x.shape)


def attend(q, k, v, scale, n_new):
    """q [n, hq, D] the last n of the L positions of k, v [L, hkv, D]: out [n, hq, D], lse [n, hq]."""
    n, hq, _ = q.shape
    L, hkv, D = k.shape
    g = hq // hkv
    out, lse = np.zeros((n, hq, D)), np.full((n, hq), -np.inf)
    for i in range(n):
        seen = L - n_new + i + 1
        if seen <= 0:
            continue
        for h in range(hq):
            z = k[:seen, h // g] @ q[i, h] * scale
            m = z.max()
            p = np.exp(z - m)
            out[i, h] = p @ v[:seen, h // g] / p.sum()
            lse[i, h] = m + math.log(p.sum())
    return out, lse


def sample(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability, kept indices) of one row of float64 logits."""
    z = np.where(np.isnan(z), -np.inf, z)
    if not (z > -np.inf).any():
        return -1, 0.0, []
    order = np.argsort(-z, kind="stable")
    if not temperature > 0 or top_k == 1 or top_p <= 0 or min_p > 1:
        return int(order[0]), 1.0, [int(order[0])]
    m = z[order[0]]
    with np.errstate(invalid="ignore"):
        w = np.where(z == m, 1.0, 0.0) if np.isinf(m) else np.exp((z - m) / temperature)
    if 1 < top_k < len(z):
        order = order[:top_k]
    ws = w[order]
    if top_p < 1:
        before = np.concatenate(([0.0], np.cumsum(ws)[:-1]))
        order = order[:max(1, int((before < top_p * ws.sum()).sum()))]
    if min_p > 0:
        order = order[w[order] >= min_p]
    kept = np.sort(order)
    cum = np.cumsum(w[kept])
    u = 0.0 if not u > 0 else min(u, 0.99999994)
    at = min(int(np.searchsorted(cum, u * cum[-1], side="right")), len(kept) - 1)
    while w[kept[at]] == 0:
        at -= 1
    return int(kept[at]), float(w[kept[at]] / cum[-1]), [int(i) for i in kept]
