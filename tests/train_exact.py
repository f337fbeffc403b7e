"""Plain 64-bit forms of the operators of training, for their tests (not a test module)."""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])


def balance(logits, ids, mask, offsets):
    """logits [T][E] float64, ids [T][k], mask [T] bool, offsets [S+1] -> dict with the gradient's parts."""
    T, E = logits.shape
    k, S = ids.shape[1], len(offsets) - 1
    top = logits.max(1, keepdims=True) if T else np.zeros((0, 1))
    alive = np.isfinite(top[:, 0])
    ex = np.exp(logits - np.where(alive[:, None], top, 0.0))
    p = ex / np.where(alive, ex.sum(1), 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(alive, np.where(alive, top[:, 0], 0.0) + np.log(ex.sum(1)), -np.inf)
    counts, mean = np.zeros((S, E), np.int64), np.zeros((S, E))
    n, seg = np.zeros(S, np.int64), np.full(T, -1)
    for s in range(S):
        at = [t for t in range(offsets[s], offsets[s + 1]) if mask[t] and alive[t]]
        seg[at] = s
        n[s] = len(at)
        for t in at:
            for i in ids[t]:
                if 0 <= i < E:
                    counts[s, i] += 1
        if at:
            mean[s] = p[at].mean(0)
    held, total = int((n > 0).sum()), int(n.sum())
    bal = sum(E / (k * n[s]) * (counts[s] * mean[s]).sum() for s in range(S) if n[s]) / max(held, 1)
    z = (lse[seg >= 0] ** 2).sum() / max(total, 1)
    lse = np.where(seg >= 0, lse, -np.inf)
    return dict(losses=np.array([bal, z]), counts=counts, prob_mean=mean, tokens=np.concatenate([n, [total, held]]),
                lse=lse, p=p, seg=seg, n=n, held=held, total=total)


def route_gradient(logits, ids, gates, dgates, d, dlosses):
    """(the gradient, the sum of its terms' magnitudes)"""
    T, E = logits.shape
    k = ids.shape[1]
    g, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s = d["seg"][t]
        if dlosses is not None and s >= 0:
            p, c = d["p"][t], d["counts"][s] / d["n"][s]
            kb, kz = dlosses[0] * E / (k * d["held"] * d["n"][s]), dlosses[1] * 2 / d["total"] * d["lse"][t]
            g[t] += kb * p * (c - (p * c).sum()) + kz * p
            size[t] += abs(kb) * p * (c + (p * c).sum()) + abs(kz) * p
        if dgates is not None:
            for j in range(k):
                if 0 <= ids[t, j] < E:
                    g[t, ids[t, j]] += gates[t, j] * (dgates[t, j] - (gates[t] * dgates[t]).sum())
                    size[t, ids[t, j]] += gates[t, j] * (abs(dgates[t, j]) + abs(gates[t] * dgates[t]).sum())
    return g, size


def nearest(grid, v):
    """Indices of the grid values nearest to v >= 0, ties to the even index, at most the last."""
    hi = np.clip(np.searchsorted(grid, v, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    below, above = v - grid[lo], grid[hi] - v
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def tensor_scale(x):
    amax = np.abs(x).max()
    if amax == 0:
        return 1.0
    g = 2.0 ** -126
    while g * 2688 < amax:
        g *= 2
    return g


def quantise(x, fmt, g=1.0, rnd=None):
    """x [rows][cols] float64 -> (codes [rows][cols], scale bytes [rows][cols/B], x / d)."""
    B = 16 if fmt == "nvfp4" else 32
    b = x.reshape(x.shape[0], -1, B)
    amax = np.abs(b).max(2)
    if fmt == "nvfp4":
        byte = nearest(E4M3, amax / (6 * g))
        d = E4M3[byte] * g
        byte, d = np.where(d >= 2.0 ** -126, byte, 0), np.where(d >= 2.0 ** -126, d, 0.0)
    else:
        e = np.frexp(amax)[1] - 1
        byte = np.where(amax >= 2.0 ** -126, np.clip(e - 2 + 127, 0, 254), 0)
        d = np.ldexp(1.0, byte - 127)
    v = np.where(d[..., None] > 0, np.abs(b) / np.where(d > 0, d, 1.0)[..., None], 0.0)
    if rnd is None:
        mag = nearest(E2M1, v)
    else:
        lo = np.clip(np.searchsorted(E2M1, v, side="right") - 1, 0, 7)
        hi = np.minimum(lo + 1, 7)
        part = np.where(hi > lo, (v - E2M1[lo]) / np.where(hi > lo, E2M1[hi] - E2M1[lo], 1.0), 0.0)
        mag = np.where(part > (rnd.reshape(b.shape) + 0.5) / 256, hi, lo)
    codes = mag + 8 * np.signbit(b)
    return codes.reshape(x.shape), byte, v.reshape(x.shape)


def pack(codes):
    return (codes[:, ::2] | codes[:, 1::2] << 4).astype(np.uint8)


def unpack(q):
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)


def values(q, scale, fmt, g=1.0):
    """Packed codes and scale bytes -> float64 values."""
    c = unpack(q).astype(np.int64)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = E4M3[np.minimum(scale, 126)] if fmt == "nvfp4" else np.ldexp(1.0, scale.astype(np.int64) - 127)
    return v * np.repeat(s, 16 if fmt == "nvfp4" else 32, axis=1) * g


def transposed(x):
    """x^T with its rows filled up to a multiple of 128 by zeros."""
    out = np.zeros((x.shape[1], -(-x.shape[0] // 128) * 128), x.dtype)
    out[:, :x.shape[0]] = x.T
    return out
