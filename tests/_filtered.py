"""Plain 64-bit statements of MXFP4 and of filtered sampling, for the tests (numpy, host)."""
import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_quantize(x):
    """(codes uint8 [rows][kp / 2], scales uint8 [rows][kp / 32]) of float64 rows."""
    rows, d = x.shape
    kp = (d + 127) // 128 * 128
    p = np.zeros((rows, kp))
    p[:, :d] = x
    codes = np.zeros((rows, kp), dtype=np.uint8)
    scales = np.zeros((rows, kp // 32), dtype=np.uint8)
    for b in range((d + 31) // 32):
        y = p[:, 32 * b:32 * b + 32]
        bad = ~np.isfinite(y).all(axis=1)
        y = np.where(bad[:, None], 0.0, y)
        top = np.abs(y).max(axis=1)
        _, e = np.frexp(top)
        e = np.where(top > 0, np.maximum(e - 3, -127), -127)
        a = np.minimum(np.abs(y) / np.exp2(e.astype(float))[:, None], 6.0)
        dist = np.abs(a[:, :, None] - GRID)
        near = dist == dist.min(axis=2, keepdims=True)
        # of two equally near magnitudes the even code
        code = np.where(near.sum(axis=2) == 1, near.argmax(axis=2),
                        (near & (np.arange(8) % 2 == 0)).argmax(axis=2))
        code = code + 8 * np.signbit(y)
        codes[:, 32 * b:32 * b + 32] = np.where(bad[:, None], 0, code)
        scales[:, b] = np.where(bad, 255, e + 127)
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8), scales


def mx_values(codes, scales, d):
    rows = codes.shape[0]
    c = np.stack([codes & 15, codes >> 4], axis=2).reshape(rows, -1)
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(float) - 127.0))
    return (v * np.repeat(s, 32, axis=1))[:, :d]


def filtered(z, t=1.0, k=0, p=1.0, m=0.0):
    """Weights in id order (0: not kept) and size of the kept set of one float64 row."""
    z = np.where(np.isnan(z), -np.inf, z)
    w = np.zeros(z.shape)
    if z.max() == -np.inf:
        return w, 0
    ids = np.flatnonzero(z > -np.inf)
    ids = ids[np.lexsort((ids, -z[ids]))]
    if t == 0:
        w[ids[0]] = 1.0
        return w, 1
    if 0 < k < len(ids):
        ids = ids[:k]
    top = z[ids[0]]
    with np.errstate(invalid="ignore"):
        wt = np.where(z[ids] == top, 1.0, np.exp((z[ids] - top) / t))
    n = len(ids)
    if p < 1:
        n = min(n, int(np.searchsorted(np.cumsum(wt), p * np.sum(wt), side="left")) + 1)
    if m > 0:
        n = min(n, int(np.count_nonzero(wt >= min(m, 1.0))))
    n = max(n, 1)
    w[ids[:n]] = wt[:n]
    return w, n


def draw(w, u):
    """Smallest id with weight whose running weight passes u times the total; -1 without any."""
    ids = np.flatnonzero(w > 0)
    if len(ids) == 0:
        return -1
    c = np.cumsum(w[ids])
    return int(ids[min(int(np.searchsorted(c, u * c[-1], side="right")), len(ids) - 1)])


def near_border(w, u, tol):
    """Whether u times the total lies within tol of the total from a step of the running sum."""
    c = np.cumsum(w[w > 0])
    return bool(len(c)) and bool(np.min(np.abs(c[:-1] - u * c[-1]), initial=np.inf) <= tol * c[-1])


def accept(z, zq, tokens, lens, offsets, u_accept, u_resample, settings):
    """accept_len, next_token of sd_accept_filtered; settings[r] = (t, k, p, m)."""
    B, g = tokens.shape
    out_a, out_t = [], []
    for r in range(B):
        a, L, base = None, lens[r], offsets[r]
        for j in range(L):
            wp, _ = filtered(z[base + j], *settings[r])
            wq, _ = filtered(zq[r, j], *settings[r])
            x = tokens[r, j]
            ok = False
            if 0 <= x < z.shape[1] and wp[x] > 0:
                ratio = (wp[x] / wp.sum()) / (wq[x] / wq.sum()) if wq[x] > 0 else math.inf
                ok = u_accept[r, j] < min(1.0, ratio)
            if not ok:
                a = j
                break
        if a is None:
            a = L
        wp, _ = filtered(z[base + a], *settings[r])
        w = wp
        if a < L and wp.sum() > 0:
            wq, _ = filtered(zq[r, a], *settings[r])
            q = wq / wq.sum() if wq.sum() > 0 else wq
            w = np.maximum(wp / wp.sum() - q, 0.0)
            if w.sum() == 0:
                w = wp
        out_a.append(a)
        out_t.append(draw(w, float(u_resample[r, a])))
    return np.array(out_a, dtype=np.int32), np.array(out_t, dtype=np.int32)
