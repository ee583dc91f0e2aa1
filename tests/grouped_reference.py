"""Float64 references of the rotary calls and of grouped and differential attention, and the bound that
each output is held to.

A rounding to bf16 is off by at most 2^-8 of the value, one to float32 by 2^-24.

Rotary: x cos a - y sin a.  The angle comes as a float32 fraction of a half turn below 1 (2^-25) of a
product cut to 2^-32 turns: off by at most pi 2^-25 + 2 pi 2^-32 radians; sincospi by 2^-22; the three
float32 operations by 3 2^-24 of |x| + |y|: all below 2^-20 (|x| + |y|), then one rounding to bf16.

Attention: a score's float32 dot product of D bf16 products (exact) is off by at most D 2^-23 of the sum
of their magnitudes (the tensor cores may cut instead of rounding), its scaling, the subtraction of the
maximum and exp2 by a few float32 roundings of numbers no larger than |s| + |max|: together d_j.  A
probability goes to the product as its rounding to bf16 and the rounding of what that left: 2^-16.
Sums over n tokens in float32, in any order: n 2^-23.  So with weights w_j = softmax(s)_j, each off by
(2^-16 + 2 d + n 2^-23) of itself,
    |out - ref| <= (2^-16 + 2 d + 2 n 2^-23) sum_j w_j |v_j| + 2^-8 |ref|,   |lse - ref| <= d + n 2^-23 + 2^-22 |ref|.
The difference of two maps adds their bounds; the norm divides by the root mean square, itself off by at
most the root mean square of the bound."""
import math

import numpy as np

HALF_BF16, EPS32 = 2.0 ** -8, 2.0 ** -24


def rotate(x, pos, freq, axes, neighbours):
    """x [T, heads, dim] float64, pos [A, T], freq [R / 2], axes [R / 2] -> (rotated, bound)."""
    R = 2 * len(freq)
    a = np.asarray(pos, np.float64)[np.asarray(axes)].T * np.asarray(freq)[None, :]
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    u, v = (x[..., 0:R:2], x[..., 1:R:2]) if neighbours else (x[..., :R // 2], x[..., R // 2:R])
    out, tol = x.copy(), np.zeros_like(x)
    w = 2.0 ** -20 * (np.abs(u) + np.abs(v))
    if neighbours:
        out[..., 0:R:2], out[..., 1:R:2] = u * c - v * s, v * c + u * s
        tol[..., 0:R:2] = tol[..., 1:R:2] = w
    else:
        out[..., :R // 2], out[..., R // 2:R] = u * c - v * s, v * c + u * s
        tol[..., :R // 2] = tol[..., R // 2:R] = w
    tol[..., :R] += HALF_BF16 * np.abs(out[..., :R])
    return out, tol


def attend(q, k, v, scale, lo, hi):
    """One row: q [G, D] over tokens lo .. hi - 1 of k [n, D], v [n, Dv] -> (out, bound, lse, bound)."""
    G, D, Dv = q.shape[0], q.shape[1], v.shape[1]
    if hi <= lo:
        return np.zeros((G, Dv)), np.zeros((G, Dv)), np.full(G, -math.inf), np.zeros(G)
    k, v, n = k[lo:hi], v[lo:hi], hi - lo
    s = q @ k.T * scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(1, keepdims=True)
    w = p / total
    out, lse = w @ v, (m + np.log(total))[:, 0]
    d = (D * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(k).T) + 4 * EPS32 * (np.abs(s) + np.abs(m)) + 2.0 ** -22).max(1)
    sums = n * 2.0 ** -23
    tol = (HALF_BF16 ** 2 + 2 * d + 2 * sums)[:, None] * (w @ np.abs(v)) + HALF_BF16 * np.abs(out)
    return out, tol, lse, d + sums + 2.0 ** -22 * np.abs(lse)


def attention(q, k, v, scale, ind, row_len, table, P, window=0, lam=None, gain=None, eps=1e-5):
    """q [T, H, maps, D], k [N, Hkv, maps, D], v [N, Hkv, Dv] float64; table [B, pages] sub-page ids.
    Returns (out, bound, lse [T, H, maps], bound); rows behind the last request are NaN."""
    T, H, maps, D = q.shape
    Hkv, Dv = k.shape[1], v.shape[2]
    G = H // Hkv
    out, tol = np.full((T, H, Dv), np.nan), np.zeros((T, H, Dv))
    lse, ltol = np.full((T, H, maps), np.nan), np.zeros((T, H, maps))
    for b in range(len(ind) - 1):
        for r in range(ind[b], ind[b + 1]):
            n = int(row_len[r])
            lo = max(0, n - window) if window else 0
            j = np.arange(max(n, 0))
            at = np.asarray(table)[b][j // P].astype(np.int64) * P + j % P
            for g in range(Hkv):
                h = slice(g * G, (g + 1) * G)
                o = [attend(q[r, h, m], k[at, g, m], v[at, g], scale, lo, n) for m in range(maps)]
                for m in range(maps):
                    lse[r, h, m], ltol[r, h, m] = o[m][2], o[m][3]
                if maps == 1:
                    out[r, h], tol[r, h] = o[0][0], o[0][1]
                    continue
                L = np.asarray(lam, np.float64)[h][:, None]
                y = o[0][0] - L * o[1][0]
                e = o[0][1] + np.abs(L) * o[1][1] - HALF_BF16 * (np.abs(o[0][0]) + np.abs(L) * np.abs(o[1][0]))
                if gain is not None:   # (y + e) / (rms + rms(e)), to first order
                    rms = np.sqrt((y ** 2).mean(1, keepdims=True) + eps)
                    rel = np.sqrt((e ** 2).mean(1, keepdims=True)) / rms
                    y, e = y / rms * gain, (e / rms + rel * np.abs(y) / rms + 4 * EPS32) * np.abs(gain) * (1 + 2 * rel)
                out[r, h], tol[r, h] = y, e + HALF_BF16 * np.abs(y)
    return out, tol, lse, ltol
