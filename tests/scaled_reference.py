"""Plain float64 / integer references of the paged 8-bit cache's operators, on the host, and the
bounds their results are held to.  Nothing here comes from the package."""
import numpy as np

import oracle

CODE_VALUE = oracle.e4m3_table()            # value of every e4m3 code
_MAG = CODE_VALUE[:127]                     # non-negative finite values, ascending with the code


def local_index(g, W, I):
    return (g // I) % W, (g // (I * W)) * I + g % I


def local_len(n, W, rank, I):
    return sum(1 for g in range(n) if local_index(g, W, I)[0] == rank) if n < 4096 else \
        (n // (I * W)) * I + min(max(n % (I * W) - rank * I, 0), I)


def update_tables(prev, seq, ind, table, ring, state, bs, T, W=1, rank=0, I=1):
    """(table, ring, state, slots) after the call; sequential, block by block."""
    table, ring = table.copy(), ring.copy()
    C, (head, count) = len(ring), state
    old_ring = ring.copy()
    held = [-(-local_len(int(n), W, rank, I) // bs) for n in prev]
    need = [-(-local_len(int(n), W, rank, I) // bs) for n in seq]
    dealt = back = 0
    for b in range(len(seq)):
        for e in range(held[b], need[b]):
            table[b, e] = old_ring[(head + dealt) % C] if dealt < count else -1
            dealt += 1
        for e in range(need[b], held[b]):
            ring[(head + count + back) % C] = table[b, e]
            back += 1
    took = min(dealt, count)
    slots = np.full(T, -1, np.int32)
    for b in range(len(seq)):
        q0, q1 = int(ind[b]), int(ind[b + 1])
        for r in range(q0, q1):
            owner, j = local_index(int(seq[b]) - q1 + r, W, I)
            if owner == rank and table[b, j // bs] >= 0:
                slots[r] = table[b, j // bs] * bs + j % bs
    return table, ring, ((head + took) % C, count - took + back), slots


def encode(x):
    """Nearest e4m3 code of every value (ties to the even code), saturating; NaN -> 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_MAG, np.nan_to_num(a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = np.nan_to_num(a) - _MAG[lo], _MAG[hi] - np.nan_to_num(a)
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code) | (np.signbit(x) & ~np.isnan(x)) * 128
    return code.astype(np.uint8)


def write_scaled(x, slots, codes, scales, G):
    """The write, unit by unit.  x [T, 576].  x / scale and code * (old / scale) are float32 values, as
    mla_write_kv's are, before they are rounded to e4m3: exact for the powers of two that the write
    chooses; for another writer's scale the quotient can round onto a code's midpoint (0.010253906 /
    2.1 = 0.004882812722 becomes 0.0048828125 = 2.5 steps of 2^-9)."""
    f32 = np.float32
    codes, scales = codes.copy(), scales.astype(np.float64).copy()
    units = {}
    for r, s in enumerate(slots):
        if s >= 0:
            units.setdefault(s // G, []).append((s, r))
    for block, rows in units.items():
        f = min(s for s, _ in rows) % G
        new = np.abs(np.stack([x[r] for _, r in rows]))
        top = new[np.isfinite(new)].max(initial=0.0)
        k = -100
        while top > 448.0 * 2.0 ** k:
            k += 1
        want = 2.0 ** k
        old = scales[block]
        scale = max(old, want) if f else want
        if f and scale > old:
            before = slice(block * G, block * G + f)
            codes[before] = encode(f32(CODE_VALUE[codes[before]]) * (f32(old) / f32(scale)))
        for s, r in rows:
            codes[s] = encode(f32(x[r]) / f32(scale))
        scales[block] = scale
    return codes, scales


def attention(q, codes, scales, G, ind, row_len, sub, P, sm):
    """(out, lse, mass, far) in float64: mass[t, h, d] = sum_j softmax_j |v_jd|; far[t, h, d] = the largest
    softmax_j a_j of the row times sum_j |code_jd|.  row_len [T], sub [B, width]."""
    T, H, _ = q.shape
    out = np.zeros((T, H, 512))
    mass = np.zeros((T, H, 512))
    far = np.zeros((T, H, 512))
    lse = np.full((T, H), -np.inf)
    for b in range(len(ind) - 1):
        for t in range(int(ind[b]), int(ind[b + 1])):
            n = int(row_len[t])
            if n <= 0:
                continue
            j = np.arange(n)
            at = sub[b, j // P].astype(np.int64) * P + j % P
            a = np.maximum(scales[at // G].astype(np.float64), 2.0 ** -100)
            k = CODE_VALUE[codes[at]] * a[:, None]
            s = q[t] @ k.T * sm
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(1, keepdims=True)
            out[t] = p @ k[:, :512] / total
            mass[t] = p @ np.abs(k[:, :512]) / total
            far[t] = (p * a / total).max(1)[:, None] * np.abs(CODE_VALUE[codes[at]][:, :512]).sum(0)[None]
            lse[t] = (m + np.log(total))[:, 0]
    return out, lse, mass, far


def out_bound(out, mass, far):
    """What an output may be off: each probability is held to 2^-7 of itself (two terms of three
    significant bits), a split part and the result are rounded to bf16 (2^-8 each, a part's size
    being at most its mass), and 2^-12 of the mass covers the float32 scores and sums.  A weight
    softmax_j a_j far below the row's largest is held to an absolute step instead: e5m2 ends at
    2^-16, half of which is 2^-28 of the reference weight 2^11, and that is at most the largest one."""
    return (2.0 ** -7 + 2.0 ** -8 + 2.0 ** -12) * mass + 2.0 ** -8 * np.abs(out) + 2.0 ** -28 * far + 1e-37
