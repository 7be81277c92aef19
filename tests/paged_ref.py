"""Plain 64-bit definitions of the paged-cache operators, for the tests: E4M3 rounding,
the page-scaled FP8 store, the page plan and attention over decoded rows."""

import math

import numpy as np


def e4m3_value(codes):
    """E4M3 bytes -> float64 (0x7F and 0xFF are NaN)."""
    c = np.asarray(codes, dtype=np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def e4m3_code(x):
    """float64 -> nearest E4M3 byte (ties to the even code), saturating, sign kept."""
    mags = e4m3_value(np.arange(127))
    mids = (mags[1:] + mags[:-1]) / 2
    a = np.abs(x)
    lo = np.searchsorted(mids, a, side="left")  # codes whose upper midpoint is >= a
    tie = (lo < 126) & (mids[np.minimum(lo, 125)] == a) & (lo % 2 == 1)
    return ((lo + tie) | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def pow2_scale(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    while amax > 448 * s:
        s *= 2
    return s


def page_store(codes, scale, x, slots, bs):
    """In place: rows x [T, H, D] into codes [slots, H, D] u8, scale [blocks, H] f32."""
    T, H, _ = x.shape
    t = 0
    while t < T:
        if slots[t] < 0 or slots[t] >= codes.shape[0]:
            t += 1
            continue
        pg, n = slots[t] // bs, 1
        while t + n < T and slots[t + n] >= 0 and slots[t + n] // bs == pg:
            n += 1
        mine = slots[t:t + n]
        for h in range(H):
            s0 = float(scale[pg, h])
            if (mine % bs == 0).any() or not (s0 > 0 and math.isfinite(s0)):
                s0 = 0.0
            s = max(s0, pow2_scale(np.abs(x[t:t + n, h]).max()))
            rows = codes[pg * bs:(pg + 1) * bs, h]
            if s > s0 > 0:
                nan = (rows & 127) == 127
                rows[:] = np.where(nan, rows, e4m3_code(np.nan_to_num(e4m3_value(rows)) * (s0 / s)))
            rows[mine % bs] = e4m3_code(x[t:t + n, h] / s)
            scale[pg, h] = s
        t += n


def plan(cached, new, free, bs, table, max_tokens):
    """(table, seq_lens, starts, slots, positions, used, status) of a page plan."""
    table = table.copy()
    lens, starts, at, first, used, status = [], [0], 0, 0, 0, 0
    slots, pos = np.full(max_tokens, -1, np.int64), np.full(max_tokens, -1, np.int32)
    for s, (c, n) in enumerate(zip(map(int, cached), map(int, new))):
        bad = c < 0 or n < 0 or c + n > table.shape[1] * bs
        rows = max(n, 0)
        ok = not bad and at + n <= max_tokens
        need = -(-(c + n) // bs) - -(-c // bs) if ok else 0
        fits = need == 0 or first + need <= len(free)
        status |= 8 if bad else 0 if ok and fits else 32
        if ok and fits:
            held = -(-c // bs)
            for j in range(need):
                table[s, held + j] = free[first + j]
            for i in range(n):
                blk = table[s, (c + i) // bs]
                slots[at + i] = int(blk) * bs + (c + i) % bs if blk >= 0 else -1
                status |= 2 if blk < 0 else 0
                pos[at + i] = c + i
            if need:
                used = first + need
        lens.append(c + n if ok and fits else -1)
        first += need
        at += rows
        starts.append(min(at, max_tokens))
    return table, np.array(lens, np.int32), np.array(starts, np.int32), slots, pos, used, status


def attention(q, K, V, lens, starts, scale, softcap=0.0, slopes=None, window=0, prefix=None, key_starts=None):
    """q [T, Hq, D], K / V per sequence [len, H, D], all float64 -> (out, largest |logit| a row sees)."""
    out = np.full(q.shape, np.nan)
    top = np.zeros(q.shape[:2])
    for s in range(len(lens)):
        n, L = starts[s + 1] - starts[s], lens[s]
        g = q.shape[1] // K[s].shape[1]
        t = np.arange(L)
        for i in range(n):
            r, p = starts[s] + i, L - n + i
            hi = max(p + 1, min(prefix[s], L) if prefix is not None else 0)
            lo = max(0, p + 1 - window if window else 0, key_starts[r] if key_starts is not None else 0)
            for qh in range(q.shape[1]):
                if lo >= hi:
                    out[r, qh] = 0
                    continue
                x = K[s][lo:hi, qh // g] @ q[r, qh] * scale
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                if slopes is not None:
                    x = x + slopes[qh] * (t[lo:hi] - p)
                top[r, qh] = np.abs(x).max()
                w = np.exp(x - x.max())
                out[r, qh] = w @ V[s][lo:hi, qh // g] / w.sum()
    return out, top
