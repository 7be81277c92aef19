"""Plain definitions of the sparse step's operators, for the tests: the append (binary32 where
the definition rounds to it), the block selection and attention over listed blocks in 64 bits."""

import math

import numpy as np
import torch

import paged_ref as R

PAGE, ROW8, NVFP4 = 5, 3, 1
F = np.float32
E2M1_MIDS = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])


def angles(positions, rot, base=10000.0):
    """[positions, rot] float32: cosines, then sines."""
    a = np.arange(positions, dtype=np.float64)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return torch.tensor(np.concatenate((np.cos(a), np.sin(a)), 1), dtype=torch.float32)


def turned(x, rows, pairs):
    """float32 rows x [T, heads, D] turned by the angles rows [T, rot], each operation rounded once."""
    rot = rows.shape[1]
    c, s = rows[:, None, :rot // 2].astype(F), rows[:, None, rot // 2:].astype(F)
    one = slice(0, rot, 2) if pairs else slice(0, rot // 2)
    two = slice(1, rot, 2) if pairs else slice(rot // 2, rot)
    y = x.astype(F).copy()
    a, b = x[..., one].astype(F), x[..., two].astype(F)
    y[..., one] = a * c - b * s
    y[..., two] = b * c + a * s
    return y


def e2m1_code(q):
    a = np.abs(q.astype(np.float64))
    i = np.searchsorted(E2M1_MIDS, a, side="left")
    i = i + ((i < 7) & (E2M1_MIDS[np.minimum(i, 6)] == a) & (i % 2 == 1))
    return (i | np.where(np.signbit(q), 8, 0)).astype(np.uint8)


def _scaled(x, s):
    """x * (1 / s), x / s where 1 / s overflows, signed zeros where s is 0; all binary32."""
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inv = np.where(s != 0, F(1) / s, F(0)).astype(F)
        return np.where(np.isinf(inv), x / s, x * inv).astype(F)


def row_codes(x, fmt):
    """(codes, block scales or None, row scales) of float32 rows x [..., D]."""
    amax = np.abs(x).max(-1)
    if fmt == ROW8:
        s = (amax / F(448)).astype(F)
        return R.e4m3_code(np.clip(_scaled(x, s[..., None]), -448, 448).astype(np.float64)), None, s
    s = (amax / F(2688)).astype(F)
    b = x.reshape(*x.shape[:-1], -1, 16)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(s[..., None] != 0, ((np.abs(b).max(-1) / F(6)).astype(F) / s[..., None]).astype(F), F(0))
    bsc = R.e4m3_code(np.minimum(t, F(448)).astype(np.float64))
    f = (R.e4m3_value(bsc).astype(F) * s[..., None]).astype(F)
    code = e2m1_code(_scaled(b, f[..., None])).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), bsc, s


def bf16(x):
    return torch.tensor(np.ascontiguousarray(x)).to(torch.bfloat16).float().numpy()


def append(planes, fmts, bs, k, v, slots, bounds=None, rows=None, pairs=False):
    """In place: planes ((codes, bscale, scale) of K and of V, numpy); bounds float32 [blocks, H, 2, D].
    Slots below 0 are skipped."""
    slots = np.asarray(slots)
    if k is not None and rows is not None:
        k = turned(k, rows, pairs)
    live = slots >= 0
    for x, (codes, bsc, scale), fmt in ((k, planes[0], fmts[0]), (v, planes[1], fmts[1])):
        if x is None:
            continue
        if fmt == PAGE:
            R.page_store(codes, scale, x.astype(np.float64), slots, bs)
            continue
        c, b, s = row_codes(x[live].astype(F), fmt)
        codes[slots[live]], scale[slots[live]] = c, s
        if b is not None:
            bsc[slots[live]] = b
    if bounds is None:
        return
    kb = bf16(k)
    for pg in dict.fromkeys((slots[live] // bs).tolist()):
        mine = live & (slots // bs == pg)
        lo, hi = kb[mine].min(0), kb[mine].max(0)
        if not (slots[mine] % bs == 0).any():
            lo, hi = np.minimum(lo, bounds[pg, :, 0]), np.maximum(hi, bounds[pg, :, 1])
        bounds[pg, :, 0], bounds[pg, :, 1] = lo, hi


def scores(q, bounds, table_row, vis, H):
    """float64 [H, vis] of one query row q [Hq, D]; NaN where the table entry is outside."""
    g = q.shape[0] // H
    qq = q.reshape(H, g, -1).astype(np.float64)
    plus, minus = np.where(qq < 0, 0, qq).sum(1), np.where(qq > 0, 0, qq).sum(1)
    blk = np.asarray(table_row[:vis]).astype(np.int64)
    ok = (blk >= 0) & (blk < bounds.shape[0])
    b = bounds[np.where(ok, blk, 0)].astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        x = np.einsum("hd,bhd->hb", plus, b[:, :, 1]) + np.einsum("hd,bhd->hb", minus, b[:, :, 0])
    return x, ok


def select(q, bounds, table, lens, starts, bs, topk, first, last, out):
    """In place: out [T, H, topk]."""
    H = bounds.shape[1]
    for s in range(len(lens)):
        n = starts[s + 1] - starts[s]
        for i in range(n):
            vis = (lens[s] - n + i) // bs + 1
            x, ok = scores(q[starts[s] + i], bounds, table[s], vis, H)
            for h in range(H):
                forced = (np.arange(vis) < first) | (np.arange(vis) >= vis - last)
                # (class, score): forced, numbers, NaN, no block
                rank = np.where(forced, 3, np.where(~ok, 0, np.where(np.isnan(x[h]), 1, 2)))
                y = np.where(rank == 2, x[h], 0)
                order = sorted(range(vis), key=lambda b: (-rank[b], -y[b], b))[:topk]
                row = sorted(order)
                out[starts[s] + i, h] = row + [-1] * (topk - len(row))
    return out


def sparse_attention(q, K, V, lens, starts, selected, bs, scale, softcap=0.0):
    """q [T, Hq, D], K / V per sequence [len, H, D], float64 -> (out, largest |logit|, largest |v| a row sees)."""
    out, top, vmax = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    H = selected.shape[1]
    g = q.shape[1] // H
    for s in range(len(lens)):
        n = starts[s + 1] - starts[s]
        for i in range(n):
            r, p = starts[s] + i, lens[s] - n + i
            for h in range(H):
                t = np.concatenate([np.arange(b * bs, min(b * bs + bs, p + 1)) for b in selected[r, h].astype(np.int64)
                                    if 0 <= b and b * bs <= p] or [np.zeros(0, np.int64)])
                if not len(t):
                    continue
                x = q[r, h * g:(h + 1) * g] @ K[s][t, h].T * scale
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                w = np.exp(x - x.max(1, keepdims=True))
                out[r, h * g:(h + 1) * g] = w @ V[s][t, h] / w.sum(1, keepdims=True)
                top[r, h * g:(h + 1) * g] = np.abs(x).max(1)
                vmax[r, h * g:(h + 1) * g] = np.abs(V[s][t, h]).max()
    return out, top, vmax


def close(got, ref, top, vmax, D, softcap=0.0):
    """The accuracy that the header promises, doubled as in the tests of kvq_attention: one rounding
    of P to f16 (2^-11, doubled), one of the output to bf16 (2^-9 of it, doubled), and 4 vmax times the
    logits' error: 2^-20 softcap + 2^-21 |logit| + 2^-22 sqrt(D)."""
    d = 2.0 ** -20 * softcap + 2.0 ** -21 * top + 2.0 ** -22 * math.sqrt(D)
    bound = 2.0 ** -8 * np.abs(ref) + ((2.0 ** -10 + 4 * d) * vmax)[..., None]
    err = np.abs(got - ref)
    assert (err <= bound).all(), np.nanmax(err / np.maximum(bound, 1e-30))
