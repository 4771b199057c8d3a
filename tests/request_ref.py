"""Plain forms of the operators on requests of many lengths, one sequence, head
and row at a time (float64; lists for the page tables), with the error bounds the
tests hold the kernels to (block_ref.py has the attention's)."""

from __future__ import annotations

import numpy as np

from block_ref import E, U, slot_rows


def clamp(v, lo, hi):
    return max(lo, min(hi, int(v)))


def pages(lengths, counts, now, held, free_count, table, free_pages, page, rows=0, positions=None,
          weights=None):
    """(table, held, free_pages, free_count, row_starts, row_positions, row_slots, positions,
    weights) after ctconv_cache_pages, on copies."""
    table, free = np.array(table), [int(v) for v in free_pages]
    P, (B, cols) = len(free), table.shape
    cap = cols * page
    need = [-(-clamp(n, 0, cap) // page) for n in lengths]
    held = [clamp(h, 0, cols) for h in held]
    top = clamp(free_count, 0, P)
    for b in range(B):
        for p in table[b, need[b]:held[b]]:
            if 0 <= p < P and top < P:
                free[top] = int(p)
                top += 1
        held[b] = min(held[b], max(need[b], 0)) if held[b] > need[b] else held[b]
    for b in range(B):
        for j in range(held[b], need[b]):
            if top > 0:
                top -= 1
                table[b, j] = free[top]
                held[b] += 1
            else:
                table[b, j] = -1
    out = [table, np.array(held), np.array(free), top]
    if counts is None:
        return out
    positions = None if positions is None else positions.copy()
    weights = None if weights is None else weights.copy()
    starts, at, to = [0], np.full(rows, -1), np.full(rows, -1)
    for b in range(B):
        n = int(lengths[b])
        c = clamp(counts[b], 0, max(n, 0))
        seen = n if now is None else int(now[b])
        for i in range(min(c, max(0, rows - starts[-1]))):
            r, t = starts[-1] + i, n - c + i
            at[r] = seen - c + i
            if t >= cap:
                continue
            p = table[b, t // page]
            if 0 <= p < P:
                to[r] = p * page + t % page
            if positions is not None:
                positions[b, :, t] = at[r]
            if weights is not None:
                weights[b, :, t] = 0
        starts.append(min(starts[-1] + c, 2 ** 31 - 1))
    return out + [np.array(starts), at, to, positions, weights]


def turned(x, positions, frequencies, layout, scale, dt):
    """x [rows, H, D] turned (layout 0: halves, 1: pairs), and the bound of its error.

    The angle's turns carry three roundings of fp64 (position * frequency / 2 pi, its
    fraction); their fraction, at most 1/2, is rounded to fp32 (off by at most pi e in
    radians, e = 2^-24); sine and cosine of that are off by a few ulp (8 e), the magnitude,
    two products and a sum by e each of what they add up: 20 e in all, and the output's own
    rounding."""
    R = 2 * len(frequencies)
    a = positions[:, None].astype(np.float64) * frequencies[None, :]
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    y, bound = x.copy(), np.zeros(x.shape)
    first = slice(0, R // 2) if layout == 0 else slice(0, R, 2)
    second = slice(R // 2, R) if layout == 0 else slice(1, R, 2)
    u, v = x[..., first], x[..., second]
    y[..., first], y[..., second] = scale * (u * c - v * s), scale * (v * c + u * s)
    off = 20 * E + np.abs(a)[:, None, :] * 4 * 2.0 ** -53
    for part in (first, second):
        bound[..., part] = U[dt] * np.abs(y[..., part]) + off * abs(scale) * (np.abs(u) + np.abs(v))
    return y, bound


def seen_rows(q, k, v, seen, scale, dt):
    """Attention of rows q [M, D] to k, v [n, D] where seen [M, n]: (out, lse, p) and their bounds,
    those of block_ref.attend row by row."""
    M, D = q.shape
    count = seen.sum(1)
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    size = np.where(seen, np.abs(q) @ np.abs(k).T, 0.0)
    ds = (D + 4) * E * abs(scale) * (size.max(1) if k.shape[0] else np.zeros(M))
    top = s.max(1, initial=-np.inf)
    ex = np.exp(s - np.where(np.isinf(top), 0.0, top)[:, None])
    tot = ex.sum(1)
    p = ex / np.where(tot == 0, 1.0, tot)[:, None]
    with np.errstate(divide="ignore"):
        lse = top + np.log(tot)
    out = p @ v
    dp = 2 * ds + (count + 32) * E
    rnd = 0.0 if dt == "f32" else U[dt]
    big = np.array([np.abs(v[r]).max(0) if r.any() else np.zeros(D) for r in seen]).reshape(M, D)
    tiny = count[:, None] * 2.0 ** -25 * big / np.where(tot == 0, 1.0, tot)[:, None] if dt == "f16" else 0.0
    b_out = U[dt] * np.abs(out) + (dp + rnd + count * E)[:, None] * (p @ np.abs(v)) + tiny + 1e-30
    b_lse = np.where(count > 0, dp + 4 * E * np.abs(np.where(count > 0, lse, 0)) + 4 * E, 0.0)
    return (out, lse, p), (b_out, b_lse, dp[:, None] * p + 2.0 ** -126)


def chunk(q, kc, vc, table, lengths, counts, page, window, scale, dt, max_length=None):
    """q: a list of [counts[b], Hq, D], caches [P, H, page, D]: lists of (out, lse) and bounds per
    sequence, added weights [B, H, slots] and their bound."""
    B, H = len(q), kc.shape[1]
    cap = table.shape[1] * page
    most = cap if max_length is None else min(cap, max_length)
    w, wb = np.zeros((B, H, cap)), np.zeros((B, H, cap))
    res = []
    for b in range(B):
        n, Hq, D = q[b].shape
        G = Hq // H
        L = clamp(lengths[b], 0, most)
        out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
        bo, bl = np.zeros((n, Hq, D)), np.zeros((n, Hq))
        at = np.arange(L)
        end = L - int(counts[b]) + np.arange(n)[:, None] + 1
        seen = (at[None, :] < end) & (at[None, :] >= (end - window if window else 0))
        for h in range(H):
            kr, ok = slot_rows(kc, table, page, b, h, at)
            vr, _ = slot_rows(vc, table, page, b, h, at)
            for j in range(h * G, (h + 1) * G):
                (o, l, p), (eo, el, ep) = seen_rows(q[b][:, j], kr[ok], vr[ok], seen[:, ok], scale, dt)
                out[:, j], lse[:, j], bo[:, j], bl[:, j] = o, l, eo, el
                # the weights are taken again, against a rounded log2 of the sum
                with np.errstate(divide="ignore"):
                    arg = np.where(p > 0, np.abs(np.log2(np.where(p > 0, p, 1.0))), 0)
                level = np.where(np.isinf(l), 0.0, np.abs(l))
                again = (1.5 * level[:, None] + arg + 8) * E
                w[b, h, at[ok]] += p.sum(0)
                wb[b, h, at[ok]] += (ep + again * p).sum(0)
        res.append((out, lse, bo, bl))
    rows = sum(x.shape[0] * x.shape[1] // H for x in q)
    return res, w, wb + (rows + 2) * E * w
