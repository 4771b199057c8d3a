"""Plain float64 forms of the decoder-block operators (numpy, one sequence and
head at a time), with the error bounds the tests hold the kernels to.

Bounds.  With u the unit roundoff of the element type and e = 2^-24:
 - a score is a sum of D products in fp32, scaled once: off by at most
   ds = (D + 4) e |scale| sum |q||k|;
 - a weight p = exp(s - lse) is then off by a factor of at most
   1 + dp, dp = 2 ds (its own score and the ones in lse) + (n + 32) e for the
   sum over n slots and for exp2 and the rescaling by powers (each a few ulp
   and at most two rescalings per block; 32 covers them);
 - the output adds u (weights rounded to the element type; none in fp32) and
   n e (the sum over slots) relative to sum p |v|, and u |out| for its own
   rounding."""

from __future__ import annotations

import math

import numpy as np

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
E = 2.0 ** -24


def attend(q, k, v, scale, dt):
    """q [M, D], k, v [n, D] float64: out, lse, p [M, n] and their error bounds."""
    M, D = q.shape
    n = k.shape[0]
    if n == 0:
        z = np.zeros((M, D))
        inf = np.full(M, -np.inf)
        return (z, inf, np.zeros((M, 0))), (z, np.zeros(M), np.zeros((M, 0)))
    s = scale * (q @ k.T)
    ds = (D + 4) * E * abs(scale) * (np.abs(q) @ np.abs(k).T).max(1)
    top = s.max(1, keepdims=True)
    ex = np.exp(s - top)
    tot = ex.sum(1, keepdims=True)
    p = ex / tot
    lse = (top + np.log(tot))[:, 0]
    out = p @ v
    dp = 2 * ds + (n + 32) * E
    pv = p @ np.abs(v)
    rnd = 0.0 if dt == "f32" else U[dt]
    # f16 weights below 2^-14 of the running maximum are subnormal: off by 2^-25 of it
    tiny = n * 2.0 ** -25 * np.abs(v).max(0, keepdims=True) / tot if dt == "f16" else 0.0
    b_out = U[dt] * np.abs(out) + (dp[:, None] + rnd + n * E) * pv + tiny * 1.0 + 1e-30
    b_lse = dp + 4 * E * np.abs(lse) + 4 * E
    b_p = dp[:, None] * p + 2.0 ** -126
    return (out, lse, p), (b_out, b_lse, b_p)


def slot_rows(cache, table, page, b, h, slots):
    """Rows of head h of sequence b at `slots` and which of them have a page."""
    pg = table[b, slots // page]
    ok = (pg >= 0) & (pg < cache.shape[0])
    return cache[np.where(ok, pg, 0), h, slots % page], ok


def paged(q, kc, vc, table, lengths, page, window, scale, dt):
    """q [B, Hq, D], caches [P, H, page, D]: out, lse, added weights and bounds."""
    B, Hq, D = q.shape
    H = kc.shape[1]
    G = Hq // H
    cap = table.shape[1] * page
    res = [np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf), np.zeros((B, H, cap))]
    bnd = [np.zeros((B, Hq, D)), np.zeros((B, Hq)), np.zeros((B, H, cap))]
    for b in range(B):
        n = int(min(max(lengths[b], 0), cap))
        first = max(0, n - window) if window else 0
        at = np.arange(first, n)
        for h in range(H):
            kr, ok = slot_rows(kc, table, page, b, h, at)
            vr, _ = slot_rows(vc, table, page, b, h, at)
            r = slice(h * G, (h + 1) * G)
            (o, l, p), (bo, bl, bp) = attend(q[b, r], kr[ok], vr[ok], scale, dt)
            res[0][b, r], res[1][b, r] = o, l
            bnd[0][b, r], bnd[1][b, r] = bo, bl
            res[2][b, h, at[ok]] = p.sum(0)
            bnd[2][b, h, at[ok]] = bp.sum(0) + G * E * p.sum(0)
    return res, bnd


def cross(q, k, v, lengths, mask, scale, dt):
    B, Lq, Hq, D = q.shape
    Lk, H = k.shape[1], k.shape[2]
    out, lse = np.zeros(q.shape), np.full((B, Hq, Lq), -np.inf)
    bo, bl = np.zeros(q.shape), np.zeros((B, Hq, Lq))
    for b in range(B):
        n = Lk if lengths is None else int(min(max(lengths[b], 0), Lk))
        at = np.arange(n)
        if mask is not None:
            at = at[mask[b, :n] != 0]
        for h in range(Hq):
            g = h // (Hq // H)
            (o, l, _), (eo, el, _) = attend(q[b, :, h], k[b, at, g], v[b, at, g], scale, dt)
            out[b, :, h], lse[b, h], bo[b, :, h], bl[b, h] = o, l, eo, el
    return (out, lse), (bo, bl)


def append(kn, vn, kc, vc, table, lengths, counts, now, page, positions=None, weights=None):
    """In place on copies; returns (kc, vc, positions, weights)."""
    kc, vc = kc.copy(), vc.copy()
    positions = None if positions is None else positions.copy()
    weights = None if weights is None else weights.copy()
    B, n = kn.shape[:2]
    for b in range(B):
        ln = max(int(lengths[b]), 0)
        c = min(max(n if counts is None else int(counts[b]), 0), n, ln)
        seen = int(lengths[b] if now is None else now[b])
        for i in range(c):
            t = ln - c + i
            if t >= table.shape[1] * page:
                continue
            if positions is not None:
                positions[b, :, t] = seen - c + i
            if weights is not None:
                weights[b, :, t] = 0
            pg = table[b, t // page]
            if 0 <= pg < kc.shape[0]:
                kc[pg, :, t % page], vc[pg, :, t % page] = kn[b, i], vn[b, i]
    return kc, vc, positions, weights


def evict(kc, vc, table, lengths, now, weights, positions, page, keep, sink, recent):
    """(kc, vc, weight_out, positions_out, lengths_out, source) by sorting."""
    kc, vc = kc.copy(), vc.copy()
    B, H, cap = weights.shape
    w_out = np.zeros((B, H, keep), np.float32)
    p_out, source = np.full((B, H, keep), -1, np.int32), np.full((B, H, keep), -1, np.int32)
    l_out = np.zeros(B, np.int32)
    for b in range(B):
        n = int(min(max(lengths[b], 0), cap))
        m = min(n, keep)
        l_out[b] = m
        seen = int(lengths[b] if now is None else now[b])
        for h in range(H):
            pos = np.arange(n) if positions is None else positions[b, h, :n].astype(np.int64)
            w = weights[b, h, :n].astype(np.float64)
            w = np.where(np.isnan(w), -np.inf, np.minimum(w, np.finfo(np.float32).max))
            safe = (pos < sink) | (pos >= seen - recent)
            page_of = table[b, np.arange(n) // page]
            gap = (page_of < 0) | (page_of >= kc.shape[0])  # stays below m, given up from m on
            group = np.where(gap, np.where(np.arange(n) < m, 0, 3), np.where(safe, 1, 2))
            order = sorted(range(n), key=lambda t: (group[t], -w[t] if group[t] == 2 else 0.0, t))
            kept = np.zeros(n, bool)
            kept[order[:m]] = True
            src = np.arange(m)
            holes = np.flatnonzero(~kept[:m])
            src[holes] = m + np.flatnonzero(kept[m:])
            source[b, h, :m] = src
            w_out[b, h, :m] = weights[b, h, src]
            p_out[b, h, :m] = src if positions is None else positions[b, h, src]
            for j in holes:
                p1, p0 = table[b, j // page], table[b, src[j] // page]
                kc[p1, h, j % page] = kc[p0, h, src[j] % page]
                vc[p1, h, j % page] = vc[p0, h, src[j] % page]
    return kc, vc, w_out, p_out, l_out, source


def norm(u, kind, w, b, eps):
    if kind == 0:
        return u
    if kind == 2:
        u = u - u.mean(-1, keepdims=True)
    u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    u = u if w is None else u * w
    return u if b is None else u + b


def norm_residual(x, h, post, pw, pb, scale, gate, fn, per, pre, nw, nb, eps):
    f = norm(h, post, pw, pb, eps)
    if scale is not None:
        f = f * scale
    if fn:
        g = gate[np.arange(x.shape[0]) // per]
        with np.errstate(over="ignore"):
            g = [None, g, 1 / (1 + np.exp(-g)), np.tanh(g)][fn]
        f = f * g
    xo = x + f
    return xo, (norm(xo, pre, nw, nb, eps) if pre else None)


def check(got, ref, bound, what=""):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities differ"
    diff = np.where(inf, 0.0, np.abs(np.where(inf, 0.0, got) - np.where(inf, 0.0, ref)))
    bad = ~(diff <= np.broadcast_to(bound, ref.shape))
    worst = float(np.max(diff / np.maximum(np.broadcast_to(bound, ref.shape), 1e-300))) if ref.size else 0.0
    print(f"  {what} max |err| / bound = {worst:.3f} over {ref.size}", flush=True)
    if bad.any():
        i = np.unravel_index(int(np.argmax(bad)), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {ref.size} outside the bound; first at "
                             f"{tuple(int(v) for v in i)}: got {got[i]!r} ref {ref[i]!r} "
                             f"bound {np.broadcast_to(bound, ref.shape)[i]!r}")
