"""GPU: the operators on requests of many lengths (page tables and row maps,
rotary positions alone and on the way into the cache, attention of a chunk of
new rows) against their plain forms (request_ref.py).  Slots and rows that must
not be used hold NaN."""

import numpy as np
import pytest

import block_ref as R
import request_ref as Q
from gpu_util import say, to_host, torch_dtype
from test_gpu_block import Cache, cc, dev, guarded, ints  # noqa: F401

pytestmark = pytest.mark.gpu

DTS = ["f32", "bf16", "f16"]


# ---------------------------------------------------------------------------
# Page tables and row maps
# ---------------------------------------------------------------------------


def requests(rng, B, page, cols, new, kind):
    """(lengths, counts, held before) of sequences that go on, end, are new or were cut back."""
    cap = cols * page
    lengths, counts, held = [], [], []
    for b in range(B):
        old = int(rng.integers(0, cap + 1))
        part = rng.integers(0, 4) if kind == "mixed" else 0
        if part == 1:
            n, c = 0, 0
        elif part == 2:
            old, c = 0, int(rng.integers(0, min(new, cap) + 1))
            n = c
        elif part == 3:
            c = 0
            n = int(rng.integers(0, old + 1))
        else:
            c = int(min(rng.integers(0, new + 1), cap))
            old = min(old, cap - c)
            n = old + c
        lengths.append(n)
        counts.append(c)
        held.append(-(-old // page))
    return np.array(lengths), np.array(counts), np.array(held)


def tables(rng, held, cols, P):
    order = rng.permutation(P)
    table = np.full((len(held), cols), -1)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    free = np.full(P, -9)
    free[:P - at] = order[at:]
    return table, free, P - at


PAGES = [
    # B, page, cols, new, kind, spare pages, heads
    (1, 16, 1, 1, "on", 0, 0),
    (1, 1, 5, 3, "mixed", 1, 1),
    (5, 7, 9, 20, "mixed", 2, 3),
    (48, 16, 40, 1, "on", 20, 8),
    (64, 16, 30, 200, "mixed", 0, 2),
    (64, 16, 30, 200, "mixed", -40, 2),
    (1024, 8, 6, 5, "mixed", 3, 1),
    (1025, 3, 11, 40, "mixed", -100, 0),
    (3000, 4, 4, 2, "mixed", 10, 0),
    (7, 64, 20, 1280, "mixed", 5, 4),
]


@pytest.mark.parametrize("case", PAGES, ids=[str(i) for i in range(len(PAGES))])
@pytest.mark.parametrize("room", [0, 5, -3], ids=["exact", "padded", "short"])
def test_cache_pages(cc, case, room):  # noqa: F811
    import torch

    B, page, cols, new, kind, spare, heads = case
    say(f"pages {case} room={room}")
    rng = np.random.default_rng(B * 31 + page)
    lengths, counts, held = requests(rng, B, page, cols, new, kind)
    need = -(-lengths // page)
    P = int(max(held.sum(), need.sum() + spare, 1))
    table, free, count = tables(rng, held, cols, P)
    now = lengths + rng.integers(0, 100, B)
    rows = max(0, int(counts.sum()) + room)
    positions = weights = pd = wd = None
    if heads:
        positions = rng.integers(-5, 5, (B, heads, cols * page)).astype(np.int32)
        weights = rng.random((B, heads, cols * page)).astype(np.float32)
        pd, wd = ints(positions), torch.from_numpy(weights).cuda()
    ref = Q.pages(lengths, counts, now, held, count, table, free, page, rows, positions, weights)
    # results apart from the state: twice the same, the state as it was
    td, fd, hd, cd = ints(table), ints(free), ints(held), ints([count])
    ld, nd, kd = ints(lengths), ints(now), ints(counts)
    ho, co = torch.empty_like(hd), torch.empty_like(cd)
    rs, rp, rl = (torch.full((k,), -77, dtype=torch.int32, device="cuda")
                  for k in (B + 1, rows, rows))
    plan = cc.CachePages(B, rows, P, page, cols, Hkv=max(heads, 1))
    s = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        plan(ld.data_ptr(), kd.data_ptr(), nd.data_ptr(), hd.data_ptr(), cd.data_ptr(),
             td.data_ptr(), fd.data_ptr(), ho.data_ptr(), co.data_ptr(), rs.data_ptr(),
             rp.data_ptr(), rl.data_ptr(), None if pd is None else pd.data_ptr(),
             None if wd is None else wd.data_ptr(), s)
        torch.cuda.synchronize()
        got = [td, ho, fd, co, rs, rp, rl, pd, wd]
        for name, g, r in zip(("table", "held", "free", "count", "starts", "positions", "slots",
                               "slot positions", "slot weights"), got, ref):
            if r is not None:
                assert np.array_equal(g.cpu().numpy().ravel(), np.asarray(r).ravel()), name
        assert np.array_equal(hd.cpu().numpy(), held) and int(cd) == count
    # in place, through the helper
    td, fd, hd, cd = ints(table), ints(free), ints(held), ints([count])
    maps = cc.cache_pages(td, hd, fd, cd, ld, page_size=page, counts=kd, now=nd, rows=rows)
    torch.cuda.synchronize()
    for g, r in zip([td, hd, fd, cd, *maps], ref):
        assert np.array_equal(g.cpu().numpy().ravel(), np.asarray(r).ravel())


def test_cache_pages_wild_state(cc):  # noqa: F811
    """Lengths, counts and holdings outside their ranges, table entries that are no pages, a
    stack that is full, no counts, no now, strided tables and slot arrays."""
    import torch

    say("pages, wild state")
    rng = np.random.default_rng(3)
    B, page, cols, P = 6, 4, 5, 24
    lengths = np.array([25, -3, 2 ** 31 - 1, 7, 0, 20])
    counts = np.array([30, 5, 3, -2, 4, 2 ** 31 - 1])
    held = np.array([9, 3, 0, 5, -1, 2])
    table = rng.permutation(B * cols)[:B * cols].reshape(B, cols) % P
    table[1, 1], table[3, 4] = -1, 10 ** 6
    for free_count in (0, 3, P, P + 9, -2):
        free = rng.permutation(P)
        rows = 40
        ref = Q.pages(lengths, counts, None, held, free_count, table, free, page, rows,
                      np.zeros((B, 2, 20), np.int32), np.ones((B, 2, 20), np.float32))
        big = torch.full((B, cols + 3), -55, dtype=torch.int32, device="cuda")
        big[:, :cols] = ints(table)
        wide = torch.full((B, 2, 27), -5, dtype=torch.int32, device="cuda")
        pos, w = wide[..., :20], torch.full((B, 2, 27), 5.0, device="cuda")[..., :20]
        pos.zero_()
        w.fill_(1.0)
        hd, fd, cd = ints(held), ints(free), ints([free_count])
        maps = cc.cache_pages(big[:, :cols], hd, fd, cd, ints(lengths), page_size=page,
                              counts=ints(counts), rows=rows, positions=pos, weight_sum=w)
        torch.cuda.synchronize()
        for g, r in zip([big[:, :cols], hd, fd, cd, *maps, pos, w], ref):
            assert np.array_equal(g.cpu().numpy().ravel(), np.asarray(r).ravel()), free_count
        assert bool((big[:, cols:] == -55).all()) and bool((wide[..., 20:] == -5).all())
        # the table alone
        td, hd, fd, cd = ints(table), ints(held), ints(free), ints([free_count])
        assert cc.cache_pages(td, hd, fd, cd, ints(lengths), page_size=page) is None
        for g, r in zip([td, hd, fd, cd], ref):
            assert np.array_equal(g.cpu().numpy().ravel(), np.asarray(r).ravel())


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

ROTARY = [
    # rows, Hq, Hk, D, R, layout, scale, far
    (1, 1, 1, 8, 8, 0, 1.0, 10),
    (1, 1, 0, 8, 2, 1, 1.0, 10),
    (3, 4, 2, 64, 64, 0, 1.0, 1000),
    (9, 8, 8, 64, 64, 1, 1.2, 2000000),
    (300, 6, 2, 128, 128, 0, 1.0, 2 ** 31 - 1),
    (37, 5, 1, 80, 32, 0, 0.7, 500),
    (37, 5, 1, 80, 40, 0, 0.7, 500),   # halves of 20 values
    (37, 3, 1, 96, 38, 0, 1.0, 500),   # of 19
    (37, 3, 1, 96, 4, 0, 1.0, 500),
    (37, 3, 1, 96, 38, 1, -1.0, 500),
    (5, 0, 3, 256, 256, 0, 1.0, 100000),
    (2100, 2, 1, 40, 24, 0, 1.0, 7),
    (4, 130, 1, 16, 12, 0, 1.0, 7),
    (1500, 3, 3, 24, 6, 1, 1.0, 7),
]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", ROTARY, ids=[str(i) for i in range(len(ROTARY))])
def test_rotary(cc, case, dt):  # noqa: F811
    import torch

    rows, Hq, Hk, D, R_, layout, scale, far = case
    say(f"rotary {case} {dt}")
    rng = np.random.default_rng(rows + D)
    f = cc.rotary_frequencies(R_, 10000.0, device="cuda")
    f64 = to_host(f)
    assert np.allclose(f64, 10000.0 ** (-np.arange(R_ // 2) * 2 / R_), rtol=1e-14)
    pos = rng.integers(0, far + 1, rows)
    pos[rng.random(rows) < 0.2] = -1
    pd = ints(pos)
    live = (pos >= 0)[:, None, None]
    # q and k behind each other in a row, as one product leaves them
    both, b64 = dev(rng.standard_normal((rows, Hq + Hk, D)), dt)
    q, k = (both[:, :Hq] if Hq else None), (both[:, Hq:] if Hk else None)
    want, bound = Q.turned(b64, pos, f64, layout, scale, dt)
    sentinel = guarded(torch.full((rows, Hq + Hk, D), 9.0, dtype=both.dtype, device="cuda"))
    q_out, k_out = (sentinel[:, :Hq] if Hq else None), (sentinel[:, Hq:] if Hk else None)
    cc.rotary(q, k, pd, f, layout, scale, q_out, k_out)
    torch.cuda.synchronize()
    R.check(to_host(sentinel), np.where(live, want, 9.0), np.where(live, bound, 0.0), "apart")
    cc.rotary(q, k, pd, f, layout, scale, q, k)  # in place
    torch.cuda.synchronize()
    R.check(to_host(both), np.where(live, want, b64), np.where(live, bound, 0.0), "in place")
    # backwards by the negative frequencies; two roundings on the way
    if scale == 1.0:
        a, b = cc.rotary(q, k, pd, -f, layout, scale)
        torch.cuda.synchronize()
        got = np.concatenate([to_host(t) for t in (a, b) if t is not None], 1)
        back, more = Q.turned(to_host(both), pos, -f64, layout, scale, dt)
        R.check(np.where(live, got, 0), np.where(live, back, 0), more + 1e-30, "back")


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "dims", "turns"])
@pytest.mark.parametrize("R_", [2, 64, 126])
def test_rotary_frequencies(cc, scaling, R_):  # noqa: F811
    i = np.arange(R_ // 2)
    base, factor, L = 50000.0, 4.0, 2048.0
    kind = {"none": cc.ROTARY_NONE, "linear": cc.ROTARY_LINEAR, "base": cc.ROTARY_BASE,
            "dims": cc.ROTARY_RAMP_DIMS, "turns": cc.ROTARY_RAMP_TURNS}[scaling]
    low, high = (1.0, 32.0) if scaling == "dims" else (1.0, 4.0)
    got = cc.rotary_frequencies(R_, base, kind, factor, L, low, high).numpy()
    f = base ** (-2.0 * i / R_)
    if scaling == "linear":
        f = f / factor
    elif scaling == "base" and R_ > 2:
        f = (base * factor ** (R_ / (R_ - 2))) ** (-2.0 * i / R_)
    elif scaling == "dims":
        def at(t):
            return R_ * np.log(L / (2 * np.pi * t)) / (2 * np.log(base))

        a, b = max(np.floor(at(high)), 0), min(np.ceil(at(low)), R_ - 1)
        k = 1 - np.clip((i - a) / max(b - a, 0.001), 0, 1)
        f = f * k + f / factor * (1 - k)
    elif scaling == "turns":
        k = np.clip((L * f / (2 * np.pi) - low) / (high - low), 0, 1)
        f = f * k + f / factor * (1 - k)
    assert np.allclose(got, f, rtol=1e-13)


APPEND = [
    # rows, Hq, Hkv, D, R, layout, page, cache layout
    (1, 1, 1, 8, 8, 0, 1, "library"),
    (48, 8, 2, 128, 128, 0, 16, "library"),
    (77, 3, 3, 80, 40, 0, 7, "slots"),
    (1030, 4, 2, 64, 64, 1, 24, "library"),
    (33, 0, 5, 256, 64, 0, 64, "both"),
    (50, 7, 1, 40, 38, 0, 3, "slots"),
]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
def test_rotary_append(cc, case, dt):  # noqa: F811
    import torch

    rows, Hq, H, D, R_, layout, page, order = case
    say(f"rotary append {case} {dt}")
    rng = np.random.default_rng(rows * 3 + D)
    f = cc.rotary_frequencies(R_, 10000.0, device="cuda")
    pos = rng.integers(0, 5000, rows)
    pos[rng.random(rows) < 0.1] = -1
    P = -(-rows // page) + 2
    slots = rng.permutation(P * page)[:rows]
    wild = rng.random(rows)
    slots = np.where(wild < 0.05, -1, np.where(wild < 0.1, P * page, np.where(wild < 0.12, 2 ** 31 - 1, slots)))
    qkv, x64 = dev(rng.standard_normal((rows, Hq + 2 * H, D)), dt)
    q, k, v = (qkv[:, :Hq] if Hq else None), qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    kc = torch.full((P, H, page, D), 5.0, dtype=torch_dtype(dt), device="cuda")
    vc = torch.full_like(kc, 6.0)
    if order == "slots":
        kc, vc = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kc, vc))
    elif order == "both":
        pair = torch.stack((kc, vc), 1)
        kc, vc = pair[:, 0], pair[:, 1]
    q_out = None if q is None else guarded(torch.full((rows, Hq, D), 9.0, dtype=q.dtype, device="cuda"))
    y = cc.rotary_append(q, k, v, ints(pos), ints(slots), f, kc, vc, layout, 1.1, q_out=q_out)
    torch.cuda.synchronize()
    live = pos >= 0
    want, bound = Q.turned(x64, pos, to_host(f), layout, 1.1, dt)
    if q is not None:
        R.check(to_host(y), np.where(live[:, None, None], want[:, :Hq], 9.0),
                np.where(live[:, None, None], bound[:, :Hq], 0.0), "q")
    kw, vw, kb = np.full((P, H, page, D), 5.0), np.full((P, H, page, D), 6.0), np.zeros((P, H, page, D))
    for r in np.flatnonzero(live & (slots >= 0) & (slots < P * page)):
        p, at = slots[r] // page, slots[r] % page
        kw[p, :, at], kb[p, :, at] = want[r, Hq:Hq + H], bound[r, Hq:Hq + H]
        vw[p, :, at] = x64[r, Hq + H:]
    R.check(to_host(kc), kw, kb, "k")
    assert np.array_equal(to_host(vc), vw)


# ---------------------------------------------------------------------------
# Attention of a chunk of new rows
# ---------------------------------------------------------------------------

CHUNK = [
    # counts, lengths, most rows, Hq, Hkv, D, page, window, cache layout
    ([1], [1], 1, 1, 1, 8, 1, 0, "library"),
    ([2, 0, 1], [250, 3, 0], 2, 8, 8, 64, 16, 0, "library"),
    ([8, 5, 8], [513, 255, 8], 8, 8, 2, 128, 16, 0, "library"),
    ([4], [700], 4, 6, 3, 80, 64, 333, "slots"),
    ([3, 4], [1300, 2049], 4, 6, 1, 128, 24, 0, "both"),
    ([2, 3], [129, 64], 3, 20, 1, 96, 7, 0, "slots"),
    ([3, 1], [260, 31], 4, 2, 2, 256, 128, 0, "library"),
    ([2], [301], 2, 17, 1, 40, 5, 1, "library"),
    ([5, 3], [95, 3], 5, 2, 1, 200, 3, 2, "slots"),
    ([64, 40, 1], [64, 300, 77], 64, 1, 1, 64, 16, 0, "library"),
    # more rows than one tile takes
    ([65], [65], 65, 1, 1, 64, 16, 0, "library"),
    ([130, 1, 0, 33], [130, 400, 5, 600], 130, 2, 2, 64, 16, 0, "library"),
    ([50, 17], [190, 17], 50, 8, 2, 128, 24, 0, "slots"),
    ([129], [500], 129, 3, 1, 80, 7, 100, "library"),
    ([100, 1], [700, 650], 100, 4, 4, 96, 64, 1, "both"),
    ([70, 128], [333, 128], 128, 2, 1, 128, 1, 64, "library"),
    ([40], [300], 40, 4, 1, 256, 16, 0, "library"),
    ([30, 33], [100, 33], 33, 7, 1, 200, 8, 50, "slots"),
    ([90], [90], 90, 5, 1, 32, 256, 0, "library"),
    ([70], [40], 70, 2, 1, 64, 16, 0, "library"),  # rows before the first slot see nothing
]

# Many rows and heads: in 16 bits most of these take the tiled kernel.
MANY = [
    ([330, 329], [330, 420], 330, 8, 8, 128, 16, 0, "library"),
    ([700, 1, 0, 257], [700, 1500, 5, 900], 700, 16, 4, 64, 24, 0, "slots"),
    ([500, 3], [1500, 1601], 500, 12, 4, 96, 7, 200, "both"),
    ([601], [700], 601, 24, 8, 80, 64, 0, "library"),
    ([300, 190], [420, 190], 300, 18, 6, 256, 8, 0, "slots"),
    ([400], [1000], 400, 32, 4, 200, 1, 64, "library"),
    ([900, 65], [903, 3000], 900, 7, 7, 32, 256, 0, "library"),
    ([800], [790], 800, 8, 8, 40, 16, 0, "library"),
    ([17] * 24, [1100 + 10 * i for i in range(24)], 17, 16, 8, 128, 16, 0, "library"),
    ([200], [1600], 200, 32, 8, 128, 32, 0, "library"),
    ([210, 3], [1700, 1500], 210, 32, 8, 96, 16, 1200, "slots"),
]


def chunk_inputs(rng, case, dt, cols=None):
    counts, lengths, n, Hq, H, D, page, window, order = case
    c = Cache(rng, len(counts), H, D, page, lengths, dt, order, cols=cols)
    return c, [rng.standard_normal((k, Hq, D)) * 1.5 for k in counts]


def packed(rows, pad, dt):
    """The sequences' rows one behind the other, `pad` rows of NaN behind them."""
    flat = np.concatenate([*rows, np.full((pad, *rows[0].shape[1:]), np.nan)])
    starts = np.cumsum([0] + [len(r) for r in rows])
    q, q64 = dev(flat, dt)
    return q, ints(starts), [q64[a:b] for a, b in zip(starts[:-1], starts[1:])]


def compare(got, lse, ref, what):
    out = np.concatenate([r[0] for r in ref])
    R.check(got, out, np.concatenate([r[2] for r in ref]), what + " out")
    R.check(lse, np.concatenate([r[1] for r in ref]), np.concatenate([r[3] for r in ref]), what + " lse")


# And over keys enough that the tiled kernel is the faster one in this type, too.
LONG = [
    ("bf16", ([400], [3000], 400, 8, 2, 256, 8, 0, "library")),
    ("f16", ([400, 9], [2800, 2500], 400, 8, 2, 200, 16, 0, "slots")),
    ("f32", ([128], [8000], 128, 32, 8, 128, 16, 0, "library")),
    ("f32", ([128, 1], [8100, 9000], 128, 32, 8, 96, 24, 0, "both")),
    ("f32", ([256], [8100], 256, 32, 8, 64, 64, 5000, "library")),
    ("f32", ([400], [6100], 400, 32, 8, 32, 16, 0, "slots")),
    ("f32", ([300], [6100], 300, 32, 8, 40, 16, 0, "library")),
    ("f32", ([200], [6100], 200, 32, 8, 80, 1, 0, "library")),
    ("f32", ([128], [8000], 128, 32, 8, 120, 16, 0, "library")),
    ("bf16", ([400], [3000], 400, 16, 4, 120, 16, 0, "library")),
    ("f16", ([401, 300], [3000, 1700], 401, 16, 4, 104, 16, 0, "both")),
]


@pytest.mark.parametrize("case", LONG, ids=[str(i) for i in range(len(LONG))])
def test_chunk_attention_long(cc, case):  # noqa: F811
    test_chunk_attention(cc, case[1], case[0], True)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", CHUNK + MANY, ids=[str(i) for i in range(len(CHUNK + MANY))])
@pytest.mark.parametrize("weights", [False, True])
def test_chunk_attention(cc, case, dt, weights):  # noqa: F811
    import torch

    counts, lengths, n, Hq, H, D, page, window, order = case
    B = len(counts)
    say(f"chunk {case} {dt} weights={weights}")
    rng = np.random.default_rng(sum(lengths) + D)
    c, rows = chunk_inputs(rng, case, dt, cols=-(-max(max(lengths), 1) // page) + 1)
    q, starts, q64 = packed(rows, 3, dt)
    cap = c.table.shape[1] * page
    w0 = rng.random((B, H, cap)).astype(np.float32)
    scale = 0.7 * D ** -0.5
    ref, w, wb = Q.chunk(q64, c.k, c.v, c.table, lengths, counts, page, window, scale, dt)
    total = sum(counts)
    out = guarded(torch.full((total + 3, Hq, D), 9.0, dtype=q.dtype, device="cuda"))
    lse = torch.full((total + 3, Hq), 9.0, device="cuda")
    wd = torch.from_numpy(w0).cuda() if weights else None
    cc.chunk_attention(q, c.kd, c.vd, c.td, c.ld, row_starts=starts, n=n, window=window,
                       scale=scale, weight_sum=wd, out=out, lse=lse)
    torch.cuda.synchronize()
    compare(to_host(out)[:total], to_host(lse)[:total], ref, "packed")
    assert bool((out[total:] == 9).all()) and bool((lse[total:] == 9).all())
    if weights:
        R.check(to_host(wd), w0 + w, wb + 2.0 ** -24 * (w0 + w), "weights")
        assert np.array_equal(to_host(wd)[w == 0], w0.astype(np.float64)[w == 0])
        return
    # padded
    full = np.full((B, n, Hq, D), np.nan)
    for b in range(B):
        full[b, :counts[b]] = q64[b]
    qp, _ = dev(full, dt)
    out = torch.full((B, n, Hq, D), 9.0, dtype=q.dtype, device="cuda")
    _, lse = cc.chunk_attention(qp, c.kd, c.vd, c.td, c.ld, counts=ints(counts), window=window,
                                scale=scale, out=out)
    torch.cuda.synchronize()
    o, l = to_host(out), to_host(lse)
    compare(np.concatenate([o[b, :counts[b]] for b in range(B)]),
            np.concatenate([l[b, :counts[b]] for b in range(B)]), ref, "padded")
    for b in range(B):
        assert (o[b, counts[b]:] == 9).all()


@pytest.mark.parametrize("n,Hq", [(3, 4), (2000, 8)])
def test_chunk_offsets_past_32_bits(cc, n, Hq):  # noqa: F811
    """A pool of few pages a long stride apart: written by rotary_append, read by
    chunk_attention with few rows and with many."""
    import torch

    D, page, L = 64, 512, 2010
    say(f"chunk far pages n={n}")
    rng = np.random.default_rng(12)
    stride = (1 << 31) + 64  # elements; page 3 starts past 2^32 elements
    pool = torch.empty(3 * stride + page * D, dtype=torch.bfloat16, device="cuda")
    kd = pool.as_strided((4, 1, page, D), (stride, page * D, D, 1))
    k, k64 = dev(rng.standard_normal((4, 1, page, D)), "bf16")
    kd.copy_(k)
    table = np.array([[3, 1, 2, 0]], np.int32)
    q, q64 = dev(rng.standard_normal((n, Hq, D)), "bf16")
    w = torch.zeros(1, 1, 4 * page, device="cuda")
    out, lse = cc.chunk_attention(q, kd, kd, ints(table), ints([L]), row_starts=ints([0, n]),
                                  weight_sum=w)
    torch.cuda.synchronize()
    ref, rw, rb = Q.chunk([q64], k64, k64, table, [L], [n], page, 0, D ** -0.5, "bf16")
    compare(to_host(out), to_host(lse), ref, "far")
    R.check(to_host(w), rw, rb, "weights")
    f = cc.rotary_frequencies(D, device="cuda")
    rows, r64 = dev(rng.standard_normal((3, 2, D)), "bf16")
    slots, pos = [3 * page + 5, 7, 4 * page - 1], np.array([9, 200, 31])
    v = torch.zeros(4, 1, page, D, dtype=torch.bfloat16, device="cuda")
    v = pool.new_empty(3 * stride + page * D).as_strided(kd.shape, kd.stride()).copy_(v)
    cc.rotary_append(None, rows[:, :1], rows[:, 1:], ints(pos), ints(slots), f, kd, v)
    want, bound = Q.turned(r64, pos, to_host(f), 0, 1.0, "bf16")
    kw, kb, vw = k64.copy(), np.zeros(k64.shape), np.zeros(k64.shape)
    for i, t in enumerate(slots):
        kw[t // page, :, t % page], kb[t // page, :, t % page] = want[i, :1], bound[i, :1]
        vw[t // page, :, t % page] = r64[i, 1:]
    R.check(to_host(kd), kw, kb, "k")
    assert np.array_equal(to_host(v), vw)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("n,Hq,H,D", [(5, 4, 2, 64), (300, 16, 4, 128), (330, 32, 8, 96)])
def test_chunk_rows_that_do_not_exist(cc, dt, n, Hq, H, D):  # noqa: F811
    """row_starts that go on past the rows of the call: those that exist have the places that
    their sequence's full count gives them."""
    import torch

    say(f"chunk cut rows {dt} n={n}")
    rng = np.random.default_rng(n)
    lengths, counts, page, cut = [n + 900, n + 20], [n - 1, n], 16, n // 2
    c = Cache(rng, 2, H, D, page, lengths, dt)
    x = rng.standard_normal((sum(counts), Hq, D))
    live = sum(counts) - cut
    q, q64 = dev(x[:live], dt)
    w = torch.zeros(2, H, c.table.shape[1] * page, device="cuda")
    out = guarded(torch.full((live, Hq, D), 9.0, dtype=q.dtype, device="cuda"))
    lse = guarded(torch.full((live, Hq), 9.0, device="cuda"))
    cc.chunk_attention(q, c.kd, c.vd, c.td, c.ld, row_starts=ints([0, n - 1, 2 * n - 1]), n=n,
                       weight_sum=w, out=out, lse=lse)
    torch.cuda.synchronize()
    ref, rw, rb = Q.chunk([q64[:n - 1], q64[n - 1:]], c.k, c.v, c.table, lengths, counts, page, 0,
                          D ** -0.5, dt)
    compare(to_host(out), to_host(lse), ref, "cut")
    R.check(to_host(w), rw, rb, "weights")


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("n,Hq,H,extra", [(6, 4, 2, 0), (90, 4, 2, 0), (150, 32, 16, 992)])
def test_chunk_attention_missing_pages_and_long_lengths(cc, dt, n, Hq, H, extra):  # noqa: F811
    """Table entries outside the pool, lengths outside the table, a negative scale, strided rows
    of q and out, a bound max_length, row starts outside the rows."""
    import torch

    say(f"chunk missing pages {dt} n={n}")
    B, D, page = 5, 64, 16
    cap = 160 + extra
    rng = np.random.default_rng(5)
    c = Cache(rng, B, H, D, page, np.full(B, cap), dt)
    c.table[0, 3], c.table[2, 0], c.table[2, 9] = -1, -2 ** 31, 2 ** 31 - 1
    c.table[1, :] = 10 ** 6
    td = ints(c.table)
    given = np.array([cap, cap, 2 ** 31 - 1, -5, cap + 1], np.int32)
    counts = [n, n - 1, n, 2, n]
    big, b64 = dev(rng.standard_normal((B, n, 3 * Hq, D)), dt)
    q = big[:, :, Hq:2 * Hq]
    q64 = [b64[b, :counts[b], Hq:2 * Hq] for b in range(B)]
    for most in (cap, cap - 10):
        ref, w, wb = Q.chunk(q64, c.k, c.v, c.table, given, counts, page, 0, -0.1, dt, most)
        wide = torch.full((B, n, 2 * Hq, D), 9.0, dtype=q.dtype, device="cuda")
        wd = torch.zeros(B, H, cap, device="cuda")
        _, lse = cc.chunk_attention(q, c.kd, c.vd, td, ints(given), counts=ints(counts),
                                    max_length=most, scale=-0.1, weight_sum=wd,
                                    out=wide[:, :, Hq:])
        torch.cuda.synchronize()
        o, l = to_host(wide), to_host(lse)
        compare(np.concatenate([o[b, :counts[b], Hq:] for b in range(B)]),
                np.concatenate([l[b, :counts[b]] for b in range(B)]), ref, "strided")
        assert (o[:, :, :Hq] == 9).all()
        R.check(to_host(wd), w, wb, "weights")
    # starts outside the rows: nothing of those sequences exists, the rest is as it was
    flat = q[0].contiguous()
    starts = ints([-n, 0, n, n + 5, 2 ** 31 - 1, -2 ** 31])
    out = torch.full_like(flat, 9.0)
    cc.chunk_attention(flat, c.kd, c.vd, ints(np.roll(c.table, 1, 0)), ints([cap] * B),
                       row_starts=starts, n=n, scale=-0.1, out=out)
    torch.cuda.synchronize()
    ref, _, _ = Q.chunk([to_host(flat)], c.k, c.v, c.table[:1], [cap], [n], page, 0, -0.1, dt)
    R.check(to_host(out), ref[0][0], ref[0][2], "first only")


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("n,G,window", [(7, 2, 0), (9, 1, 4), (100, 1, 0), (40, 4, 0), (90, 2, 20),
                                        (700, 16, 0), (900, 16, 150)])
def test_chunk_attention_odd_values_reach_only_who_sees_them(cc, dt, n, G, window):  # noqa: F811
    """Infinities and NaN in keys and values of new slots: rows before them are as without."""
    import torch

    say(f"chunk odd values {dt} n={n} G={G} window={window}")
    rng = np.random.default_rng(n)
    D, page, H = 64, 16, 1
    L = n + 100
    c = Cache(rng, 1, H, D, page, [L], dt)
    q, starts, q64 = packed([rng.standard_normal((n, G * H, D))], 0, dt)
    ref, _, _ = Q.chunk(q64, c.k, c.v, c.table, [L], [n], page, window, 0.1, dt)
    at = L - n // 2 - 1  # seen from row n - n // 2 - 1 on, for `window` rows
    p, o = c.table[0, at // page], at % page
    first = n - n // 2 - 1
    last = n if not window else min(n, first + window)
    for what in ("nan v", "inf v", "-inf v", "nan k"):
        k, v = c.kd.clone(), c.vd.clone()
        (k if what == "nan k" else v)[p, 0, o, 5] = float(what.split()[0])
        out, lse = cc.chunk_attention(q, k, v, c.td, c.ld, row_starts=starts, n=n, window=window,
                                      scale=0.1)
        torch.cuda.synchronize()
        got = to_host(out)
        mine = np.zeros(n, bool)
        mine[first:last] = True
        assert np.isfinite(got[~mine]).all(), what
        R.check(got[~mine], ref[0][0][~mine], ref[0][2][~mine], what)
        if what == "nan k":
            assert np.isnan(got[mine]).all()
        elif what == "nan v":
            assert np.isnan(got[mine][..., 5]).all()
        else:
            assert (got[mine][..., 5] == float(what.split()[0])).all()
        if what != "nan k":
            rest = np.delete(got, 5, -1)
            R.check(rest, np.delete(ref[0][0], 5, -1), np.delete(ref[0][2], 5, -1), what)


# ---------------------------------------------------------------------------
# Together, captured, on other streams
# ---------------------------------------------------------------------------


def test_steps_of_a_serving_batch(cc):  # noqa: F811
    """Requests come with prompts, go on row by row, end; their pages come from one pool: every
    row's attention is that of the whole history in float64, and eviction takes it from there."""
    import torch

    say("serving steps")
    dt, Hq, H, D, page, cols, P, S = "f32", 4, 2, 64, 8, 8, 40, 6
    rng = np.random.default_rng(8)
    f = cc.rotary_frequencies(D, 10000.0, device="cuda")
    f64 = to_host(f)
    kc = torch.full((P, H, page, D), float("nan"), device="cuda")
    vc = kc.clone()
    table = torch.full((S, cols), -1, dtype=torch.int32, device="cuda")
    held, lengths, now = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(3))
    free = torch.arange(P, dtype=torch.int32, device="cuda")
    count = torch.tensor([P], dtype=torch.int32, device="cuda")
    pos = torch.zeros(S, H, cols * page, dtype=torch.int32, device="cuda")
    wsum = torch.full((S, H, cols * page), 7.0, device="cuda")
    past = [[np.zeros((0, H, D)), np.zeros((0, H, D))] for _ in range(S)]
    drawn = [np.zeros((H, cols * page)) for _ in range(S)]
    seen = [0] * S
    plan = [[9, 3, 0, 20, 0, 1], [1, 1, 5, 1, 0, 1], [1, -1, 1, 1, 30, 1], [2, 17, 1, -1, 1, 1],
            [1, 1, 1, 12, 1, 1], [-1, 1, 1, 1, 1, 40], [1, 1, 1, 1, 1, 1]]
    rows = 64
    for step in plan:
        new = [max(v, 0) for v in step]
        for b, v in enumerate(step):
            if v < 0:  # ended
                past[b], seen[b] = [np.zeros((0, H, D)), np.zeros((0, H, D))], 0
                drawn[b][:] = 0
                lengths[b] = 0
                now[b] = 0
        lengths += ints(new)
        now += ints(new)
        starts, at, to = cc.cache_pages(table, held, free, count, lengths, page_size=page,
                                        counts=ints(new), now=now, rows=rows, positions=pos,
                                        weight_sum=wsum)
        qkv, x = dev(rng.standard_normal((rows, Hq + 2 * H, D)), dt)
        q = cc.rotary_append(qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], at, to, f, kc, vc)
        out, lse = cc.chunk_attention(q, kc, vc, table, lengths, row_starts=starts, n=40,
                                      weight_sum=wsum)
        torch.cuda.synchronize()
        assert np.array_equal(held.cpu().numpy(), -(-lengths.cpu().numpy() // page))
        used = np.concatenate([table[b, :int(held[b])].cpu().numpy() for b in range(S)])
        rest = free[:int(count)].cpu().numpy()
        assert sorted([*used, *rest]) == list(range(P))
        r = 0
        for b, n in enumerate(new):
            where = np.arange(seen[b], seen[b] + n)
            x_q, _ = Q.turned(x[r:r + n, :Hq], where, f64, 0, 1.0, dt)
            x_k, _ = Q.turned(x[r:r + n, Hq:Hq + H], where, f64, 0, 1.0, dt)
            past[b] = [np.concatenate([past[b][0], x_k]), np.concatenate([past[b][1], x[r:r + n, Hq + H:]])]
            for i in range(n):
                e = seen[b] + i + 1
                for h in range(H):
                    g = slice(h * 2, h * 2 + 2)
                    (o, l, p), (bo, bl, _) = R.attend(x_q[i, g], past[b][0][:e, h], past[b][1][:e, h],
                                                      D ** -0.5, dt)
                    # the turned queries and keys are off by 20 e of |u| + |v| each: the scores by
                    # 2 * 2 * 20 e sum |q||k| at most
                    ds = 80 * R.E * D ** -0.5 * (np.abs(x_q[i, g]) @ np.abs(past[b][0][:e, h]).T).max() * 2
                    more = 2 * ds * (p @ np.abs(past[b][1][:e, h]))
                    R.check(to_host(out[r + i, g]), o, bo + more, "")
                    R.check(to_host(lse[r + i, g]), l, bl + ds, "")
                    drawn[b][h, :e] += p.sum(0)
            seen[b] += n
            r += n
    for b in range(S):
        n = seen[b]
        got = to_host(wsum)[b, :, :n]
        assert np.allclose(got, drawn[b][:, :n], rtol=1e-4, atol=1e-5)
        assert np.array_equal(pos.cpu().numpy()[b, :, :n], np.broadcast_to(np.arange(n), (H, n)))
    before = [int(v) for v in lengths]
    cc.cache_evict(kc, vc, table, lengths, wsum, 10, positions=pos, now=now, sink=1, recent=4)
    free_before = int(count)
    cc.cache_pages(table, held, free, count, lengths, page_size=page)
    torch.cuda.synchronize()
    assert [int(v) for v in lengths] == [min(10, v) for v in before]
    assert int(count) == free_before + sum(-(-v // page) - -(-min(10, v) // page) for v in before)


def test_captured_and_on_another_stream(cc):  # noqa: F811
    """The calls of a step recorded into a graph and replayed with other lengths; two calls with
    workspaces of their own on two streams at once."""
    import torch

    say("captured")
    dt, B, Hq, H, D, page, cols, n = "bf16", 3, 8, 2, 64, 16, 40, 40
    rng = np.random.default_rng(2)
    lengths = [600, 333, 90]
    c = Cache(rng, B, H, D, page, [cols * page] * B, dt)
    f = cc.rotary_frequencies(D, 10000.0, device="cuda")
    rows = 100
    x, _ = dev(rng.standard_normal((rows, Hq + 2 * H, D)), dt)
    P = c.kd.shape[0]
    held, ld, kd = ints([cols] * B), ints(lengths), ints([40, 3, 40])
    free, count = ints(np.arange(P)), ints([0])
    ho, co = torch.empty_like(held), torch.empty_like(count)
    starts, at, to = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (B + 1, rows, rows))
    td = c.td.clone()
    qo = torch.zeros(rows, Hq, D, dtype=x.dtype, device="cuda")
    out, lse = torch.zeros_like(qo), torch.zeros(rows, Hq, device="cuda")
    kc, vc = c.kd.clone(), c.vd.clone()
    code = cc.CTCONV_BF16
    row = tuple(x.stride()[:2])
    tables_ = cc.CachePages(B, rows, P, page, cols)
    turn = cc.RotaryAppend(rows, Hq, H, D, P, page, dtype=code, q_strides=row, new_strides=row)
    attend = cc.ChunkAttention(B, rows, n, Hq, H, D, P, page, cols, dtype=code)
    ws = torch.empty(max(attend.workspace_bytes, 16), dtype=torch.uint8, device="cuda")
    es = x.element_size()

    def step():
        s = torch.cuda.current_stream().cuda_stream
        tables_(ld.data_ptr(), kd.data_ptr(), None, held.data_ptr(), count.data_ptr(),
                td.data_ptr(), free.data_ptr(), ho.data_ptr(), co.data_ptr(), starts.data_ptr(),
                at.data_ptr(), to.data_ptr(), None, None, s)
        turn(x.data_ptr(), x.data_ptr() + Hq * D * es, x.data_ptr() + (Hq + H) * D * es,
             at.data_ptr(), to.data_ptr(), f.data_ptr(), qo.data_ptr(), kc.data_ptr(),
             vc.data_ptr(), s)
        attend(qo.data_ptr(), kc.data_ptr(), vc.data_ptr(), td.data_ptr(), ld.data_ptr(),
               starts.data_ptr(), None, out.data_ptr(), lse.data_ptr(), None, ws.data_ptr(),
               ws.numel(), s)

    def eager(lens, counts):
        ld.copy_(ints(lens))
        kd.copy_(ints(counts))
        kc.copy_(c.kd)
        vc.copy_(c.vd)
        out.zero_()
        step()
        torch.cuda.synchronize()
        return out.clone(), kc.clone()

    cases = [([600, 333, 90], [40, 3, 40]), ([100, 640, 64], [40, 1, 20]), ([640, 1, 40], [1, 1, 40])]
    want = [eager(*v) for v in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for turn_ in range(2):
        for (lens, counts), (o, k) in zip(cases, want):
            ld.copy_(ints(lens))
            kd.copy_(ints(counts))
            kc.copy_(c.kd)
            vc.copy_(c.vd)
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, o) and torch.equal(torch.nan_to_num(kc), torch.nan_to_num(k))
    # two streams
    ld.copy_(ints(cases[0][0]))
    kd.copy_(ints(cases[0][1]))
    kc.copy_(c.kd)
    vc.copy_(c.vd)
    step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        res = [cc.chunk_attention(qo, kc, vc, td, ld, row_starts=starts, n=n, stream=s) for s in streams]
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for o, _ in res:
            assert torch.equal(o[:83], want[0][0][:83])


def test_helpers_refuse(cc):  # noqa: F811
    import torch

    z = torch.zeros
    t32 = dict(dtype=torch.int32, device="cuda")
    q, k = z(4, 2, 64, device="cuda"), z(3, 2, 8, 64, device="cuda")
    table, one, four = z(1, 3, **t32), z(1, **t32), z(4, **t32)
    f = cc.rotary_frequencies(64, device="cuda")
    bad = [
        lambda: cc.cache_pages(table.cpu(), one, one, one, one),
        lambda: cc.cache_pages(table, four, one, one, one),
        lambda: cc.cache_pages(table, one, one, four, one),
        lambda: cc.cache_pages(table, one, one, one, None),
        lambda: cc.cache_pages(table, one, one, one, one, counts=one),
        lambda: cc.cache_pages(table, one, one, one, one, weight_sum=z(1, 1, 48, device="cuda")),
        lambda: cc.cache_pages(table, one, one, one, one, counts=one, rows=1,
                               weight_sum=z(1, 1, 47, device="cuda")),
        lambda: cc.rotary(None, None, four, f),
        lambda: cc.rotary(q, q[:3], four, f),
        lambda: cc.rotary(q, q, one, f),
        lambda: cc.rotary(q, q, four, f.float()),
        lambda: cc.rotary(q, q, four, f.cpu()),
        lambda: cc.rotary(q, q, four, f, q_out=z(4, 2, 32, device="cuda")),
        lambda: cc.rotary(q, q.half(), four, f),
        lambda: cc.rotary(q.transpose(1, 2), None, four, f),
        lambda: cc.rotary_append(q, None, q, four, four, f, k, k),
        lambda: cc.rotary_append(q, q, q[:, :1], four, four, f, k, k),
        lambda: cc.rotary_append(q, q, q, four, None, f, k, k),
        lambda: cc.rotary_append(q, q, q, four, four, f, k[:, :1], k[:, :1]),
        lambda: cc.rotary_append(q, q, q, four, four, f, k, k.half()),
        lambda: cc.chunk_attention(q.cpu(), k, k, table, one, row_starts=z(2, **t32)),
        lambda: cc.chunk_attention(q, k, k, table, one),
        lambda: cc.chunk_attention(q, k, k, table, one, row_starts=one),
        lambda: cc.chunk_attention(q, k, k, table, one, row_starts=z(2, **t32), counts=one),
        lambda: cc.chunk_attention(q, k, k, table, four, row_starts=z(2, **t32)),
        lambda: cc.chunk_attention(q[None].repeat(2, 1, 1, 1), k, k, table, one),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            say(f"accepted {i}")
    with pytest.raises(cc.CtconvError):
        cc.rotary(q, q, four, f, layout=2)
    with pytest.raises(cc.CtconvError):
        cc.chunk_attention(q, k, k, table, one, row_starts=z(2, **t32), max_length=25)
    with pytest.raises(cc.CtconvError):
        cc.rotary_frequencies(63)
    with pytest.raises(cc.CtconvError):
        cc.rotary_frequencies(64, scaling=cc.ROTARY_RAMP_TURNS, low=4.0, high=4.0)
