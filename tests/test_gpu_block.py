"""GPU: the decoder-block operators against their plain float64 forms
(block_ref.py), at the sizes, masks, strides and orders where they can go
wrong.  Slots and rows that must not be used hold NaN."""

import numpy as np
import pytest

import block_ref as R
from gpu_util import say, to_host, torch_dtype

pytestmark = pytest.mark.gpu

DTS = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def cc():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from vision_upsampler_decoders_amd import ctconv

    ctconv.load()
    return ctconv


def dev(a, dt):
    """numpy -> device tensor of type dt, and the float64 values it holds."""
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a)).to(torch_dtype(dt)).cuda()
    return t, to_host(t)


def ints(a):
    import torch

    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def guarded(t, pad=4096):
    """t inside a NaN-filled buffer (same strides order, contiguous)."""
    import torch

    buf = torch.full((t.numel() + 2 * pad,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[pad:pad + t.numel()].view(t.shape)
    v.copy_(t)
    return v


class Cache:
    """A paged cache with its pages in random order, every unused slot NaN."""

    def __init__(self, rng, B, H, D, page, lengths, dt, layout="library", spare=2, cols=None):
        import torch

        self.page, self.lengths = page, np.asarray(lengths, np.int64)
        need = int(max(1, -(-int(max(self.lengths.max(), 1)) // page)))
        cols = need if cols is None else cols
        P = B * cols + spare
        self.table = rng.permutation(P)[:B * cols].reshape(B, cols).astype(np.int32)
        k = np.full((P, H, page, D), np.nan)
        v = np.full((P, H, page, D), np.nan)
        for b in range(B):
            for t in range(min(int(self.lengths[b]), cols * page)):
                k[self.table[b, t // page], :, t % page] = rng.standard_normal((H, D))
                v[self.table[b, t // page], :, t % page] = rng.standard_normal((H, D))
        self.kd, self.k = dev(k, dt)
        self.vd, self.v = dev(v, dt)
        if layout == "slots":  # [pages, page, H, D] in memory
            self.kd, self.vd = (t.transpose(1, 2).contiguous().transpose(1, 2)
                                for t in (self.kd, self.vd))
        elif layout == "both":  # k and v of a page side by side
            both = torch.stack((self.kd, self.vd), 1)
            self.kd, self.vd = both[:, 0], both[:, 1]
        self.td = ints(self.table)
        self.ld = ints(self.lengths)


PAGED = [
    # B, Hq, Hkv, D, page, lengths, window, layout
    (1, 1, 1, 8, 1, [1], 0, "library"),
    (3, 8, 8, 64, 16, [250, 0, 1], 0, "library"),
    (2, 8, 8, 64, 16, [1000, 37], 250, "slots"),
    (3, 32, 8, 128, 16, [513, 255, 256], 0, "library"),
    (2, 12, 2, 128, 24, [1300, 2049], 0, "both"),
    (2, 40, 2, 96, 7, [129, 64], 0, "slots"),
    (1, 6, 3, 80, 64, [700], 333, "library"),
    (2, 4, 4, 256, 128, [260, 31], 0, "library"),
    (1, 17, 1, 40, 5, [301], 0, "library"),
    (2, 64, 1, 32, 256, [5000, 4097], 0, "library"),
    (2, 2, 1, 200, 3, [95, 96], 1, "slots"),
]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", PAGED, ids=[str(i) for i in range(len(PAGED))])
@pytest.mark.parametrize("weights", [False, True])
def test_paged_attention(cc, case, dt, weights):
    import torch

    B, Hq, H, D, page, lengths, window, layout = case
    say(f"paged {case} {dt} weights={weights}")
    rng = np.random.default_rng(abs(hash((B, Hq, D, page))) % 1000 + 1)
    c = Cache(rng, B, H, D, page, lengths, dt, layout, cols=-(-max(lengths) // page) + 1)
    q, q64 = dev(rng.standard_normal((B, Hq, D)) * 1.5, dt)
    cap = c.table.shape[1] * page
    w0 = rng.random((B, H, cap)).astype(np.float32)
    w = torch.from_numpy(w0).cuda() if weights else None
    scale = 0.7 * D ** -0.5
    out, lse = cc.paged_attention(q, c.kd, c.vd, c.td, c.ld, window=window, scale=scale,
                                  weight_sum=w)
    torch.cuda.synchronize()
    (o, l, p), (bo, bl, bp) = R.paged(q64, c.k, c.v, c.table, c.lengths, page, window, scale, dt)
    R.check(to_host(out), o, bo, "out")
    R.check(to_host(lse), l, bl, "lse")
    if weights:
        R.check(to_host(w), w0 + p, bp + 2.0 ** -24 * (w0 + p), "weights")
        untouched = p == 0
        assert np.array_equal(to_host(w)[untouched], w0.astype(np.float64)[untouched])


@pytest.mark.parametrize("dt", DTS)
def test_paged_attention_missing_pages_and_long_lengths(cc, dt):
    """Table entries outside the pool, lengths outside the table, a negative
    scale, rows of q and out with their own strides, and a bound max_length."""
    import torch

    B, Hq, H, D, page = 5, 8, 2, 64, 16
    say(f"paged missing pages {dt}")
    rng = np.random.default_rng(5)
    lengths = np.array([160, 160, 160, 160, 160])
    c = Cache(rng, B, H, D, page, lengths, dt)
    c.table[0, 3] = -1
    c.table[1, :] = 10 ** 6
    c.table[2, 0] = -2 ** 31
    c.table[2, 9] = 2 ** 31 - 1
    td = ints(c.table)
    given = np.array([160, 160, 2 ** 31 - 1, -5, 161], np.int32)
    big, q64 = dev(rng.standard_normal((B, 3 * Hq, D)), dt)
    q, q64 = big[:, 1::3], q64[:, 1::3]
    whole = torch.full((B, 2 * Hq, D), 7.0, dtype=q.dtype, device="cuda")
    out = whole[:, ::2]
    got, lse = cc.paged_attention(q, c.kd, c.vd, td, ints(given), scale=-0.2, out=out)
    torch.cuda.synchronize()
    (o, l, _), (bo, bl, _) = R.paged(q64, c.k, c.v, c.table, given, page, 0, -0.2, dt)
    R.check(to_host(got), o, bo, "out")
    R.check(to_host(lse), l, bl, "lse")
    assert bool((whole[:, 1::2] == 7).all())
    got, _ = cc.paged_attention(q, c.kd, c.vd, td, ints(given), scale=-0.2, max_length=33)
    (o, _, _), (bo, _, _) = R.paged(q64, c.k, c.v, c.table, np.minimum(given, 33), page, 0, -0.2, dt)
    R.check(to_host(got), o, bo, "bounded")


def test_paged_attention_large_scores(cc):
    """Scores over +-10^4 with the largest ones late: the running maximum moves
    in steps that overflow any fixed reference."""
    import torch

    B, H, D, page, n = 1, 2, 64, 16, 1500
    rng = np.random.default_rng(9)
    say("paged large scores")
    c = Cache(rng, B, H, D, page, [n], "f32")
    ramp = np.linspace(-1.0, 1.0, n)
    q64 = np.ones((B, H, D))
    k = np.zeros_like(c.k)
    for t in range(n):
        k[c.table[0, t // page], :, t % page] = np.float32(160.0 * ramp[t])
    kd, k = dev(k, "f32")
    q, q64 = dev(q64, "f32")
    out, lse = cc.paged_attention(q, kd, c.vd, c.td, c.ld, scale=1.0)
    torch.cuda.synchronize()
    (o, l, _), (bo, bl, _) = R.paged(q64, k, c.v, c.table, c.lengths, page, 0, 1.0, "f32")
    R.check(to_host(out), o, bo, "out")
    R.check(to_host(lse), l, bl, "lse")


def test_paged_attention_offsets_past_32_bits(cc):
    """Pages whose byte and element offsets pass 2^32: a pool with few pages a
    long stride apart."""
    import torch

    B, Hq, H, D, page = 1, 4, 1, 64, 64
    say("paged far pages")
    rng = np.random.default_rng(11)
    stride = (1 << 31) + 64  # elements; page 3 starts past 2^32 elements
    pool = torch.empty(3 * stride + H * page * D, dtype=torch.bfloat16, device="cuda")
    kd = pool.as_strided((4, H, page, D), (stride, page * D, D, 1))
    k, k64 = dev(rng.standard_normal((4, H, page, D)), "bf16")
    kd.copy_(k)
    vpool = kd  # the same rows serve as values
    table = np.array([[3, 1, 2, 0]], np.int32)
    q, q64 = dev(rng.standard_normal((B, Hq, D)), "bf16")
    out, lse = cc.paged_attention(q, kd, vpool, ints(table), ints([250]))
    torch.cuda.synchronize()
    (o, l, _), (bo, bl, _) = R.paged(q64, k64, k64, table, [250], page, 0, D ** -0.5, "bf16")
    R.check(to_host(out), o, bo, "out")
    R.check(to_host(lse), l, bl, "lse")
    # the same pool through append
    new, new64 = dev(rng.standard_normal((1, 3, H, D)), "bf16")
    cc.cache_append(new, new, kd, kd, ints(table), ints([250]))
    want = k64.copy()
    for i, t in enumerate((247, 248, 249)):
        want[table[0, t // page], :, t % page] = new64[0, i]
    assert np.array_equal(to_host(kd), want)


def test_paged_attention_streams_workspace_and_repeats(cc):
    """Another stream than the inputs', a caller's workspace full of NaN, the
    same bits every time."""
    import torch

    B, Hq, H, D, page = 4, 16, 4, 128, 16
    rng = np.random.default_rng(13)
    say("paged streams")
    c = Cache(rng, B, H, D, page, [3000, 17, 1024, 2500], "bf16")
    q, _ = dev(rng.standard_normal((B, Hq, D)), "bf16")
    cap = c.table.shape[1] * page
    need = cc.ctconv_paged_attention_workspace_bytes(B, Hq, H, D, cap, 0, True, cc.CTCONV_BF16)
    outs = []
    side = torch.cuda.Stream()
    for rep in range(4):
        ws = torch.full((need // 4 + 1,), float("nan"), device="cuda").view(torch.uint8)
        w = torch.zeros((B, H, cap), device="cuda")
        o, l = cc.paged_attention(q, c.kd, c.vd, c.td, c.ld, weight_sum=w, workspace=ws,
                                  stream=side if rep % 2 else None)
        torch.cuda.synchronize()
        outs.append((o.clone(), l.clone(), w.clone()))
    for o in outs[1:]:
        assert all(torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                               b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))
                   for a, b in zip(o, outs[0]))
    with pytest.raises(ValueError, match="workspace"):
        cc.paged_attention(q, c.kd, c.vd, c.td, c.ld, weight_sum=w, workspace=ws[:need - 16])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("layout", ["library", "slots", "both"])
def test_cache_append(cc, dt, layout):
    import torch

    rng = np.random.default_rng(17)
    for B, n, H, D, page, lengths, counts, now in [
        (1, 1, 1, 8, 1, [1], None, None),
        (4, 1, 8, 64, 16, [17, 16, 1, 40], None, [117, 16, 1, 41]),
        (5, 37, 3, 96, 7, [40, 37, 20, 100, 0], [37, 0, 30, -4, 9], [40, 90, 20, 100, 3]),
        (2, 300, 2, 256, 64, [300, 512], [299, 1000], None),
        (3, 9, 12, 40, 24, [9, 50, 11], None, None),
    ]:
        say(f"append {dt} {layout} B={B} n={n} H={H} D={D} page={page}")
        cols = 7 if B == 5 else -(-max(lengths) // page)  # B = 5: slots past the table
        c = Cache(rng, B, H, D, page, lengths, dt, layout, cols=cols)
        if B == 5:
            c.table[0, 5] = -1
        kn, kn64 = dev(rng.standard_normal((B, n, H, D)), dt)
        vn, vn64 = dev(rng.standard_normal((B, n, H, D)), dt)
        cap = cols * page
        pos = rng.integers(0, 99, (B, H, cap)).astype(np.int32)
        w = rng.random((B, H, cap)).astype(np.float32)
        pd, wd = ints(pos), torch.from_numpy(w).cuda()
        cc.cache_append(guarded(kn), guarded(vn), c.kd, c.vd, ints(c.table), c.ld,
                        None if counts is None else ints(counts),
                        None if now is None else ints(now), pd, wd)
        torch.cuda.synchronize()
        k, v, p2, w2 = R.append(kn64, vn64, c.k, c.v, c.table, lengths, counts, now, page, pos, w)
        assert np.array_equal(to_host(c.kd), k, equal_nan=True)
        assert np.array_equal(to_host(c.vd), v, equal_nan=True)
        assert np.array_equal(pd.cpu().numpy(), p2)
        assert np.array_equal(wd.cpu().numpy(), w2)


EVICT = [
    # B, H, D, page, lengths, keep, sink, recent, kind of weights
    (1, 1, 8, 1, [1], 1, 0, 0, "random"),
    (4, 8, 64, 16, [320, 256, 257, 0], 256, 4, 32, "random"),
    (3, 2, 64, 16, [1000, 999, 128], 100, 0, 0, "ties"),
    (2, 3, 96, 24, [2000, 1500], 640, 10, 64, "level"),
    (2, 2, 128, 64, [1100, 1024], 1024, 0, 1024, "nan"),
    (2, 1, 40, 7, [130, 129], 64, 200, 0, "random"),
    (2, 2, 16, 256, [9000, 8191], 8000, 4, 128, "random"),
    (1, 2, 8, 512, [45000], 30000, 1, 100, "ties"),
    (1, 1, 8, 1024, [70001], 69000, 0, 7, "random"),
    (2, 2, 32, 16, [100, 90], 160, 0, 0, "random"),
    (2, 2, 64, 16, [513, 600], 1, 0, 0, "level"),
    (1, 1, 8, 512, [9500], 4100, 0, 0, "close"),
    (1, 1, 8, 512, [9500], 4100, 0, 0, "level"),
    (2, 1, 8, 512, [30000, 29000], 9000, 4, 9, "close"),
    (1, 1, 8, 1024, [200001], 100000, 4, 9, "ties"),
]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", EVICT, ids=[str(i) for i in range(len(EVICT))])
def test_cache_evict(cc, case, dt):
    import torch

    B, H, D, page, lengths, keep, sink, recent, kind = case
    say(f"evict {case} {dt}")
    rng = np.random.default_rng(23)
    layout = "slots" if B == 3 else "library"
    c = Cache(rng, B, H, D, page, lengths, dt, layout)
    cap = c.table.shape[1] * page
    if kind == "ties":
        w = rng.integers(0, 5, (B, H, cap)).astype(np.float32) * np.float32(0.25) - 0.5
        w[w == 0] = np.where(rng.random(int((w == 0).sum())) < 0.5, 0.0, -0.0)
    elif kind == "level":
        w = np.full((B, H, cap), 0.125, np.float32)
    elif kind == "close":  # the same upper three digits, many equal
        w = (0x3F123400 + rng.integers(0, 256, (B, H, cap))).astype(np.int32).view(np.float32)
    else:
        w = (rng.random((B, H, cap)) ** 8 * 50).astype(np.float32)
    if kind == "nan":
        at = rng.random(w.shape)
        w[at < 0.1] = np.nan
        w[(at > 0.1) & (at < 0.2)] = np.inf
        w[(at > 0.2) & (at < 0.3)] = -np.inf
        w[(at > 0.3) & (at < 0.31)] = np.finfo(np.float32).max
    pos = np.stack([rng.permutation(cap) for _ in range(B * H)]).reshape(B, H, cap).astype(np.int32)
    now = np.asarray(lengths, np.int32) + (0 if kind == "random" else 50)
    use_pos = kind != "level"
    want = R.evict(c.k, c.v, c.table, lengths, now if use_pos else None, w,
                   pos if use_pos else None, page, keep, sink, recent)
    plan = cc.CacheEvict(B, H, D, c.kd.shape[0], page, c.table.shape[1], keep, max(lengths), sink,
                         recent, {"f32": 0, "bf16": 1, "f16": 2}[dt],
                         kv_strides=(c.kd.stride(0), c.kd.stride(2), c.kd.stride(1)))
    wd, pd = torch.from_numpy(w).cuda(), ints(pos)
    wo = torch.full((B, H, keep), 3.0, device="cuda")
    po, so = ints(np.full((B, H, keep), 9)), ints(np.full((B, H, keep), 9))
    lo, nd = ints(np.full(B, 9)), ints(now)
    plan(c.kd.data_ptr(), c.vd.data_ptr(), c.td.data_ptr(), c.ld.data_ptr(),
         nd.data_ptr() if use_pos else None, wd.data_ptr(), pd.data_ptr() if use_pos else None,
         wo.data_ptr(), po.data_ptr(), lo.data_ptr(), so.data_ptr(),
         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for name, g, r in [("source", so, want[5]), ("positions", po, want[3]), ("lengths", lo, want[4])]:
        assert np.array_equal(g.cpu().numpy(), r), name
    assert np.array_equal(wo.cpu().numpy(), want[2], equal_nan=True)
    assert np.array_equal(to_host(c.kd), want[0], equal_nan=True)
    assert np.array_equal(to_host(c.vd), want[1], equal_nan=True)


# rows of slots that start anywhere and end inside a group of four; short ones beside long ones
EVICT_ODD = [
    (4, 1, 8, 7, [1030, 2, 3, 5], 1, 0, 0, "random"),
    (6, 1, 8, 7, [1030, 2, 3, 4, 1, 0], 2, 1, 0, "ties"),
    (2, 3, 8, 7, [4099, 1025], 1000, 4, 32, "nan"),
    (3, 1, 8, 13, [1039, 1037, 1038], 1030, 0, 0, "ties"),
    (1, 2, 8, 5, [8190], 4097, 3, 5, "close"),
    (2, 2, 8, 3, [4097, 2050], 2049, 0, 0, "level"),
]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", EVICT_ODD, ids=[str(i) for i in range(len(EVICT_ODD))])
def test_cache_evict_odd_rows(cc, case, dt):
    test_cache_evict(cc, case, dt)


def test_cache_evict_in_place_and_missing_pages(cc):
    """The helper's in-place form: weights, positions and lengths are updated
    in their buffers, slots from keep on stay; rows without a page do not move."""
    import torch

    B, H, D, page, keep = 3, 4, 64, 16, 200
    lengths = np.array([333, 200, 250], np.int32)
    rng = np.random.default_rng(29)
    say("evict in place")
    c = Cache(rng, B, H, D, page, lengths, "bf16")
    c.table[0, 2] = -1
    c.table[2, 14] = 10 ** 7
    cap = c.table.shape[1] * page
    w = rng.random((B, H, cap)).astype(np.float32)
    pos = np.tile(np.arange(cap, dtype=np.int32), (B, H, 1))
    want = R.evict(c.k, c.v, c.table, lengths, None, w, pos, page, keep, 4, 16)
    wd, pd, ld = torch.from_numpy(w).cuda(), ints(pos), ints(lengths)
    src = cc.cache_evict(c.kd, c.vd, ints(c.table), ld, wd, keep, positions=pd, sink=4, recent=16)
    torch.cuda.synchronize()
    assert np.array_equal(src.cpu().numpy(), want[5])
    assert np.array_equal(ld.cpu().numpy(), want[4])
    for b in range(B):
        m = want[4][b]
        assert np.array_equal(wd.cpu().numpy()[b, :, :m], want[2][b, :, :m])
        assert np.array_equal(pd.cpu().numpy()[b, :, :m], want[3][b, :, :m])
    assert np.array_equal(wd.cpu().numpy()[:, :, keep:], w[:, :, keep:])
    assert np.array_equal(to_host(c.kd), want[0], equal_nan=True)
    assert np.array_equal(to_host(c.vd), want[1], equal_nan=True)


CROSS = [
    # B, Lq, Lk, Hq, Hkv, D, lengths, mask
    (1, 1, 1, 1, 1, 8, None, None),
    (3, 1, 700, 16, 16, 64, [700, 0, 333], None),
    (2, 1, 1501, 12, 4, 128, None, "random"),
    (2, 5, 77, 8, 8, 64, [77, 3], "random"),
    (2, 33, 129, 6, 2, 96, None, "row"),
    (1, 100, 300, 4, 4, 128, None, None),
    (2, 257, 65, 3, 1, 80, [64, 1], None),
    (1, 63, 1000, 2, 2, 256, None, "random"),
    (1, 300, 190, 8, 2, 32, [190], "head"),
    (2, 4, 0, 2, 2, 64, None, None),
    (1, 3, 4100, 8, 1, 40, None, "random"),
    (1, 130, 2500, 2, 1, 128, [2300], None),
    (1, 17, 64, 2, 2, 200, None, None),
]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", CROSS, ids=[str(i) for i in range(len(CROSS))])
def test_cross_attention(cc, case, dt):
    import torch

    B, Lq, Lk, Hq, H, D, lengths, mask = case
    say(f"cross {case} {dt}")
    rng = np.random.default_rng(31)
    q, q64 = dev(rng.standard_normal((B, Lq, Hq, D)) * 1.5, dt)
    k, v = rng.standard_normal((2, B, Lk, H, D))
    m = None
    if mask is not None:
        m = rng.random((B, Lk)) < 0.6
        if mask == "row":
            m[0] = False
        if mask == "head":
            m[:, :100] = False
    gone = np.zeros((B, Lk), bool)
    if lengths is not None:
        gone |= np.arange(Lk)[None] >= np.asarray(lengths)[:, None]
    if m is not None:
        gone |= ~m
    k[gone], v[gone] = np.nan, np.inf
    (kd, k64), (vd, v64) = dev(k, dt), dev(v, dt)
    out, lse = cc.cross_attention(guarded(q), guarded(kd), guarded(vd),
                                  None if lengths is None else ints(lengths),
                                  None if m is None else torch.from_numpy(m).cuda())
    torch.cuda.synchronize()
    (o, l), (bo, bl) = R.cross(q64, k64, v64, lengths, m, D ** -0.5, dt)
    R.check(to_host(out), o, bo, "out")
    R.check(to_host(lse), l, bl, "lse")


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("Lq", [1, 150])
def test_cross_attention_strides_and_repeats(cc, dt, Lq):
    """q, k and v as slices of one projection, heads before rows in the output,
    a mask with a stride of its own; the same bits twice."""
    import torch

    B, Lk, H, D = 2, 333, 4, 64
    rng = np.random.default_rng(37)
    say(f"cross strides {dt} {Lq}")
    kv, kv64 = dev(rng.standard_normal((B, Lk, 3, H, D)), dt)
    qq, qq64 = dev(rng.standard_normal((Lq, B, 2 * H, D)), dt)
    q, q64 = qq.transpose(0, 1)[:, :, H:], qq64.transpose(1, 0, 2, 3)[:, :, H:]
    m = rng.random((B, 2 * Lk + 1)) < 0.5
    md = torch.from_numpy(m).cuda()
    got = []
    for _ in range(2):
        buf = torch.full((B, H, Lq, D), float("nan"), dtype=q.dtype, device="cuda")
        out, lse = cc.cross_attention(q, kv[:, :, 0], kv[:, :, 2], mask=md[:, 3:3 + Lk], scale=-0.3,
                                      out=buf.transpose(1, 2))
        torch.cuda.synchronize()
        got.append((buf, lse))
    (o, l), (bo, bl) = R.cross(q64, kv64[:, :, 0], kv64[:, :, 2], None, m[:, 3:3 + Lk], -0.3, dt)
    R.check(to_host(out), o, bo, "out")
    R.check(to_host(lse), l, bl, "lse")
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


NORM = [
    # rows, C, post, pre, gate_fn, rows_per_gate
    (1, 1, 1, 2, 0, 1), (8, 512, 0, 2, 0, 1), (5, 64, 2, 1, 1, 1), (7, 65, 1, 2, 2, 3),
    (3, 2048, 1, 1, 2, 1), (9, 1000, 2, 2, 3, 4), (2, 4097, 2, 1, 2, 5), (3, 8192, 1, 2, 1, 1),
    (2, 16384, 2, 2, 2, 1), (300, 24, 0, 0, 3, 7), (4, 16383, 1, 1, 0, 1), (6, 520, 1, 0, 2, 2),
    (2, 4104, 0, 1, 0, 1), (3, 1032, 2, 1, 1, 2), (257, 7, 1, 2, 2, 100),
]


def _norm_bound(dt, C, ref, mag):
    """One rounding of the result and, relative to the magnitudes that went
    into it, (C + 64) e for the fp32 sums behind a norm and the functions."""
    return R.U[dt] * np.abs(ref) + (C + 64) * R.E * mag + 1e-30


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", NORM, ids=[str(i) for i in range(len(NORM))])
def test_norm_residual(cc, case, dt):
    import torch

    rows, C, post, pre, fn, per = case
    say(f"norm {case} {dt}")
    rng = np.random.default_rng(41)
    x, x64 = dev(rng.standard_normal((rows, C)) * 3, dt)
    h, h64 = dev(rng.standard_normal((rows, C)) + 2, dt)
    g, g64 = dev(rng.standard_normal((-(-rows // per), C)) * 4, dt) if fn else (None, None)
    some = rows % 2 == 1  # leave some channel arrays out
    par = [dev(1 + 0.1 * rng.standard_normal(C), dt) for _ in range(5)]
    pw, pb, sc, nw, nb = [None if i == (1 if some else 2) else t for i, t in enumerate(par)]
    d = lambda t: None if t is None else t[0]  # noqa: E731
    a = lambda t: None if t is None else t[1]  # noqa: E731
    xo, y = cc.norm_residual(x, h, post, d(pw), d(pb), d(sc), g, fn, per, pre, d(nw), d(nb), 1e-5)
    torch.cuda.synchronize()
    rx, ry = R.norm_residual(x64, h64, post, a(pw), a(pb), a(sc), g64, fn, per, pre, a(nw), a(nb),
                             1e-5)
    f = np.abs(rx - x64) + (0 if pb is None or not post else np.abs(a(pb))) + 1.0
    bx = _norm_bound(dt, C, rx, np.abs(x64) + 2 * f)
    R.check(to_host(xo), rx, bx, "x_out")
    if pre:
        # y scales x_out's fp32 error (before its rounding) by weight / deviation
        dev_x = np.sqrt(((rx - (rx.mean(-1, keepdims=True) if pre == 2 else 0)) ** 2)
                        .mean(-1, keepdims=True) + 1e-5)
        wmax = 1.0 if nw is None else np.abs(a(nw)).max()
        mag = (np.abs(x64) + 2 * f).max(-1, keepdims=True) / dev_x * wmax * 4 + np.abs(ry)
        R.check(to_host(y), ry, _norm_bound(dt, C, ry, mag), "y")
    # in place, another stream: the same bits
    s = torch.cuda.Stream()
    xi, hi = x.clone(), h.clone()
    cc.norm_residual(xi, hi, post, d(pw), d(pb), d(sc), g, fn, per, pre, d(nw), d(nb), 1e-5,
                     x_out=xi, y=hi if pre else None, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(xi, xo) and (not pre or torch.equal(hi, y))


def test_large_rows_past_the_caches(cc):
    """Enough rows that norms and appended rows are written past the L2 caches."""
    import torch

    say("large norm")
    g = torch.Generator(device="cuda").manual_seed(5)
    rows, C = 4200, 4104
    x, h, gate = (torch.randn(rows, C, generator=g, device="cuda").bfloat16() for _ in range(3))
    xo, y = cc.norm_residual(x, h, cc.NORM_RMS, gate=gate, gate_fn=cc.GATE_SIGMOID, pre=cc.NORM_RMS)
    pick = torch.tensor([0, 1, 63, 64, 2047, 4199], device="cuda")
    rx, ry = R.norm_residual(to_host(x[pick]), to_host(h[pick]), 1, None, None, None,
                             to_host(gate[pick]), 2, 1, 1, None, None, 1e-5)
    R.check(to_host(xo[pick]), rx, _norm_bound("bf16", C, rx, np.abs(rx) + 20), "x_out")
    R.check(to_host(y[pick]), ry, _norm_bound("bf16", C, ry, np.abs(ry) + 40), "y")
    small = cc.norm_residual(x[:64], h[:64], cc.NORM_RMS, gate=gate[:64], gate_fn=cc.GATE_SIGMOID,
                             pre=cc.NORM_RMS)
    assert torch.equal(small[0], xo[:64]) and torch.equal(small[1], y[:64])
    say("large append")
    B, n, H, D, page = 2, 2100, 8, 256, 64
    kn, vn = (torch.randn(B, n, H, D, generator=g, device="cuda") for _ in range(2))
    cols = -(-n // page)
    table = torch.randperm(B * cols).int().view(B, cols).cuda()
    k, v = (torch.zeros(B * cols, H, page, D, device="cuda") for _ in range(2))
    cc.cache_append(kn, vn, k, v, table, ints([n, n]))
    for new, cache in ((kn, k), (vn, v)):
        rows = cache[table.long()].transpose(2, 3).reshape(B, cols * page, H, D)
        assert torch.equal(rows[:, :n], new) and not bool(rows[:, n:].any())


def test_cross_attention_far_rows(cc):
    """Key and value rows so far apart that a tile of them spans over 4 GiB."""
    import torch

    B, Lq, Lk, H, D = 1, 130, 70, 1, 64
    say("cross far rows")
    rng = np.random.default_rng(53)
    stride = (1 << 26) + 64  # bf16: 64 rows span 8 GiB
    pool = torch.empty((Lk - 1) * stride + D, dtype=torch.bfloat16, device="cuda")
    kd = pool.as_strided((B, Lk, H, D), (0, stride, D, 1))
    k, k64 = dev(rng.standard_normal((B, Lk, H, D)), "bf16")
    kd.copy_(k)
    q, q64 = dev(rng.standard_normal((B, Lq, H, D)), "bf16")
    out, lse = cc.cross_attention(q, kd, kd)
    torch.cuda.synchronize()
    (o, l), (bo, bl) = R.cross(q64, k64, k64, None, None, D ** -0.5, "bf16")
    R.check(to_host(out), o, bo, "out")
    R.check(to_host(lse), l, bl, "lse")


def test_norm_residual_row_strides(cc):
    """Rows apart from each other, by strides that keep and that break the
    16-byte starts: the same bits as dense rows, nothing written between."""
    import torch

    rng = np.random.default_rng(43)
    for stride in (264, 259):
        say(f"norm strides {stride}")
        rows, C = 6, 256
        x, h, g = (torch.from_numpy(rng.standard_normal((rows, stride)).astype(np.float32))
                   .to(torch.bfloat16).cuda() for _ in range(3))
        xo, y = (torch.full((rows, stride), 7.0, dtype=torch.bfloat16, device="cuda")
                 for _ in range(2))
        plan = cc.NormResidual(rows, C, cc.NORM_RMS, cc.NORM_LAYER, cc.GATE_TANH, 1, 1e-6,
                               cc.CTCONV_BF16, (stride,) * 5)
        plan(x.data_ptr(), h.data_ptr(), None, None, None, g.data_ptr(), None, None,
             xo.data_ptr(), y.data_ptr(), torch.cuda.current_stream().cuda_stream)
        a, b = cc.norm_residual(x[:, :C], h[:, :C], cc.NORM_RMS, gate=g[:, :C].contiguous(),
                                gate_fn=cc.GATE_TANH, pre=cc.NORM_LAYER, eps=1e-6)
        torch.cuda.synchronize()
        assert bool((xo[:, C:] == 7).all()) and bool((y[:, C:] == 7).all())
        ra, rb = R.norm_residual(to_host(x[:, :C]), to_host(h[:, :C]), 1, None, None, None,
                                 to_host(g[:, :C]), 3, 1, 2, None, None, 1e-6)
        for got, dense, ref in ((xo, a, ra), (y, b, rb)):
            R.check(to_host(got[:, :C]), ref, 2.0 ** -8 * np.abs(ref) + 1e-4, "strided")
            R.check(to_host(dense), ref, 2.0 ** -8 * np.abs(ref) + 1e-4, "dense")


def test_graph_replay(cc):
    """A decode step captured once and replayed with new contents: append,
    attention with weights, cross attention, the seam and eviction take their
    lengths from the device."""
    import torch

    B, Hq, H, D, page, cols, C, Lk = 2, 8, 4, 64, 16, 20, 512, 90
    rng = np.random.default_rng(47)
    say("graph")
    dt = torch.bfloat16
    pool = B * cols
    table = ints(rng.permutation(pool).reshape(B, cols))
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dt).cuda()  # noqa: E731
    k0, v0 = mk(pool, H, page, D), mk(pool, H, page, D)
    ek, ev = mk(B, Lk, H, D), mk(B, Lk, H, D)
    w0 = torch.rand((B, H, cols * page), device="cuda")
    q, kn, vn, x, hh = mk(B, Hq, D), mk(B, 1, H, D), mk(B, 1, H, D), mk(B, C), mk(B, C)

    def state():
        return dict(k=k0.clone(), v=v0.clone(), w=w0.clone(), l=ints([300, 41]),
                    x=x.clone(), lo=ints([0, 0]))

    def step(s):
        cc.cache_append(kn, vn, s["k"], s["v"], table, s["l"], weight_sum=s["w"])
        a, lse = cc.paged_attention(q, s["k"], s["v"], table, s["l"], weight_sum=s["w"])
        c, _ = cc.cross_attention(a[:, None], ek, ev)
        xo, y = cc.norm_residual(s["x"], c.reshape(B, C))
        s["x"].copy_(xo)
        src = cc.cache_evict(s["k"], s["v"], table, s["l"], s["w"], 256, recent=16)
        s["l"].add_(1)
        return [a, lse, c, xo, y, src]

    eager, s1 = [], state()
    for _ in range(4):
        eager.append([t.clone() for t in step(s1)] + [s1[n].clone() for n in "kvwl"])
    s2 = state()
    step(state())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(s2)
    for n, t in state().items():
        s2[n].copy_(t)
    for r in range(4):
        g.replay()
        torch.cuda.synchronize()
        got = outs + [s2[n] for n in "kvwl"]
        for i, (a, b) in enumerate(zip(got, eager[r])):
            assert torch.equal(a, b), (r, i)


def test_helpers_refuse(cc):
    """Arguments that do not fit are refused before any launch."""
    import torch

    B, H, D, page, cols = 2, 2, 32, 8, 4
    cache = torch.zeros((10, H, page, D), device="cuda")
    table = ints(np.zeros((B, cols)))
    lengths = ints(np.zeros(B))
    rows = torch.zeros((B, 1, H, D), device="cuda")
    q = torch.zeros((B, H, D), device="cuda")
    x = torch.zeros((3, D), device="cuda")
    slots = torch.zeros((B, H, cols * page), device="cuda")
    enc = torch.zeros((B, 5, H, D), device="cuda")
    bad = [
        (ValueError, lambda: cc.cache_append(rows, rows, cache, cache, table, None)),
        (TypeError, lambda: cc.cache_append(rows, rows, cache, cache, table, lengths.long())),
        (ValueError, lambda: cc.cache_append(rows, rows[:, :, :1], cache, cache, table, lengths)),
        (ValueError, lambda: cc.cache_append(rows, rows, cache, cache[:, :1], table, lengths)),
        (ValueError, lambda: cc.cache_append(rows, rows, cache, cache, table[:1], lengths)),
        (ValueError, lambda: cc.cache_append(rows, rows, cache, cache, table, lengths,
                                             positions=ints(np.zeros((B, H, 3))))),
        (ValueError, lambda: cc.paged_attention(q, cache, cache, table, None)),
        (TypeError, lambda: cc.paged_attention(q.half(), cache, cache, table, lengths)),
        (ValueError, lambda: cc.paged_attention(q[..., :16], cache, cache, table, lengths)),
        (ValueError, lambda: cc.paged_attention(q, cache, cache, table, lengths.cpu())),
        (cc.CtconvError, lambda: cc.paged_attention(q, cache, cache, table, lengths, window=-1)),
        (cc.CtconvError, lambda: cc.paged_attention(q, cache, cache, table, lengths,
                                                    max_length=cols * page + 1)),
        (cc.CtconvError, lambda: cc.paged_attention(q, cache, cache, table, lengths,
                                                    scale=float("nan"))),
        (ValueError, lambda: cc.cache_evict(cache, cache, table, lengths, None, 4)),
        (ValueError, lambda: cc.cache_evict(cache, cache, table, lengths, slots, 0)),
        (ValueError, lambda: cc.cache_evict(cache, cache, table, lengths, slots, 33)),
        (TypeError, lambda: cc.cache_evict(cache, cache, table, lengths, slots.double(), 4)),
        (ValueError, lambda: cc.cross_attention(q[:, None], enc, enc[:, :4])),
        (ValueError, lambda: cc.cross_attention(q[:, None], enc, enc, mask=slots[0, :, :5] > 0,
                                                lengths=lengths[:1])),
        (TypeError, lambda: cc.cross_attention(q[:, None], enc, enc, mask=enc[:, :, 0, 0])),
        (ValueError, lambda: cc.norm_residual(x, x[:2])),
        (ValueError, lambda: cc.norm_residual(x, x, gate=x)),
        (ValueError, lambda: cc.norm_residual(x, x, gate=x, gate_fn=cc.GATE_TANH,
                                              rows_per_gate=2)),
        (ValueError, lambda: cc.norm_residual(x, x, x_out=torch.zeros((D, 3), device="cuda").t())),
        (cc.CtconvError, lambda: cc.norm_residual(x, x, eps=-1.0)),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            say(f"not refused: {i}")
