"""GPU: eviction where slots have no page.  Such a slot has no row: it stays
where it is or is given up, and every slot that is left with a page holds the
key, value, weight and position of one and the same row."""

import numpy as np
import pytest

import block_ref as R
from gpu_util import say, to_host
from test_gpu_block import DTS, Cache, cc, dev, ints  # noqa: F401 (cc: a fixture)

pytestmark = pytest.mark.gpu


def kept_rows(has_page, weights, positions, n, keep, sink, seen, recent):
    """The slots that stay, of n, as the rule says it: as many as fit, of those
    with a page, protected ones first, then by weight, ties by the lower slot."""
    m = min(n, keep)
    fixed = [t for t in range(m) if not has_page[t]]
    free = [t for t in range(n) if has_page[t]]
    safe = [t for t in free if positions[t] < sink or positions[t] >= seen - recent]
    rest = [t for t in free if not (positions[t] < sink or positions[t] >= seen - recent)]
    rest.sort(key=lambda t: (-float(weights[t]), t))
    return set(fixed) | set((safe + rest)[:m - len(fixed)])


GAPS = [
    # B, H, D, page, lengths, keep, sink, recent, share of the pages missing
    (3, 2, 64, 16, [333, 200, 250], 200, 4, 16, 0.3),    # one kernel, one slot per thread
    (2, 2, 32, 7, [700, 699], 500, 0, 90, 0.5),
    (2, 1, 16, 1, [900, 1000], 300, 2, 0, 0.4),          # single slots missing
    (2, 2, 64, 16, [3000, 1500], 1000, 4, 64, 0.2),      # four slots per thread
    (1, 2, 8, 3, [9001], 4000, 1, 100, 0.6),             # two kernels, pages end inside a group
    (2, 1, 8, 512, [40000, 5], 9000, 0, 600, 0.3),
    (2, 2, 16, 16, [300, 280], 200, 0, 8, 1.0),          # no page at all
    (1, 1, 8, 1, [6000], 3000, 5000, 0, 0.3),            # more protected than stay
]


def run(cc, c, td, w, pos, now, lengths, keep, sink, recent, page, place):  # noqa: F811
    import torch

    B, H, cap = w.shape
    D = c.kd.shape[3]
    code = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[c.kd.dtype]
    wd, pd, ld, nd = torch.from_numpy(w).cuda(), ints(pos), ints(lengths), ints(now)
    so = ints(np.full((B, H, keep), 9))
    if place:
        wo, po, lo, out = wd, pd, ld, (H * cap, cap)
    else:
        wo, po, lo, out = (torch.full((B, H, keep), 3.0, device="cuda"),
                           ints(np.full((B, H, keep), 9)), ints(np.full(B, 9)), None)
    plan = cc.CacheEvict(B, H, D, c.kd.shape[0], page, td.shape[1], keep, max(lengths), sink, recent,
                         code, out_slot_strides=out)
    plan(c.kd.data_ptr(), c.vd.data_ptr(), td.data_ptr(), ld.data_ptr(), nd.data_ptr(),
         wd.data_ptr(), pd.data_ptr(), wo.data_ptr(), po.data_ptr(), lo.data_ptr(), so.data_ptr(),
         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return wo, po, lo, so


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("place", [False, True])
@pytest.mark.parametrize("case", GAPS, ids=[str(i) for i in range(len(GAPS))])
def test_evict_without_pages(cc, case, place, dt):  # noqa: F811
    B, H, D, page, lengths, keep, sink, recent, share = case
    say(f"evict gaps {case} in place={place} {dt}")
    rng = np.random.default_rng(61)
    c = Cache(rng, B, H, D, page, lengths, dt)
    P, cols = c.kd.shape[0], c.table.shape[1]
    cap = cols * page
    lost = rng.random((B, cols)) < share
    c.table[lost] = rng.choice([-1, -2 ** 31, P, 2 ** 31 - 1], int(lost.sum()))
    has = np.repeat((c.table >= 0) & (c.table < P), page, 1)
    w = rng.integers(0, 2000, (B, H, cap)).astype(np.float32)  # some equal
    w[rng.random(w.shape) < 0.02] = -np.inf
    w[~np.broadcast_to(has[:, None], w.shape)] += 10 ** 6      # the heaviest have no page
    pos = np.stack([rng.permutation(cap) for _ in range(B * H)]).reshape(B, H, cap).astype(np.int32)
    now = np.asarray(lengths, np.int32)
    wo, po, lo, so = run(cc, c, ints(c.table), w, pos, now, lengths, keep, sink, recent, page, place)
    src, gw, gp = so.cpu().numpy(), wo.cpu().numpy(), po.cpu().numpy()
    k, v = to_host(c.kd), to_host(c.vd)
    kept_k = c.k.copy()
    kept_v = c.v.copy()
    for b, n in enumerate(lengths):
        m = min(n, keep)
        assert lo.cpu().numpy()[b] == m
        at = np.arange(m)
        for h in range(H):
            s = src[b, h, :m]
            assert set(s.tolist()) == kept_rows(has[b], w[b, h], pos[b, h], n, keep, sink, n, recent)
            moved = s != at
            assert has[b, at[moved]].all() and has[b, s[moved]].all()
            assert (s[moved] >= m).all() and (np.diff(s[moved]) > 0).all()
            assert np.array_equal(gw[b, h, :m], w[b, h, s])
            assert np.array_equal(gp[b, h, :m], pos[b, h, s])
            assert (src[b, h, m:] == -1).all()
            if not place:
                assert (gw[b, h, m:] == 0).all() and (gp[b, h, m:] == -1).all()
            for j in at[moved]:
                p1, p0 = c.table[b, j // page], c.table[b, s[j] // page]
                kept_k[p1, h, j % page] = c.k[p0, h, s[j] % page]
                kept_v[p1, h, j % page] = c.v[p0, h, s[j] % page]
    # moved rows and nothing else
    assert np.array_equal(k, kept_k, equal_nan=True) and np.array_equal(v, kept_v, equal_nan=True)


def test_attention_after_eviction_without_pages(cc):  # noqa: F811
    """What attention sees after the eviction are the rows that stayed."""
    import torch

    B, H, D, page, keep, n = 1, 2, 64, 16, 128, 250
    say("attention after eviction with gaps")
    rng = np.random.default_rng(67)
    c = Cache(rng, B, H, D, page, [n], "f32")
    c.table[0, 3] = -1
    c.table[0, 14] = 10 ** 6  # slots 224 .. 239: recent ones are lost
    has = np.repeat((c.table[0] >= 0) & (c.table[0] < c.kd.shape[0]), page)
    cap = has.size
    w = rng.random((B, H, cap)).astype(np.float32)
    td, ld, wd = ints(c.table), ints([n]), torch.from_numpy(w).cuda()
    cc.cache_evict(c.kd, c.vd, td, ld, wd, keep, recent=20)
    q, q64 = dev(rng.standard_normal((B, H, D)), "f32")
    out, _ = cc.paged_attention(q, c.kd, c.vd, td, ld)
    torch.cuda.synchronize()
    for h in range(H):
        rows = [t for t in sorted(kept_rows(has, w[0, h], np.arange(n), n, keep, 0, n, 20)) if has[t]]
        k = np.stack([c.k[c.table[0, t // page], h, t % page] for t in rows])
        v = np.stack([c.v[c.table[0, t // page], h, t % page] for t in rows])
        (o, _, _), (bo, _, _) = R.attend(q64[0, h:h + 1], k, v, D ** -0.5, "f32")
        R.check(to_host(out)[0, h:h + 1], o, bo, "out")
