"""GPU: a NaN that attention does see reaches every result that depends on it,
whichever kernel runs and however the keys are split, and no other result."""

import numpy as np
import pytest

import block_ref as R
from gpu_util import say, to_host, torch_dtype
from test_gpu_block import DTS, cc, dev, ints  # noqa: F401 (cc: a fixture)

pytestmark = pytest.mark.gpu

CROSS = [
    # B, Lq, Lk, Hq, Hkv, D: one workgroup a row tile; split over keys; the join of many rows
    # (4096 of them); many query rows, in one piece and split
    (2, 1, 200, 4, 2, 64),
    (1, 3, 4100, 4, 1, 40),
    (64, 1, 2500, 64, 8, 64),
    (2, 100, 300, 4, 4, 128),
    (1, 130, 2500, 2, 1, 128),
]


def cross(cc, q, k, v, lengths=None, mask=None):  # noqa: F811
    import torch

    out, lse = cc.cross_attention(q, k, v, lengths, mask)
    torch.cuda.synchronize()
    return to_host(out), to_host(lse)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", CROSS, ids=[str(i) for i in range(len(CROSS))])
def test_cross_attention_nan(cc, case, dt):  # noqa: F811
    import torch

    B, Lq, Lk, Hq, H, D = case
    say(f"cross nan {case} {dt}")
    rng = np.random.default_rng(71)
    q, q64 = dev(rng.standard_normal((B, Lq, Hq, D)), dt)
    # every sequence sees the same states
    k, k64 = dev(rng.standard_normal((1, Lk, H, D)), dt)
    v, v64 = dev(rng.standard_normal((1, Lk, H, D)), dt)
    ex = lambda t: t.expand(B, Lk, H, D)  # noqa: E731
    some = min(B, 3)  # sequences that are compared value by value
    (o, l), (bo, bl) = R.cross(q64[:some], np.repeat(k64, some, 0), np.repeat(v64, some, 0), None,
                               None, D ** -0.5, dt)

    # one value of one query row
    qn = q.clone()
    qn[0, Lq // 2, Hq - 1, 3] = float("nan")
    out, lse = cross(cc, qn, ex(k), ex(v))
    assert np.isnan(out[0, Lq // 2, Hq - 1]).all() and np.isnan(lse[0, Hq - 1, Lq // 2])
    hit = np.zeros(out.shape[:3], bool)
    hit[0, Lq // 2, Hq - 1] = True
    out[hit], lse[hit.transpose(0, 2, 1)] = 0, 0
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    keep = ~hit[:some]
    R.check(out[:some][keep], o[keep], bo[keep], "the others' out")
    keep = keep.transpose(0, 2, 1)
    R.check(lse[:some][keep], l[keep], bl[keep], "the others' lse")

    # a key of head 0: its query heads, and only they; the first one, the last one, and whole
    # stretches of keys that are seen, with nothing but hidden ones before them
    G = Hq // H
    for at in (slice(0, 1), slice(Lk - 1, Lk), slice(0, Lk), slice(0, min(Lk, 64)),
               slice(Lk // 2, Lk)):
        kn = k.clone()
        kn[:, at, 0, 5] = float("nan")
        out, lse = cross(cc, q, ex(kn), ex(v))
        assert np.isnan(out[:, :, :G]).all() and np.isnan(lse[:, :G]).all(), at
        assert np.isfinite(out[:, :, G:]).all() and np.isfinite(lse[:, G:]).all(), at
        mask = torch.zeros((B, Lk), dtype=torch.bool, device="cuda")
        mask[:, at] = True
        out, lse = cross(cc, q, ex(kn), ex(v), mask=mask)
        assert np.isnan(out[:, :, :G]).all() and np.isnan(lse[:, :G]).all(), at
        assert np.isfinite(out[:, :, G:]).all() and np.isfinite(lse[:, G:]).all(), at
        # hidden, it is not seen
        out, lse = cross(cc, q, ex(kn), ex(v), mask=~mask)
        assert np.isfinite(out).all(), at
        assert np.isfinite(lse).all() or (at == slice(0, Lk) and (lse == -np.inf).all()), at

    # a value: its column
    vn = v.clone()
    vn[:, Lk // 3, H - 1, D - 1] = float("nan")
    out, lse = cross(cc, q, ex(k), ex(vn))
    assert np.isnan(out[:, :, Hq - G:, D - 1]).all() and np.isfinite(lse).all()
    out[:, :, Hq - G:, D - 1] = 0
    assert np.isfinite(out).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("n", [100, 3000, 70000])
def test_paged_attention_nan(cc, n, dt):  # noqa: F811
    """With weights added: a NaN row makes the weights of every slot that its cache head sees NaN,
    and leaves those without a page and past the length as they were."""
    import torch

    B, Hq, H, D, page = 2, 6, 2, 64, 50
    say(f"paged nan {n} {dt}")
    g = torch.Generator(device="cuda").manual_seed(73)
    cols = n // page + 1
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch_dtype(dt))  # noqa: E731
    k, v = mk(B * cols, H, page, D), mk(B * cols, H, page, D)
    table = torch.randperm(B * cols).view(B, cols).int()
    table[0, cols // 2] = -1
    td, ld = table.cuda(), ints([n, n])
    for where in ("query", "first key", "all keys"):
        q, kn = mk(B, Hq, D), k.clone()
        if where == "query":
            q[0, 1] = float("nan")
        elif where == "first key":
            kn[int(table[0, 0]), 0, 0, 1] = float("nan")
        else:
            kn[table[0][table[0] >= 0].long(), 0, :, 1] = float("nan")
        w0 = torch.rand((B, H, cols * page), generator=g, device="cuda")
        for weights in (False, True):
            w = w0.clone() if weights else None
            out, lse = cc.paged_attention(q, kn, v, td, ld, weight_sum=w)
            torch.cuda.synchronize()
            bad = torch.zeros((B, Hq), dtype=torch.bool, device="cuda")
            bad[0, 1 if where == "query" else slice(0, 3)] = True
            assert torch.equal(torch.isnan(lse), bad), (where, weights)
            assert torch.equal(torch.isnan(out), bad[..., None].expand(out.shape)), (where, weights)
            if weights:
                seen = (torch.arange(cols * page) < n).expand(B, -1) & (table >= 0).repeat_interleave(
                    page, 1)
                want = torch.zeros((B, H, cols * page), dtype=torch.bool)
                want[0, 0] = seen[0]
                assert torch.equal(torch.isnan(w).cpu(), want), where
                gone = ~seen[:, None].expand(want.shape).cuda()
                assert torch.equal(w[gone], w0[gone]), where
