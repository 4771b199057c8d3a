"""Norms of rows in which one value holds nearly all of the mean and of the mean
square: lost or counted twice, it changes every value of the row by a large
factor.  The value stands at each end of what a lane, a wave or a workgroup of
the kernel holds, one place per row.

Bound.  A statistic is a sum of at most 64 values per lane, 6 steps over the
lanes and 16 over the waves, in fp32: below 100 roundings.  The result is off
by 4 times that, relative to its own size and to what the largest value of the
row becomes (a mean that is off moves all values alike), and by its rounding."""

import numpy as np
import pytest

import block_ref as R
from gpu_util import say, to_host
from test_gpu_block import DTS, cc, dev  # noqa: F401 (cc: a fixture)

# up to 64, 128 and 256 16-byte pieces for a wave, 512 and 1024 for 256 lanes, 2048 and 4096 for
# 1024 lanes, and rows taken value by value: both sides of every limit
WIDTHS = [7, 65, 256, 264, 512, 513, 520, 1000, 1024, 1032, 2048, 2049, 2056, 4096, 4097, 4104, 8192,
          8200, 16383, 16384]


def places(C):
    """Values at the ends of pieces of 1, 4 and 8 values, of lanes, waves and workgroups."""
    at = {0, 1, C // 2, C - 1}
    for n in (4, 8, 64, 256, 512, 1024, 2048, 4096, 8192):
        for p in (n - 1, n, C - n, C - n - 1, C // n * n, C // n * n - 1):
            if 0 <= p < C:
                at.add(p)
    return sorted(at)


def rows(rng, C):
    u = rng.standard_normal((len(places(C)), C))
    for i, p in enumerate(places(C)):
        u[i, p] = 4 * np.sqrt(C) * (1 if i % 2 else -1)
    return u


def bound(u, y, kind, dt):
    """u: what is normed, y: the reference result (without weights)."""
    d = u - u.mean(-1, keepdims=True) if kind == 2 else u
    top = np.abs(u).max(-1, keepdims=True) / np.sqrt((d * d).mean(-1, keepdims=True))
    return R.U[dt] * np.abs(y) + 400 * R.E * (np.abs(y) + top) + 1e-30


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("C", WIDTHS)
def test_one_value_holds_the_row(cc, C, kind, dt):  # noqa: F811
    import torch

    say(f"norm rows {C} {kind} {dt}")
    rng = np.random.default_rng(103)
    u, u64 = dev(rows(rng, C), dt)
    none = torch.zeros_like(u)
    want = R.norm(u64, kind, None, None, 1e-5)
    b = bound(u64, want, kind, dt)
    # the norm after the block, then the one before the next
    post, _ = cc.norm_residual(none, u, post=kind, pre=cc.NORM_NONE)
    _, pre = cc.norm_residual(u, none, pre=kind)
    torch.cuda.synchronize()
    R.check(to_host(post), want, b, "post")
    R.check(to_host(pre), want, b, "pre")


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("C", WIDTHS)
def test_the_bound_tells_a_lost_value(C, kind):
    """Statistics that miss or repeat any one of those values, by the bound of the widest type."""
    u = rows(np.random.default_rng(107), C)
    want = R.norm(u, kind, None, None, 1e-5)
    b = bound(u, want, kind, "bf16")
    for i, p in enumerate(places(C)):
        for times in (0, 2):
            w = np.ones(C)
            w[p] = times
            mean = (w * u[i]).sum() / C if kind == 2 else 0.0
            d = u[i] - mean
            y = d / np.sqrt((w * d * d).sum() / C + 1e-5)
            assert (np.abs(y - want[i]) > b[i]).mean() > 0.5, (p, times)
