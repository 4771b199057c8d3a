"""GPU: page tables of as many sequences as a call takes, and steps that give back and take
more pages than the kernel moves in one round (4 entries of each of 1024 threads)."""

import numpy as np
import pytest

import request_ref as Q
from gpu_util import say
from test_gpu_block import cc, ints  # noqa: F401
from test_gpu_requests import requests, tables

pytestmark = pytest.mark.gpu

NAMES = ("table", "held", "free", "count", "starts", "positions", "slots", "slot positions",
         "slot weights")


def run(cc, lengths, counts, held, page, cols, P, rows, heads, seed, stack=None):  # noqa: F811
    import torch

    rng = np.random.default_rng(seed)
    table, free, count = tables(rng, held, cols, P)
    if stack is not None:
        count = stack(count)
    B = len(lengths)
    now = lengths + rng.integers(0, 100, B)
    positions = weights = pd = wd = None
    if heads:
        positions = rng.integers(-5, 5, (B, heads, cols * page)).astype(np.int32)
        weights = rng.random((B, heads, cols * page)).astype(np.float32)
        pd, wd = ints(positions), torch.from_numpy(weights).cuda()
    ref = Q.pages(lengths, counts, now, held, count, table, free, page, rows, positions, weights)
    td, fd, hd, cd = ints(table), ints(free), ints(held), ints([count])
    maps = cc.cache_pages(td, hd, fd, cd, ints(lengths), page_size=page, counts=ints(counts),
                          now=ints(now), rows=rows, positions=pd, weight_sum=wd)
    torch.cuda.synchronize()
    for name, g, r in zip(NAMES, [td, hd, fd, cd, *maps, pd, wd], ref):
        if r is not None:
            assert np.array_equal(g.cpu().numpy().ravel(), np.asarray(r).ravel()), name
    return ref


# (16 bytes of LDS each: from 48 KiB on the launch raises the limit)
@pytest.mark.parametrize("B,page,cols,new,spare,heads", [
    (3100, 4, 4, 2, 10, 1), (4097, 3, 5, 9, -50, 0),
    (8191, 2, 3, 2, -5, 2), (8192, 16, 2, 30, 40, 0), (8192, 1, 1, 1, 0, 1)])
def test_many_sequences(cc, B, page, cols, new, spare, heads):  # noqa: F811
    say(f"pages of many sequences {B} {page} {cols} {new} {spare} {heads}")
    rng = np.random.default_rng(B + page)
    lengths, counts, held = requests(rng, B, page, cols, new, "mixed")
    P = int(max(held.sum(), (-(-lengths // page)).sum() + spare, 1))
    run(cc, lengths, counts, held, page, cols, P, int(counts.sum()) + 3, heads, B)


@pytest.mark.parametrize("B,page,cols,left", [(100, 4, 400, 0), (100, 4, 400, 900), (9, 1, 3000, 5),
                                              (2, 2, 10000, -1)])
def test_many_pages(cc, B, page, cols, left):  # noqa: F811
    """Half of the sequences end, the other half come with prompts; `left` pages stay on the stack
    (-1: it is empty before the last are served)."""
    say(f"many pages {B} {page} {cols} {left}")
    rng = np.random.default_rng(B)
    order = rng.permutation(B)
    old = np.where(order % 2 == 0, rng.integers(cols * page // 2, cols * page + 1, B), 0)
    lengths = np.where(order % 2 == 0, 0, rng.integers(cols * page // 2, cols * page + 1, B))
    counts = lengths.copy()
    held = -(-old // page)
    need = -(-lengths // page)
    P = int(max(held.sum(), need.sum()) + max(left, 0))
    ref = run(cc, lengths, counts, held, page, cols, P, int(counts.sum()), 0, B,
              stack=(lambda n: 0) if left < 0 else None)
    given, taken = int(held.sum()), int(need.sum())
    assert given + taken > 13000
    if left < 0:
        assert ref[3] == max(given - taken, 0)
