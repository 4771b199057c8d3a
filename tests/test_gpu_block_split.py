"""GPU: one query row per sequence and head at both sides of the limits by which
its keys are split over workgroups and waves: few keys on many heads, many keys
on few, in one workgroup or several."""

import numpy as np
import pytest

import block_ref as R
from gpu_util import say, to_host, torch_dtype
from test_gpu_block import DTS, cc, ints  # noqa: F401 (cc: a fixture)

pytestmark = pytest.mark.gpu

# sequences, heads, keys, D
CASES = [
    (64, 16, 5, 64), (64, 16, 129, 32), (128, 64, 1, 16), (32, 8, 300, 64), (33, 8, 300, 64),
    (1, 8, 512, 64), (1, 8, 513, 64), (16, 16, 1024, 24), (16, 16, 1025, 24), (8, 15, 1000, 40),
    (2, 4, 256, 256), (2, 4, 257, 200), (1, 8, 500, 256), (1, 8, 384, 144), (1, 8, 385, 144), (16, 16, 700, 136), (64, 16, 140, 128),
    (41, 25, 140, 104), (16, 8, 128, 128), (16, 8, 129, 128), (16, 16, 65, 48),
    (16, 17, 512, 64), (16, 17, 513, 64), (16, 17, 1025, 64),
]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_one_row_however_it_is_split(cc, case, dt):  # noqa: F811
    import torch

    B, H, n, D = case
    page = 16
    say(f"split {case} {dt}")
    g = torch.Generator(device="cuda").manual_seed(109)
    cols = -(-n // page)
    kind = torch_dtype(dt)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(kind)  # noqa: E731
    k, v, q = rnd(B * cols, H, page, D), rnd(B * cols, H, page, D), rnd(B, H, D)
    table = torch.randperm(B * cols, generator=g, device="cuda").int().view(B, cols)
    rows = [t[table.long()].transpose(2, 3).reshape(B, cols * page, H, D)[:, :n] for t in (k, v)]
    out, lse = cc.paged_attention(q, k, v, table, ints([n] * B), max_length=n)
    w = torch.zeros((B, H, cols * page), device="cuda")
    out_w, lse_w = cc.paged_attention(q, k, v, table, ints([n] * B), max_length=n, weight_sum=w)
    crossed, clse = cc.cross_attention(q[:, None], *(t.contiguous() for t in rows))
    torch.cuda.synchronize()
    got = [to_host(t) for t in (out, lse, out_w, lse_w, crossed[:, 0], clse[..., 0], w)]
    q64, (k64, v64) = to_host(q), (to_host(t) for t in rows)
    pick = {(0, 0), (B - 1, H - 1)} | {(int(b), int(h)) for b, h in
                                       np.random.default_rng(113).integers(0, [B, H], (30, 2))}
    for b, h in sorted(pick):
        (o, l, p), (bo, bl, bp) = R.attend(q64[b, h:h + 1], k64[b, :, h], v64[b, :, h], D ** -0.5, dt)
        for i in (0, 2, 4):
            R.check(got[i][b, h:h + 1], o, bo, "out")
            R.check(got[i + 1][b, h:h + 1], l, bl, "lse")
        R.check(got[6][b, h, :n], p[0], bp[0] + R.E * p[0], "weights")
    # every head: the kernels' forms against each other, and whole sums of weights
    tol = 4 * R.U[dt] if dt != "f32" else 1e-4
    assert np.abs(got[0] - got[4]).max() < tol * np.abs(got[0]).max()
    assert np.abs(got[6].sum(-1) - 1).max() < 1e-4
