"""GPU: what attention loses to 16 bits besides the roundings of its inputs and
of its result.

With few query rows the weights meet the values in two 16-bit parts, the second
one what the first leaves over: a weight is off by u^2 of itself (u the type's
unit roundoff), so that values that cancel leave a result with its own digits.
The rest of the bound is the one of block_ref.attend: fp32 scores, weights and
sums."""

import numpy as np
import pytest

import block_ref as R
from gpu_util import say, to_host, torch_dtype
from test_gpu_block import Cache, cc, dev, ints  # noqa: F401 (cc: a fixture)

pytestmark = pytest.mark.gpu


def attend(q, k, v, scale, dt):
    """q [M, D], k, v [n, D] float64: out and its bound."""
    D, n = q.shape[1], k.shape[0]
    s = scale * (q @ k.T)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    out, pv = p @ v, p @ np.abs(v)
    ds = (D + 4) * R.E * abs(scale) * (np.abs(q) @ np.abs(k).T).max(1)
    dp = 2 * ds + (n + 32) * R.E
    # f16 weights end at 2^-24 of their reference, which a wave's largest one reaches; a wave
    # has at most 512 keys
    tiny = min(n, 512) * 2.0 ** -25 * np.abs(v).max(0) if dt == "f16" else 0.0
    return out, R.U[dt] * np.abs(out) + (dp[:, None] + R.U[dt] ** 2 + n * R.E) * pv + tiny


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n", [2, 3, 5, 40, 300, 2600])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_few_rows_keep_the_weights(cc, n, D, dt):  # noqa: F811
    import torch

    say(f"weights n={n} D={D} {dt}")
    rng = np.random.default_rng(79)
    B, Hq, H, page = 2, 32, 4, 16
    c = Cache(rng, B, H, D, page, [n, n], dt)
    # values in pairs of opposite signs, so that most of every sum cancels
    sign = np.where(np.arange(c.table.shape[1] * page) % 2, -1.0, 1.0)
    v = np.full_like(c.v, np.nan)
    for b in range(B):
        for t in range(n):
            v[c.table[b, t // page], :, t % page] = sign[t] * (1 + 0.02 * rng.random((H, D)))
    vd, v = dev(v, dt)
    q, q64 = dev(rng.standard_normal((B, Hq, D)) * 0.3, dt)
    out, _ = cc.paged_attention(q, c.kd, vd, c.td, c.ld)
    at = np.arange(n)
    rows = lambda x, b: np.stack([x[c.table[b, at // page], h, at % page]  # noqa: E731
                                  for h in range(H)], 1)
    kk, vv = (np.stack([rows(x, b) for b in range(B)]) for x in (c.k, v))
    dense = [torch.from_numpy(x).to(torch_dtype(dt)).cuda() for x in (kk, vv)]
    cross, _ = cc.cross_attention(q[:, None], *dense)
    torch.cuda.synchronize()
    G = Hq // H
    for b in range(B):
        for h in range(H):
            r = slice(h * G, (h + 1) * G)
            o, bound = attend(q64[b, r], kk[b, :, h], vv[b, :, h], D ** -0.5, dt)
            R.check(to_host(out)[b, r], o, bound, "paged")
            R.check(to_host(cross)[b, 0, r], o, bound, "cross")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("masked", [False, True])
def test_many_small_weights_add_up(cc, masked, dt):  # noqa: F811
    """One key that takes nearly all the weight, first, and 60000 keys of e^-18 of it each: the
    values are theirs alone.  f16 weights are held against a reference of 2^-5 of the largest, so
    that they end at 2^-30 of it (half a step of 2^-24 there), not at 2^-25."""
    import torch

    B, Lq, Lk, Hq, H, D = 16, 128, 60001, 16, 1, 64
    say(f"small weights masked={masked} {dt}")
    kind = torch_dtype(dt)
    q = torch.zeros((B, Lq, Hq, D), dtype=kind, device="cuda")
    q[..., 0] = 4.0
    k = torch.zeros((1, Lk, H, D), dtype=kind, device="cuda")
    k[:, 0, :, 0] = 4.5
    v = torch.ones((1, Lk, H, D), dtype=kind, device="cuda")
    v[:, 0] = 0.0
    mask = None
    n = Lk - 1
    if masked:
        mask = torch.ones((B, Lk), dtype=torch.bool, device="cuda")
        mask[:, 1::3] = False
        n = int(mask[0, 1:].sum())
    ex = lambda t: t.expand(B, Lk, H, D)  # noqa: E731
    out, lse = cc.cross_attention(q, ex(k), ex(v), mask=mask, scale=1.0)
    torch.cuda.synchronize()
    p = np.exp(-18.0)
    want = n * p / (1 + n * p)
    dp = 2 * (D + 4) * R.E * 18 + (n + 32) * R.E
    bound = (2 * R.U[dt] + dp + n * R.E) * want + (n * 2.0 ** -30 if dt == "f16" else 0.0)
    R.check(to_host(out), np.full(out.shape, want), bound, "out")
    R.check(to_host(lse), np.full(lse.shape, 18 + np.log1p(n * p)), dp + 8 * R.E * 18, "lse")
