"""GPU: chunk attention's tiled kernel in fp32 (sequences of different rows, every cache
layout, rows that do not exist, missing pages), at sizes for which it is the one that is
chosen, and 16-bit weights in two parts in the streaming kernel."""

import numpy as np
import pytest

import block_ref as R
import request_cases as cases
import test_gpu_requests as T
from gpu_util import say, to_host, torch_dtype
from test_gpu_block import Cache, cc, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", cases.TILED, ids=[str(i) for i in range(len(cases.TILED))])
@pytest.mark.parametrize("weights", [False, True])
def test_tiled(cc, case, weights):  # noqa: F811
    T.test_chunk_attention(cc, case[1], case[0], weights)


@pytest.mark.parametrize("case", cases.NARROW, ids=[str(i) for i in range(len(cases.NARROW))])
def test_tiled_narrow_heads(cc, case):  # noqa: F811
    T.test_chunk_attention(cc, case[1], case[0], True)


@pytest.mark.parametrize("dt,n,Hq,H,D", cases.CUT)
def test_tiled_rows_that_do_not_exist(cc, dt, n, Hq, H, D):  # noqa: F811
    T.test_chunk_rows_that_do_not_exist(cc, dt, n, Hq, H, D)


@pytest.mark.parametrize("dt,n,Hq,H,extra", cases.MISSING)
def test_tiled_missing_pages_and_long_lengths(cc, dt, n, Hq, H, extra):  # noqa: F811
    T.test_chunk_attention_missing_pages_and_long_lengths(cc, dt, n, Hq, H, extra)


def two_parts(q, k, v, seen, scale, dt):
    """(out, bound, the same out from weights rounded to the type) of rows q [M, D].

    As in block_ref, but a weight p keeps its rounded rest: the rest is U p at most and is rounded
    to the type, so that U^2 p is lost.  The two products and the sums over the slots add twice as
    many numbers as one product.  f16 ends at 2^-24: the rest of a small weight is off by half of
    that, 2^-25, of the weight of the maximum (which the kernel's reference never passes)."""
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    ds = (q.shape[1] + 4) * R.E * scale * (np.where(seen, np.abs(q) @ np.abs(k).T, 0.0)).max(1)
    ex = np.exp(s - s.max(1, keepdims=True))
    tot, count = ex.sum(1, keepdims=True), seen.sum(1)
    out, pv = ex @ v / tot, ex @ np.abs(v) / tot
    tiny = count[:, None] * 2.0 ** -25 * np.abs(v).max(0) / tot if dt == "f16" else 0.0
    lost = 2 * ds + (count + 32) * R.E + R.U[dt] ** 2 + 2 * count * R.E
    rounded = torch_rounded(ex, dt) @ v / tot
    return out, R.U[dt] * np.abs(out) + lost[:, None] * pv + tiny + 1e-30, rounded


def torch_rounded(x, dt):
    import torch

    return to_host(torch.from_numpy(x).to(torch_dtype(dt)))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,G,D,L", [(1, 1, 64, 40), (1, 16, 128, 64), (4, 4, 128, 57),
                                     (16, 1, 80, 70), (3, 5, 256, 33), (2, 8, 32, 50)])
def test_weights_keep_both_parts_with_up_to_16_rows(cc, dt, n, G, D, L):  # noqa: F811
    """Values whose weighted sums vanish for every row: the output's own rounding is small, and
    what rounded weights would leave is several times the bound."""
    say(f"two parts {dt} {n} {G} {D} {L}")
    rng = np.random.default_rng(L)
    scale = 1.28 / D
    c = Cache(rng, 1, 1, D, 16, [L], dt)
    q, starts, (q64,) = T.packed([rng.standard_normal((n, G, D))], 0, dt)
    rows = q64.reshape(n * G, D)
    slots = np.arange(L)
    k, _ = R.slot_rows(c.k, c.table, 16, 0, 0, slots)
    seen = slots < L - n + np.repeat(np.arange(n), G)[:, None] + 1
    ex = np.where(seen, np.exp(scale * (rows @ k.T)), 0.0)
    v, _ = R.slot_rows(c.v, c.table, 16, 0, 0, slots)
    v = v - ex.T @ np.linalg.solve(ex @ ex.T, ex @ v)
    c.v[c.table[0, slots // 16], 0, slots % 16] = v
    c.vd, c.v = dev(c.v, dt)
    v, _ = R.slot_rows(c.v, c.table, 16, 0, 0, slots)
    want, bound, rounded = two_parts(rows, k, v, seen, scale, dt)
    assert (np.abs(rounded - want) / bound).max() > 3  # the test tells the two apart
    out, _ = cc.chunk_attention(q, c.kd, c.vd, c.td, c.ld, row_starts=starts, n=n, scale=scale)
    R.check(to_host(out).reshape(n * G, D), want, bound, "two parts")
