"""GPU: chunk attention under bounds far above what the call holds: n past the rows of
the call, and one sequence with many rows among sequences with one."""

import numpy as np
import pytest

import request_ref as Q
import block_ref as R
from gpu_util import say, to_host
from test_gpu_block import Cache, cc, guarded, ints  # noqa: F401
from test_gpu_requests import compare, packed

pytestmark = pytest.mark.gpu

DTS = ["f32", "bf16", "f16"]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("Hq,H,D,window", [(2, 2, 256, 0), (8, 2, 64, 0), (6, 1, 80, 1500)])
def test_chunk_n_past_the_rows(cc, dt, Hq, H, D, window):  # noqa: F811
    """n = rows, and 4096 of 4 rows: the same plan and the same bits."""
    import torch

    say(f"chunk n past the rows {dt} {Hq} {H} {D} {window}")
    rng = np.random.default_rng(D)
    lengths, counts, page = [9001, 2, 5000], [2, 1, 1], 16
    c = Cache(rng, 3, H, D, page, lengths, dt)
    q, starts, q64 = packed([rng.standard_normal((k, Hq, D)) for k in counts], 0, dt)
    ref, w, wb = Q.chunk(q64, c.k, c.v, c.table, lengths, counts, page, window, D ** -0.5, dt)
    res = []
    for n in (2, 4, 4096):
        out = guarded(torch.full((4, Hq, D), 9.0, dtype=q.dtype, device="cuda"))
        lse = guarded(torch.full((4, Hq), 9.0, device="cuda"))
        weights = torch.zeros(3, H, c.table.shape[1] * page, device="cuda")
        cc.chunk_attention(q, c.kd, c.vd, c.td, c.ld, row_starts=starts, n=n, window=window,
                           weight_sum=weights, out=out, lse=lse)
        torch.cuda.synchronize()
        compare(to_host(out), to_host(lse), ref, f"n={n}")
        R.check(to_host(weights), w, wb, f"weights n={n}")
        res.append((out, lse, weights))
    for a, b in zip(res[1], res[2]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", DTS)
def test_chunk_counts_past_the_rows_of_the_call(cc, dt):  # noqa: F811
    """A sequence whose row_starts go past all rows of the call, under an n that does, too: the
    rows that exist keep the places that the full count gives them."""
    import torch

    say(f"chunk counts past the rows {dt}")
    rng = np.random.default_rng(3)
    Hq, H, D, page, L, count, live = 4, 2, 64, 16, 700, 90, 3
    c = Cache(rng, 1, H, D, page, [L], dt)
    for window in (0, 100):
        q, _, q64 = packed([rng.standard_normal((live, Hq, D))], 0, dt)
        out = guarded(torch.full((live, Hq, D), 9.0, dtype=q.dtype, device="cuda"))
        lse = guarded(torch.full((live, Hq), 9.0, device="cuda"))
        cc.chunk_attention(q, c.kd, c.vd, c.td, c.ld, row_starts=ints([0, count]), n=1000,
                           window=window, out=out, lse=lse)
        torch.cuda.synchronize()
        ref, _, _ = Q.chunk(q64, c.k, c.v, c.table, [L], [count], page, window, D ** -0.5, dt)
        compare(to_host(out), to_host(lse), ref, f"window {window}")


@pytest.mark.parametrize("dt,Hq,H,D", [("f32", 8, 8, 256), ("bf16", 12, 12, 64), ("f32", 4, 4, 64)])
def test_chunk_one_long_among_single_rows(cc, dt, Hq, H, D):  # noqa: F811
    """20 sequences, of which one has most of the rows: the streaming kernel's grid is mostly
    workgroups without rows."""
    import torch

    say(f"chunk one long among single rows {dt} {Hq} {H} {D}")
    rng = np.random.default_rng(H)
    B, page, cap = 20, 64, 4000
    counts = [1] * B
    counts[7] = 400 if H < 12 else 180
    lengths = [int(v) for v in rng.integers(1, cap + 1, B)]
    lengths[7] = cap
    c = Cache(rng, B, H, D, page, lengths, dt)
    q, starts, q64 = packed([rng.standard_normal((k, Hq, D)) for k in counts], 2, dt)
    rows = sum(counts)
    out = guarded(torch.full((rows + 2, Hq, D), 9.0, dtype=q.dtype, device="cuda"))
    lse = guarded(torch.full((rows + 2, Hq), 9.0, device="cuda"))
    cc.chunk_attention(q, c.kd, c.vd, c.td, c.ld, row_starts=starts, n=max(counts), out=out,
                       lse=lse)
    torch.cuda.synchronize()
    ref, _, _ = Q.chunk(q64, c.k, c.v, c.table, lengths, counts, page, 0, D ** -0.5, dt)
    compare(to_host(out)[:rows], to_host(lse)[:rows], ref, "mixed")
    assert bool((out[rows:] == 9).all()) and bool((lse[rows:] == 9).all())
