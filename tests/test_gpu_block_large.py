"""GPU: calls of more workgroups than one row of a launch grid holds (2^32
threads): each operator at a little more than its kernels' limit."""

import pytest

from gpu_util import say
from test_gpu_block import cc  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("C", [8, 7])
def test_norm_rows(cc, C):  # noqa: F811
    """4 rows of 8 (or 7) values per workgroup of 256: the same as in parts."""
    import torch

    rows = (1 << 26) + 4099
    say(f"norm {rows} x {C}")
    g = torch.Generator(device="cuda").manual_seed(83)
    x, h = (torch.empty(rows, C, dtype=torch.float16, device="cuda").normal_(generator=g)
            for _ in range(2))
    xo, y = cc.norm_residual(x, h, cc.NORM_RMS)
    part = 1 << 24  # rows, on 16 bytes also where C is odd
    for r in range(0, rows, part):
        a, b = cc.norm_residual(x[r:r + part], h[r:r + part], cc.NORM_RMS)
        assert torch.equal(a, xo[r:r + part]) and torch.equal(b, y[r:r + part]), r
    assert bool((xo[-1] != x[-1]).any())


def test_cache_append_sequences(cc):  # noqa: F811
    import torch

    B, H, D = (1 << 24) + 77, 1, 8
    say(f"append {B}")
    new = torch.arange(B * D, device="cuda").view(B, 1, H, D).remainder(2039).half()
    k, v = (torch.zeros(B, H, 1, D, dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.arange(B, device="cuda").flip(0).int()[:, None]
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    w = torch.ones(B, H, 1, device="cuda")
    cc.cache_append(new, new, k, v, table, one, weight_sum=w)
    assert torch.equal(k.flip(0)[:, 0], new[:, 0]) and torch.equal(v, k) and not bool(w.any())


@pytest.mark.parametrize("weights", [False, True])
def test_paged_attention_sequences(cc, weights):  # noqa: F811
    """One slot each: out is its value, its weight 1."""
    import torch

    B, H, D, pool = (1 << (24 if weights else 22)) + 77, 1, 8, 1021
    say(f"paged {B} weights={weights}")
    g = torch.Generator(device="cuda").manual_seed(89)
    q = torch.randn(B, H, D, generator=g, device="cuda").half()
    k, v = (torch.randn(pool, H, 1, D, generator=g, device="cuda").half() for _ in range(2))
    table = torch.randint(0, pool, (B, 1), generator=g, device="cuda", dtype=torch.int32)
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    w = torch.full((B, H, 1), 2.0, device="cuda") if weights else None
    out, lse = cc.paged_attention(q, k, v, table, one, scale=0.5, weight_sum=w)
    at = table[:, 0].long()
    assert torch.equal(out[:, 0], v[at][:, 0, 0])
    s = 0.5 * (q[:, 0].float() * k[at][:, 0, 0].float()).sum(-1)
    assert float((lse[:, 0] - s).abs().max()) < 1e-4
    if weights:
        assert float((w - 3).abs().max()) < 1e-5


@pytest.mark.parametrize("fused", [False, True])
def test_cache_evict_sequences(cc, fused):  # noqa: F811
    """Two slots each, the heavier one stays."""
    import torch

    B, H, D = (1 << (22 if fused else 24)) + 77, 1, 8
    say(f"evict {B} fused={fused}")
    g = torch.Generator(device="cuda").manual_seed(97)
    k = torch.arange(2 * B * D, device="cuda").view(2 * B, H, 1, D).remainder(2039).half()
    v = k.clone()
    table = torch.arange(2 * B, device="cuda", dtype=torch.int32).view(B, 2)
    lengths = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    w = torch.rand(B, H, 2, generator=g, device="cuda")
    want = torch.where((w[:, 0, 1] > w[:, 0, 0])[:, None], k[1::2, 0, 0], k[0::2, 0, 0])
    best = w.amax(2)
    if fused:  # results and lengths of their own: one kernel
        wo = torch.empty(B, H, 1, device="cuda")
        lo, src = torch.empty_like(lengths), torch.empty(B, H, 1, dtype=torch.int32, device="cuda")
        cc.CacheEvict(B, H, D, 2 * B, 1, 2, 1, dtype=cc.CTCONV_F16)(
            k.data_ptr(), v.data_ptr(), table.data_ptr(), lengths.data_ptr(), None, w.data_ptr(),
            None, wo.data_ptr(), None, lo.data_ptr(), src.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
    else:
        cc.cache_evict(k, v, table, lengths, w, 1)
        wo, lo = w[:, :, :1], lengths
    torch.cuda.synchronize()
    assert torch.equal(k[0::2, 0, 0], want) and torch.equal(v[0::2, 0, 0], want)
    assert torch.equal(wo[:, :, 0], best) and bool((lo == 1).all())


def test_cross_attention_row_tiles(cc):  # noqa: F811
    """65 rows per sequence, one workgroup each: all sequences alike."""
    import torch

    B, Lq, Lk, H, D = (1 << 24) + 13, 65, 3, 1, 8
    say(f"cross {B}")
    g = torch.Generator(device="cuda").manual_seed(101)
    q = torch.randn(1, Lq, H, D, generator=g, device="cuda").half()
    k, v = (torch.randn(1, Lk, H, D, generator=g, device="cuda").half() for _ in range(2))
    one, lse1 = cc.cross_attention(q, k, v)
    out, lse = cc.cross_attention(q.expand(B, Lq, H, D), k.expand(B, Lk, H, D),
                                  v.expand(B, Lk, H, D))
    for b in range(0, B, 1 << 21):
        assert torch.equal(out[b:b + (1 << 21)], one.expand_as(out[b:b + (1 << 21)])), b
        assert torch.equal(lse[b:b + (1 << 21)], lse1.expand_as(lse[b:b + (1 << 21)])), b
