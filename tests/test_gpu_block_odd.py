"""GPU: an infinite value in cross attention whose keys are divided among workgroups: every row
sees it, and its column is that infinity for all of them, whichever division holds it."""

import numpy as np
import pytest

from gpu_util import say, torch_dtype
from test_gpu_block import cc  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,Lq,Lk,Hq,H,D,splits", [(1, 2048, 2500, 2, 2, 64, 5), (1, 700, 4000, 8, 2, 128, 5),
                                                   (2, 600, 1500, 4, 4, 96, 4), (2, 600, 6000, 4, 4, 96, 6),
                                                   (1, 2048, 4000, 2, 2, 64, 7)])
def test_an_infinite_value_in_any_split(cc, dt, B, Lq, Lk, Hq, H, D, splits):  # noqa: F811
    import torch

    say(f"infinite value {dt} {B} {Lq} {Lk} {Hq} {H} {D}")
    nb = cc.ctconv_cross_attention_workspace_bytes(B, Lq, Lk, Hq, H, D, cc.dtype_code_of(dt))
    assert nb // (B * Lq * Hq * (D + 2) * 4) == splits
    g = torch.Generator(device="cuda").manual_seed(Lk)
    kind = torch_dtype(dt)
    q = torch.randn((B, Lq, Hq, D), generator=g, device="cuda").to(kind)
    k, v = (torch.randn((B, Lk, H, D), generator=g, device="cuda").to(kind) for _ in range(2))
    clean, level = cc.cross_attention(q, k, v, scale=0.1)
    torch.cuda.synchronize()
    G = Hq // H
    for at in (0, Lk // 2, Lk - 1):
        for value in (np.inf, -np.inf):
            odd = v.clone()
            odd[B - 1, at, H - 1, 3] = value
            out, lse = cc.cross_attention(q, k, odd, scale=0.1)
            torch.cuda.synchronize()
            hit = out[B - 1, :, Hq - G:, 3]
            assert bool((hit == value).all()), (at, value)
            hit.copy_(clean[B - 1, :, Hq - G:, 3])
            assert torch.equal(out, clean) and torch.equal(lse, level), (at, value)
