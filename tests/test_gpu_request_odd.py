"""GPU: infinities and NaN in the tiled kernel of chunk attention: in slots that no row of
the call may see, in a page of another request, and in slots that some rows see."""

import numpy as np
import pytest

import block_ref as R
import request_ref as Q
from gpu_util import say, to_host, torch_dtype
from test_gpu_block import Cache, cc, ints  # noqa: F401
from test_gpu_requests import packed

pytestmark = pytest.mark.gpu

DTS = ["f32", "bf16", "f16"]


def test_another_request_s_nan_costs_nothing(cc):  # noqa: F811
    """Keys that a short tile lacks are read from page 0.  What it holds (NaN of another request)
    changes neither results nor time: the values that some rows see are not gone over again.
    (Where they were, the call below took 2.4 times as long.)"""
    import torch

    say("nan in page 0")
    B, n, Hq, H, D, page, L = 2, 128, 32, 8, 128, 16, 8000
    cols = L // page
    k = torch.randn(B * cols + 1, H, page, D, device="cuda").to(torch.bfloat16)
    v = torch.randn_like(k)
    q = torch.randn(B * n, Hq, D, device="cuda").to(torch.bfloat16)
    table = (torch.randperm(B * cols, device="cuda") + 1).int().view(B, cols)
    lengths, starts = ints([L, L - 1]), ints([0, n, 2 * n])
    plan = cc.ChunkAttention(B, B * n, n, Hq, H, D, B * cols + 1, page, cols, dtype=cc.CTCONV_BF16)
    ws = torch.empty(max(plan.workspace_bytes, 16), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(B * n, Hq, device="cuda")
    odd_k, odd_v = k.clone(), v.clone()
    odd_k[0], odd_v[0] = float("inf"), float("nan")
    s = torch.cuda.current_stream().cuda_stream
    times, results = ([], []), []
    for i in range(20):
        for j, (kk, vv) in enumerate(((k, v), (odd_k, odd_v))):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            plan(q.data_ptr(), kk.data_ptr(), vv.data_ptr(), table.data_ptr(), lengths.data_ptr(),
                 starts.data_ptr(), None, out.data_ptr(), lse.data_ptr(), None, ws.data_ptr(),
                 ws.numel(), s)
            b.record()
            torch.cuda.synchronize()
            times[j].append(a.elapsed_time(b))
            if i == 0:
                results.append((out.clone(), lse.clone()))
    for x, y in zip(*results):
        assert torch.equal(x, y) and bool(torch.isfinite(x).all())
    assert min(times[1]) < 1.5 * min(times[0]), (min(times[0]), min(times[1]))
