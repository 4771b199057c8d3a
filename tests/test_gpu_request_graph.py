"""GPU: calls that a graph records, replayed several times with the program's own work between
the replays: page maps in two launches, rotary positions in place, attention with weights in
every kernel and split; two graphs in turn, each with a workspace of its own."""

import numpy as np
import pytest

from gpu_util import say, torch_dtype
from test_gpu_block import cc, ints  # noqa: F401

pytestmark = pytest.mark.gpu


def record(step):
    import torch

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    return graph


def test_page_maps_of_many_rows(cc):  # noqa: F811
    """More rows than the first kernel maps: the second launch, and lengths that change."""
    import torch

    say("graph: pages")
    B, page, cols, rows = 40, 16, 60, 9000
    P = B * cols
    rng = np.random.default_rng(4)
    ld, kd, hd, cd = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, B, B, 1))
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(P, dtype=torch.int32, device="cuda")
    starts, at, to = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B + 1, rows, rows))
    plan = cc.CachePages(B, rows, P, page, cols)

    def step():
        plan(ld.data_ptr(), kd.data_ptr(), None, hd.data_ptr(), cd.data_ptr(), table.data_ptr(),
             free.data_ptr(), hd.data_ptr(), cd.data_ptr(), starts.data_ptr(), at.data_ptr(),
             to.data_ptr(), None, None, torch.cuda.current_stream().cuda_stream)

    def fresh(lengths, counts):
        ld.copy_(ints(lengths))
        kd.copy_(ints(counts))
        hd.zero_()
        cd.fill_(P)
        free.copy_(torch.arange(P, device="cuda"))
        table.fill_(-1)

    cases = []
    for _ in range(3):
        lengths = rng.integers(100, cols * page + 1, B)
        cases.append((lengths, np.minimum(rng.integers(0, 400, B), lengths)))
    want = []
    for c in cases:
        fresh(*c)
        step()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (table, hd, cd, free, starts, at, to)])
    graph = record(step)
    for c, w in list(zip(cases, want)) * 2:
        fresh(*c)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((table, hd, cd, free, starts, at, to), w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,Hq,H,D,L,window", [(2, 4, 2, 64, 3000, 0), (300, 16, 2, 128, 3000, 0),
                                               (500, 8, 8, 64, 700, 200)])
def test_attention_with_weights(cc, dt, n, Hq, H, D, L, window):  # noqa: F811
    import torch

    say(f"graph: attention {dt} {n} {Hq} {H} {D} {L}")
    B, page = 3, 16
    cols = -(-L // page)
    g = torch.Generator(device="cuda").manual_seed(n)
    kind = torch_dtype(dt)
    k, v = (torch.randn((B * cols, H, page, D), generator=g, device="cuda").to(kind) for _ in range(2))
    q = torch.randn((B * n, Hq, D), generator=g, device="cuda").to(kind)
    table = torch.randperm(B * cols, generator=g, device="cuda").int().view(B, cols)
    f = cc.rotary_frequencies(D, device="cuda")
    position = torch.arange(B * n, dtype=torch.int32, device="cuda")
    rotary = cc.Rotary(B * n, Hq, 0, D, dtype=cc.dtype_code_of(dt))
    plan = cc.ChunkAttention(B, B * n, n, Hq, H, D, B * cols, page, cols, window=window,
                             max_length=L, weights=True, dtype=cc.dtype_code_of(dt))

    class Run:
        def __init__(self):
            self.q = torch.zeros_like(q)
            self.out, self.lse = torch.zeros_like(q), torch.zeros(B * n, Hq, device="cuda")
            self.w = torch.zeros(B, H, cols * page, device="cuda")
            self.lengths, self.starts = ints([L, L // 2, n]), ints([0, n, 2 * n, 3 * n])
            self.ws = torch.empty(max(plan.workspace_bytes, 16), dtype=torch.uint8, device="cuda")

        def step(self):
            s = torch.cuda.current_stream().cuda_stream
            rotary(self.q.data_ptr(), None, position.data_ptr(), f.data_ptr(), self.q.data_ptr(),
                   None, s)
            plan(self.q.data_ptr(), k.data_ptr(), v.data_ptr(), table.data_ptr(),
                 self.lengths.data_ptr(), self.starts.data_ptr(), None, self.out.data_ptr(),
                 self.lse.data_ptr(), self.w.data_ptr(), self.ws.data_ptr(), self.ws.numel(), s)

        def fresh(self, lengths, starts):
            self.lengths.copy_(ints(lengths))
            self.starts.copy_(ints(starts))
            self.q.copy_(q)
            for t in (self.out, self.lse, self.w):
                t.zero_()

    cases = [([L, L // 2 + n, n], [0, n, n + 1, 2 * n]), ([n, L, 0], [0, 1, n + 1, n + 1]),
             ([L, L, L], [0, n, 2 * n, 3 * n])]
    eager, runs = Run(), [Run(), Run()]
    want = []
    for c in cases:
        eager.fresh(*c)
        eager.step()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (eager.out, eager.lse, eager.w)])
    graphs = [record(r.step) for r in runs]
    for i in range(6):
        for j, (r, graph) in enumerate(zip(runs, graphs)):
            r.fresh(*cases[(i + j) % 3])
            graph.replay()
        eager.fresh(*cases[i % 3])
        eager.step()
        torch.cuda.synchronize()
        for j, r in enumerate(runs):
            for a, b in zip((r.out, r.lse, r.w), want[(i + j) % 3]):
                assert torch.equal(a, b), (i, j)
