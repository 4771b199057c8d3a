"""GPU: infinities and NaN in the tiled kernel of chunk attention: in slots that no row of
the call may see, in a page of another request, and in slots that some rows see."""

import numpy as np
import pytest

import block_ref as R
import request_cases as cases
import request_ref as Q
from gpu_util import say, to_host, torch_dtype
from test_gpu_block import cc, ints  # noqa: F401

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


class Chunk:
    """The inputs of a chunk call, packed, made on the GPU; slots past the lengths are NaN."""

    def __init__(self, dt, counts, lengths, H, G, D, page=16):
        import torch

        g = torch.Generator(device="cuda").manual_seed(sum(lengths) + D)
        B, cols = len(counts), -(-max(lengths) // page)
        self.dt, self.counts, self.lengths, self.page, self.G = dt, counts, lengths, page, G
        kind = torch_dtype(dt)
        self.table = torch.randperm(B * cols + 2, generator=g, device="cuda")[:B * cols].view(B, cols)
        shape = (B * cols + 2, H, page, D)
        at = torch.arange(cols * page, device="cuda").view(1, cols, page)
        unused = at >= torch.tensor(lengths, device="cuda").view(-1, 1, 1)
        self.k, self.v = (torch.randn(shape, generator=g, device="cuda").to(kind) for _ in range(2))
        for t in (self.k, self.v):
            used = t[self.table]  # [B, cols, H, page, D]
            used[unused[:, :, None, :, None].expand_as(used)] = float("nan")
            t.fill_(float("nan"))
            t[self.table] = used
        self.q = torch.randn((sum(counts), H * G, D), generator=g, device="cuda").to(kind)
        self.starts = np.cumsum([0, *counts])
        self.window = 0

    def place(self, b, t):
        return int(self.table[b, t // self.page]), t % self.page

    def call(self, cc, k, v, scale):  # noqa: F811
        import torch

        out, lse = cc.chunk_attention(self.q, k, v, self.table.int(), ints(self.lengths),
                                      row_starts=ints(self.starts), n=max(self.counts),
                                      max_length=max(self.lengths), window=self.window, scale=scale)
        torch.cuda.synchronize()
        return out, lse

    def seen_by(self, b, t):
        """Rows of the call, as truth values, that see slot t of sequence b."""
        n, L = self.counts[b], self.lengths[b]
        at = np.arange(n) + L - n
        mine = (at >= t) & ((at < t + self.window) if self.window else True)
        res = np.zeros(len(self.q), bool)
        res[self.starts[b]:self.starts[b + 1]] = mine
        return res

    def check(self, out, lse, scale, rng, skip=None):
        """Some rows of every sequence against float64 (none of those of `skip`)."""
        H = self.k.shape[1]
        for b, (n, L) in enumerate(zip(self.counts, self.lengths)):
            if n == 0:
                continue
            rows = np.unique(np.concatenate([[0, n - 1], rng.integers(0, n, 12)]))
            if skip is not None:
                rows = rows[~skip[self.starts[b] + rows]]
            slots = np.arange(L)
            end = L - n + rows[:, None] + 1
            seen = (slots < end) & (slots >= (end - self.window if self.window else 0))
            r = self.starts[b] + rows
            got, level = to_host(out[r]), to_host(lse[r])
            q = to_host(self.q[r])
            for h in range(H):
                kr, vr = (to_host(t[self.table[b], h].reshape(-1, t.shape[-1])[:L])
                          for t in (self.k, self.v))
                for j in range(h * self.G, (h + 1) * self.G):
                    (o, l, _), (eo, el, _) = Q.seen_rows(q[:, j], kr, vr, seen, scale, self.dt)
                    R.check(got[:, j], o, eo, f"sequence {b} out")
                    R.check(level[:, j], l, el, f"sequence {b} lse")


@pytest.mark.parametrize("case", cases.ODD, ids=[str(i) for i in range(len(cases.ODD))])
def test_odd_values_reach_only_the_rows_that_see_them(cc, case):  # noqa: F811
    """An infinity or a NaN in a new slot, at the first, in the middle and at the last of those
    that not every row sees, and in one that all see: who sees it has it, in its column (of a key:
    in all); everything else has the same bits as without (of a
    value) or is as far from the definition (of a key)."""
    import torch

    dt, counts, lengths, H, G, D, window, kernel, split = case
    say(f"chunk odd values {case}")
    rng = np.random.default_rng(len(cases.ODD))
    c = Chunk(dt, counts, lengths, H, G, D)
    c.window = window
    scale = 0.1
    out, lse = c.call(cc, c.k, c.v, scale)
    c.check(out, lse, scale, rng)
    clean = out.cpu()
    mine = slice((H - 1) * G, H * G)  # the query heads of the head that is touched
    for b, (n, L) in enumerate(zip(counts, lengths)):
        slots = sorted({L - n, L - n + 1, L - n // 2 - 1, L - 1, max(L - n - 1, 0)})
        for i, t in enumerate(slots):
            p, o = c.place(b, t)
            col = (5, D - 1, 0, D // 2)[i % 4]
            for what in ("nan v", "inf v", "-inf v", "nan k"):
                if what == "-inf v" and i % 2 or what == "nan k" and not i % 2:
                    continue
                k, v = c.k, c.v.clone()
                if what == "nan k":
                    k = c.k.clone()
                value = float(what.split()[0])
                (k if what == "nan k" else v)[p, H - 1, o, col] = value
                got, level = c.call(cc, k, v, scale)
                note = f"{what} at {t} of sequence {b}"
                sees = torch.from_numpy(c.seen_by(b, t))
                got = got.cpu()
                hit = got[sees][:, mine]
                assert torch.equal(got[:, :mine.start], clean[:, :mine.start]), note
                if what == "nan k":
                    # (a row's softmax reference moves with those of its wave's other rows, so
                    # that these are the same numbers in other roundings)
                    assert bool(torch.isfinite(got[~sees]).all()), note
                    c.check(got, level, scale, rng, skip=sees.numpy())
                    assert bool(torch.isnan(hit).all()), note
                    assert bool(torch.isnan(level.cpu()[sees][:, mine]).all()), note
                    continue
                assert torch.equal(got[~sees], clean[~sees]), note
                if what == "nan v":
                    assert bool(torch.isnan(hit[..., col]).all()), note
                else:
                    assert bool((hit[..., col] == value).all()), note
                rest = [d for d in range(D) if d != col]
                assert torch.equal(hit[..., rest], clean[sees][:, mine][..., rest]), note
                assert torch.equal(level.cpu(), lse.cpu()), note
    # several in one sequence at once: opposite infinities meet in a NaN
    n, L = counts[0], lengths[0]
    v = c.v.clone()
    first, second = L - n + 1, L - 1
    for t, value in ((first, float("inf")), (second, float("-inf"))):
        p, o = c.place(0, t)
        v[p, H - 1, o, 3] = value
    got = c.call(cc, c.k, v, scale)[0].cpu()
    one, two = (torch.from_numpy(c.seen_by(0, t)) for t in (first, second))
    assert bool((got[one & ~two][:, mine, 3] == float("inf")).all())
    assert bool((got[two & ~one][:, mine, 3] == float("-inf")).all())
    assert bool(torch.isnan(got[one & two][:, mine, 3]).all())
    assert torch.equal(got[~one & ~two], clean[~one & ~two])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("n,G,L,window", [(8, 2, 600, 50), (900, 16, 1400, 100), (2000, 8, 2112, 300)])
def test_odd_rows_reach_only_the_weights_of_slots_they_see(cc, dt, n, G, L, window):  # noqa: F811
    """A NaN in a query, or in a key, makes NaN of the weights of the slots that its rows see; the
    others stay what they are, up to the roundings of the other rows' lse (a few 2^-24 of scores
    below 2^5)."""
    import torch

    say(f"odd weights {dt} {n} {G} {L} {window}")
    H, D, page = 2, 64, 16
    c = Chunk(dt, [n], [L], H, G, D)
    cap = c.table.shape[1] * page

    def weights(q, k):
        w = torch.full((1, H, cap), 0.25, device="cuda")
        cc.chunk_attention(q, k, c.v, c.table.int(), ints([L]), row_starts=ints([0, n]), n=n,
                           window=window, scale=0.1, weight_sum=w)
        torch.cuda.synchronize()
        return w.cpu()

    clean = weights(c.q, c.k)
    assert bool(torch.isfinite(clean).all())
    at = np.arange(L)
    for what in ("query", "key"):
        q, k = c.q.clone(), c.k.clone()
        row = n // 2
        own = L - n + row  # the slot of that row
        hit = np.zeros(cap, bool)
        if what == "query":
            q[row, G - 1, 3] = float("nan")
            hit[:L] = (at <= own) & (at > own - window)
        else:
            p, o = c.place(0, own)
            k[p, 0, o, 3] = float("nan")
            # rows own .. own + window - 1 see it, and so do the slots around them
            last = min(own + window - 1, L - 1)
            hit[:L] = (at <= last) & (at > own - window)
        got = weights(q, k)
        hit = torch.from_numpy(hit)
        assert bool(torch.isnan(got[0, 0, hit]).all()), what
        assert torch.equal(got[0, 1], clean[0, 1]), what
        assert torch.allclose(got[0, 0, ~hit], clean[0, 0, ~hit], rtol=1e-5, atol=0), what
