"""Cases of the operators that take requests of many lengths into the paged
cache: page tables and row maps from request lengths, rotary positions (alone,
and on the way into the cache), and attention of a chunk of new rows.

Each pass runs either the library's kernels (`own`) or the plain form of the
same operator in elementary torch operations; `exact` is the definition in 64
bits, written apart from the plain form."""

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"f32": 0, "bf16": 1, "f16": 2}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}

# scaled frequencies: every position's angles as within this factor of a shorter context
FACTOR, ORIGINAL, LOW, HIGH = 8.0, 4096, 1.0, 4.0
RAMP_LOW, RAMP_HIGH = 1.0, 32.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one step of a serving batch, a row for each sequence: the smallest call, all latency
        dict(name="pages step", op="pages", B=48, page=16, longest=8192, new=1, Hkv=8, spare=50,
             turnover=False, slots=True),
        # a third of the requests has ended, a third is new with its whole prompt, a third goes on
        dict(name="pages turnover", op="pages", B=96, page=16, longest=4096, new=4096, Hkv=8,
             spare=100, turnover=True, slots=False),
        # frames of a few streams, fp32, pairs side by side
        dict(name="rotary frames", op="rotary", dtype="f32", rows=8, Hq=8, Hk=8, D=64, R=64,
             layout="pairs", scaling="none", far=1000),
        # long prompts, far positions of a stretched context
        dict(name="rotary prompts", op="rotary", dtype="bf16", rows=32768, Hq=32, Hk=8, D=128,
             R=128, layout="half", scaling="dims", far=1000000),
        # a serving step's rows on their way into the cache
        dict(name="rotary append step", op="append", dtype="bf16", rows=48, Hq=32, Hk=8, D=128,
             R=128, layout="half", scaling="turns", far=8192, page=16),
        # packed prompts, half of each head turned, a few rows of padding behind them
        dict(name="rotary append prompts", op="append", dtype="f16", rows=16397, Hq=24, Hk=8,
             D=128, R=64, layout="half", scaling="linear", far=100000, page=64),
        # two frames at a time of one stream, a window of 250 of its slots, fp32
        dict(name="chunk frames", op="chunk", dtype="f32", B=1, n=2, Hq=8, Hkv=8, D=64, page=16,
             longest=1000, window=250, fill="full", weights=False),
        # a batch that proposes eight rows each and attends to all of them at once
        dict(name="chunk proposals", op="chunk", dtype="bf16", B=24, n=8, Hq=32, Hkv=8, D=128,
             page=16, longest=8192, window=0, fill="ragged", weights=False),
        # prompts of different lengths, packed, with what the cache held before them
        dict(name="chunk prompts", op="chunk", dtype="bf16", B=8, n=4099, Hq=32, Hkv=8, D=128,
             page=16, longest=8192, window=0, fill="ragged", weights=False),
        # one long prompt's next piece among sequences that go on by one row
        dict(name="chunk mixed", op="chunk", dtype="bf16", B=48, n=2048, Hq=32, Hkv=8, D=128,
             page=16, longest=16384, window=0, fill="mixed", weights=False),
        # a prompt into a cache that is bounded by the weights which its slots have drawn
        dict(name="chunk weights", op="chunk", dtype="f16", B=2, n=4096, Hq=24, Hkv=4, D=128,
             page=64, longest=32768, window=0, fill="full", weights=True),
        # the same with narrow heads in fp32 and a window
        dict(name="chunk window", op="chunk", dtype="f32", B=4, n=1723, Hq=8, Hkv=8, D=64, page=24,
             longest=4001, window=1000, fill="ragged", weights=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["pages", "rotary", "append", "chunk", "chunk", "chunk"])
    page = rng.choice([1, 8, 16, 16, 24, 64, 128, 256])
    if op == "pages":
        longest = max(page, _log(rng, 1, 16384))
        turnover = rng.random() < 0.5
        return dict(op=op, B=_log(rng, 1, 256), page=page, longest=longest,
                    new=_log(rng, 1, longest) if turnover or rng.random() < 0.4 else 1,
                    Hkv=rng.choice([1, 2, 4, 8]), spare=rng.choice([-3, 0, 7, 200]),
                    turnover=turnover, slots=rng.random() < 0.5)
    dtype = rng.choice(["f32", "bf16", "f16"])
    D = rng.choice([32, 64, 64, 80, 96, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 8, 12])
    G = rng.choice([1, 1, 2, 4, 6, 8])
    if op != "chunk":
        part = rng.choice([1.0, 1.0, 0.5, 0.25, 0.4])
        c = dict(op=op, dtype=dtype, rows=_log(rng, 1, 40000), Hq=Hkv * G, Hk=Hkv, D=D,
                 R=2 * max(1, int(D * part) // 2), layout=rng.choice(["half", "half", "pairs"]),
                 scaling=rng.choice(["none", "linear", "base", "dims", "turns"]),
                 far=_log(rng, 1, 2000000))
        if op == "append":
            c["page"] = page
        return c
    longest = _log(rng, 1, 65536)
    fill = rng.choice(["full", "ragged", "ragged", "mixed"])
    return dict(op=op, dtype=dtype, B=_log(rng, 1, 48), n=_log(rng, 1, min(longest, 5000)),
                Hq=Hkv * G, Hkv=Hkv, D=D, page=page, longest=longest,
                window=_log(rng, 1, longest) if rng.random() < 0.3 else 0, fill=fill,
                weights=rng.random() < 0.3)


def _memory(c):
    """Values that the plain form holds at once, more or less."""
    if c["op"] == "pages":
        return c["B"] * (-(-c["longest"] // c["page"]) + c["new"] + c["slots"] * c["Hkv"] * c["longest"])
    if c["op"] == "chunk":
        return c["Hq"] * c["n"] * c["longest"] + 2 * c["B"] * c["Hkv"] * c["longest"] * c["D"]
    return c["rows"] * (c["Hq"] + c["Hk"]) * c["D"]


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["op"], [0, 0, 0])
        t[0] = max(t[0], w["bytes"])
        t[1] = max(t[1], w["flops"])
        t[2] = max(t[2], _memory(c))
    while True:
        c = _drawn(rng)
        w, t = work(c), top[c["op"]]
        if w["bytes"] > t[0] or w["flops"] > t[1] or _memory(c) > t[2]:
            continue
        if c["op"] == "chunk" and c["dtype"] == "f32" and w["flops"] > t[1] / 16:
            continue
        return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


class State:
    pass


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 6007 + 29)


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _filled(g, shape, dtype):
    """Normal values for the large buffers, generated in slices (the fp32 temporary stays small)."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    flat = t.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda"))
    return t


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _lengths(c):
    """A case's lengths are the same for every seed, in another order (the buffers' sizes follow
    from their sums); they are on the host too: a scheduler knows its requests' lengths."""
    return random.Random(str((c["op"], c["B"], c["longest"])))


def _shuffled(g, items):
    return [items[i] for i in torch.randperm(len(items), generator=g, device="cuda").tolist()]


def _pages_state(s, c, g):
    B, page = c["B"], c["page"]
    s.cols = -(-c["longest"] // page)
    rng, requests = _lengths(c), []  # (slots before, new rows, slots after)
    for b in range(B):
        part = b % 3 if c["turnover"] else 2
        past, more = rng.randint(0, c["longest"]), rng.randint(1, c["new"])
        if part == 0:  # ended
            requests.append((past, 0, 0))
        elif part == 1:  # new
            requests.append((0, more, more))
        else:  # going on, by a row or a few
            n = 1 if c["turnover"] else more
            past = min(past, c["longest"] - n)
            requests.append((past, n, past + n))
    old, counts, lengths = zip(*_shuffled(g, requests))
    evicted = torch.randint(0, 501, (B,), generator=g, device="cuda", dtype=torch.int32)
    held = [-(-v // page) for v in old]
    need = [-(-v // page) for v in lengths]
    s.num_pages = max(sum(held), sum(need) + c["spare"], 1)
    order = torch.randperm(s.num_pages, generator=g, device="cuda").int()
    at = torch.arange(s.cols, device="cuda")[None, :]
    h = _ints(held)
    first = torch.cumsum(h, 0) - h
    index = (first[:, None] + at).clamp(max=s.num_pages - 1)
    s.table = torch.where(at < h[:, None], order[index], -1).int().contiguous()
    free = s.num_pages - sum(held)
    s.free_pages = torch.full((s.num_pages,), -1, dtype=torch.int32, device="cuda")
    s.free_pages[:free] = order[sum(held):]
    s.free_count, s.held = _ints([free]), h
    s.lengths, s.counts = _ints(lengths), _ints(counts)
    s.now = s.lengths + evicted
    s.rows = sum(counts) + 5  # the step's buffers have room for a few rows more
    s.held_out, s.free_count_out = torch.empty_like(s.held), torch.empty_like(s.free_count)
    s.row_starts = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    s.row_positions, s.row_slots = (torch.empty(s.rows, dtype=torch.int32, device="cuda")
                                    for _ in range(2))
    s.positions = s.weights = None
    if c["slots"]:
        shape = (B, c["Hkv"], s.cols * page)
        s.positions = torch.full(shape, -7, dtype=torch.int32, device="cuda")
        s.weights = torch.rand(shape, generator=g, device="cuda")


def _rotary_state(s, c, g):
    dt = DTYPES[c["dtype"]]
    rows, D = c["rows"], c["D"]
    # q, k and v of a row lie behind each other, as one product with the weights leaves them
    qkv = _filled(g, (rows, c["Hq"] + 2 * c["Hk"], D), dt)
    s.q, s.k, s.v = qkv.split((c["Hq"], c["Hk"], c["Hk"]), 1)
    s.positions = torch.randint(0, c["far"] + 1, (rows,), generator=g, device="cuda",
                                dtype=torch.int32)
    if rows > 8:
        s.positions[-5:] = -1  # padding
    s.q_out = torch.zeros((rows, c["Hq"], D), dtype=dt, device="cuda")
    s.scale = 0.1 * math.log(FACTOR) + 1 if c["scaling"] == "dims" else 1.0
    if c["op"] == "rotary":
        s.k_out = torch.zeros((rows, c["Hk"], D), dtype=dt, device="cuda")
        return
    s.num_pages = -(-rows // c["page"]) + 3
    # runs of slots within pages, the pages in any order
    run = torch.arange(rows, device="cuda")
    pages = torch.randperm(s.num_pages, generator=g, device="cuda")
    slots = pages[run // c["page"]] * c["page"] + run % c["page"]
    s.slots = torch.where(s.positions < 0, -1, slots).int()
    shape = (s.num_pages, c["Hk"], c["page"], D)
    s.k_cache, s.v_cache = (torch.zeros(shape, dtype=dt, device="cuda") for _ in range(2))


def _chunk_state(s, c, g):
    dt = DTYPES[c["dtype"]]
    B, n, page = c["B"], c["n"], c["page"]
    if c["fill"] == "full":
        s.n_new = [n] * B
        s.n_all = [c["longest"]] * B
    else:
        rng = _lengths(c)
        new = [1 if c["fill"] == "mixed" else rng.randint(0, n) for _ in range(B - 1)] + [n]
        past = [rng.randint(0, c["longest"] - n) for _ in range(B)]
        past[0] = c["longest"] - new[0]
        s.n_new, s.n_all = zip(*_shuffled(g, [(m, p + m) for m, p in zip(new, past)]))
    s.cols = -(-c["longest"] // page)
    s.pool = B * s.cols + 2
    order = torch.randperm(s.pool, generator=g, device="cuda")[:B * s.cols]
    s.table = order.to(torch.int32).view(B, s.cols).contiguous()
    shape = (s.pool, c["Hkv"], page, c["D"])
    s.k, s.v = (_filled(g, shape, dt) for _ in range(2))
    s.rows = sum(s.n_new) + (0 if c["fill"] == "full" else 3)
    s.q = _filled(g, (s.rows, c["Hq"], c["D"]), dt)
    s.lengths = _ints(s.n_all)
    starts = [0]
    for v in s.n_new:
        starts.append(starts[-1] + v)
    s.row_starts = _ints(starts)
    s.starts = starts
    s.out = torch.zeros_like(s.q)
    s.lse = torch.zeros((s.rows, c["Hq"]), device="cuda")
    s.weights = (torch.rand((B, c["Hkv"], s.cols * page), generator=g, device="cuda")
                 if c["weights"] else None)


STATES = {"pages": _pages_state, "rotary": _rotary_state, "append": _rotary_state,
          "chunk": _chunk_state}


def _frequencies(c):
    """Radians per position of every pair, in 64 bits."""
    R, base = c["R"], 10000.0
    i = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    if c["scaling"] == "base" and R > 2:
        base *= FACTOR ** (R / (R - 2))
    f = base ** (-2 * i / R)
    if c["scaling"] == "linear":
        f = f / FACTOR
    if c["scaling"] == "turns":
        keep = ((ORIGINAL * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / FACTOR
    if c["scaling"] == "dims":
        def pair(turns):  # that makes so many turns in the original context
            return R * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo = max(math.floor(pair(RAMP_HIGH)), 0)
        hi = min(math.ceil(pair(RAMP_LOW)), R - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / FACTOR
    return f


def _plan(s, c):
    """The library's plan, workspace and frequencies, which a program keeps from call to call."""
    from vision_upsampler_decoders_amd import ctconv as C

    s.ws = None
    if c["op"] == "pages":
        s.plan = C.CachePages(c["B"], s.rows, s.num_pages, c["page"], s.cols, Hkv=c["Hkv"])
        return
    dt = CODES[c["dtype"]]
    if c["op"] == "chunk":
        s.plan = C.ChunkAttention(c["B"], s.rows, c["n"], c["Hq"], c["Hkv"], c["D"], s.pool,
                                  c["page"], s.cols, max_length=c["longest"], window=c["window"],
                                  weights=c["weights"], dtype=dt)
        if s.plan.workspace_bytes:
            s.ws = torch.empty(s.plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        return
    kind = {"none": C.ROTARY_NONE, "linear": C.ROTARY_LINEAR, "base": C.ROTARY_BASE,
            "dims": C.ROTARY_RAMP_DIMS, "turns": C.ROTARY_RAMP_TURNS}[c["scaling"]]
    low, high = (RAMP_LOW, RAMP_HIGH) if c["scaling"] == "dims" else (LOW, HIGH)
    s.frequencies = C.rotary_frequencies(c["R"], 10000.0, kind, FACTOR, ORIGINAL, low, high,
                                         device="cuda")
    layout = C.ROTARY_HALF if c["layout"] == "half" else C.ROTARY_PAIRS
    row = tuple(s.q.stride()[:2])
    if c["op"] == "rotary":
        s.plan = C.Rotary(c["rows"], c["Hq"], c["Hk"], c["D"], R=c["R"], layout=layout,
                          scale=s.scale, dtype=dt, q_strides=row, k_strides=row)
    else:
        s.plan = C.RotaryAppend(c["rows"], c["Hq"], c["Hk"], c["D"], s.num_pages, c["page"],
                                R=c["R"], layout=layout, scale=s.scale, dtype=dt, q_strides=row,
                                new_strides=row)


def prepare(case, seed):
    s = State()
    s.case = case
    g = _gen(seed)
    STATES[case["op"]](s, case, g)
    if own:
        _plan(s, case)
    elif case["op"] in ("rotary", "append"):
        s.frequencies = _frequencies(case)
    return s


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------


def _p(t):
    return None if t is None else t.data_ptr()


def _run_own(s):
    stream = torch.cuda.current_stream().cuda_stream
    op = s.case["op"]
    if op == "pages":
        s.plan(s.lengths.data_ptr(), s.counts.data_ptr(), s.now.data_ptr(), s.held.data_ptr(),
               s.free_count.data_ptr(), s.table.data_ptr(), s.free_pages.data_ptr(),
               s.held_out.data_ptr(), s.free_count_out.data_ptr(), s.row_starts.data_ptr(),
               s.row_positions.data_ptr(), s.row_slots.data_ptr(), _p(s.positions), _p(s.weights),
               stream)
        return _pages_out(s)
    if op == "rotary":
        s.plan(s.q.data_ptr(), s.k.data_ptr(), s.positions.data_ptr(), s.frequencies.data_ptr(),
               s.q_out.data_ptr(), s.k_out.data_ptr(), stream)
        return [s.q_out, s.k_out]
    if op == "append":
        s.plan(s.q.data_ptr(), s.k.data_ptr(), s.v.data_ptr(), s.positions.data_ptr(),
               s.slots.data_ptr(), s.frequencies.data_ptr(), s.q_out.data_ptr(),
               s.k_cache.data_ptr(), s.v_cache.data_ptr(), stream)
        return [s.q_out, s.k_cache, s.v_cache]
    ws = s.ws
    s.plan(s.q.data_ptr(), s.k.data_ptr(), s.v.data_ptr(), s.table.data_ptr(),
           s.lengths.data_ptr(), s.row_starts.data_ptr(), None, s.out.data_ptr(), s.lse.data_ptr(),
           _p(s.weights), _p(ws), 0 if ws is None else ws.numel(), stream)
    return [s.out, s.lse] + ([s.weights] if s.weights is not None else [])


def _pages_out(s):
    out = [s.table, s.held_out, s.free_pages, s.free_count_out, s.row_starts, s.row_positions,
           s.row_slots]
    return out + ([s.positions, s.weights] if s.positions is not None else [])


# ---------------------------------------------------------------------------
# The plain forms: elementary torch operations, fp32 (angles in 64 bits)
# ---------------------------------------------------------------------------


def _plain_pages(s):
    c = s.case
    page = c["page"]
    at = torch.arange(s.cols, device="cuda")[None, :]
    held = s.held.clamp(0, s.cols).long()
    need = (s.lengths.clamp(0, s.cols * page).long() + page - 1) // page
    # what is given back goes on the stack, sequence by sequence
    back = s.table[(at >= need[:, None]) & (at < held[:, None])]
    top = s.free_count.long() + back.numel()
    s.free_pages[s.free_count.long() + torch.arange(back.numel(), device="cuda")] = back
    # what is taken comes from its top, sequence by sequence
    grow = (need - held).clamp(min=0)
    first = torch.cumsum(grow, 0) - grow
    nth = first[:, None] + at - held[:, None]
    taken = s.free_pages[(top - 1 - nth).clamp(0, s.num_pages - 1)]
    taken = torch.where(nth < top, taken, -1)
    s.table.copy_(torch.where((at >= held[:, None]) & (at < need[:, None]), taken, s.table))
    got = torch.minimum(grow, (top - first).clamp(min=0))
    s.held_out.copy_(torch.minimum(held, need) + got)
    s.free_count_out.copy_(top - got.sum())
    s.row_starts[0] = 0
    s.row_starts[1:] = torch.cumsum(s.counts, 0)
    r = torch.arange(s.rows, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s.row_starts[1:], r, right=True)
    there = b < c["B"]
    b = b.clamp(max=c["B"] - 1)
    back = s.row_starts[1:][b] - r
    s.row_positions.copy_(torch.where(there, s.now[b] - back, -1))
    t = (s.lengths[b] - back).long().clamp(min=0)
    p = s.table[b, (t // page).clamp(max=s.cols - 1)]
    s.row_slots.copy_(torch.where(there & (p >= 0), p * page + t % page, -1))
    if s.positions is not None:
        b, t, at_row = b[there], t[there], s.row_positions[there]
        s.positions[b, :, t] = at_row[:, None].expand(-1, c["Hkv"])
        s.weights[b, :, t] = 0.0
    return _pages_out(s)


def _turned(x, s):
    """x [rows, H, D] turned by the rows' angles, in fp32."""
    c = s.case
    R = c["R"]
    angle = s.positions.double()[:, None] * s.frequencies[None, :]
    cos, sin = ((f(angle) * s.scale).float()[:, None, :] for f in (torch.cos, torch.sin))
    x = x.float()
    out = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        out[..., :R // 2], out[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        out[..., 0:R:2], out[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    return out


def _plain_rotary(s):
    there = (s.positions >= 0)[:, None, None]
    s.q_out.copy_(torch.where(there, _turned(s.q, s), s.q_out.float()))
    s.k_out.copy_(torch.where(there, _turned(s.k, s), s.k_out.float()))
    return [s.q_out, s.k_out]


def _plain_append(s):
    page = s.case["page"]
    there = s.positions >= 0
    s.q_out.copy_(torch.where(there[:, None, None], _turned(s.q, s), s.q_out.float()))
    there = there & (s.slots >= 0)
    slot = s.slots[there].long()
    s.k_cache[slot // page, :, slot % page] = _turned(s.k, s)[there].to(s.k_cache.dtype)
    s.v_cache[slot // page, :, slot % page] = s.v[there]
    return [s.q_out, s.k_cache, s.v_cache]


def _plain_chunk(s):
    c = s.case
    Hkv, D = c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    for b, (n, L) in enumerate(zip(s.n_new, s.n_all)):
        if n == 0:
            continue
        rows = slice(s.starts[b], s.starts[b + 1])
        pages = s.table[b, :-(-L // c["page"])].long()
        k, v = (t[pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].float() for t in (s.k, s.v))
        q = s.q[rows].float().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
        scores = torch.matmul(q * D ** -0.5, k.transpose(1, 2)).view(Hkv, G, n, L)
        end = torch.arange(L - n + 1, L + 1, device="cuda")[:, None]
        at = torch.arange(L, device="cuda")[None, :]
        hidden = at >= end
        if c["window"]:
            hidden = hidden | (at < end - c["window"])
        scores.masked_fill_(hidden, -math.inf)
        top = scores.amax(-1, keepdim=True)
        p = scores.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        p.div_(total)
        o = torch.matmul(p.view(Hkv, G * n, L), v).view(Hkv, G, n, D)
        s.out[rows] = o.permute(2, 0, 1, 3).reshape(n, Hkv * G, D).to(s.out.dtype)
        s.lse[rows] = (top + torch.log(total)).view(Hkv * G, n).T
        if s.weights is not None:
            s.weights[b, :, :L] += p.sum((1, 2))
    return [s.out, s.lse] + ([s.weights] if s.weights is not None else [])


def run(state):
    if own:
        return _run_own(state)
    return {"pages": _plain_pages, "rotary": _plain_rotary, "append": _plain_append,
            "chunk": _plain_chunk}[state.case["op"]](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_pages(s, c):
    """The stack of free pages as a list, one sequence after the other."""
    page = c["page"]
    table, held = s.table.tolist(), s.held.tolist()
    lengths, counts, now = s.lengths.tolist(), s.counts.tolist(), s.now.tolist()
    stack = s.free_pages.tolist()
    count = s.free_count.tolist()[0]
    need = [-(-n // page) for n in lengths]
    for b in range(c["B"]):
        for p in table[b][need[b]:held[b]]:
            stack[count] = p
            count += 1
        held[b] = min(held[b], need[b]) if held[b] > need[b] else held[b]
    for b in range(c["B"]):
        for j in range(held[b], need[b]):
            if count > 0:
                count -= 1
                table[b][j] = stack[count]
                held[b] += 1
            else:
                table[b][j] = -1
    starts, positions, slots = [0], [], []
    pos = s.positions.cpu() if c["slots"] else None
    weights = s.weights.double().cpu() if c["slots"] else None
    for b in range(c["B"]):
        starts.append(starts[-1] + counts[b])
        for i in range(counts[b]):
            t = lengths[b] - counts[b] + i
            p = table[b][t // page]
            positions.append(now[b] - counts[b] + i)
            slots.append(p * page + t % page if p >= 0 else -1)
        if c["slots"]:
            span = slice(lengths[b] - counts[b], lengths[b])
            pos[b, :, span] = torch.arange(now[b] - counts[b], now[b], dtype=torch.int32)
            weights[b, :, span] = 0
    rest = [-1] * (s.rows - len(slots))
    out = [_ints(v) for v in (table, held, stack, [count], starts, positions + rest, slots + rest)]
    return out + ([pos.cuda(), weights.cuda()] if c["slots"] else [])


def _exact_turned(x, positions, c, scale):
    """Each pair as a complex number times e^(i angle)."""
    R, half = c["R"], c["R"] // 2
    turn = torch.polar(torch.full((), scale, dtype=torch.float64, device="cuda"),
                       torch.outer(positions.double(), _frequencies(c)))[:, None, :]
    y = x.double()
    if c["layout"] == "half":
        z = torch.complex(y[..., :half], y[..., half:R]) * turn
        return torch.cat([z.real, z.imag, y[..., R:]], -1)
    z = torch.view_as_complex(y[..., :R].reshape(*y.shape[:-1], half, 2).contiguous()) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), y[..., R:]], -1)


def _exact_rotary(s, c):
    live = s.positions >= 0
    out = []
    for x in (s.q, s.k):
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        y[live] = _exact_turned(x[live], s.positions[live], c, s.scale)
        out.append(y)
    if c["op"] == "rotary":
        return out
    rows = torch.nonzero(live).view(-1)
    p, at = s.slots[rows].long() // c["page"], s.slots[rows].long() % c["page"]
    k, v = (torch.zeros(s.k_cache.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for h in range(c["Hk"]):
        k[p, h, at] = out[1][rows, h]
        v[p, h, at] = s.v[rows, h].double()
    return [out[0], k, v]


def _exact_chunk(s, c):
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    out = torch.zeros(s.out.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s.lse.shape, dtype=torch.float64, device="cuda")
    weights = s.weights.double() if s.weights is not None else None
    for b, (n, L) in enumerate(zip(s.n_new, s.n_all)):
        slot = torch.arange(L, device="cuda")
        where = (s.table[b].long()[slot // page], slot % page)
        last = slot[L - n:, None]  # the slot of each new row itself
        seen = slot <= last
        if c["window"]:
            seen &= slot > last - c["window"]
        for h in range(Hkv if n else 0):
            k, v = s.k[where[0], h, where[1]].double(), s.v[where[0], h, where[1]].double()
            for j in range(h * G, (h + 1) * G):
                r = slice(s.starts[b], s.starts[b] + n)
                t = (s.q[r, j].double() @ k.T) / math.sqrt(D)
                t = torch.where(seen, t, -math.inf)
                lse[r, j] = torch.logsumexp(t, 1)
                p = torch.exp(t - lse[r, j, None])
                out[r, j] = p @ v
                if weights is not None:
                    weights[b, h, :L] += p.sum(0)
    return [out, lse] + ([weights] if weights is not None else [])


def exact(case, seed):
    if case["op"] == "chunk" and work(case)["flops"] > 2e13:
        return None
    s = State()
    STATES[case["op"]](s, case, _gen(seed))
    return {"pages": _exact_pages, "rotary": _exact_rotary, "append": _exact_rotary,
            "chunk": _exact_chunk}[case["op"]](s, case)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "pages":
        third = c["B"] / 3
        if c["turnover"]:
            rows = third * (c["new"] + 1) / 2 + third
            moved = third * (c["longest"] + c["new"]) / 2 / c["page"] + third / c["page"]
        else:
            rows = c["B"] * (c["new"] + 1) / 2
            moved = rows / c["page"]
        per_row = 8 + 4 / c["page"] + (8 * c["Hkv"] if c["slots"] else 0)
        return {"bytes": 24 * c["B"] + 8 * moved + rows * per_row, "flops": 0}
    e = ESIZE[c["dtype"]]
    if c["op"] != "chunk":
        heads = c["Hq"] + c["Hk"] * (2 if c["op"] == "append" else 1)
        index = 4 if c["op"] == "rotary" else 8
        return {"bytes": c["rows"] * (2 * heads * c["D"] * e + index) + 4 * c["R"],
                "flops": 3.0 * c["rows"] * (c["Hq"] + c["Hk"]) * c["R"]}
    B, n = c["B"], c["n"]
    if c["fill"] == "full":
        part = [(B, n, c["longest"])]
    else:  # (how many, their new rows, all their rows), in the mean
        past = (c["longest"] - n) / 2
        new = 1 if c["fill"] == "mixed" else n / 2
        part = [(B - 1, new, past + new), (1, n, past + n)]
    flops = rows = read = 0.0
    for m, new, length in part:
        seen = length - new / 2
        if c["window"]:
            seen = min(seen, c["window"])
        flops += m * new * seen * c["Hq"] * c["D"] * (6.0 if c["weights"] else 4.0)
        rows += m * new
        read += m * (min(length, c["window"] + new) if c["window"] else length)
    row = e * c["D"] * c["Hkv"]
    return {"bytes": 2 * read * row + rows * c["Hq"] * (2 * c["D"] * e + 4)
            + (8 * read * c["Hkv"] if c["weights"] else 0), "flops": flops}
