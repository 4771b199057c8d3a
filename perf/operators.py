"""Cases of the decoder-block operators: the paged cache (append, one-token
attention, eviction), cross attention and the normalised gated residual.

Each pass runs either the library's kernels (`own`) or the plain form of the
same operator in elementary fp32 torch operations; `exact` is the definition
in 64 bits, written apart from the plain form."""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"f32": 0, "bf16": 1, "f16": 2}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one 80 ms frame of one stream: a codec decoder's block with a sliding window of 250
        # frames, in fp32 as such decoders run; the smallest call, all latency
        dict(name="paged frame", op="paged", dtype="f32", B=1, Hq=8, Hkv=8, D=64, page=16,
             longest=1000, ragged=False, window=250, weights=False),
        # a serving batch of streams of very different ages, grouped heads
        dict(name="paged serving batch", op="paged", dtype="bf16", B=48, Hq=32, Hkv=8, D=128,
             page=16, longest=8192, ragged=True, window=0, weights=False),
        # few long sessions whose cache is kept bounded: the weights are accumulated too
        dict(name="paged long weights", op="paged", dtype="f16", B=3, Hq=24, Hkv=4, D=128, page=64,
             longest=100003, ragged=True, window=0, weights=True),
        # the step's own row of every stream of a batch
        dict(name="append step", op="append", dtype="bf16", B=48, Hkv=8, D=128, page=16, n=1,
             longest=8192, ragged=False),
        # prompts of different lengths entering the cache
        dict(name="append prompts", op="append", dtype="f16", B=8, Hkv=8, D=128, page=64, n=4099,
             longest=16384, ragged=True),
        # a frame-by-frame decoder that lets its cache grow by 64 frames and cuts it back
        dict(name="evict frames", op="evict", dtype="f32", B=4, Hkv=8, D=64, page=16, longest=320,
             keep=256, sink=4, recent=32, ragged=False),
        # long sessions cut back to a budget
        dict(name="evict sessions", op="evict", dtype="f16", B=8, Hkv=8, D=128, page=64,
             longest=40001, keep=32768, sink=4, recent=1024, ragged=True),
        # one token of each stream against its text encoder's states
        dict(name="cross token", op="cross", dtype="bf16", B=16, Lq=1, Lk=1500, Hq=16, Hkv=16, D=64,
             ragged=True, masked=False),
        # a whole sequence against another one: matrix products on both sides
        dict(name="cross sequences", op="cross", dtype="bf16", B=4, Lq=4000, Lk=2000, Hq=16, Hkv=16,
             D=128, ragged=False, masked=False),
        # the two branches of a separation model's decoder, fp32, padded states masked
        dict(name="cross branches", op="cross", dtype="f32", B=2, Lq=1723, Lk=431, Hq=8, Hkv=8, D=64,
             ragged=True, masked=True),
        # the seam between two blocks for one frame of a few streams
        dict(name="norm frame", op="norm", dtype="bf16", rows=8, C=512, post="none", pre="layer",
             gate="none", per=1),
        # the same seam over long prompts, with a norm and a gate on the block's output
        dict(name="norm prompts", op="norm", dtype="bf16", rows=32768, C=2048, post="rms",
             pre="rms", gate="sigmoid", per=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["paged", "paged", "append", "evict", "cross", "cross", "norm"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, 40000),
                    C=8 * _log(rng, 8, 512) if rng.random() < 0.7 else _log(rng, 65, 6000),
                    post=rng.choice(["none", "rms", "layer"]),
                    pre=rng.choice(["none", "rms", "layer"]),
                    gate=rng.choice(["none", "linear", "sigmoid", "tanh"]),
                    per=rng.choice([1, 1, 7, 100]))
    D = rng.choice([32, 64, 64, 80, 96, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 8, 12])
    G = rng.choice([1, 1, 2, 4, 6, 8, 16])
    page = rng.choice([1, 8, 16, 16, 24, 64, 128, 256])
    if op == "cross":
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 32),
                    Lq=1 if rng.random() < 0.35 else _log(rng, 2, 4000), Lk=_log(rng, 1, 9000),
                    Hq=Hkv * G, Hkv=Hkv, D=D, ragged=rng.random() < 0.5,
                    masked=rng.random() < 0.4)
    longest = _log(rng, 1, 100000)
    c = dict(op=op, dtype=dtype, B=_log(rng, 1, 64))
    if op == "paged":
        c.update(Hq=Hkv * G, Hkv=Hkv, D=D, page=page, longest=longest,
                 ragged=rng.random() < 0.7,
                 window=_log(rng, 1, longest) if rng.random() < 0.3 else 0,
                 weights=rng.random() < 0.5)
    elif op == "append":
        c.update(Hkv=Hkv, D=D, page=page, n=1 if rng.random() < 0.4 else _log(rng, 2, 5000),
                 ragged=rng.random() < 0.6)
        c["longest"] = max(longest, c["n"])
    else:
        longest = max(longest, 16)
        keep = max(8, int(longest * rng.uniform(0.4, 1.02)))
        c.update(Hkv=Hkv, D=D, page=page, longest=longest, keep=keep, sink=rng.choice([0, 1, 4]),
                 recent=_log(rng, 1, max(1, keep // 4)), ragged=rng.random() < 0.6)
    return c


def _memory(c):
    """Values that the plain form holds at once, more or less."""
    if c["op"] == "norm":
        return 4 * c["rows"] * c["C"]
    if c["op"] == "cross":
        return (c["B"] * c["Hq"] * c["Lq"] * c["Lk"] + 2 * c["B"] * c["Hq"] * (c["Lq"] + c["Lk"])
                * c["D"])
    return 2 * c["B"] * c["Hkv"] * c["D"] * (c["longest"] + c["page"])


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
        if c["op"] == "cross" and c["dtype"] == "f32" and w["flops"] > t[1] / 8:
            continue
        return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


class State:
    pass


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


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


def _lengths(g, c, low, high):
    if not c["ragged"]:
        return torch.full((c["B"],), high, dtype=torch.int32, device="cuda")
    n = torch.randint(low, high + 1, (c["B"],), generator=g, device="cuda", dtype=torch.int32)
    n[0] = high
    return n


def _cache(s, c, g):
    """A pool of pages, every sequence's pages scattered over it, two pages of the pool unused."""
    s.cols = -(-c["longest"] // c["page"])
    s.pool = c["B"] * s.cols + 2
    order = torch.randperm(s.pool, generator=g, device="cuda")[:c["B"] * s.cols]
    s.table = order.to(torch.int32).view(c["B"], s.cols).contiguous()
    shape = (s.pool, c["Hkv"], c["page"], c["D"])
    s.k, s.v = (_filled(g, shape, DTYPES[c["dtype"]]) for _ in range(2))
    s.cap = s.cols * c["page"]


def _paged_state(s, c, g):
    dt = DTYPES[c["dtype"]]
    _cache(s, c, g)
    s.q = _normal(g, (c["B"], c["Hq"], c["D"]), dt)
    s.lengths = _lengths(g, c, 1, c["longest"])
    s.weights = (torch.rand((c["B"], c["Hkv"], s.cap), generator=g, device="cuda")
                 if c["weights"] else None)
    s.out = torch.empty_like(s.q)
    s.lse = torch.empty((c["B"], c["Hq"]), device="cuda")


def _append_state(s, c, g):
    dt = DTYPES[c["dtype"]]
    _cache(s, c, g)
    s.k_new, s.v_new = (_normal(g, (c["B"], c["n"], c["Hkv"], c["D"]), dt) for _ in range(2))
    s.counts = _lengths(g, c, 0, c["n"])
    past = (torch.rand((c["B"],), generator=g, device="cuda") * (c["longest"] - c["n"] + 1)).int()
    s.lengths = torch.minimum(past, torch.full_like(past, c["longest"] - c["n"])) + s.counts
    s.now = s.lengths + 5
    s.positions = torch.arange(s.cap, device="cuda", dtype=torch.int32).repeat(c["B"], c["Hkv"], 1)
    s.weights = torch.rand((c["B"], c["Hkv"], s.cap), generator=g, device="cuda")


def _evict_state(s, c, g):
    _cache(s, c, g)
    s.lengths = _lengths(g, c, min(c["longest"], max(1, c["keep"] // 2)), c["longest"])
    s.now = s.lengths + 100
    # a few positions with most of the weight, many with hardly any
    s.weights = torch.rand((c["B"], c["Hkv"], s.cap), generator=g, device="cuda").pow(8) * 50
    # earlier evictions have filled holes out of order and dropped 100 positions
    at = torch.arange(s.cap, device="cuda", dtype=torch.int32).repeat(c["B"], c["Hkv"], 1)
    turned = 2 * (s.lengths // 4)[:, None, None]
    s.positions = torch.where(at < turned, at ^ 1, at + 100).int()
    s.weights_out = torch.empty((c["B"], c["Hkv"], c["keep"]), device="cuda")
    s.positions_out, s.source = (torch.empty((c["B"], c["Hkv"], c["keep"]), device="cuda",
                                             dtype=torch.int32) for _ in range(2))
    s.lengths_out = torch.empty_like(s.lengths)


def _cross_state(s, c, g):
    dt = DTYPES[c["dtype"]]
    s.q = _normal(g, (c["B"], c["Lq"], c["Hq"], c["D"]), dt)
    s.k, s.v = (_normal(g, (c["B"], c["Lk"], c["Hkv"], c["D"]), dt) for _ in range(2))
    s.lengths = _lengths(g, c, 0, c["Lk"]) if c["ragged"] else None
    s.mask = ((torch.rand((c["B"], c["Lk"]), generator=g, device="cuda") < 0.8).to(torch.uint8)
              if c["masked"] else None)
    s.out = torch.empty_like(s.q)
    s.lse = torch.empty((c["B"], c["Hq"], c["Lq"]), device="cuda")


def _norm_state(s, c, g):
    dt = DTYPES[c["dtype"]]
    rows, C = c["rows"], c["C"]
    s.x, s.h = _normal(g, (rows, C), dt, 2.0), _normal(g, (rows, C), dt)
    s.gate = _normal(g, (-(-rows // c["per"]), C), dt) if c["gate"] != "none" else None
    s.scale = _normal(g, (C,), dt, 0.1)

    def norm(kind):
        w = None if kind == "none" else (1 + _normal(g, (C,), dt, 0.1)).to(dt)
        return w, _normal(g, (C,), dt, 0.1) if kind == "layer" else None

    s.post_w, s.post_b = norm(c["post"])
    s.pre_w, s.pre_b = norm(c["pre"])
    s.x_out = torch.empty_like(s.x)
    s.y = torch.empty_like(s.x) if c["pre"] != "none" else None


def _plan(s, c):
    """The library's plan and workspace, which a program keeps from call to call."""
    from vision_upsampler_decoders_amd import ctconv as C

    op, dt = c["op"], CODES[c["dtype"]]
    if op == "paged":
        s.plan = C.PagedAttention(c["B"], c["Hq"], c["Hkv"], c["D"], s.pool, c["page"], s.cols,
                                  max_length=c["longest"], window=c["window"],
                                  weights=c["weights"], dtype=dt)
    elif op == "append":
        s.plan = C.CacheAppend(c["B"], c["n"], c["Hkv"], c["D"], s.pool, c["page"], s.cols,
                               dtype=dt)
    elif op == "evict":
        s.plan = C.CacheEvict(c["B"], c["Hkv"], c["D"], s.pool, c["page"], s.cols, c["keep"],
                              max_length=c["longest"], sink=c["sink"], recent=c["recent"],
                              dtype=dt)
    elif op == "cross":
        s.plan = C.CrossAttention(c["B"], c["Lq"], c["Lk"], c["Hq"], c["Hkv"], c["D"], dtype=dt)
    else:
        kinds = {"none": C.NORM_NONE, "rms": C.NORM_RMS, "layer": C.NORM_LAYER}
        gates = {"none": C.GATE_NONE, "linear": C.GATE_LINEAR, "sigmoid": C.GATE_SIGMOID,
                 "tanh": C.GATE_TANH}
        s.plan = C.NormResidual(c["rows"], c["C"], post=kinds[c["post"]], pre=kinds[c["pre"]],
                                gate=gates[c["gate"]], rows_per_gate=c["per"], eps=1e-5, dtype=dt)
    need = getattr(s.plan, "workspace_bytes", 0)
    s.ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None


def prepare(case, seed):
    s = State()
    s.case = case
    g = _gen(seed)
    {"paged": _paged_state, "append": _append_state, "evict": _evict_state, "cross": _cross_state,
     "norm": _norm_state}[case["op"]](s, case, g)
    if own:
        _plan(s, case)
    return s


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------


def _p(t):
    return None if t is None else t.data_ptr()


def _run_own(s):
    stream = torch.cuda.current_stream().cuda_stream
    op = s.case["op"]
    if op == "paged":
        ws = s.ws
        s.plan(s.q.data_ptr(), s.k.data_ptr(), s.v.data_ptr(), s.table.data_ptr(),
               s.lengths.data_ptr(), s.out.data_ptr(), s.lse.data_ptr(), _p(s.weights), _p(ws),
               0 if ws is None else ws.numel(), stream)
        return [s.out, s.lse] + ([s.weights] if s.weights is not None else [])
    if op == "append":
        s.plan(s.k_new.data_ptr(), s.v_new.data_ptr(), s.k.data_ptr(), s.v.data_ptr(),
               s.table.data_ptr(), s.lengths.data_ptr(), s.counts.data_ptr(), s.now.data_ptr(),
               s.positions.data_ptr(), s.weights.data_ptr(), stream)
        return [s.k, s.v, s.positions, s.weights]
    if op == "evict":
        s.plan(s.k.data_ptr(), s.v.data_ptr(), s.table.data_ptr(), s.lengths.data_ptr(),
               s.now.data_ptr(), s.weights.data_ptr(), s.positions.data_ptr(),
               s.weights_out.data_ptr(), s.positions_out.data_ptr(), s.lengths_out.data_ptr(),
               s.source.data_ptr(), stream)
        return [s.k, s.v, s.weights_out, s.positions_out, s.lengths_out, s.source]
    if op == "cross":
        ws = s.ws
        s.plan(s.q.data_ptr(), s.k.data_ptr(), s.v.data_ptr(), _p(s.lengths), _p(s.mask),
               s.out.data_ptr(), s.lse.data_ptr(), _p(ws), 0 if ws is None else ws.numel(), stream)
        return [s.out, s.lse]
    s.plan(s.x.data_ptr(), s.h.data_ptr(), _p(s.post_w), _p(s.post_b), s.scale.data_ptr(),
           _p(s.gate), _p(s.pre_w), _p(s.pre_b), s.x_out.data_ptr(), _p(s.y), stream)
    return [s.x_out] + ([s.y] if s.y is not None else [])


# ---------------------------------------------------------------------------
# The plain forms: elementary torch operations in fp32
# ---------------------------------------------------------------------------


def _attend(q, k, v, seen, scale):
    """q [B, H, M, D], k and v [B, H, L, D], seen [B, 1, 1, L]: out, log-sum-exp and weights in
    fp32; rows that see nothing give zeros and minus infinity."""
    scores = torch.matmul(q * scale, k.transpose(2, 3)).masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    return torch.matmul(p, v), (top + torch.log(total)).squeeze(-1), p


def _plain_paged(s):
    c = s.case
    B, Hkv, D, L = c["B"], c["Hkv"], c["D"], s.cap
    G = c["Hq"] // Hkv
    rows = s.table.long()
    k, v = (t[rows].transpose(1, 2).reshape(B, Hkv, L, D).float() for t in (s.k, s.v))
    at = torch.arange(L, device="cuda")[None, :]
    n = s.lengths[:, None]
    seen = at < n
    if c["window"]:
        seen = seen & (at >= n - c["window"])
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    o, lse, p = _attend(s.q.float().view(B, Hkv, G, D), k, v, seen[:, None, None, :],
                        1 / math.sqrt(D))
    s.out.copy_(o.reshape(B, Hkv * G, D))
    got = [s.out, lse.reshape(B, Hkv * G)]
    if s.weights is not None:
        s.weights += p.sum(2)
        got.append(s.weights)
    return got


def _plain_append(s):
    c = s.case
    i = torch.arange(c["n"], device="cuda")[None, :]
    new = i < s.counts[:, None]
    b, i = torch.nonzero(new, as_tuple=True)
    back = s.counts[b] - i
    slot = (s.lengths[b] - back).long()
    page, off = s.table[b, slot // c["page"]].long(), slot % c["page"]
    s.k[page, :, off] = s.k_new[b, i]
    s.v[page, :, off] = s.v_new[b, i]
    s.positions[b, :, slot] = (s.now[b] - back)[:, None].int().expand(-1, c["Hkv"])
    s.weights[b, :, slot] = 0.0
    return [s.k, s.v, s.positions, s.weights]


def _plain_evict(s):
    c = s.case
    B, H, L, keep, page = c["B"], c["Hkv"], s.cap, c["keep"], c["page"]
    at = torch.arange(L, device="cuda")
    n = s.lengths[:, None, None]
    live = at < n
    w = s.weights.clamp(max=torch.finfo(torch.float32).max)
    w = torch.where(torch.isnan(w), torch.full_like(w, -math.inf), w)
    safe = (s.positions < c["sink"]) | (s.positions >= s.now[:, None, None] - c["recent"])
    w = torch.where(safe, torch.full_like(w, math.inf), w)
    w = torch.where(live, w, torch.full_like(w, -math.inf))
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(-1, order, at.expand(B, H, L))
    m = n.clamp(max=keep)
    kept = rank < m
    holes = ~kept & (at < m)
    spare = kept & (at >= m)
    spares = torch.sort((~spare).int(), dim=-1, stable=True)[1]
    nth = (torch.cumsum(holes.int(), -1) - 1).clamp(min=0)
    src = torch.where(holes, spares.gather(-1, nth), at.expand(B, H, L))
    if L < keep:
        more = torch.arange(L, keep, device="cuda").expand(B, H, keep - L)
        src = torch.cat([src, more], -1)
    src, to = src[..., :keep], torch.arange(keep, device="cuda")
    there = to < m
    src = torch.where(there, src, torch.zeros_like(src))
    s.weights_out.copy_(torch.where(there, s.weights.gather(-1, src), torch.zeros((), device="cuda")))
    s.positions_out.copy_(torch.where(there, s.positions.gather(-1, src).long(), -1))
    s.source.copy_(torch.where(there, src, -1))
    s.lengths_out.copy_(m.view(-1))
    b, h, j = torch.nonzero(there & (src != to), as_tuple=True)
    i = src[b, h, j]
    p0, p1 = s.table[b, i // page].long(), s.table[b, j // page].long()
    s.k[p1, h, j % page] = s.k[p0, h, i % page]
    s.v[p1, h, j % page] = s.v[p0, h, i % page]
    return [s.k, s.v, s.weights_out, s.positions_out, s.lengths_out, s.source]


def _plain_cross(s):
    c = s.case
    B, Lq, Lk, Hkv, D = c["B"], c["Lq"], c["Lk"], c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    q = s.q.float().view(B, Lq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Lq, D)
    k, v = (t.float().transpose(1, 2).contiguous() for t in (s.k, s.v))
    seen = torch.ones((B, Lk), dtype=torch.bool, device="cuda")
    if s.lengths is not None:
        seen = seen & (torch.arange(Lk, device="cuda")[None, :] < s.lengths[:, None])
    if s.mask is not None:
        seen = seen & (s.mask != 0)
    o, lse, _ = _attend(q, k, v, seen[:, None, None, :], 1 / math.sqrt(D))
    s.out.copy_(o.view(B, Hkv, G, Lq, D).permute(0, 3, 1, 2, 4).reshape(B, Lq, Hkv * G, D))
    return [s.out, lse.view(B, Hkv * G, Lq)]


def _normed(x, kind, w, b, eps):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    return x + b.float() if b is not None else x


def _plain_norm(s):
    c = s.case
    h = s.h.float()
    if c["post"] != "none":
        h = _normed(h, c["post"], s.post_w, s.post_b, 1e-5)
    h = h * s.scale.float()
    if s.gate is not None:
        t = s.gate.float()
        t = torch.sigmoid(t) if c["gate"] == "sigmoid" else torch.tanh(t) if c["gate"] == "tanh" else t
        h = h * t.repeat_interleave(c["per"], 0)[:c["rows"]]
    x = s.x.float() + h
    s.x_out.copy_(x)
    if s.y is None:
        return [s.x_out]
    s.y.copy_(_normed(x, c["pre"], s.pre_w, s.pre_b, 1e-5))
    return [s.x_out, s.y]


def run(state):
    if own:
        return _run_own(state)
    return {"paged": _plain_paged, "append": _plain_append, "evict": _plain_evict,
            "cross": _plain_cross, "norm": _plain_norm}[state.case["op"]](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits, one sequence and head at a time
# ---------------------------------------------------------------------------


def _softmax_rows(q, k, v, scale):
    """q [M, D], k and v [n, D] in 64 bits: out, log-sum-exp, weights."""
    if k.shape[0] == 0:
        return (torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=q.dtype,
                                                device=q.device), q.new_zeros(q.shape[0], 0))
    t = (q @ k.T) * scale
    lse = torch.logsumexp(t, -1)
    p = torch.exp(t - lse[:, None])
    return p @ v, lse, p


def _slots(s, c, b, slots):
    return s.table[b].long()[slots // c["page"]], slots % c["page"]


def _exact_paged(s, c):
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Hq), dtype=torch.float64, device="cuda")
    weights = s.weights.double() if s.weights is not None else None
    for b, n in enumerate(s.lengths.tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        page, off = _slots(s, c, b, torch.arange(first, n, device="cuda"))
        for h in range(Hkv):
            r = slice(h * G, (h + 1) * G)
            out[b, r], lse[b, r], p = _softmax_rows(s.q[b, r].double(), s.k[page, h, off].double(),
                                                    s.v[page, h, off].double(), D ** -0.5)
            if weights is not None:
                weights[b, h, first:n] += p.sum(0)
    return [out, lse] + ([weights] if weights is not None else [])


def _exact_append(s, c):
    k, v, positions, weights = s.k.double(), s.v.double(), s.positions.clone(), s.weights.double()
    for b, (n, m, now) in enumerate(zip(s.lengths.tolist(), s.counts.tolist(), s.now.tolist())):
        page, off = _slots(s, c, b, torch.arange(n - m, n, device="cuda"))
        for h in range(c["Hkv"]):
            k[page, h, off] = s.k_new[b, :m, h].double()
            v[page, h, off] = s.v_new[b, :m, h].double()
        positions[b, :, n - m:n] = torch.arange(now - m, now, device="cuda", dtype=torch.int32)
        weights[b, :, n - m:n] = 0
    return [k, v, positions, weights]


def _exact_evict(s, c):
    k, v = s.k.double(), s.v.double()
    w_out = torch.zeros_like(s.weights_out, dtype=torch.float64)
    p_out, source = torch.full_like(s.positions_out, -1), torch.full_like(s.source, -1)
    l_out = s.lengths.clamp(max=c["keep"])
    for b, (n, now) in enumerate(zip(s.lengths.tolist(), s.now.tolist())):
        m = min(n, c["keep"])
        for h in range(c["Hkv"]):
            w, pos = s.weights[b, h, :n].double(), s.positions[b, h, :n]
            safe = (pos < c["sink"]) | (pos >= now - c["recent"])
            score = torch.where(safe, torch.full_like(w, math.inf), w)
            # the m best: those above the m-th largest score, then the first ones equal to it
            edge = torch.sort(score)[0][n - m]
            sure = score > edge
            level = torch.nonzero(score == edge).view(-1)[:m - int(sure.sum())]
            sure[level] = True
            src = torch.arange(m, device="cuda")
            src[~sure[:m]] = torch.nonzero(sure[m:]).view(-1) + m
            w_out[b, h, :m], p_out[b, h, :m], source[b, h, :m] = w[src], pos[src], src.int()
            p0, o0 = _slots(s, c, b, src)
            p1, o1 = _slots(s, c, b, torch.arange(m, device="cuda"))
            k[p1, h, o1] = s.k[p0, h, o0].double()
            v[p1, h, o1] = s.v[p0, h, o0].double()
    return [k, v, w_out, p_out, l_out, source]


def _exact_cross(s, c):
    B, Lq, Lk, Hq, Hkv, D = (c[n] for n in ("B", "Lq", "Lk", "Hq", "Hkv", "D"))
    out = torch.zeros((B, Lq, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Hq, Lq), dtype=torch.float64, device="cuda")
    n = s.lengths.tolist() if s.lengths is not None else [Lk] * B
    for b in range(B):
        at = torch.arange(n[b], device="cuda")
        if s.mask is not None:
            at = at[s.mask[b, :n[b]] != 0]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            out[b, :, h], lse[b, h], _ = _softmax_rows(s.q[b, :, h].double(),
                                                       s.k[b, at, g].double(),
                                                       s.v[b, at, g].double(), D ** -0.5)
    return [out, lse]


def _exact_norm(s, c):
    def norm(x, kind, w, b):
        if kind == "rms":
            return x / torch.sqrt(x.square().mean(1) + 1e-5)[:, None] * w.double()
        var, mean = torch.var_mean(x, 1, correction=0)
        return (x - mean[:, None]) / torch.sqrt(var + 1e-5)[:, None] * w.double() + b.double()

    h = s.h.double()
    if c["post"] != "none":
        h = norm(h, c["post"], s.post_w, s.post_b)
    factor = s.scale.double()[None, :]
    if s.gate is not None:
        t = s.gate.double()
        t = {"linear": lambda u: u, "sigmoid": lambda u: 1 / (1 + torch.exp(-u)),
             "tanh": torch.tanh}[c["gate"]](t)
        factor = factor * t[torch.arange(c["rows"], device="cuda") // c["per"]]
    x = s.x.double() + factor * h
    return [x] if c["pre"] == "none" else [x, norm(x, c["pre"], s.pre_w, s.pre_b)]


def exact(case, seed):
    s = State()
    g = _gen(seed)
    {"paged": _paged_state, "append": _append_state, "evict": _evict_state, "cross": _cross_state,
     "norm": _norm_state}[case["op"]](s, case, g)
    return {"paged": _exact_paged, "append": _exact_append, "evict": _exact_evict,
            "cross": _exact_cross, "norm": _exact_norm}[case["op"]](s, case)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    c = case
    e = ESIZE[c["dtype"]]
    if c["op"] == "norm":
        gate = 0 if c["gate"] == "none" else -(-c["rows"] // c["per"])
        moved = 3 + (c["pre"] != "none")
        return {"bytes": e * c["C"] * (moved * c["rows"] + gate + 5), "flops": 12.0 * c["rows"] * c["C"]}
    if c["op"] == "cross":
        half = 0.5 if c["ragged"] else 1.0
        row = e * c["D"]
        return {"bytes": c["B"] * (2 * c["Lq"] * c["Hq"] * row + 2 * half * c["Lk"] * c["Hkv"] * row
                                   + 4 * c["Hq"] * c["Lq"]),
                "flops": 4.0 * half * c["B"] * c["Hq"] * c["Lq"] * c["Lk"] * c["D"]}
    row = e * c["D"] * c["Hkv"]
    mean = c["longest"] * (0.5 + 0.5 / c["B"] if c["ragged"] else 1.0)
    if c["op"] == "paged":
        if c["window"]:
            mean = min(mean, c["window"])
        acc = 8 * c["Hkv"] * mean if c["weights"] else 0
        return {"bytes": c["B"] * (2 * mean * row + acc + 2 * c["Hq"] * c["D"] * e),
                "flops": 4.0 * c["B"] * mean * c["Hq"] * c["D"]}
    if c["op"] == "append":
        n = c["n"] * (0.5 + 0.5 / c["B"] if c["ragged"] else 1.0)
        return {"bytes": c["B"] * n * (4 * row + 8 * c["Hkv"]), "flops": 0}
    low = min(c["longest"], max(1, c["keep"] // 2))
    mean = (low + c["longest"]) / 2 if c["ragged"] else c["longest"]
    # sequences past the budget lose the excess; the kept share of it moves into holes
    span = max(1, c["longest"] - low) if c["ragged"] else 1
    over = max(0.0, c["longest"] - c["keep"])
    share = min(1.0, over / span) * 0.5 if c["ragged"] else 1.0
    moved = share * over * min(1.0, c["keep"] / c["longest"])
    return {"bytes": c["B"] * (c["Hkv"] * (8 * mean + 12 * min(mean, c["keep"])) + 4 * moved * row),
            "flops": 0}
