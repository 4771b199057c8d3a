"""Host-only checks of the C entry points of the operators on requests of many
lengths: argument validation before any launch, workspace sizes, the table form
and the Python plans' refusals (no device call is made by any of these)."""

import ctypes
import math

import pytest

from test_block_abi_host import (ALIGN, DTYPE, NULL, P, PARAM, SHAPE, WORKSPACE, arr,  # noqa: F401
                                 lib)
from vision_upsampler_decoders_amd import ctconv as C


def _arr(v):
    return None if v is None else arr(*v)


NAMES = ("lengths", "counts", "now", "held", "free_count", "table", "free", "held_out",
         "count_out", "starts", "at", "to", "positions", "weights")


def _pages(lib, B=2, rows=6, H=4, pages=10, page=16, cols=5, ts=5, slot=(320, 80), **kw):
    bufs = dict(zip(NAMES, [*P, 0x100000, 0x110000]))
    bufs.update(kw)
    return lib.ctconv_cache_pages(*[bufs[n] for n in NAMES], B, rows, H, pages, page, cols, ts,
                                  _arr(slot), None)


def test_pages_validation(lib):  # noqa: F811
    assert _pages(lib, B=0, lengths=None, table=None) == 0
    for name in ("lengths", "held", "free_count", "table", "free", "held_out", "count_out",
                 "starts", "at", "to", "slot"):
        assert _pages(lib, **{name: None}) == NULL, name
    for kw in (dict(B=-1), dict(B=8193), dict(rows=-1), dict(rows=1 << 31), dict(H=0),
               dict(H=65536), dict(pages=0), dict(page=0), dict(cols=0), dict(ts=-1), dict(ts=4),
               dict(page=1 << 20, cols=1 << 12), dict(pages=1 << 30), dict(page=1 << 24, pages=200),
               dict(B=8192, cols=1 << 18, page=1), dict(slot=(-1, 80)), dict(slot=(320, 79)),
               dict(slot=(319, 80)), dict(slot=(1 << 62, 80))):
        assert _pages(lib, **kw) == SHAPE, kw
    for name in NAMES:
        assert _pages(lib, **{name: 0x10002}) == ALIGN, name


def _rotary(lib, q=P[0], k=P[1], pos=P[2], f=P[3], qo=P[4], ko=P[5], rows=7, Hq=4, Hk=2, D=64, R=64,
            qs=(384, 64), ks=(384, 64), qos=(256, 64), kos=(128, 64), layout=0, scale=1.0, dt=1):
    return lib.ctconv_rotary(q, k, pos, f, qo, ko, rows, Hq, Hk, D, R, _arr(qs), _arr(ks),
                             _arr(qos), _arr(kos), layout, scale, dt, None)


ROTARY_SHAPES = (dict(rows=-1), dict(rows=1 << 31), dict(Hq=-1), dict(Hq=65536), dict(D=60),
                 dict(D=264), dict(D=0), dict(R=0), dict(R=63), dict(R=66), dict(R=-2),
                 dict(qs=(-384, 64)), dict(qos=(255 // 8 * 8, 64)), dict(qos=(256, 56)),
                 dict(qos=(0, 64)), dict(qos=(1 << 62, 64)))


def test_rotary_validation(lib):  # noqa: F811
    assert _rotary(lib, rows=0, q=None, pos=None) == 0
    for name in ("q", "k", "pos", "f", "qo", "ko", "qs", "ks", "qos", "kos"):
        assert _rotary(lib, **{name: None}) == NULL, name
    for kw in ROTARY_SHAPES + (dict(Hq=0, Hk=0), dict(kos=(127 // 8 * 8, 64)), dict(Hk=70000)):
        assert _rotary(lib, **kw) == SHAPE, kw
    for kw in (dict(layout=2), dict(layout=-1), dict(scale=math.inf), dict(scale=math.nan),
               dict(qo=P[0]), dict(ko=P[1])):  # in place with other strides
        assert _rotary(lib, **kw) == PARAM, kw
    for dt in (3, -1):
        assert _rotary(lib, dt=dt) == DTYPE
    for kw in (dict(q=0x1008), dict(ko=0x1004), dict(f=0x1008), dict(pos=0x1002),
               dict(qs=(388, 64)), dict(kos=(128, 68))):
        assert _rotary(lib, **kw) == ALIGN, kw
    # what a call without queries or keys does not use
    assert _rotary(lib, Hq=0, q=None, qo=None, qs=None, qos=None, f=None) == NULL
    assert _rotary(lib, Hk=0, k=None, ko=None, ks=None, kos=None, R=63) == SHAPE


def _rappend(lib, q=P[0], k=P[1], v=P[2], pos=P[3], slots=P[4], f=P[5], qo=P[6], kc=P[7], vc=P[8],
             rows=7, Hq=4, Hk=2, D=64, R=64, pages=10, page=16, qs=(512, 64), new=(512, 64),
             qos=(256, 64), kv=(2048, 64, 1024), layout=0, scale=1.0, dt=1):
    return lib.ctconv_rotary_append(q, k, v, pos, slots, f, qo, kc, vc, rows, Hq, Hk, D, R, pages,
                                    page, _arr(qs), _arr(new), _arr(qos), _arr(kv), layout, scale,
                                    dt, None)


def test_rotary_append_validation(lib):  # noqa: F811
    assert _rappend(lib, rows=0, k=None) == 0
    for name in ("q", "k", "v", "pos", "slots", "f", "qo", "kc", "vc", "qs", "new", "qos", "kv"):
        assert _rappend(lib, **{name: None}) == NULL, name
    for kw in ROTARY_SHAPES + (dict(Hk=0), dict(pages=0), dict(page=0), dict(pages=1 << 30),
                               dict(new=(-512, 64)), dict(kv=(2048, 64, 0)),
                               dict(kv=(2040, 64, 1024)), dict(kv=(0, 64, 1024)),
                               dict(kv=(1 << 62, 64, 1024))):
        assert _rappend(lib, **kw) == SHAPE, kw
    for kw in (dict(layout=5), dict(scale=math.nan), dict(qo=P[0])):
        assert _rappend(lib, **kw) == PARAM, kw
    assert _rappend(lib, dt=9) == DTYPE
    for kw in (dict(v=0x1008), dict(vc=0x1004), dict(slots=0x1001), dict(new=(516, 64)),
               dict(kv=(2048, 66, 1024))):
        assert _rappend(lib, **kw) == ALIGN, kw
    assert _rappend(lib, Hq=0, q=None, qo=None, qs=None, qos=None, slots=None) == NULL


def test_frequencies_validation(lib):  # noqa: F811
    out = (ctypes.c_double * 128)()
    f = lib.ctconv_rotary_frequencies
    at = ctypes.addressof(out)
    good = dict(R=64, base=1e4, kind=3, factor=8.0, original=4096.0, low=1.0, high=32.0, out=at)

    def call(**kw):
        a = {**good, **kw}
        return f(a["R"], a["base"], a["kind"], a["factor"], a["original"], a["low"], a["high"],
                 a["out"])

    assert call() == 0 and out[0] == 1.0
    for R in (0, 1, 63, 258, -2, 1 << 40):
        assert call(R=R) == SHAPE
    for kw in (dict(kind=5), dict(kind=-1), dict(base=0.0), dict(base=-1.0), dict(base=math.inf),
               dict(base=1.0), dict(factor=0.0), dict(factor=math.nan), dict(original=0.0),
               dict(low=0.0), dict(high=1.0), dict(high=math.inf), dict(kind=4, high=0.5),
               dict(kind=4, original=math.nan)):
        assert call(**kw) == PARAM, kw
    assert call(kind=0, original=-1.0, low=9.0, high=1.0, base=0.5) == 0  # not used
    assert call(out=None) == NULL


def _chunk(lib, q=P[0], k=P[1], v=P[2], table=P[3], lengths=P[4], starts=P[9], counts=None,
           out=P[5], lse=P[6], w=None, B=2, rows=9, n=6, Hq=8, H=4, D=64, pages=10, page=16, cols=5,
           maxlen=80, window=0, qs=(0, 512, 64), kv=(4096, 64, 1024), os_=(0, 512, 64), ts=5,
           slot=(320, 80), scale=0.1, dt=1, ws=P[8], nb=1 << 40):
    return lib.ctconv_chunk_attention(q, k, v, table, lengths, starts, counts, out, lse, w, B, rows,
                                      n, Hq, H, D, pages, page, cols, maxlen, window, _arr(qs),
                                      _arr(kv), _arr(os_), ts, _arr(slot), scale, dt, ws, nb, None)


def test_chunk_attention_validation(lib):  # noqa: F811
    for kw in (dict(B=0), dict(rows=0), dict(n=0)):
        assert _chunk(lib, q=None, out=None, **kw) == 0
    for name in ("q", "k", "v", "table", "lengths", "out", "qs", "kv", "os_"):
        assert _chunk(lib, **{name: None}) == NULL, name
    assert _chunk(lib, w=P[7], slot=None) == NULL
    padded = dict(starts=None, rows=10, n=5, qs=(2560, 512, 64), os_=(2560, 512, 64))
    for kw in (dict(B=-1), dict(rows=-1), dict(n=-1), dict(Hq=0), dict(Hq=6), dict(H=0), dict(D=60),
               dict(D=512), dict(pages=0), dict(maxlen=81), dict(maxlen=-1), dict(window=-1),
               dict(kv=(-1, 64, 1024)), dict(qs=(0, -512, 64)), dict(os_=(0, 1 << 62, 64)),
               dict(os_=(0, 511 // 8 * 8, 64)), dict(os_=(0, 0, 64)), dict(ts=-5),
               dict(n=1 << 29), dict(w=P[7], slot=(1, -1)), dict(w=P[7], slot=(0, 80)),
               dict(w=P[7], slot=(320, 40)), {**padded, "rows": 9}, {**padded, "rows": 11},
               {**padded, "os_": (2048, 512, 64)}, {**padded, "os_": (0, 512, 64)}):
        assert _chunk(lib, **kw) == SHAPE, kw
    for s in (math.inf, math.nan, -math.inf):
        assert _chunk(lib, scale=s) == PARAM
    assert _chunk(lib, dt=-1) == DTYPE
    for kw in (dict(q=8), dict(k=0x1001), dict(v=0x1008), dict(out=0x1002), dict(ws=0x1008),
               dict(qs=(0, 512, 60)), dict(kv=(4097, 64, 1024)), {**padded, "qs": (2561, 512, 64)}):
        assert _chunk(lib, **kw) == ALIGN, kw
    need = C.ctconv_chunk_attention_workspace_bytes(2, 9, 6, 8, 4, 64, 80, 0, True, 1)
    assert need >= 9 * 8 * 4
    assert _chunk(lib, w=P[7], ws=None) == WORKSPACE
    assert _chunk(lib, w=P[7], nb=need - 1) == WORKSPACE


def test_chunk_attention_index_alignment_and_most_rows(lib):  # noqa: F811
    for kw in (dict(table=P[3] + 2), dict(lengths=P[4] + 1), dict(starts=P[9] + 2),
               dict(lse=P[6] + 2), dict(w=P[7] + 2),
               dict(starts=None, rows=10, n=5, qs=(2560, 512, 64), os_=(2560, 512, 64),
                    counts=P[9] + 2)):
        assert _chunk(lib, **kw) == ALIGN, kw
    # the kernels step past the last row: no int32 may end there
    for weights in (False, True):
        with pytest.raises(C.CtconvError) as e:
            C.ctconv_chunk_attention_workspace_bytes(1, 9, 2 ** 31 - 1, 1, 1, 64, 80, 0, weights, 1)
        assert e.value.status == SHAPE
        with pytest.raises(C.CtconvError) as e:
            C.ctconv_chunk_attention_workspace_bytes(1, 9, 2 ** 29 - 1, 4, 1, 64, 80, 0, weights, 1)
        assert e.value.status == SHAPE
    assert C.ctconv_chunk_attention_workspace_bytes(1, 9, 2 ** 20, 1, 1, 64, 80, 0, False, 1) == 0


def test_chunk_attention_workspace(lib):  # noqa: F811
    f = C.ctconv_chunk_attention_workspace_bytes
    assert f(0, 0, 1, 8, 4, 64, 10000, 0, False, 1) == 0
    assert f(1, 2, 2, 8, 8, 64, 250, 0, False, 0) == 0         # one workgroup per head: no join
    long = f(1, 2, 2, 8, 8, 128, 100000, 0, False, 1)
    assert long >= 2 * 8 * 2 * (128 + 2) * 4                    # split
    assert f(1, 2, 2, 8, 8, 128, 100000, 200, False, 1) == 0    # the window bounds it
    assert f(1, 2, 2, 8, 8, 128, 100000, 0, True, 1) == long + 64
    assert lib.ctconv_chunk_attention_workspace_bytes(1, 1, 1, 8, 8, 128, 1, 0, 0, 1, None) == NULL
    for a in ((1, 1, 1, 8, 3, 64, 1, 0, 0, 1), (1, 1, 1, 8, 8, 4, 1, 0, 0, 1),
              (1, 1, 1, 8, 8, 64, -1, 0, 0, 1), (1, -1, 1, 8, 8, 64, 1, 0, 0, 1)):
        with pytest.raises(C.CtconvError) as e:
            f(*a)
        assert e.value.status == SHAPE


def test_table_form_reaches_each_function(lib):  # noqa: F811
    run = lib.ctconv_block_run
    bufs = (ctypes.c_void_p * 14)(*P, 0x100000, 0x110000)

    def bits(x):
        return ctypes.c_int64.from_buffer_copy(ctypes.c_double(x)).value

    pages = [2, 6, 4, 10, 16, 5, 5, 320, 80]
    rotary = [7, 4, 2, 64, 64, 384, 64, 384, 64, 256, 64, 128, 64, 0, bits(1.0), 1]
    rappend = [7, 4, 2, 64, 64, 10, 16, 512, 64, 512, 64, 256, 64, 2048, 64, 1024, 0, bits(1.0), 1]
    chunk = [2, 9, 6, 8, 4, 64, 10, 16, 5, 80, 0, 0, 512, 64, 4096, 64, 1024, 0, 512, 64, 5, 320, 80,
             bits(0.1), 1]

    def call(op, z, **kw):
        z = list(z)
        for i, v in kw.items():
            z[int(i[1:])] = v
        return run(op, arr(*z), bufs, None, 0, None)

    for op in (5, 6, 15, 20):
        assert call(op, chunk) == PARAM
    for op, z in ((17, rotary), (18, rappend), (19, chunk)):
        for bad in (3, -1, 1 << 40):
            assert call(op, z, **{f"_{len(z) - 1}": bad}) == DTYPE, (op, bad)
    assert call(16, pages, _0=0) == 0
    assert call(16, pages, _6=4) == SHAPE
    assert call(16, pages, _8=79) == SHAPE
    assert call(17, rotary, _4=63) == SHAPE
    assert call(17, rotary, _12=68) == ALIGN
    assert call(17, rotary, _13=-1) == PARAM
    assert call(17, rotary, _14=bits(math.nan)) == PARAM
    assert call(18, rappend, _6=0) == SHAPE
    assert call(18, rappend, _15=1028) == ALIGN
    assert call(18, rappend, _16=1 << 33) == PARAM
    assert call(19, chunk) == WORKSPACE  # a weight_sum is among the buffers
    assert call(19, chunk, _19=63) == ALIGN
    assert call(19, chunk, _23=bits(math.inf)) == PARAM
    assert call(19, chunk, _22=1) == SHAPE


def test_plans_raise_the_function_s_error():
    for plan, args, name in (
            (C.CachePages(2, 4, 8, 16, 3), (None,) * 14, "ctconv_cache_pages"),
            (C.Rotary(4, 2, 2, 64), (None,) * 6, "ctconv_rotary"),
            (C.RotaryAppend(4, 2, 2, 64, 8, 16), (None,) * 9, "ctconv_rotary_append"),
            (C.ChunkAttention(2, 4, 2, 2, 2, 64, 8, 16, 3), (None,) * 11 + (0,),
             "ctconv_chunk_attention")):
        with pytest.raises(C.CtconvError, match=name) as e:
            plan(*args, 0)
        assert e.value.status == NULL


def test_helpers_refuse_host_tensors():
    import torch

    t = torch.zeros(2, 2, 8, 8)
    with pytest.raises(ValueError, match="device"):
        C.cache_pages(t, t, t, t, t)
    with pytest.raises(ValueError, match="device"):
        C.rotary(t, t, t, t)
    with pytest.raises(ValueError, match="device"):
        C.rotary_append(t, t, t, t, t, t, t, t)
    with pytest.raises(ValueError, match="device"):
        C.chunk_attention(t, t, t, t, t)
