"""Host-only checks of the decoder-block operators' C entry points: argument
validation before any launch, workspace sizes, and the Python plans'
refusals (no device call is made by any of these)."""

import ctypes
import os

import pytest

from vision_upsampler_decoders_amd import ctconv as C

NULL, SHAPE, PARAM, DTYPE, ALIGN, WORKSPACE = 1, 2, 3, 4, 5, 7


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(C.LIB_PATH):
        from vision_upsampler_decoders_amd import build

        build.build()
    return C.load()


def arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


P = [0x10000 * (i + 1) for i in range(12)]  # aligned, never dereferenced by a refused call


def _append(lib, kn=P[0], vn=P[1], k=P[2], v=P[3], table=P[4], lengths=P[5], pos=P[8], w=P[9], B=2,
            n=3, H=4, D=64, pages=10, page=16, cols=5, new=(768, 256, 64), kv=(4096, 64, 1024),
            ts=5, slot=(320, 80), dt=1):
    return lib.ctconv_cache_append(kn, vn, k, v, table, lengths, None, None, pos, w, B, n, H, D,
                                   pages, page, cols, None if new is None else arr(*new),
                                   None if kv is None else arr(*kv), ts,
                                   None if slot is None else arr(*slot), dt, None)


def test_append_validation(lib):
    assert _append(lib, B=0, kn=None) == 0
    assert _append(lib, n=0, kn=None, table=None) == 0
    for name in ("kn", "vn", "k", "v", "table", "lengths", "new", "kv", "slot"):
        assert _append(lib, **{name: None}) == NULL, name
    for kw in (dict(B=-1), dict(n=-1), dict(H=0), dict(D=0), dict(D=12), dict(D=264),
               dict(pages=0), dict(page=0), dict(cols=0), dict(page=1 << 20, cols=1 << 12),
               dict(ts=-1), dict(kv=(4096, -64, 1024)), dict(kv=(1 << 62, 64, 1024)),
               dict(new=(1 << 62, 256, 64)), dict(slot=(-1, 80)), dict(B=1 << 20, n=1 << 20)):
        assert _append(lib, **kw) == SHAPE, kw
    assert _append(lib, dt=5) == DTYPE
    for kw in (dict(kn=0x1008), dict(v=0x1004), dict(new=(768, 260, 64)), dict(kv=(4096, 66, 1024))):
        assert _append(lib, **kw) == ALIGN, kw


def _paged(lib, q=P[0], k=P[1], v=P[2], table=P[3], lengths=P[4], out=P[5], lse=P[6], w=None, B=2,
           Hq=8, H=4, D=64, pages=10, page=16, cols=5, maxlen=80, window=0, qs=(512, 64),
           kv=(4096, 64, 1024), os_=(512, 64), ts=5, slot=(320, 80), scale=0.1, dt=1, ws=P[8],
           nb=1 << 30):
    return lib.ctconv_paged_attention(q, k, v, table, lengths, out, lse, w, B, Hq, H, D, pages, page,
                                      cols, maxlen, window, None if qs is None else arr(*qs),
                                      None if kv is None else arr(*kv),
                                      None if os_ is None else arr(*os_), ts,
                                      None if slot is None else arr(*slot), scale, dt, ws, nb, None)


def test_paged_attention_validation(lib):
    assert _paged(lib, B=0, q=None) == 0
    for name in ("q", "k", "v", "table", "lengths", "out", "qs", "kv", "os_"):
        assert _paged(lib, **{name: None}) == NULL, name
    assert _paged(lib, w=P[7], slot=None) == NULL
    for kw in (dict(B=-1), dict(Hq=0), dict(Hq=6), dict(H=0), dict(D=60), dict(D=512),
               dict(pages=0), dict(maxlen=81), dict(maxlen=-1), dict(window=-1),
               dict(kv=(-1, 64, 1024)), dict(qs=(-512, 64)), dict(os_=(1 << 62, 64)),
               dict(ts=-5), dict(B=1 << 30, Hq=1 << 10, H=4), dict(w=P[7], slot=(1, -1))):
        assert _paged(lib, **kw) == SHAPE, kw
    for s in (float("inf"), float("nan"), float("-inf")):
        assert _paged(lib, scale=s) == PARAM
    assert _paged(lib, dt=-1) == DTYPE
    for kw in (dict(q=8), dict(k=0x1001), dict(v=0x1008), dict(out=0x1002), dict(ws=0x1008),
               dict(qs=(512, 60)), dict(kv=(4097, 64, 1024))):
        assert _paged(lib, **kw) == ALIGN, kw
    need = C.ctconv_paged_attention_workspace_bytes(2, 8, 4, 64, 80, 0, True, 1)
    assert need > 0
    assert _paged(lib, w=P[7], ws=None) == WORKSPACE
    assert _paged(lib, w=P[7], nb=need - 1) == WORKSPACE


def test_paged_attention_workspace(lib):
    f = C.ctconv_paged_attention_workspace_bytes
    assert f(0, 8, 4, 64, 10000, 0, False, 1) == 0
    assert f(1, 8, 8, 64, 250, 0, False, 0) == 0          # one workgroup per head: no join
    long = f(1, 8, 8, 128, 100000, 0, False, 1)
    assert long >= 8 * 2 * (128 + 2) * 4                   # split
    assert f(1, 8, 8, 128, 100000, 200, False, 1) == 0     # the window bounds it
    assert f(1, 8, 8, 128, 100000, 0, True, 1) >= long + 8 * 100000 * 4  # the scores too
    assert lib.ctconv_paged_attention_workspace_bytes(1, 8, 8, 128, 1, 0, 0, 1, None) == NULL
    for a in ((1, 8, 3, 64, 1, 0, 0, 1), (1, 8, 8, 4, 1, 0, 0, 1), (1, 8, 8, 64, -1, 0, 0, 1)):
        with pytest.raises(C.CtconvError) as e:
            f(*a)
        assert e.value.status == SHAPE


def _evict(lib, k=P[0], v=P[1], table=P[2], lengths=P[3], w=P[4], pos=P[5], wo=P[6], po=P[7],
           lo=P[8], src=P[9], B=2, H=4, D=64, pages=10, page=16, cols=5, maxlen=80, keep=64, sink=4,
           recent=8, kv=(4096, 64, 1024), ts=5, slot=(320, 80), out=(256, 64), dt=1):
    return lib.ctconv_cache_evict(k, v, table, lengths, None, w, pos, wo, po, lo, src, B, H, D,
                                  pages, page, cols, maxlen, keep, sink, recent,
                                  None if kv is None else arr(*kv), ts,
                                  None if slot is None else arr(*slot),
                                  None if out is None else arr(*out), dt, None)


def test_evict_validation(lib):
    assert _evict(lib, B=0, k=None) == 0
    for name in ("k", "v", "table", "lengths", "w", "wo", "po", "src", "kv", "slot", "out"):
        assert _evict(lib, **{name: None}) == NULL, name
    for kw in (dict(keep=0), dict(sink=-1), dict(recent=-1),
               dict(wo=P[4]), dict(po=P[5])):  # in place needs the same strides
        assert _evict(lib, **kw) == PARAM, kw
    for kw in (dict(B=-2), dict(H=0), dict(D=20), dict(maxlen=81),
               dict(page=1 << 10, cols=1 << 10, maxlen=262145, slot=(1 << 22, 1 << 20),
                    kv=(1 << 18, 64, 1 << 16)), dict(slot=(-1, 80)),
               dict(out=(256, -1)), dict(kv=(4096, 64, -1)), dict(keep=1 << 31),
               dict(B=1 << 16, H=1 << 15)):
        assert _evict(lib, **kw) == SHAPE, kw
    assert _evict(lib, dt=3) == DTYPE
    assert _evict(lib, k=0x1008) == ALIGN
    assert _evict(lib, kv=(4096, 65, 1024)) == ALIGN


def _cross(lib, q=P[0], k=P[1], v=P[2], mask=None, out=P[3], B=2, Lq=5, Lk=7, Hq=8, H=4, D=64,
           qs=(2560, 512, 64), ks=(1792, 256, 64), vs=(1792, 256, 64), os_=(2560, 512, 64), ms=7,
           scale=0.1, dt=2, ws=P[4], nb=1 << 30):
    a = [None if s is None else arr(*s) for s in (qs, ks, vs, os_)]
    return lib.ctconv_cross_attention(q, k, v, None, mask, out, None, B, Lq, Lk, Hq, H, D, *a, ms,
                                      scale, dt, ws, nb, None)


def test_cross_attention_validation(lib):
    assert _cross(lib, B=0, q=None) == 0
    assert _cross(lib, Lq=0, q=None, out=None) == 0
    for name in ("q", "k", "v", "out", "qs", "ks", "vs", "os_"):
        assert _cross(lib, **{name: None}) == NULL, name
    for kw in (dict(B=-1), dict(Lq=-1), dict(Lk=-1), dict(Hq=7), dict(H=0), dict(D=4), dict(D=260),
               dict(mask=P[5], ms=-1), dict(ks=(1792, -256, 64)), dict(qs=(1 << 62, 512, 64)),
               dict(Lq=1 << 30, Hq=16)):
        assert _cross(lib, **kw) == SHAPE, kw
    assert _cross(lib, scale=float("nan")) == PARAM
    assert _cross(lib, dt=4) == DTYPE
    for kw in (dict(q=0x1008), dict(v=0x1002), dict(out=0x1004), dict(ws=0x1001),
               dict(vs=(1792, 257, 64)), dict(os_=(2560, 516, 64))):
        assert _cross(lib, **kw) == ALIGN, kw
    need = C.ctconv_cross_attention_workspace_bytes(1, 1, 9000, 8, 8, 64, 2)
    assert need > 0
    kw = dict(B=1, Lq=1, Lk=9000, Hq=8, H=8, qs=(512, 512, 64), ks=(4608000, 512, 64),
              vs=(4608000, 512, 64), os_=(512, 512, 64))
    assert _cross(lib, ws=None, **kw) == WORKSPACE
    assert _cross(lib, nb=need - 1, **kw) == WORKSPACE
    assert lib.ctconv_cross_attention_workspace_bytes(1, 1, 1, 1, 1, 8, 0, None) == NULL


def _norm(lib, x=P[0], h=P[1], gate=P[2], xo=P[3], y=P[4], pw=None, sc=None, nw=None, rows=4, Cn=64,
          st=(64,) * 5, per=1, post=1, pre=2, fn=2, eps=1e-5, dt=0):
    return lib.ctconv_norm_residual(x, h, pw, None, sc, gate, nw, None, xo, y, rows, Cn,
                                    None if st is None else arr(*st), per, post, pre, fn, eps, dt,
                                    None)


def test_norm_residual_validation(lib):
    assert _norm(lib, rows=0, x=None) == 0
    for name in ("x", "h", "gate", "xo", "y", "st"):
        assert _norm(lib, **{name: None}) == NULL, name
    for kw in (dict(post=3), dict(post=-1), dict(pre=9), dict(fn=4), dict(fn=-2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert _norm(lib, **kw) == PARAM, kw
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(Cn=0), dict(Cn=16385), dict(per=0),
               dict(st=(64, -1, 64, 64, 64)), dict(st=(64, 64, 64, 63, 64)),
               dict(st=(64, 64, 64, 64, 0)), dict(st=(1 << 62, 64, 64, 64, 64))):
        assert _norm(lib, **kw) == SHAPE, kw
    assert _norm(lib, dt=7) == DTYPE
    for kw in (dict(x=4), dict(gate=0x1008), dict(y=0x1008), dict(pw=0x1004), dict(sc=0x1004),
               dict(nw=0x1002)):
        assert _norm(lib, **kw) == ALIGN, kw


def test_python_helpers_refuse_host_tensors():
    import torch

    t = torch.zeros(2, 2, 8)
    with pytest.raises(ValueError, match="device"):
        C.paged_attention(t, t, t, t, t)
    with pytest.raises(ValueError, match="device"):
        C.cross_attention(t, t, t)
    with pytest.raises(ValueError, match="device"):
        C.norm_residual(t, t)
    with pytest.raises(ValueError, match="device"):
        C.cache_append(t, t, t, t, t, t)
    with pytest.raises(ValueError, match="device"):
        C.cache_evict(t, t, t, t, t, 1)


def test_block_run_reaches_each_function(lib):
    """The table form refuses what the functions refuse, with their statuses."""
    run = lib.ctconv_block_run
    bufs = (ctypes.c_void_p * 12)(*P)

    def sizes(*v):
        return (ctypes.c_int64 * 24)(*v)

    one = ctypes.c_int64.from_buffer_copy(ctypes.c_double(0.1)).value
    nan = ctypes.c_int64.from_buffer_copy(ctypes.c_double(float("nan"))).value
    append = [2, 3, 4, 64, 10, 16, 5, 768, 256, 64, 4096, 64, 1024, 5, 320, 80, 1]
    paged = [2, 8, 4, 64, 10, 16, 5, 80, 0, 512, 64, 4096, 64, 1024, 512, 64, 5, 320, 80, one, 1]
    evict = [2, 4, 64, 10, 16, 5, 80, 64, 4, 8, 4096, 64, 1024, 5, 320, 80, 320, 80, 1]
    cross = [2, 5, 7, 8, 4, 64, 2560, 512, 64, 1792, 256, 64, 1792, 256, 64, 2560, 512, 64, 7, one, 1]
    norm = [4, 64, 64, 64, 64, 64, 64, 1, 1, 2, 2, one, 0]

    def call(op, z, **kw):
        z = list(z)
        for i, v in kw.items():
            z[int(i[1:])] = v
        return run(op, sizes(*z), bufs, None, 0, None)

    assert run(5, sizes(), bufs, None, 0, None) == PARAM
    assert run(-1, sizes(), bufs, None, 0, None) == PARAM
    assert run(0, None, bufs, None, 0, None) == NULL
    assert run(0, sizes(*append), None, None, 0, None) == NULL
    for op, z in enumerate((append, paged, evict, cross, norm)):
        last = len(z) - 1
        for bad in (3, -1, 1 << 40):
            assert call(op, z, **{f"_{last}": bad}) == DTYPE, (op, bad)
    assert call(0, append, _3=12) == SHAPE
    assert call(0, append, _11=66) == ALIGN
    assert call(1, paged, _19=nan) == PARAM
    assert call(1, paged) == WORKSPACE  # a weight_sum is among the buffers
    assert call(2, evict, _7=0) == PARAM
    assert call(3, cross, _19=nan) == PARAM
    assert call(3, cross, _10=257) == ALIGN
    assert call(4, norm, _8=7) == PARAM
    assert call(4, norm, _10=-3) == PARAM
    assert call(4, norm, _11=nan) == PARAM
    assert call(4, norm, _0=0) == 0


def test_plans_raise_the_function_s_error():
    with pytest.raises(C.CtconvError, match="ctconv_norm_residual") as e:
        C.NormResidual(4, 64)(None, P[1], None, None, None, None, None, None, P[2], P[3], 0)
    assert e.value.status == NULL
    with pytest.raises(C.CtconvError, match="ctconv_cache_evict") as e:
        C.CacheEvict(1, 1, 8, 4, 4, 4, keep=0)(*P[:11], 0)
    assert e.value.status == PARAM
