"""Host-only checks: what the decoder-block operators write must fit the arrays
they are given and lie apart in them, and is refused before any launch where it
does not."""

import pytest

from test_block_abi_host import (P, PARAM, SHAPE, WORKSPACE, _append, _cross, _evict,  # noqa: F401
                                 _paged, lib)
from vision_upsampler_decoders_amd import ctconv as C


def test_evict_output_rows_hold_keep_slots(lib):  # noqa: F811
    # 2 sequences of 4 heads, 64 slots kept: rows of fewer values run into the next head's
    for out in ((256, 63), (256, 0), (0, 64), (255, 64), (64, 127), (252, 64)):
        assert _evict(lib, out=out) == SHAPE, out
    # heads before sequences hold them too, and a dimension of one takes no step: these get as
    # far as the strides of an update in place
    for kw in (dict(out=(64, 128)), dict(out=(0, 64), B=1), dict(out=(64, 0), H=1)):
        assert _evict(lib, wo=P[4], **kw) == PARAM, kw


def test_evict_in_place_keeps_no_more_than_the_table_holds(lib):  # noqa: F811
    # weights and positions of 5 pages of 16 slots, updated in place
    place = dict(wo=P[4], po=P[5])
    for kw in (dict(), dict(wo=P[6]), dict(po=P[7])):
        for slot in ((320, 80), (1000, 200)):
            kw2 = {**place, **kw, "slot": slot, "out": slot}
            assert _evict(lib, keep=81, **kw2) == SHAPE, kw2
            assert _evict(lib, keep=1 << 20, **kw2) == SHAPE, kw2
    # one sequence and head: nothing else tells that the row is too long
    one = dict(B=1, H=1, slot=(80, 80), out=(80, 80), kv=(1024, 64, 1024))
    assert _evict(lib, keep=81, **place, **one) == SHAPE
    assert _evict(lib, keep=81, pos=None, po=None, wo=P[4], **one) == SHAPE
    with pytest.raises(C.CtconvError, match="ctconv_cache_evict") as e:
        C.CacheEvict(1, 1, 8, 4, 4, 4, keep=17)(
            P[0], P[1], P[2], P[3], None, P[4], P[5], P[4], P[5], P[3], P[9], 0)
    assert e.value.status == SHAPE


# pages, slots and heads of [10, 4, 16, 64] caches that meet: nothing steps over the pages, a slot
# or head within a row of 64, pages within a page's heads
MEET = [(0, 64, 1024), (4096, 0, 1024), (4096, 56, 1024), (4096, 64, 0), (4096, 64, 960),
        (4032, 64, 1024), (4096, 256, 256), (8, 64, 1024)]


def test_written_caches_lie_apart(lib):  # noqa: F811
    for kv in MEET:
        assert _append(lib, kv=kv) == SHAPE, kv
        assert _evict(lib, kv=kv) == SHAPE, kv
        # read only there: as far as the workspace
        assert _paged(lib, w=P[7], kv=kv, ws=None) == WORKSPACE, kv
    for kv in ((4096, 64, 1024), (4096, 256, 64), (8192, 128, 2048), (64, 640, 10240)):
        # in place with other strides is refused last
        assert _evict(lib, wo=P[4], kv=kv) == PARAM, kv


def test_written_slot_arrays_lie_apart(lib):  # noqa: F811
    for slot in ((0, 80), (320, 0), (320, 79), (316, 80), (40, 80)):
        assert _append(lib, slot=slot) == SHAPE, slot
        assert _append(lib, slot=slot, pos=None) == SHAPE, slot
        assert _paged(lib, w=P[7], slot=slot) == SHAPE, slot
    for slot in ((320, 80), (80, 160), (1000, 200)):
        assert _paged(lib, w=P[7], slot=slot, ws=None) == WORKSPACE, slot
    # no slot past max_length is written
    assert _paged(lib, w=P[7], slot=(280, 70), maxlen=70, ws=None) == WORKSPACE
    assert _paged(lib, w=P[7], slot=(0, 80), B=1, ws=None) == WORKSPACE


def test_written_outputs_lie_apart(lib):  # noqa: F811
    for o in ((0, 64), (512, 0), (512, 32), (448, 64), (8, 64)):
        assert _paged(lib, w=P[7], os_=o, ws=None) == SHAPE, o
    for o in ((512, 64), (64, 128), (1024, 128)):
        assert _paged(lib, w=P[7], os_=o, ws=None) == WORKSPACE, o
    long = dict(B=2, Lq=1, Lk=9000, H=8, ks=(4608000, 512, 64), vs=(4608000, 512, 64), ws=None)
    for o in ((0, 512, 64), (512, 512, 0), (512, 512, 56), (448, 512, 64)):
        assert _cross(lib, os_=o, **long) == SHAPE, o
    for o in ((512, 0, 64), (64, 512, 128)):
        assert _cross(lib, os_=o, **long) == WORKSPACE, o
    for o in ((2560, 0, 64), (2560, 448, 64), (64, 512, 64), (2560, 512, 48)):
        assert _cross(lib, os_=o) == SHAPE, o
