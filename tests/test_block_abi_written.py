"""Host-only checks: what an eviction writes must fit the arrays it is given,
and is refused before any launch where it does not."""

import pytest

from test_block_abi_host import P, PARAM, SHAPE, _evict, arr, lib  # noqa: F401 (lib: a fixture)
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
