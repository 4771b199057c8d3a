"""Host-only checks of the Python helpers of the operators on requests of many lengths."""

import math
import resource

import pytest

from test_block_abi_host import SHAPE
from vision_upsampler_decoders_amd import ctconv as C


@pytest.mark.parametrize("R", [-2, 0, 1, 257, 258, 1 << 33, 1 << 40])
def test_rotary_frequencies_refuse_a_width_without_room_for_it(R):
    """The library refuses a width; nothing of that size is allocated before."""
    C.rotary_frequencies(2)  # (torch and the library are loaded)
    soft, hard = resource.getrlimit(resource.RLIMIT_AS)
    now = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
    resource.setrlimit(resource.RLIMIT_AS, (now + (4 << 30), hard))
    try:
        with pytest.raises(C.CtconvError) as e:
            C.rotary_frequencies(R)
    finally:
        resource.setrlimit(resource.RLIMIT_AS, (soft, hard))
    assert e.value.status == SHAPE


@pytest.mark.parametrize("R", [2, 64, 256])
def test_rotary_frequencies_have_their_number(R):
    f = C.rotary_frequencies(R, 100.0)
    assert tuple(f.shape) == (R // 2,)
    assert all(math.isclose(float(v), 100.0 ** (-2 * i / R), rel_tol=1e-14) for i, v in enumerate(f))
