"""ctconv: dense transposed convolution (ConvTranspose1d/2d) on AMD MI355X,
and the operators of the transformer block that feeds it in a streaming decoder.

The computation lives in libctconv.so (HIP, gfx950); see include/ctconv.h for
the C ABI.  This package holds the build script and the ctypes binding.
"""

from .ctconv import (  # noqa: F401
    CTCONV_BF16,
    CTCONV_F16,
    CTCONV_F32,
    GATE_LINEAR,
    GATE_NONE,
    GATE_SIGMOID,
    GATE_TANH,
    NORM_LAYER,
    NORM_NONE,
    NORM_RMS,
    ROUTE_AUTO,
    ROUTE_GATHER,
    ROUTE_POLYPHASE,
    CacheAppend,
    CacheEvict,
    CrossAttention,
    CtconvError,
    NormResidual,
    PagedAttention,
    cache_append,
    cache_evict,
    cross_attention,
    elu,
    forward,
    load,
    norm_residual,
    paged_attention,
    prepack,
)
