// Attention of many query rows per cache head (attn_tile.h) to an encoder's states.

#include "attn_tile.h"

namespace ctconv {
namespace block {

namespace {

template <class TR, int DP>
hipError_t tile_d(const AttnArgs& a, hipStream_t s) {
    const int64_t items = (int64_t)a.B * a.Hkv * a.row_tiles * a.splits;
    const size_t lds = Shape<TR, DP>::LDS;
    const void* fn = a.D == DP ? reinterpret_cast<const void*>(&tile_kernel<TR, DP, true>)
                               : reinterpret_cast<const void*>(&tile_kernel<TR, DP, false>);
    if (lds > 64u << 10) {
        const hipError_t e =
            hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    AttnArgs args = a;
    void* params[] = {&args};
    return hipLaunchKernel(fn, grid_of((items + 7) / 8 * 8), dim3(kThreads), params, lds, s);
}

template <class TR>
hipError_t tile_t(const AttnArgs& a, hipStream_t s) {
    if (a.D <= 64) return tile_d<TR, 64>(a, s);
    if (a.D <= 128) return tile_d<TR, 128>(a, s);
    // fp32 rows of 1 KB: two tiles of K and of V do not fit LDS
    if constexpr (sizeof(typename TR::storage) == 2) return tile_d<TR, 256>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs& a, ctconv_dtype dt, hipStream_t s) {
    switch (dt) {
        case CTCONV_F32: return tile_t<TF32>(a, s);
        case CTCONV_BF16: return tile_t<TBF16>(a, s);
        case CTCONV_F16: return tile_t<TF16>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace block
}  // namespace ctconv
