// Attention of a chunk of new rows over the paged cache with many query rows per
// key head: the chunk form of the tile kernel (attn_tile.h), and the join of its
// splits.

#include "attn_tile.h"

namespace ctconv {
namespace block {

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kAtOnce = 4;  // splits of a row whose loads are in flight together

constexpr int kJoins = 8;   // workgroups of a row tile in the join

// Join: D / 4 lanes add a row's splits in ascending order.  Tiles of one split
// have written their results already.  With a workgroup per tile instead of eight, 4 x
// 128 rows of 8 heads over 16384 keys in 16 splits take 98 us, and 65 this way.
template <class TR>
__global__ __launch_bounds__(kThreads) void chunk_tile_join_kernel(AttnArgs a) {
    using S = typename TR::storage;
    int b, h, tile, split;
    const uint32_t number = block_number();
    if (!chunk_item(a, kThreads / 64, number / kJoins, false, b, h, tile, split)) return;
    const ChunkRows cr = chunk_rows(a, b);
    const int R = cr.live * a.G, row0 = tile * 128;
    const int last = row0 + 127 < R ? row0 + 127 : R - 1;
    int first, span;
    chunk_span(a, cr, (int)fdiv((uint32_t)row0, a.fd_G), (int)fdiv((uint32_t)last, a.fd_G), first,
               span);
    if (span <= a.chunk) return;
    const int n = (span + a.chunk - 1) / a.chunk;
    const int pieces = a.D / 4, together = kThreads / pieces;
    const int grp = threadIdx.x / pieces, d = (threadIdx.x - grp * pieces) * 4;
    if (grp >= together) return;
    constexpr int kRows = 128 / kJoins;
    const int from = row0 + (int)(number % kJoins) * kRows;
    const int to = from + kRows - 1 < last ? from + kRows - 1 : last;
    for (int row = from + grp; row <= to; row += together) {
        const int lq = (int)fdiv((uint32_t)row, a.fd_G), hq = h * a.G + (row - lq * a.G);
        const int64_t at = (cr.row0 + lq) * a.Hq + hq, p0 = at * a.splits;
        const float* ml = a.part_ml + 2 * p0;
        const float* po = a.part_o + p0 * a.D + d;
        float top = -__builtin_huge_valf(), sum = 0.f;
        f32x4 o{0.f, 0.f, 0.f, 0.f};
        for (int s0 = 0; s0 < n; s0 += kAtOnce) {
            // every load clamped to a split that exists, none behind a branch
            f32x2 v[kAtOnce];
            f32x4 x[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int64_t s = s0 + i < n ? s0 + i : n - 1;
                v[i] = *reinterpret_cast<const f32x2*>(ml + 2 * s);
                x[i] = *reinterpret_cast<const f32x4*>(po + s * a.D);
            }
            float up = top;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) up = fmaxf(up, v[i][0]);
            // nothing seen yet: weights 0, whatever is subtracted
            const float ref = up == -__builtin_huge_valf() ? 0.f : up;
            const float old = exp2_fast(top - ref);
            top = up;
            sum *= old;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] *= old;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                // (read twice: 0 as a result, too, as 0 times an infinite one is NaN)
                const bool is = s0 + i < n;
                const float f = is ? exp2_fast(v[i][0] - ref) : 0.f;
                sum = fmaf(f, v[i][1], sum);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = fmaf(f, is ? x[i][e] : 0.f, o[e]);
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        S* out = static_cast<S*>(a.out) + (a.row_starts ? cr.row0 * a.o_row : b * a.o_b) +
                 lq * a.o_row + (int64_t)hq * a.o_head + d;
        if constexpr (sizeof(S) == 2) {
            u32x2 w{mfma::pack2<TR>(o[0] * inv, o[1] * inv),
                    mfma::pack2<TR>(o[2] * inv, o[3] * inv)};
            *reinterpret_cast<u32x2*>(out) = w;
        } else {
            *reinterpret_cast<f32x4*>(out) = o * inv;
        }
        if (d == 0) write_lse(a, at, top, sum);
    }
}

template <class TR, int DP, int DU = DP>
hipError_t tile_d(const AttnArgs& a, hipStream_t s) {
    using Sh = Shape<TR, DP, DU>;
    const size_t lds = Sh::LDS + 4 * Sh::KT * sizeof(int64_t) + sizeof(int);
    const void* fn = reinterpret_cast<const void*>(&tile_kernel<TR, DP, false, true, DU>);
    if constexpr (DU == DP)
        if (a.D == DP) fn = reinterpret_cast<const void*>(&tile_kernel<TR, DP, true, true>);
    if (lds > 64u << 10) {
        const hipError_t e =
            hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    AttnArgs args = a;
    void* params[] = {&args};
    return hipLaunchKernel(fn, grid_of((int64_t)a.row_tiles * a.splits * a.Hkv), dim3(kThreads),
                           params, lds, s);
}

template <class TR>
hipError_t tile_t(const AttnArgs& a, hipStream_t s) {
    if (a.D <= 32) return tile_d<TR, 64, 32>(a, s);
    if (a.D <= 64) return tile_d<TR, 64>(a, s);
    if (a.D <= 96) return tile_d<TR, 128, 96>(a, s);
    if (a.D <= 128) return tile_d<TR, 128>(a, s);
    // fp32 rows of 1 KB: two tiles of K and of V do not fit LDS
    if constexpr (sizeof(typename TR::storage) == 2) return tile_d<TR, 256>(a, s);
    return hipErrorInvalidValue;
}

template <class TR>
hipError_t join_t(const AttnArgs& a, hipStream_t s) {
    chunk_tile_join_kernel<TR>
        <<<grid_of((int64_t)a.row_tiles * a.Hkv * kJoins), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk_tile(const AttnArgs& a, ctconv_dtype dt, hipStream_t s) {
    switch (dt) {
        case CTCONV_F32: return tile_t<TF32>(a, s);
        case CTCONV_BF16: return tile_t<TBF16>(a, s);
        case CTCONV_F16: return tile_t<TF16>(a, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_chunk_tile_join(const AttnArgs& a, ctconv_dtype dt, hipStream_t s) {
    switch (dt) {
        case CTCONV_F32: return join_t<TF32>(a, s);
        case CTCONV_BF16: return join_t<TBF16>(a, s);
        case CTCONV_F16: return join_t<TF16>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace block
}  // namespace ctconv
