// Attention of few query rows per cache head (attn_stream.h) for one-row paged
// calls and dense calls, and the joins of split calls.

#include "attn_stream.h"

namespace ctconv {
namespace block {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

// Join.  A row's outputs are its splits' outputs weighted by 2^(m - maximum),
// over the sum of their sums weighted the same.
//  - Few splits of many rows: D / 4 lanes add a row's splits in ascending
//    order, 256 / (D / 4) rows per workgroup.  A whole call with it and with a
//    workgroup per row: 4096 rows of 3 splits 212 us against 219, 8192 of 5
//    194 against 210; but 8 rows of 20000 keys 29 against 23.
//  - Else: a workgroup per row; each of its lane groups takes every
//    groups-th split in ascending order, then the groups are added in order.
// The workgroups past those add the weights to weight_sum: 1024 slots each.
// They need the sums of all splits, hence a second kernel: 9.8 us after 75 to 83
// for 3 ragged sequences up to 100003 (24 heads on 4, f16; 416 MB in all).
constexpr int kFewSplits = 16, kManyRows = 4096;
constexpr int kAtOnce = 4;  // splits of a row whose loads are in flight together
constexpr int kWeightSlots = 4 * kThreads;
constexpr int kLseRows = 256;
constexpr int kAhead = 8;  // score rows that a weight workgroup loads ahead

// One row's joined values of 4 value columns, and its log-sum-exp.
template <class TR>
__device__ inline void join_write(const AttnArgs& a, int b, int h, int r, int d, f32x4 o, float top,
                                  float sum) {
    using S = typename TR::storage;
    const int lq = (int)fdiv((uint32_t)r, a.fd_G);
    const int hq = h * a.G + (r - lq * a.G);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    S* to = static_cast<S*>(a.out) + b * a.o_b + lq * a.o_row + (int64_t)hq * a.o_head + d;
    if constexpr (sizeof(S) == 2) {
        u32x2 w{mfma::pack2<TR>(o[0] * inv, o[1] * inv), mfma::pack2<TR>(o[2] * inv, o[3] * inv)};
        *reinterpret_cast<u32x2*>(to) = w;
    } else {
        *reinterpret_cast<f32x4*>(to) = o * inv;
    }
    if (d == 0 && a.lse)
        a.lse[((int64_t)b * a.Hq + hq) * a.Lq + lq] = top * kLn2 + logf(sum);
}

template <class TR, bool PAGED>
__global__ __launch_bounds__(kThreads) void join_few_kernel(AttnArgs a) {
    const int pieces = a.D / 4, rows = kThreads / pieces;
    const int grp = threadIdx.x / pieces, d = (threadIdx.x - grp * pieces) * 4;
    const int64_t i = (int64_t)block_number() * rows + grp;
    if (grp >= rows || i >= (int64_t)a.B * a.Hkv * a.R) return;
    const int bh = (int)(i / a.R), r = (int)(i - (int64_t)bh * a.R);
    const int b = bh / a.Hkv, h = bh - b * a.Hkv;
    int first, span;
    visible<PAGED>(a, b, first, span);
    const int n = (span + a.chunk - 1) / a.chunk;
    const int64_t p0 = (int64_t)bh * a.splits * a.R + r;
    // every load clamped to a split that exists, none behind a branch
    const float* ml = a.part_ml + 2 * p0;
    const float* po = a.part_o + p0 * a.D + d;
    const int64_t step = (int64_t)a.R;
    float top = -__builtin_huge_valf(), sum = 0.f;
    f32x4 o{0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < n; s0 += kAtOnce) {
        f32x2 v[kAtOnce];
        f32x4 x[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int64_t s = s0 + i < n ? s0 + i : n - 1;
            v[i] = *reinterpret_cast<const f32x2*>(ml + 2 * s * step);
            x[i] = *reinterpret_cast<const f32x4*>(po + s * step * a.D);
        }
        float up = top;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) up = fmaxf(up, v[i][0]);
        const float ref = reference_of(up), old = exp2_fast(top - ref);
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
    join_write<TR>(a, b, h, r, d, o, top, sum);
}

// A slot's weight; none where it is hidden, whatever the row's sum is.
__device__ inline float weight_of(float s, float lse2) {
    return s == -__builtin_huge_valf() ? 0.f : exp2_fast(s - lse2);
}

template <class TR, bool PAGED>
__global__ __launch_bounds__(kThreads) void join_kernel(AttnArgs a, int out_blocks,
                                                        int weight_blocks) {
    __shared__ float part[kThreads * 4];
    const int tid = threadIdx.x, wave = tid >> 6;
    if (block_number() >= (uint32_t)out_blocks + (uint32_t)(a.B * a.Hkv * weight_blocks)) return;
    const int number = (int)block_number();
    if (number < out_blocks) {
        const int bh = number / a.R, r = number - bh * a.R;
        const int b = bh / a.Hkv, h = bh - b * a.Hkv;
        int first, span;
        visible<PAGED>(a, b, first, span);
        const int n = (span + a.chunk - 1) / a.chunk;
        const int64_t p0 = (int64_t)bh * a.splits * a.R + r;
        const float* ml = a.part_ml + 2 * p0;
        const float* const rows[1] = {ml};
        float tops[1], sums[1];
        join_stats(rows, a.R, n, tops, sums);
        const float top = tops[0], sum = sums[0];
        const int pieces = a.D / 4, groups = kThreads / pieces;
        const int grp = tid / pieces, d = (tid - grp * pieces) * 4;
        if (grp < groups) {
            f32x4 o{0.f, 0.f, 0.f, 0.f};
            for (int s = grp; s < n; s += groups) {
                const float f = exp2_fast(ml[2 * (int64_t)s * a.R] - reference_of(top));
                const f32x4 x = *reinterpret_cast<const f32x4*>(
                    a.part_o + (p0 + (int64_t)s * a.R) * a.D + d);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = fmaf(f, x[e], o[e]);
            }
            *reinterpret_cast<f32x4*>(part + 4 * tid) = o;
        }
        __syncthreads();
        if (tid < pieces) {
            f32x4 o{0.f, 0.f, 0.f, 0.f};
            for (int q = 0; q < groups; ++q)
                o += *reinterpret_cast<const f32x4*>(part + 4 * (q * pieces + tid));
            join_write<TR>(a, b, h, r, d, o, top, sum);
        }
        return;
    }
    // weights of paged calls (Lq = 1, R = G)
    const int item = number - out_blocks;
    const int bh = item / weight_blocks, blk = item - bh * weight_blocks;
    const int b = bh / a.Hkv, h = bh - b * a.Hkv;
    int first, span;
    visible<PAGED>(a, b, first, span);
    if (blk * kWeightSlots >= span) return;
    const int n = (span + a.chunk - 1) / a.chunk;
    float add[4] = {0.f, 0.f, 0.f, 0.f};
    const int i0 = blk * kWeightSlots + 4 * tid;
    const bool mine = i0 < span;
    float* w = a.weight_sum + b * a.slot_b + h * a.slot_h + first + i0;
    float old[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) old[e] = i0 + e < span ? w[e] : 0.f;
    const float* sr = a.scores + (int64_t)bh * a.R * a.score_stride + i0;
    float* lse2 = part;
    for (int r0 = 0; r0 < a.R; r0 += kLseRows) {
        const int rn = a.R - r0 < kLseRows ? a.R - r0 : kLseRows;
        // the first rows' scores are on their way while the sums are joined
        f32x4 s[kAhead];
#pragma unroll
        for (int r = 0; r < kAhead; ++r)
            if (mine && r < rn)
                s[r] = *reinterpret_cast<const f32x4*>(sr + (int64_t)(r0 + r) * a.score_stride);
        __syncthreads();
        const float* ml = a.part_ml + 2 * ((int64_t)bh * a.splits * a.R + r0);
        for (int r = wave; r < rn; r += 2 * kWaves) {
            const int r2 = r + kWaves < rn ? r + kWaves : r;
            const float* const rows[2] = {ml + 2 * r, ml + 2 * r2};
            float top[2], sum[2];
            join_stats(rows, a.R, n, top, sum);
            // a row without a visible slot adds nothing: exp2(s - infinity)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if ((tid & 63) == 0)
                    lse2[i ? r2 : r] = top[i] == -__builtin_huge_valf()
                                           ? __builtin_huge_valf()
                                           : top[i] + __builtin_amdgcn_logf(sum[i]);
        }
        __syncthreads();
        if (mine) {
#pragma unroll
            for (int r = 0; r < kAhead; ++r)
                if (r < rn) {
                    const float z = lse2[r];
#pragma unroll
                    for (int e = 0; e < 4; ++e) add[e] += weight_of(s[r][e], z);
                }
            for (int r = kAhead; r < rn; ++r) {
                const f32x4 t =
                    *reinterpret_cast<const f32x4*>(sr + (int64_t)(r0 + r) * a.score_stride);
                const float z = lse2[r];
#pragma unroll
                for (int e = 0; e < 4; ++e) add[e] += weight_of(t[e], z);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (i0 + e < span) w[e] = old[e] + add[e];
}

template <class TR, int DP, bool PAGED, int NW>
hipError_t stream_w(const AttnArgs& a, size_t lds, hipStream_t s) {
    const dim3 grid = grid_of((int64_t)a.B * a.Hkv * a.row_tiles * a.splits);
    const void* fn = a.D == DP
                         ? reinterpret_cast<const void*>(&stream_kernel<TR, DP, PAGED, true, NW>)
                         : reinterpret_cast<const void*>(&stream_kernel<TR, DP, PAGED, false, NW>);
    if (lds > 64u << 10) {
        const hipError_t e =
            hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    AttnArgs args = a;
    void* params[] = {&args};
    return hipLaunchKernel(fn, grid, dim3(64 * NW), params, lds, s);
}

template <class TR, int DP, bool PAGED>
hipError_t stream_d(const AttnArgs& a, hipStream_t s) {
    const int rows = a.R < 16 ? a.R : 16;
    const size_t stage = (PAGED ? (size_t)a.chunk * 8 : 0) + (size_t)(a.chunk / 32 + 2) * 4;
    const auto lds = [&](int nw) {
        const size_t merge = (size_t)(nw * rows * (DP + 4) + 2 * nw * 16) * 4;
        return stage > merge ? stage : merge;
    };
    // as many waves as the registers allow (512 per lane and SIMD)
    constexpr int WIDE = DP <= 64 ? 16 : DP <= 128 ? 8 : 4;
    if constexpr (WIDE > 4)
        if (a.wide) return stream_w<TR, DP, PAGED, WIDE>(a, lds(WIDE), s);
    return stream_w<TR, DP, PAGED, 4>(a, lds(4), s);
}

template <class TR, bool PAGED>
hipError_t stream_t(const AttnArgs& a, hipStream_t s) {
    if (a.D <= 64) return stream_d<TR, 64, PAGED>(a, s);
    if (a.D <= 128) return stream_d<TR, 128, PAGED>(a, s);
    return stream_d<TR, 256, PAGED>(a, s);
}

template <class TR, bool PAGED>
hipError_t join_t(const AttnArgs& a, hipStream_t s) {
    const int out_blocks = a.B * a.Hkv * a.R;
    if (a.splits <= kFewSplits && out_blocks >= kManyRows && !a.weight_sum) {
        const int rows = kThreads / (a.D / 4);
        join_few_kernel<TR, PAGED><<<grid_of(((int64_t)out_blocks + rows - 1) / rows),
                                     dim3(kThreads), 0, s>>>(a);
        return hipGetLastError();
    }
    const int64_t longest = a.score_stride;
    const int weight_blocks =
        a.weight_sum ? (int)((longest + kWeightSlots - 1) / kWeightSlots) : 0;
    const int64_t grid = out_blocks + (int64_t)a.B * a.Hkv * weight_blocks;
    join_kernel<TR, PAGED>
        <<<grid_of(grid), dim3(kThreads), 0, s>>>(a, out_blocks, weight_blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_stream(const AttnArgs& a, ctconv_dtype dt, bool paged, hipStream_t s) {
    switch (dt) {
        case CTCONV_F32: return paged ? stream_t<TF32, true>(a, s) : stream_t<TF32, false>(a, s);
        case CTCONV_BF16: return paged ? stream_t<TBF16, true>(a, s) : stream_t<TBF16, false>(a, s);
        case CTCONV_F16: return paged ? stream_t<TF16, true>(a, s) : stream_t<TF16, false>(a, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_attn_join(const AttnArgs& a, ctconv_dtype dt, bool paged, hipStream_t s) {
    switch (dt) {
        case CTCONV_F32: return paged ? join_t<TF32, true>(a, s) : join_t<TF32, false>(a, s);
        case CTCONV_BF16: return paged ? join_t<TBF16, true>(a, s) : join_t<TBF16, false>(a, s);
        case CTCONV_F16: return paged ? join_t<TF16, true>(a, s) : join_t<TF16, false>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace block
}  // namespace ctconv
