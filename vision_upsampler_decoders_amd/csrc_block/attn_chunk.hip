// Attention of a chunk of new rows over the paged cache: the chunk form of the
// streaming kernel (attn_stream.h) for few rows per key head, the join of its
// splits, and the weights of the slots.

#include "attn_mma.h"
#include "attn_stream.h"

namespace ctconv {
namespace block {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

// Join of a row's splits, a workgroup per row: each of its lane groups takes
// every groups-th split in ascending order, then the groups are added in order.
template <class TR>
__global__ __launch_bounds__(kThreads) void chunk_join_kernel(AttnArgs a) {
    using S = typename TR::storage;
    __shared__ float part[kThreads * 4];
    const int tid = threadIdx.x;
    const uint32_t number = block_number();
    if (number >= (uint32_t)a.B * a.Hkv * a.R) return;
    const int bh = (int)(number / a.R), r = (int)(number - (uint32_t)bh * a.R);
    const int b = bh / a.Hkv, h = bh - b * a.Hkv;
    const ChunkRows cr = chunk_rows(a, b);
    const int R = cr.live * a.G;
    if (r >= R) return;
    const int row0 = r & ~15, last = row0 + 15 < R ? row0 + 15 : R - 1;
    int first, span;
    chunk_span(a, cr, (int)fdiv((uint32_t)row0, a.fd_G), (int)fdiv((uint32_t)last, a.fd_G), first,
               span);
    if (span <= a.chunk) return;  // one workgroup wrote the result
    const int n = (span + a.chunk - 1) / a.chunk;
    const int lq = (int)fdiv((uint32_t)r, a.fd_G), hq = h * a.G + (r - lq * a.G);
    const int64_t row = (cr.row0 + lq) * a.Hq + hq, p0 = row * a.splits;
    const float* ml = a.part_ml + 2 * p0;
    const float* const rows[1] = {ml};
    float tops[1], sums[1];
    join_stats(rows, 1, n, tops, sums);
    const float top = tops[0], sum = sums[0];
    const int pieces = a.D / 4, groups = kThreads / pieces;
    const int grp = tid / pieces, d = (tid - grp * pieces) * 4;
    if (grp < groups) {
        f32x4 o{0.f, 0.f, 0.f, 0.f};
        for (int s = grp; s < n; s += groups) {
            const float f = exp2_fast(ml[2 * s] - reference_of(top));
            const f32x4 x = *reinterpret_cast<const f32x4*>(a.part_o + (p0 + s) * a.D + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(f, x[e], o[e]);
        }
        *reinterpret_cast<f32x4*>(part + 4 * tid) = o;
    }
    __syncthreads();
    if (tid >= pieces) return;
    f32x4 o{0.f, 0.f, 0.f, 0.f};
    for (int q = 0; q < groups; ++q)
        o += *reinterpret_cast<const f32x4*>(part + 4 * (q * pieces + tid));
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    S* to = static_cast<S*>(a.out) + (a.row_starts ? cr.row0 * a.o_row : b * a.o_b) +
            lq * a.o_row + (int64_t)hq * a.o_head + d;
    if constexpr (sizeof(S) == 2) {
        u32x2 w{mfma::pack2<TR>(o[0] * inv, o[1] * inv), mfma::pack2<TR>(o[2] * inv, o[3] * inv)};
        *reinterpret_cast<u32x2*>(to) = w;
    } else {
        *reinterpret_cast<f32x4*>(to) = o * inv;
    }
    if (d == 0) write_lse(a, row, top, sum);
}

// weight_sum[b][h][t] += the sum over rows and heads of exp2(score - lse2).  The
// sums of all slots have to be known before any slot can be weighed, so the
// scores are computed again.  A wave keeps its keys in registers (32 or 64 of
// them, a key per row of the matrix instruction) and walks the query rows, 32 at a
// time, the next ones on their way; a lane adds up its query column and the
// columns are added at the end.  The waves of a workgroup take keys of their own and
// the same rows (which they then find in the L1 cache), or, where that would leave
// compute units idle (apart), the same keys and every fourth rows.
template <class TR, int DP, bool EXACT>
__global__ __launch_bounds__(kThreads, DP * sizeof(typename TR::storage) > 512 ? 1 : 2) void
chunk_weights_kernel(AttnArgs a, int key_blocks, int apart) {
    using S = typename TR::storage;
    constexpr int ES = sizeof(S), VEC = 16 / ES;
    constexpr int NF = DP / (2 * VEC);
    constexpr int KG = NF <= 8 ? 2 : 1;  // groups of 32 keys of a wave
    constexpr bool AHEAD = EXACT || NF != 16;  // (registers for the next rows)
    __shared__ float parts[kWaves][KG * 32];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 31, half = lane >> 5;
    const uint32_t number = block_number();
    if (number >= (uint32_t)a.B * a.Hkv * key_blocks) return;
    const int h = (int)(number % a.Hkv), bk = (int)(number / a.Hkv);
    const int b = bk / key_blocks, kb = bk - b * key_blocks;
    const ChunkRows cr = chunk_rows(a, b);
    const int key0 = (apart ? kb : kb * kWaves + wave) * KG * 32, key_end = key0 + KG * 32;
    // rows that see some of the keys
    int lo = key0 - cr.off;
    lo = lo > 0 ? lo : 0;
    int hi = cr.live;
    if (a.window > 0) {
        const int64_t most = (int64_t)key_end - 1 - cr.off + a.window;
        hi = most < hi ? (int)most : hi;
    }
    if (lo >= hi) return;  // (apart: for all waves)

    u32x4 kf[KG][NF];
    bool there[KG];
#pragma unroll
    for (int g = 0; g < KG; ++g) {
        const int t = key0 + 32 * g + col;
        const int64_t o = t < cr.len ? slot_offset(a.pages, b, t) : -1;
        there[g] = o >= 0;
        const S* kr = static_cast<const S*>(a.k) + h * a.pages.head_stride + (o >= 0 ? o : 0);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int d = (2 * f + half) * VEC;
            kf[g][f] = u32x4{0, 0, 0, 0};
            if (there[g] && (EXACT || d < a.D)) kf[g][f] = *reinterpret_cast<const u32x4*>(kr + d);
            // the sign of the scale (the keys' pieces past a row stay 0)
            const uint32_t flip = a.negate ? (ES == 2 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) kf[g][f][i] ^= flip;
        }
    }
    f32x16 sum[KG];
#pragma unroll
    for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[g][i] = 0.f;
    const S* qb = static_cast<const S*>(a.q) + (a.row_starts ? cr.row0 * a.q_row : b * a.q_b) +
                  (int64_t)(h * a.G) * a.q_head;
    const float* lse2 = a.lse2 + cr.row0 * a.Hq + h * a.G;
    const int r_end = hi * a.G, step = apart ? 32 * kWaves : 32;
    u32x4 next[NF];
    float next_low;
    int next_end;
    // Rows past the last one are read as that one and weigh nothing.
    const auto load = [&](int r0) __attribute__((always_inline)) {
        const int r = r0 + col < r_end ? r0 + col : r_end - 1;
        const int lq = (int)fdiv((uint32_t)r, a.fd_G), hq = r - lq * a.G;
        const S* qr = qb + lq * a.q_row + hq * a.q_head;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int d = (2 * f + half) * VEC;
            next[f] = *reinterpret_cast<const u32x4*>(qr + (EXACT || d < a.D ? d : 0));
        }
        next_low = lse2[(int64_t)lq * a.Hq + hq];
        if (r0 + col >= r_end) next_low = __builtin_huge_valf();
        next_end = cr.off + lq + 1;
    };
    int r0 = lo * a.G + (apart ? 32 * wave : 0);
    if (AHEAD && r0 < r_end) load(r0);
    for (; r0 < r_end; r0 += step) {
        if (!AHEAD) load(r0);
        u32x4 qf[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) qf[f] = next[f];
        const float low = next_low;
        const int end = next_end, begin = a.window > 0 ? end - a.window : 0;
        if (AHEAD && r0 + step < r_end) load(r0 + step);
        const bool whole = __all(begin <= key0 && end >= key_end);
        f32x16 s[KG];
#pragma unroll
        for (int g = 0; g < KG; ++g)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[g][i] = 0.f;
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int g = 0; g < KG; ++g) Mma32<TR>::step(s[g], kf[g][f], qf[f]);
        if (whole) {
#pragma unroll
            for (int g = 0; g < KG; ++g)
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[g][i] += exp2_fast(fmaf(s[g][i], a.c, -low));
        } else {
#pragma unroll
            for (int g = 0; g < KG; ++g)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    // a hidden slot gets nothing, whatever the row's sum is
                    const int t = key0 + 32 * g + 8 * (i >> 2) + 4 * half + (i & 3);
                    const float p = exp2_fast(fmaf(s[g][i], a.c, -low));
                    sum[g][i] += t < end && t >= begin ? p : 0.f;
                }
        }
    }
#pragma unroll
    for (int g = 0; g < KG; ++g) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[g][i] += __shfl_xor(sum[g][i], o);
        // lane i of a half writes key 8 (i / 4) + 4 half + i % 4
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) mine = col == i ? sum[g][i] : mine;
        if (col < 16) parts[wave][32 * g + 8 * (col >> 2) + 4 * half + (col & 3)] = mine;
    }
    if (apart) __syncthreads();
    if (apart && wave > 0) return;
    asm volatile("" ::: "memory");  // (a wave's own LDS writes and reads are in order)
    // slots that some row sees: not past the last one's end, nor before the first one's window
    const int64_t from = a.window > 0 ? (int64_t)cr.off + 1 - a.window : 0;
#pragma unroll
    for (int g = 0; g < KG; ++g) {
        const int t = key0 + 32 * g + col;
        if (half != 0 || !there[g] || t >= cr.off + cr.live || t < from) continue;
        float add = parts[wave][32 * g + col];
        if (apart)
            for (int w = 1; w < kWaves; ++w) add += parts[w][32 * g + col];
        a.weight_sum[b * a.slot_b + h * a.slot_h + t] += add;
    }
}

template <class TR, int DP, int NW>
hipError_t chunk_w(const AttnArgs& a, size_t lds, hipStream_t s) {
    const dim3 grid = grid_of((int64_t)a.B * a.Hkv * a.row_tiles * a.splits);
    const void* fn =
        a.D == DP ? reinterpret_cast<const void*>(&stream_kernel<TR, DP, true, true, NW, true>)
                  : reinterpret_cast<const void*>(&stream_kernel<TR, DP, true, false, NW, true>);
    if (lds > 64u << 10) {
        const hipError_t e =
            hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    AttnArgs args = a;
    void* params[] = {&args};
    return hipLaunchKernel(fn, grid, dim3(64 * NW), params, lds, s);
}

template <class TR, int DP>
hipError_t chunk_d(const AttnArgs& a, hipStream_t s) {
    const int rows = a.R < 16 ? a.R : 16;
    const int staged = a.chunk < kPiece ? a.chunk : kPiece;
    const size_t stage = (size_t)staged * 8 + (size_t)(staged / 32 + 2) * 4;
    const auto lds = [&](int nw) {
        const size_t merge = (size_t)(nw * rows * (DP + 4) + 2 * nw * 16) * 4;
        return stage > merge ? stage : merge;
    };
    constexpr int WIDE = DP <= 64 ? 16 : DP <= 128 ? 8 : 4;
    if constexpr (WIDE > 4)
        if (a.wide) return chunk_w<TR, DP, WIDE>(a, lds(WIDE), s);
    return chunk_w<TR, DP, 4>(a, lds(4), s);
}

template <class TR, int DP>
hipError_t weights_d(const AttnArgs& a, hipStream_t s) {
    constexpr int NF = DP * (int)sizeof(typename TR::storage) / 32;
    constexpr int keys = 32 * (NF <= 8 ? 2 : 1);
    const int64_t blocks = ((int64_t)a.pages.slots + keys - 1) / keys;
    if (blocks == 0) return hipSuccess;
    const int apart = (int64_t)a.B * a.Hkv * blocks < 512 * kWaves;
    const int key_blocks = (int)(apart ? blocks : (blocks + kWaves - 1) / kWaves);
    const dim3 grid = grid_of((int64_t)a.B * a.Hkv * key_blocks);
    if (a.D == DP)
        chunk_weights_kernel<TR, DP, true><<<grid, dim3(kThreads), 0, s>>>(a, key_blocks, apart);
    else
        chunk_weights_kernel<TR, DP, false><<<grid, dim3(kThreads), 0, s>>>(a, key_blocks, apart);
    return hipGetLastError();
}

template <class TR>
hipError_t chunk_t(const AttnArgs& a, hipStream_t s) {
    if (a.D <= 64) return chunk_d<TR, 64>(a, s);
    if (a.D <= 128) return chunk_d<TR, 128>(a, s);
    return chunk_d<TR, 256>(a, s);
}

template <class TR>
hipError_t join_t(const AttnArgs& a, hipStream_t s) {
    chunk_join_kernel<TR><<<grid_of((int64_t)a.B * a.Hkv * a.R), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
}

template <class TR>
hipError_t weights_t(const AttnArgs& a, hipStream_t s) {
    if (a.D <= 64) return weights_d<TR, 64>(a, s);
    if (a.D <= 128) return weights_d<TR, 128>(a, s);
    return weights_d<TR, 256>(a, s);
}

template <class F>
hipError_t by_type(ctconv_dtype dt, F f) {
    switch (dt) {
        case CTCONV_F32: return f(TF32{});
        case CTCONV_BF16: return f(TBF16{});
        case CTCONV_F16: return f(TF16{});
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_chunk_stream(const AttnArgs& a, ctconv_dtype dt, hipStream_t s) {
    return by_type(dt, [&](auto tr) { return chunk_t<decltype(tr)>(a, s); });
}

hipError_t launch_chunk_join(const AttnArgs& a, ctconv_dtype dt, hipStream_t s) {
    return by_type(dt, [&](auto tr) { return join_t<decltype(tr)>(a, s); });
}

hipError_t launch_chunk_weights(const AttnArgs& a, ctconv_dtype dt, hipStream_t s) {
    return by_type(dt, [&](auto tr) { return weights_t<decltype(tr)>(a, s); });
}

}  // namespace block
}  // namespace ctconv
