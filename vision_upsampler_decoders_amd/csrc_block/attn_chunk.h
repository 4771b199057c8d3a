// What the kernels of a chunk call share: the rows of a sequence, what they
// see, and which of them a workgroup takes.
#pragma once

#include <type_traits>

#include "block_internal.h"

namespace ctconv {
namespace block {

namespace {

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The new rows of sequence b: row i of `count` has slot off + i; `live` of them exist.
struct ChunkRows {
    int len, count, live, off;
    int64_t row0;  // the first one's number in the call
};
__device__ inline ChunkRows chunk_rows(const AttnArgs& a, int b) {
    ChunkRows r;
    r.len = clamped(a.lengths[b], a.pages.slots);
    if (a.row_starts) {
        const int from = a.row_starts[b];
        const int64_t given = (int64_t)a.row_starts[b + 1] - from;
        r.row0 = from;
        r.count = given < 0 ? 0 : given > a.most ? a.most : (int)given;
        const int room = from >= 0 && from < a.rows ? a.rows - from : 0;
        r.live = r.count < room ? r.count : room;
    } else {
        r.row0 = (int64_t)b * a.n;
        r.live = r.count = a.counts ? clamped(a.counts[b], a.n) : a.n;
    }
    r.off = r.len - r.count;
    return r;
}
// The slots that some of the rows i0 .. i1 see: [first, first + span).
__device__ inline void chunk_span(const AttnArgs& a, const ChunkRows& r, int i0, int i1, int& first,
                                  int& span) {
    first = a.window > 0 && r.off + i0 + 1 > a.window ? r.off + i0 + 1 - a.window : 0;
    span = r.off + i1 + 1 - first;
    span = span > 0 ? span : 0;
}
// Log-sum-exp of a chunk call's row: the result, and what its weights are taken against.
__device__ inline void write_lse(const AttnArgs& a, int64_t at, float top, float sum) {
    if (a.lse) a.lse[at] = top * kLn2 + logf(sum);
    // a row without a visible slot adds nothing: exp2(s - infinity)
    if (a.lse2)
        a.lse2[at] = top == -__builtin_huge_valf() && sum == 0.f
                         ? __builtin_huge_valf()
                         : top + __builtin_amdgcn_logf(sum);
}
// Bits [0, x) of 32.
__device__ inline uint32_t low_bits(int x) {
    return x >= 32 ? 0xFFFFFFFFu : x <= 0 ? 0u : (1u << x) - 1;
}

// The infinities and NaN of packed values, set to zero; not 0 where there were any.
// (An exponent of ones is the one that carries into the sign bit.  No compare
// masks: the tile kernel's scalar registers are full.)
template <class TR>
__device__ inline uint32_t take_odd(uint32_t& w) {
    uint32_t odd;
    if constexpr (std::is_same_v<TR, TF32>) {
        odd = (uint32_t)((int32_t)((w & 0x7FFFFFFFu) + 0x00800000u) >> 31);
    } else {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
        constexpr uint16_t one = std::is_same_v<TR, TBF16> ? 0x0080 : 0x0400;
        const u16x2 t = __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu) + u16x2{one, one};
        odd = __builtin_bit_cast(uint32_t, (i16x2)(__builtin_bit_cast(i16x2, t) >> (int16_t)15));
    }
    w &= ~odd;
    return odd;
}

// The row tiles of 128 of all sequences, for calls with many rows: those of a
// sequence from the last one down (it sees the most keys), each in the same number
// of splits, the heads fastest (workgroups go to the XCDs in turn, so that a head's
// tiles meet its keys in one L2).  False behind the last one.  split_too: item
// `number` is a split of a tile, else a tile.  Called by whole workgroups of
// `waves` waves.
__device__ inline int chunk_splits(const AttnArgs& a, const ChunkRows& r) {
    int span = r.off + r.live;
    // (128 rows lie at most this far apart)
    const int most = a.window + (a.most < 128 ? a.most : 128);
    span = a.window > 0 && span > most ? most : span;
    return span > a.chunk ? (span + a.chunk - 1) / a.chunk : 1;
}
__device__ inline bool chunk_item(const AttnArgs& a, int waves, uint32_t number, bool split_too,
                                  int& b, int& h, int& tile, int& split) {
    __shared__ uint32_t sums[4], found[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t target = number / a.Hkv;
    h = (int)(number - target * a.Hkv);
    uint32_t before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64 * waves) {
        uint32_t mine = 0;
        if (b0 + tid < a.B) {
            const ChunkRows r = chunk_rows(a, b0 + tid);
            mine = (uint32_t)((r.live * a.G + 127) >> 7) * (split_too ? chunk_splits(a, r) : 1);
        }
        uint32_t to = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t w = __shfl_up(to, o);
            to += lane >= o ? w : 0;
        }
        if (lane == 63) sums[wave] = to;
        __syncthreads();
        uint32_t all = before;
        for (int w = 0; w < waves; ++w) {
            if (w == wave) to += all;
            all += sums[w];
        }
        if (target < to && target >= to - mine) {
            found[0] = b0 + tid;
            found[1] = target - (to - mine);
        }
        __syncthreads();
        if (target < all) {
            b = __builtin_amdgcn_readfirstlane((int)found[0]);
            const int at = __builtin_amdgcn_readfirstlane((int)found[1]);
            const ChunkRows r = chunk_rows(a, b);
            const int splits = split_too ? chunk_splits(a, r) : 1;
            tile = at / splits;
            split = at - tile * splits;
            tile = ((r.live * a.G + 127) >> 7) - 1 - tile;
            return true;
        }
        before = all;
    }
    return false;
}

}  // namespace
}  // namespace block
}  // namespace ctconv
