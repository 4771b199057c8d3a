// Attention of few query rows per cache head: one new row over the paged
// cache, single tokens over an encoder's states.
//
// With at most 16 query rows per tile every key and value is used once per
// tile, so the work is reading them: keys and values go from memory straight
// to registers in 16-byte pieces and never through LDS.  A wave takes blocks
// of KB keys.
//  - Scores: S^T = K Q^T by 16x16 matrix instructions, a key per row, a query
//    per column, so a lane holds 4 consecutive keys (4g .. 4g + 3 for lane
//    group g = lane / 16) of one query, lane % 16.
//  - The output is O^T = V^T P^T.  A matrix instruction sums over its k slots
//    in whatever order, so slot j of lane group g stands for exactly the keys
//    whose scores the group already holds, and P needs no exchange between
//    lanes.  V^T needs, per lane, one value column over those keys: lane c of
//    a group loads the c-th piece of VPL values of each key's row (whole rows,
//    coalesced) and turns its keys x VPL block in registers.  Output tile e
//    holds the value columns c * VPL + e.
//  - Softmax is the one-pass one, base 2, per wave: a running maximum m that
//    is only raised when a score passes it by 2^8 (the weights stay below
//    2^8, far from overflow in every type, and rescaling is rare), and the
//    sum of the weights, in fp32.  A matrix instruction takes both operands in
//    one type, so 16-bit weights meet V in two parts, the rounded weight and
//    the rounded rest: relative error 2^-16 (bf16) or 2^-22 each instead of
//    2^-8 or 2^-11, and no time (serving batch below 157.6 us against 158.0,
//    one token 16.0 against 15.9): the matrix unit waits for memory.
// The waves of a workgroup are merged in LDS, the workgroups of one row tile
// by a second kernel, both in a fixed order.
//
// Long calls are bound by memory, whole rows of 16-byte pieces in random pages:
// 48 ragged sequences up to 8192 (32 query heads on 8 cache heads, D = 128,
// bf16; 760 MB) take 147 us, 5.2 TB/s, and 7.3 for the join (a read-only sweep
// of random 4 KB pieces reaches 6.0).  Single tokens to up to 1500 states of
// 256 heads (D = 64, bf16; 50 MB) take 15 us and one frame's window of 250
// slots 8: one round of workgroups each, whose loads, merge and stores follow
// each other.

//
// Chunk calls (CHUNK: several new rows per sequence in causal order) differ in
// what a row sees.  Blocks that every row of the tile sees whole are as above;
// in the others each row hides its own keys.  A hidden key's weight is 0, but
// 0 times an infinity or a NaN is NaN, and so is an infinity times a weight in
// two parts of which one is 0.  A workgroup whose sums are not all finite goes
// over its keys once more: V's infinities and NaN are then taken out of the
// product and added to the rows that see them.
// 2 rows of 8 heads over a window of 250, fp32: 9.5 us (one row of a paged call: 8.4).
// 128 rows per key head over 24 x 8192 keys, D = 128, bf16: 560 us, and 955 with a
// head's row tiles on different XCDs; a window of 1000 over 3867 rows of 8 heads, D =
// 64, fp32: 88 us, the matrix unit 59 % busy.

#pragma once

#include "attn_chunk.h"
#include "block_internal.h"
#include "mfma_common.h"

namespace ctconv {
namespace block {

namespace {

using mfma::Mma;
using mfma::u32x2;
using mfma::u32x4;

constexpr float kRaise = 8.f;
constexpr int kPiece = 1024;

// A maximum as what weights are taken against: where nothing is seen (minus
// infinity), 0, so that the weights of hidden scores are zero and a sum that
// is NaN (no maximum is, see fmaxf) stays NaN.
__device__ inline float reference_of(float top) {
    return top == -__builtin_huge_valf() ? 0.f : top;
}

// The keys of sequence b that the call sees: [first, first + span).
template <bool PAGED>
__device__ inline void visible(const AttnArgs& a, int b, int& first, int& span) {
    const int hi = PAGED ? a.pages.slots : a.Lk;
    const int n = a.lengths ? clamped(a.lengths[b], hi) : hi;
    first = PAGED && a.window > 0 && n > a.window ? n - a.window : 0;
    span = n - first;
}

template <class TR, int DP, bool PAGED, bool EXACT, int NW, bool CHUNK = false>
__global__ __launch_bounds__(64 * NW, NW > 4 ? 1 : DP <= 64 ? 4 : DP <= 128 ? 3 : 1) void
stream_kernel(AttnArgs a) {
    using S = typename TR::storage;
    constexpr int ES = sizeof(S), VEC = 16 / ES;
    constexpr int KB = ES == 2 ? 32 : 16;  // keys per block
    constexpr int NT = KB / 16;            // score tiles per block
    constexpr int NF = DP / (4 * VEC);     // 16-byte pieces of a key per lane
    constexpr int VPL = DP / 16;           // values of a row per lane
    constexpr int VW = VPL * ES / 4;       // the same in dwords
    constexpr int VK = 4 * NT;             // keys per lane group
    constexpr int DS = DP + 4;             // LDS row of a merged output
    extern __shared__ __align__(16) char lds[];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 15, g = lane >> 4;
    // Splits slowest: workgroups go to the XCDs in turn, and the late splits
    // of ragged sequences, which are empty, must not all fall to the same
    // ones (splits fastest, 16 of them: 212 us instead of 157 for 48 ragged
    // sequences up to 8192).
    const int tiles = a.B * a.Hkv * a.row_tiles;
    if (block_number() >= (uint32_t)(tiles * a.splits)) return;
    int item = (int)block_number();
    const int split = item / tiles;
    item -= split * tiles;
    int tile, bh, b, h;
    if constexpr (CHUNK) {
        // heads fastest: the row tiles of a head, which read the same keys, follow
        // each other on one XCD
        const int bt = item / a.Hkv;
        h = item - bt * a.Hkv;
        b = bt / a.row_tiles;
        tile = bt - b * a.row_tiles;
        bh = b * a.Hkv + h;
    } else {
        tile = item % a.row_tiles;
        bh = item / a.row_tiles;
        b = bh / a.Hkv;
        h = bh - b * a.Hkv;
    }
    const int row0 = tile * 16;
    ChunkRows cr;
    if constexpr (CHUNK) {
        cr = chunk_rows(a, b);
        if (row0 >= cr.live * a.G) return;
    }
    const int R = CHUNK ? cr.live * a.G : a.R;
    const int rows = R - row0 < 16 ? R - row0 : 16;

    // Queries of this tile: lane (col, g) holds pieces 4f + g of row col.  They
    // and, where no length moves the first slot, this thread's page are asked
    // for before the length has arrived: a short call is a chain of latencies.
    u32x4 qf[NF];
    int my_end = 0, my_begin = 0;  // CHUNK: the slots that this lane's row sees
    {
        const int r = row0 + col;
        const bool live = col < rows;
        const int lq = live ? (int)fdiv((uint32_t)r, a.fd_G) : 0;
        if constexpr (CHUNK) {
            my_end = cr.off + lq + 1;
            my_begin = a.window > 0 ? my_end - a.window : 0;
        }
        const int64_t q_from =
            CHUNK && a.row_starts ? cr.row0 * a.q_row : b * a.q_b;
        const S* qr = static_cast<const S*>(a.q) + q_from + lq * a.q_row +
                      (int64_t)(h * a.G + (live ? r - lq * a.G : 0)) * a.q_head;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int d = (4 * f + g) * VEC;
            qf[f] = u32x4{0, 0, 0, 0};
            if (live && (EXACT || d < a.D)) qf[f] = *reinterpret_cast<const u32x4*>(qr + d);
        }
    }
    const int start = split * a.chunk;  // relative to the first slot
    int page0 = -1;
    if (PAGED && !CHUNK && a.window == 0 && start + tid < a.pages.slots)
        page0 = a.pages.table[b * a.pages.table_stride +
                              (int)fdiv((uint32_t)(start + tid), a.pages.fd_page)];

    int first, span;
    int all_from = 0, all_to = 0;  // CHUNK: what every row of the tile sees
    bool direct = a.direct;
    if constexpr (CHUNK) {
        const int i0 = (int)fdiv((uint32_t)row0, a.fd_G);
        const int i1 = (int)fdiv((uint32_t)(row0 + rows - 1), a.fd_G);
        chunk_span(a, cr, i0, i1, first, span);
        all_from = a.window > 0 ? cr.off + i1 + 1 - a.window : 0;
        all_to = cr.off + i0 + 1;
        if (split > 0 && start >= span) return;
        direct = span <= a.chunk;
    } else {
        visible<PAGED>(a, b, first, span);
        if (a.splits > 1 && start >= span) return;
    }
    int n = span - start;
    n = n < a.chunk ? n : a.chunk;
    n = n > 0 ? n : 0;

    // Row offsets and visibility bits of the chunk's keys.
    int64_t* offs = reinterpret_cast<int64_t*>(lds);
    // (of a chunk call: of kPiece keys at a time, its chunks may be long)
    const int staged = CHUNK && a.chunk > kPiece ? kPiece : a.chunk;
    uint32_t* seen = reinterpret_cast<uint32_t*>(lds + (PAGED ? (size_t)staged * 8 : 0));
    const auto stage = [&](int from, int to) __attribute__((always_inline)) {
        const int padded = (to - from + 63) & ~63;
        for (int i = tid; i < padded; i += (64 * NW)) {
            bool ok = i < to - from;
            const int t = first + start + from + i;
            if constexpr (PAGED) {
                int64_t o = -1;
                if (ok)
                    o = !CHUNK && a.window == 0 && i == tid ? offset_in_page(a.pages, t, page0)
                                                            : slot_offset(a.pages, b, t);
                ok = o >= 0;
                offs[i] = ok ? o : 0;  // page 0 exists: a readable row
            } else {
                if (ok && a.mask) ok = a.mask[b * a.mask_stride + t] != 0;
            }
            const uint64_t w = __ballot(ok);
            if (lane == 0) *reinterpret_cast<uint64_t*>(seen + (i >> 5)) = w;
        }
    };
    if constexpr (!CHUNK) stage(0, n);

    const S* kbase = static_cast<const S*>(a.k) +
                     (PAGED ? h * a.pages.head_stride : b * a.k_b + h * a.k_head);
    const S* vbase = static_cast<const S*>(a.v) +
                     (PAGED ? h * a.pages.head_stride : b * a.v_b + h * a.v_head);
    if constexpr (!CHUNK) __syncthreads();
    if (a.negate)
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i) qf[f][i] ^= ES == 2 ? 0x80008000u : 0x80000000u;

    f32x4 acc[VPL];
#pragma unroll
    for (int e = 0; e < VPL; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -__builtin_huge_valf(), l = 0.f;
    const int t0 = first + start;

    __shared__ int odd_sums;
    if (CHUNK && tid == 0) odd_sums = 0;
    // (CHUNK: once more, carefully, where sums are odd)
    for (bool careful = false;; careful = true) {
        int done = 0;  // keys of earlier pieces
        int n_here = n;
        do {
            if constexpr (CHUNK) {
                n_here = n - done < kPiece ? n - done : kPiece;
                if (done > 0) __syncthreads();
                stage(done, done + n_here);
                __syncthreads();
            }
            for (int kb = wave * KB; kb < n_here; kb += NW * KB) {
                uint32_t bits = seen[kb >> 5];
                if (KB == 16) bits = (bits >> (kb & 16)) & 0xFFFFu;
                const uint32_t all = KB == 32 ? 0xFFFFFFFFu : 0xFFFFu;
                if (bits == 0 && !a.scores) continue;
                u32x4 kf[NT][NF];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int i = kb + 16 * t + col;
                    int64_t o;
                    if constexpr (PAGED) o = offs[i];
                    else o = (bits >> (16 * t + col)) & 1 ? (int64_t)(t0 + i) * a.k_row : 0;
                    const S* kr = kbase + o;
#pragma unroll
                    for (int f = 0; f < NF; ++f) {
                        const int d = (4 * f + g) * VEC;
                        kf[t][f] = *reinterpret_cast<const u32x4*>(kr + (EXACT || d < a.D ? d : 0));
                    }
                }
                // Values: key slot j of this lane group is key 4g + j % 4 of score
                // tile j / 4.
                uint32_t vr[VK][VW];
#pragma unroll
                for (int j = 0; j < VK; ++j) {
                    const int i = kb + 16 * (j >> 2) + 4 * g + (j & 3);
                    int64_t o;
                    if constexpr (PAGED) o = offs[i];
                    else o = (bits >> (i - kb)) & 1 ? (int64_t)(t0 + i) * a.v_row : 0;
                    const int d = col * VPL;
                    const S* vrow = vbase + o;
                    if constexpr (VW == 2) {
                        const u32x2 w =
                            *reinterpret_cast<const u32x2*>(vrow + (EXACT || d < a.D ? d : 0));
                        vr[j][0] = w[0];
                        vr[j][1] = w[1];
                    } else {
#pragma unroll
                        for (int p = 0; p < VW / 4; ++p) {
                            const int dp = d + p * VEC;
                            const u32x4 w = *reinterpret_cast<const u32x4*>(
                                vrow + (EXACT || dp < a.D ? dp : 0));
#pragma unroll
                            for (int q = 0; q < 4; ++q) vr[j][4 * p + q] = w[q];
                        }
                    }
                }
                // CHUNK: what this lane's row sees of the block
                uint32_t mine = bits;
                bool odd = false;
                if constexpr (CHUNK) {
                    const int at = t0 + done + kb;
                    if (at < all_from || at + KB > all_to)
                        mine &= low_bits(my_end - at) & ~low_bits(my_begin - at);
                    if (careful) {
#pragma unroll
                        for (int j = 0; j < VK; ++j)
                            if ((bits >> (16 * (j >> 2) + 4 * g + (j & 3))) & 1)
#pragma unroll
                                for (int w = 0; w < VW; ++w) odd |= take_odd<TR>(vr[j][w]) != 0;
                    }
                }
                f32x4 s[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int f = 0; f < NF; ++f) {
                        u32x4 k = kf[t][f];
                        // the piece past the row was read from its start: not a product
                        if (!EXACT && (4 * f + g) * VEC >= a.D) k = u32x4{0, 0, 0, 0};
                        Mma<TR>::step(s[t], k, qf[f]);
                    }
                }
                float top = -__builtin_huge_valf();
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v = s[t][i] * a.c;
                        if (mine != all && !((mine >> (16 * t + 4 * g + i)) & 1))
                            v = -__builtin_huge_valf();
                        s[t][i] = v;
                        top = fmaxf(top, v);
                    }
                if (a.scores && col < rows) {
                    float* sr = a.scores + ((int64_t)bh * a.R + row0 + col) * a.score_stride +
                                start + kb;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        *reinterpret_cast<f32x4*>(sr + 16 * t + 4 * g) = s[t];
                }
                if (bits != all) {
                    // what a slot without a visible key holds may be NaN: zero, not 0 * NaN
#pragma unroll
                    for (int j = 0; j < VK; ++j)
                        if (!((bits >> (16 * (j >> 2) + 4 * g + (j & 3))) & 1))
#pragma unroll
                            for (int w = 0; w < VW; ++w) vr[j][w] = 0;
                }
                if (__any(top > m + kRaise)) {
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    const float up = fmaxf(m, top);
                    const float f = m == up ? 1.f : exp2_fast(m - up);
                    m = up;
                    l *= f;
#pragma unroll
                    for (int e = 0; e < VPL; ++e)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[e][i] *= f;
                }
                const float ref = reference_of(m);
                float p[VK];
#pragma unroll
                for (int j = 0; j < VK; ++j) {
                    p[j] = exp2_fast(s[j >> 2][j & 3] - ref);
                    l += p[j];
                }
                if constexpr (ES == 2) {
                    u32x4 pf, pl;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const float p0 = p[2 * w], p1 = p[2 * w + 1];
                        pf[w] = mfma::pack2<TR>(p0, p1);
                        pl[w] = mfma::pack2<TR>(p0 - TR::to_f32((uint16_t)pf[w]),
                                                p1 - TR::to_f32((uint16_t)(pf[w] >> 16)));
                    }
#pragma unroll
                    for (int e = 0; e < VPL; ++e) {
                        const unsigned sel = (e & 1) ? 0x07060302u : 0x05040100u;
                        u32x4 vf;
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            vf[w] = __builtin_amdgcn_perm(vr[2 * w + 1][e >> 1],
                                                          vr[2 * w][e >> 1], sel);
                        Mma<TR>::step(acc[e], vf, pf);
                        Mma<TR>::step(acc[e], vf, pl);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < VK; ++j)
#pragma unroll
                        for (int e = 0; e < VPL; ++e)
                            acc[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                __uint_as_float(vr[j][e]), p[j], acc[e], 0, 0, 0);
                }
                if constexpr (CHUNK)
                    if (__any(odd)) {
                        // this lane's values of output columns (4 g + i) VPL + e, row col (what
                        // lies past a row's end goes to columns that are not written)
                        constexpr int RUN = VPL < 8 ? VPL : 8;
                        for (int j = 0; j < KB; ++j) {
                            if (!((bits >> j) & 1)) continue;
                            const S* vrow = vbase + offs[kb + j];
                            const float sees = (mine >> j) & 1 ? 1.f : 0.f;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int e0 = 0; e0 < VPL; e0 += RUN) {
                                    const int d = (4 * g + i) * VPL + e0;
                                    const S* run = vrow + (EXACT || d < a.D ? d : 0);
#pragma unroll
                                    for (int e = 0; e < RUN; ++e) {
                                        const float x = TR::to_f32(run[e]);
                                        if (sees != 0.f && !(fabsf(x) <= __FLT_MAX__))
                                            acc[e0 + e][i] += x;
                                    }
                                }
                        }
                    }
            }
            done += n_here;
        } while (CHUNK && done < n);
        if constexpr (!CHUNK) break;
        // What is not finite in a sum (0 times infinity is NaN) is in it for good.
        float worst = 0.f;
#pragma unroll
        for (int e = 0; e < VPL; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) worst += 0.f * acc[e][i];
        if (!careful && __any(worst != 0.f)) odd_sums = 1;
        __syncthreads();  // offs and seen are no longer read
        if (careful || !odd_sums) break;
#pragma unroll
        for (int e = 0; e < VPL; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
        m = -__builtin_huge_valf();
        l = 0.f;
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // Merge the waves: [wave][row][DS] outputs, then [wave][row] maxima and
    // sums.  Who writes a piece of a row weighs the waves by itself: NW
    // exponentials cost less than one more barrier.
    if constexpr (!CHUNK) __syncthreads();  // offs and seen are no longer read
    float* mo = reinterpret_cast<float*>(lds);
    float* mm = mo + NW * rows * DS;
    float* ml = mm + NW * 16;
    if (col < rows) {
        float* o = mo + (wave * rows + col) * DS;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < VPL; e += 4)
                *reinterpret_cast<f32x4*>(o + (4 * g + i) * VPL + e) =
                    f32x4{acc[e][i], acc[e + 1][i], acc[e + 2][i], acc[e + 3][i]};
        if (g == 0) {
            mm[wave * 16 + col] = m;
            ml[wave * 16 + col] = l;
        }
    }
    __syncthreads();
    const int pieces = a.D / 4;
    for (int i = tid; i < rows * pieces; i += (64 * NW)) {
        const int r = i / pieces, d = (i - r * pieces) * 4;
        float top = mm[r];
#pragma unroll
        for (int w = 1; w < NW; ++w) top = fmaxf(top, mm[w * 16 + r]);
        const float low = reference_of(top);  // no key: factors 0
        float sum = 0.f;
        f32x4 o{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = exp2_fast(mm[w * 16 + r] - low);
            sum = fmaf(f, ml[w * 16 + r], sum);
            const f32x4 x = *reinterpret_cast<const f32x4*>(mo + (w * rows + r) * DS + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(f, x[e], o[e]);
        }
        if (direct) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int rr = row0 + r, lq = (int)fdiv((uint32_t)rr, a.fd_G);
            const int hq = h * a.G + (rr - lq * a.G);
            const int64_t o_from =
                CHUNK && a.row_starts ? cr.row0 * a.o_row : b * a.o_b;
            S* to = static_cast<S*>(a.out) + o_from + lq * a.o_row + (int64_t)hq * a.o_head + d;
            if constexpr (CHUNK) {
                if (d == 0) write_lse(a, (cr.row0 + lq) * a.Hq + hq, top, sum);
            } else if (d == 0 && a.lse)
                a.lse[((int64_t)b * a.Hq + hq) * a.Lq + lq] = top * kLn2 + logf(sum);
            if constexpr (ES == 2) {
                u32x2 w{mfma::pack2<TR>(o[0] * inv, o[1] * inv),
                        mfma::pack2<TR>(o[2] * inv, o[3] * inv)};
                *reinterpret_cast<u32x2*>(to) = w;
            } else {
                *reinterpret_cast<f32x4*>(to) = o * inv;
            }
        } else {
            int64_t part = ((int64_t)bh * a.splits + split) * a.R + row0 + r;
            if constexpr (CHUNK) {
                const int rr = row0 + r, lq = (int)fdiv((uint32_t)rr, a.fd_G);
                part = ((cr.row0 + lq) * a.Hq + h * a.G + (rr - lq * a.G)) * a.splits + split;
            }
            *reinterpret_cast<f32x4*>(a.part_o + part * a.D + d) = o;
            if (d == 0) {
                a.part_ml[2 * part] = top;
                a.part_ml[2 * part + 1] = sum;
            }
        }
    }
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Maximum and sum (relative to it) of each of N rows over its splits; every
// lane of the wave calls it and gets both.  Up to 128 splits, of all N rows,
// are read in one go.
template <int N>
__device__ inline void join_stats(const float* const (&ml)[N], int64_t stride, int n,
                                  float (&top)[N], float (&sum)[N]) {
    const int lane = threadIdx.x & 63;
    f32x2 v[N][2];
#pragma unroll
    for (int r = 0; r < N; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t s = lane + 64 * i < n ? lane + 64 * i : 0;
            v[r][i] = *reinterpret_cast<const f32x2*>(ml[r] + 2 * s * stride);
        }
#pragma unroll
    for (int r = 0; r < N; ++r) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane + 64 * i >= n) v[r][i] = f32x2{-__builtin_huge_valf(), 0.f};
        top[r] = fmaxf(v[r][0][0], v[r][1][0]);
        for (int s = lane + 128; s < n; s += 64) top[r] = fmaxf(top[r], ml[r][2 * s * stride]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < N; ++r) top[r] = fmaxf(top[r], __shfl_xor(top[r], o));
#pragma unroll
    for (int r = 0; r < N; ++r) {
        sum[r] = 0.f;
        const float ref = reference_of(top[r]);
#pragma unroll
        for (int i = 0; i < 2; ++i) sum[r] += exp2_fast(v[r][i][0] - ref) * v[r][i][1];
        for (int s = lane + 128; s < n; s += 64)
            sum[r] += exp2_fast(ml[r][2 * s * stride] - ref) * ml[r][2 * s * stride + 1];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < N; ++r) sum[r] += __shfl_xor(sum[r], o);
}

}  // namespace
}  // namespace block
}  // namespace ctconv
