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

#include "block_internal.h"
#include "mfma_common.h"

namespace ctconv {
namespace block {

namespace {

using mfma::Mma;
using mfma::u32x2;
using mfma::u32x4;

constexpr int kWaves = 4;  // of the join kernels
constexpr int kThreads = 64 * kWaves;
constexpr float kRaise = 8.f;

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

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

template <class TR, int DP, bool PAGED, bool EXACT, int NW>
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
    const int tile = item % a.row_tiles;
    const int bh = item / a.row_tiles;
    const int b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int row0 = tile * 16;
    const int rows = a.R - row0 < 16 ? a.R - row0 : 16;

    // Queries of this tile: lane (col, g) holds pieces 4f + g of row col.  They
    // and, where no length moves the first slot, this thread's page are asked
    // for before the length has arrived: a short call is a chain of latencies.
    u32x4 qf[NF];
    {
        const int r = row0 + col;
        const bool live = col < rows;
        const int lq = live ? (int)fdiv((uint32_t)r, a.fd_G) : 0;
        const S* qr = static_cast<const S*>(a.q) + b * a.q_b + lq * a.q_row +
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
    if (PAGED && a.window == 0 && start + tid < a.pages.slots)
        page0 = a.pages.table[b * a.pages.table_stride +
                              (int)fdiv((uint32_t)(start + tid), a.pages.fd_page)];

    int first, span;
    visible<PAGED>(a, b, first, span);
    if (a.splits > 1 && start >= span) return;
    int n = span - start;
    n = n < a.chunk ? n : a.chunk;
    n = n > 0 ? n : 0;

    // Row offsets and visibility bits of the chunk's keys.
    int64_t* offs = reinterpret_cast<int64_t*>(lds);
    uint32_t* seen = reinterpret_cast<uint32_t*>(lds + (PAGED ? (size_t)a.chunk * 8 : 0));
    const int padded = (n + 63) & ~63;
    for (int i = tid; i < padded; i += (64 * NW)) {
        bool ok = i < n;
        const int t = first + start + i;
        if constexpr (PAGED) {
            int64_t o = -1;
            if (ok)
                o = a.window == 0 && i == tid ? offset_in_page(a.pages, t, page0)
                                              : slot_offset(a.pages, b, t);
            ok = o >= 0;
            offs[i] = ok ? o : 0;  // page 0 exists: a readable row
        } else {
            if (ok && a.mask) ok = a.mask[b * a.mask_stride + t] != 0;
        }
        const uint64_t w = __ballot(ok);
        if (lane == 0) *reinterpret_cast<uint64_t*>(seen + (i >> 5)) = w;
    }

    const S* kbase = static_cast<const S*>(a.k) +
                     (PAGED ? h * a.pages.head_stride : b * a.k_b + h * a.k_head);
    const S* vbase = static_cast<const S*>(a.v) +
                     (PAGED ? h * a.pages.head_stride : b * a.v_b + h * a.v_head);
    __syncthreads();
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

    for (int kb = wave * KB; kb < n; kb += NW * KB) {
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
                const u32x2 w = *reinterpret_cast<const u32x2*>(vrow + (EXACT || d < a.D ? d : 0));
                vr[j][0] = w[0];
                vr[j][1] = w[1];
            } else {
#pragma unroll
                for (int p = 0; p < VW / 4; ++p) {
                    const int dp = d + p * VEC;
                    const u32x4 w =
                        *reinterpret_cast<const u32x4*>(vrow + (EXACT || dp < a.D ? dp : 0));
#pragma unroll
                    for (int q = 0; q < 4; ++q) vr[j][4 * p + q] = w[q];
                }
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
                if (bits != all && !((bits >> (16 * t + 4 * g + i)) & 1)) v = -__builtin_huge_valf();
                s[t][i] = v;
                top = fmaxf(top, v);
            }
        if (a.scores && col < rows) {
            float* sr = a.scores + ((int64_t)bh * a.R + row0 + col) * a.score_stride + start + kb;
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
                    vf[w] = __builtin_amdgcn_perm(vr[2 * w + 1][e >> 1], vr[2 * w][e >> 1], sel);
                Mma<TR>::step(acc[e], vf, pf);
                Mma<TR>::step(acc[e], vf, pl);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VK; ++j)
#pragma unroll
                for (int e = 0; e < VPL; ++e)
                    acc[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(vr[j][e]), p[j],
                                                                  acc[e], 0, 0, 0);
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // Merge the waves: [wave][row][DS] outputs, then [wave][row] maxima and
    // sums.  Who writes a piece of a row weighs the waves by itself: NW
    // exponentials cost less than one more barrier.
    __syncthreads();  // offs and seen are no longer read
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
        if (a.direct) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int rr = row0 + r, lq = (int)fdiv((uint32_t)rr, a.fd_G);
            const int hq = h * a.G + (rr - lq * a.G);
            S* to = static_cast<S*>(a.out) + b * a.o_b + lq * a.o_row + (int64_t)hq * a.o_head + d;
            if (d == 0 && a.lse)
                a.lse[((int64_t)b * a.Hq + hq) * a.Lq + lq] = top * kLn2 + logf(sum);
            if constexpr (ES == 2) {
                u32x2 w{mfma::pack2<TR>(o[0] * inv, o[1] * inv),
                        mfma::pack2<TR>(o[2] * inv, o[3] * inv)};
                *reinterpret_cast<u32x2*>(to) = w;
            } else {
                *reinterpret_cast<f32x4*>(to) = o * inv;
            }
        } else {
            const int64_t part = ((int64_t)bh * a.splits + split) * a.R + row0 + r;
            *reinterpret_cast<f32x4*>(a.part_o + part * a.D + d) = o;
            if (d == 0) {
                a.part_ml[2 * part] = top;
                a.part_ml[2 * part + 1] = sum;
            }
        }
    }
}

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
            const float f = s0 + i < n ? exp2_fast(v[i][0] - ref) : 0.f;
            sum = fmaf(f, v[i][1], sum);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(f, x[i][e], o[e]);
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
