// Attention of a chunk of new rows over the paged cache: the chunk form of the
// streaming kernel (attn_stream.h) for few rows per key head, the join of its
// splits (a workgroup per row, as few rows have many splits), and the weights of the
// slots.

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

// Groups of 32 keys of a wave: two where the registers allow it.
template <bool APART>
constexpr int key_groups(int pieces) {
    return pieces <= (APART ? 4 : 8) ? 2 : 1;
}

// weight_sum[b][h][t] += the sum over rows and heads of exp2(score - lse2).  The
// sums of all slots have to be known before any slot can be weighed, so the
// scores are computed again.  A wave keeps its keys in registers (32 or 64 of
// them, a key per row of the matrix instruction) and walks the query rows, 32 at a
// time; a lane adds up its query column and the columns are added at the end.  The
// rows go through LDS: read straight to the instruction's lanes, 16 bytes of each
// of 32 rows at a time, they keep the load unit busy for longer than the matrix
// instructions take (4096 rows of 24 heads over 32768 keys twice, f16: 3126 us, and
// 2005 this way; 1822 now).  The waves of a workgroup take keys of their own and the
// same rows, or, where that would leave compute units idle (APART), the same keys and
// every fourth rows: where those are at most 512 workgroups (bf16, 4 heads of 128
// channels, apart | together, the call: 4000 rows of 16 heads over 4000 keys, 500
// workgroups apart, 212 | 487 us; 500 of 32 over 8: 1000 keys, 256 workgroups,
// 53 | 98, 4000, 1000, 105 | 119, twice 4000, 2000, 198 | 176; 16 rows of 32: 21 | 22,
// 32 | 25, 52 | 33).
// 1.55 TFLOP in 1.82 ms there: 0.7 of it for the exponentials, 0.7 for the matrix
// instructions, 0.35 for two more vector instructions a score; each is busy while the
// other waits.  Tried: the scores of one group weighed between the next one's matrix
// instructions (5.6 ms the call, and 5.5 without).
template <class TR, int DP, bool EXACT, bool APART>
__global__ __launch_bounds__(kThreads, DP * sizeof(typename TR::storage) > 512 ? 1 : 2) void
chunk_weights_kernel(AttnArgs a, int key_blocks) {
    using S = typename TR::storage;
    constexpr int ES = sizeof(S), VEC = 16 / ES;
    constexpr int NF = DP / (2 * VEC), PIECES = DP / VEC, ROW = DP * ES, TILE = 32 * ROW;
    constexpr int KG = key_groups<APART>(NF);
    constexpr int LOADERS = APART ? 64 : kThreads, LOADS = TILE / 16 / LOADERS;
    static_assert(LOADERS % PIECES == 0, "a thread moves the same piece of every row");
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 31, half = lane >> 5;
    const uint32_t number = block_number();
    if (number >= (uint32_t)a.B * a.Hkv * key_blocks) return;
    const int h = (int)(number % a.Hkv), bk = (int)(number / a.Hkv);
    const int b = bk / key_blocks, kb = bk - b * key_blocks;
    const ChunkRows cr = chunk_rows(a, b);
    constexpr int KEYS = KG * 32 * (APART ? 1 : kWaves);  // of the workgroup
    const int key0 = kb * KEYS + (APART ? 0 : wave * KG * 32), key_end = key0 + KG * 32;
    // rows that see some of the workgroup's keys
    int lo = kb * KEYS - cr.off;
    lo = lo > 0 ? lo : 0;
    int hi = cr.live;
    if (a.window > 0) {
        const int64_t most = (int64_t)(kb + 1) * KEYS - 1 - cr.off + a.window;
        hi = most < hi ? (int)most : hi;
    }
    if (lo >= hi) return;

    f32x16 sum[KG];
#pragma unroll
    for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[g][i] = 0.f;
    const S* qb = static_cast<const S*>(a.q) + (a.row_starts ? cr.row0 * a.q_row : b * a.q_b) +
                  (int64_t)(h * a.G) * a.q_head;
    const float* lse2 = a.lse2 + cr.row0 * a.Hq + h * a.G;
    const float c = a.negate ? -a.c : a.c;
    const int r_first = lo * a.G + (APART ? 32 * wave : 0), r_end = hi * a.G;
    constexpr int STEP = APART ? 32 * kWaves : 32;
    // Each lane steps from row to row by additions (row r is row r / G of the
    // sequence, head r % G).  Rows past the last one are read as that one and weigh
    // nothing.
    const int by_row = (int)fdiv((uint32_t)STEP, a.fd_G), by_head = STEP - by_row * a.G;
    const int64_t q_step = by_row * a.q_row + by_head * a.q_head;
    const int64_t q_turn = a.q_row - a.G * a.q_head;
    struct Walk {
        int row, head;
    };
    const auto start = [&](int r) __attribute__((always_inline)) {
        const int row = (int)fdiv((uint32_t)r, a.fd_G);
        return Walk{row, r - row * a.G};
    };
    char* const mine = lds + (APART ? wave * 2 * TILE : 0);
    const int loader = APART ? lane : tid, piece = loader % PIECES, first = loader / PIECES;
    const S* const q_piece = qb + (EXACT || piece * VEC < a.D ? piece * VEC : 0);
    u32x4 moved[LOADS];
    int q_head[LOADS];
    const S* q_at[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const Walk w = start(r_first + first + i * (LOADERS / PIECES));
        q_head[i] = w.head;
        q_at[i] = q_piece + w.row * a.q_row + w.head * a.q_head;
    }
    const Walk end_row = start(r_end - 1), my_row = start(r_first + col);
    const S* const q_last = q_piece + end_row.row * a.q_row + end_row.head * a.q_head;
    int low_head = my_row.head, low_row = my_row.row;
    float low_next = 0.f;
    int end_next = 0;
    const auto load = [&](int r0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const bool is = r0 + first + i * (LOADERS / PIECES) < r_end;
            moved[i] = *reinterpret_cast<const u32x4*>(is ? q_at[i] : q_last);
            q_head[i] += by_head;
            q_at[i] += q_step;
            if (q_head[i] >= a.G) {
                q_head[i] -= a.G;
                q_at[i] += q_turn;
            }
        }
    };
    const auto load_low = [&](int r0) __attribute__((always_inline)) {
        const bool is = r0 + col < r_end;
        const int row = is ? low_row : end_row.row, head = is ? low_head : end_row.head;
        low_next = lse2[(int64_t)row * a.Hq + head];
        if (!is) low_next = __builtin_huge_valf();
        end_next = cr.off + row + 1;
        low_head += by_head;
        low_row += by_row;
        if (low_head >= a.G) {
            low_head -= a.G;
            ++low_row;
        }
    };
    // piece c of row r at c ^ (r % 16)
    const auto store = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = first + i * (LOADERS / PIECES);
            *reinterpret_cast<u32x4*>(mine + buf * TILE + r * ROW +
                                      ((piece ^ (r & 15 & (PIECES - 1))) << 4)) = moved[i];
        }
    };
    // (a wave's own LDS writes and reads are in order)
    const auto meet = [] __attribute__((always_inline)) {
        if constexpr (APART) asm volatile("" ::: "memory");
        else __syncthreads();
    };
    load(r_first);
    load_low(r_first);
    // slots that some row sees: not past the last one's end, nor before the first one's window
    const int64_t from = a.window > 0 ? (int64_t)cr.off + 1 - a.window : 0;
    float* const weights = a.weight_sum + b * a.slot_b + h * a.slot_h + key0 + col;
    u32x4 kf[KG][NF];
    bool there[KG], added[KG];
    float old[KG];
#pragma unroll
    for (int g = 0; g < KG; ++g) {
        const int t = key0 + 32 * g + col;
        const int64_t o = t < cr.len ? slot_offset(a.pages, b, t) : -1;
        there[g] = o >= 0;
        added[g] = there[g] && t < cr.off + cr.live && t >= from;
        old[g] = added[g] ? weights[32 * g] : 0.f;
        const S* kr = static_cast<const S*>(a.k) + h * a.pages.head_stride + (o >= 0 ? o : 0);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int d = (2 * f + half) * VEC;
            kf[g][f] = u32x4{0, 0, 0, 0};
            if (there[g] && (EXACT || d < a.D)) kf[g][f] = *reinterpret_cast<const u32x4*>(kr + d);
        }
    }
    store(0);
    load(r_first + STEP);
    meet();
    int buf = 0;
    for (int r0 = r_first; r0 < r_end; r0 += STEP, buf ^= 1) {
        const float low = low_next;
        const int end = end_next, begin = a.window > 0 ? end - a.window : 0;
        load_low(r0 + STEP);
        const bool whole = __all(begin <= key0 && end >= key_end);
        f32x16 s[KG];
#pragma unroll
        for (int g = 0; g < KG; ++g)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[g][i] = 0.f;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const u32x4 qf = *reinterpret_cast<const u32x4*>(
                mine + buf * TILE + col * ROW + (((2 * f + half) ^ (col & 15 & (PIECES - 1))) << 4));
#pragma unroll
            for (int g = 0; g < KG; ++g) Mma32<TR>::step(s[g], kf[g][f], qf);
        }
        // (read last an iteration ago)
        store(buf ^ 1);
        load(r0 + 2 * STEP);
#pragma unroll
        for (int g = 0; g < KG; ++g)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[g][i] = exp2_fast(fmaf(s[g][i], c, -low));
        if (!whole) {
#pragma unroll
            for (int g = 0; g < KG; ++g)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    // a hidden slot gets nothing, whatever the row's sum is
                    const int t = key0 + 32 * g + 8 * (i >> 2) + 4 * half + (i & 3);
                    s[g][i] = t < end && t >= begin ? s[g][i] : 0.f;
                }
        }
#pragma unroll
        for (int g = 0; g < KG; ++g)
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[g][i] += s[g][i];
        meet();
    }
    __syncthreads();  // (the rows are no longer read)
    float* parts = reinterpret_cast<float*>(lds) + wave * KG * 32;
#pragma unroll
    for (int g = 0; g < KG; ++g) {
        // Each step adds up what two lanes hold of one half of the values and leaves
        // them a half each: lane col ends with value i.
        int i = 0;
#pragma unroll
        for (int n = 8; n > 0; n >>= 1) {
            const bool upper = col & (2 * n);
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const float give = upper ? sum[g][j] : sum[g][j + n];
                const float keep = upper ? sum[g][j + n] : sum[g][j];
                sum[g][j] = keep + __shfl_xor(give, 2 * n);
            }
            i += upper ? n : 0;
        }
        const float one = sum[g][0] + __shfl_xor(sum[g][0], 1);
        if ((col & 1) == 0) parts[32 * g + 8 * (i >> 2) + 4 * half + (i & 3)] = one;
    }
    __syncthreads();
    if ((APART && wave > 0) || half != 0) return;
#pragma unroll
    for (int g = 0; g < KG; ++g) {
        if (!added[g]) continue;
        float add = parts[32 * g + col];
        if (APART)
            for (int w = 1; w < kWaves; ++w) add += parts[w * KG * 32 + 32 * g + col];
        weights[32 * g] = old[g] + add;
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

template <class TR, int DP, bool APART>
hipError_t weights_a(const AttnArgs& a, int key_blocks, hipStream_t s) {
    const void* fn =
        a.D == DP ? reinterpret_cast<const void*>(&chunk_weights_kernel<TR, DP, true, APART>)
                  : reinterpret_cast<const void*>(&chunk_weights_kernel<TR, DP, false, APART>);
    const size_t lds = 2 * 32 * DP * sizeof(typename TR::storage) * (APART ? kWaves : 1);
    if (lds > 64u << 10) {
        const hipError_t e =
            hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    AttnArgs args = a;
    void* params[] = {&args, &key_blocks};
    return hipLaunchKernel(fn, grid_of((int64_t)a.B * a.Hkv * key_blocks), dim3(kThreads), params,
                           lds, s);
}

template <class TR, int DP>
hipError_t weights_d(const AttnArgs& a, hipStream_t s) {
    constexpr int NF = DP * (int)sizeof(typename TR::storage) / 32;
    constexpr int own = 32 * key_groups<true>(NF), together = kWaves * 32 * key_groups<false>(NF);
    const auto blocks = [&](int keys) { return (int)(((int64_t)a.pages.slots + keys - 1) / keys); };
    if (a.pages.slots == 0) return hipSuccess;
    // (fp32 rows of 1 KB: the tiles of four waves do not fit LDS)
    if constexpr (NF <= 16)
        if ((int64_t)a.B * a.Hkv * blocks(own) <= 512)
            return weights_a<TR, DP, true>(a, blocks(own), s);
    return weights_a<TR, DP, false>(a, blocks(together), s);
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
