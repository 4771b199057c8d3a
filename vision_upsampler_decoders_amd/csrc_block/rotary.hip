// Rotary positions, alone and on the way into the paged cache.
//
// A workgroup takes a few rows.  Their sines and cosines, one per row and pair
// for all heads, are computed once into LDS (the angle's turns are reduced in
// fp64: position 10^6 of frequency 1 is 1.6e5 turns, of which fp32 would keep
// 1/64), while the first pieces of the rows are already on their way from
// memory.  A thread turns whole pieces: 16 bytes of first values and the 16
// bytes that they go with, each read and written once by the same thread, so
// that a call may work in place.  Rotary parts whose half is not a multiple of
// 16 bytes are taken in pieces of 8, 4 or 2 (one value).
// Long calls are bound by memory: 32768 rows of 40 heads of 128, bf16 (671 MB): 125
// us, 5.3 TB/s, the rate of a large copy; 16397 rows into the cache, f16 (336 MB), 72
// us, 4.65.  Value by value (38 of 96 values, bf16) 2.8 and 2.1 TB/s; in fp32 4.8
// and 3.6.  A step of 48 rows takes 4.8 us, a chain of latencies.

#include "block_internal.h"
#include "mfma_common.h"

namespace ctconv {
namespace block {

namespace {

using mfma::u32x2;
using mfma::u32x4;

constexpr int kThreads = 256;
constexpr int kMostRows = 8;   // rows of a workgroup
constexpr int kMostPairs = 128;
constexpr int kAtOnce = 4;     // pairs of pieces of a thread that are in flight together

template <class S, int V>
struct Piece {
    static constexpr int BYTES = V * sizeof(S);
    using Word = std::conditional_t<
        BYTES == 16, u32x4,
        std::conditional_t<BYTES == 8, u32x2, std::conditional_t<BYTES == 4, uint32_t, uint16_t>>>;
    union {
        Word word;
        S value[V];
    };
    __device__ inline void load(const S* p) { word = *reinterpret_cast<const Word*>(p); }
    __device__ inline void store(S* p) const { *reinterpret_cast<Word*>(p) = word; }
};

// V: values of a piece.
template <class TR, int V, bool PAIRS, bool APPEND>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a) {
    using S = typename TR::storage;
    __shared__ __align__(16) float cs[kMostRows * 2 * kMostPairs];  // per row: cosines, sines
    __shared__ int64_t to_slot[kMostRows];                          // cache rows, or -1
    __shared__ int live[kMostRows];
    const int tid = threadIdx.x;
    const int64_t from_row = (int64_t)block_number() * a.per;
    if (from_row >= a.rows) return;
    const int row0 = (int)from_row;
    const int rows = a.rows - row0 < a.per ? a.rows - row0 : a.per;

    // Item: two pieces of a head of q, k or v of a row.
    struct Item {
        const S* from;
        int row, head, d0, d1;
        int kind;  // 0 q, 1 k, 2 v
        bool turned, first, second;
    };
    const int q_items = a.Hq * a.units, k_items = q_items + a.Hk * a.units;
    const int total = rows * a.items;
    const auto item_of = [&](int i) {
        Item it;
        it.first = i < total;
        if (!it.first) i = 0;
        it.row = (int)fdiv((uint32_t)i, a.fd_items);
        int at = i - it.row * a.items;
        it.kind = at < q_items ? 0 : !APPEND || at < k_items ? 1 : 2;
        at -= it.kind == 0 ? 0 : it.kind == 1 ? q_items : k_items;
        int u;
        if (APPEND && it.kind == 2) {
            it.head = (int)fdiv((uint32_t)at, a.fd_v_units);
            u = at - it.head * a.v_units;
        } else {
            it.head = (int)fdiv((uint32_t)at, a.fd_units);
            u = at - it.head * a.units;
        }
        it.turned = it.kind != 2;
        if (PAIRS || it.kind == 2) {
            it.d0 = 2 * u * V;
            it.d1 = it.d0 + V;
        } else if (u * V < a.half) {
            it.d0 = u * V;
            it.d1 = it.d0 + a.half;
        } else {
            it.turned = false;
            it.d0 = 2 * u * V;
            it.d1 = it.d0 + V;
        }
        it.second = it.first && it.d1 < a.D;
        const int64_t row = row0 + it.row;
        it.from = it.kind == 0 ? static_cast<const S*>(a.q) + row * a.q_row + it.head * a.q_head
                               : static_cast<const S*>(it.kind == 1 ? a.k : a.v) + row * a.k_row +
                                     it.head * a.k_head;
        return it;
    };
    Item it[kAtOnce];
    Piece<S, V> p0[kAtOnce], p1[kAtOnce];
    const auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            it[j] = item_of(i0 + j * kThreads + tid);
            if (it[j].first) p0[j].load(it[j].from + it[j].d0);
            if (it[j].second) p1[j].load(it[j].from + it[j].d1);
        }
    };
    load(0);

    for (int i = tid; i < rows * a.half; i += kThreads) {
        const int r = (int)fdiv((uint32_t)i, a.fd_half), j = i - r * a.half;
        double turns = (double)a.positions[row0 + r] * a.frequencies[j] * 0.15915494309189533577;
        turns -= rint(turns);
        float s, c;
        sincospif(2.f * (float)turns, &s, &c);
        cs[r * 2 * a.half + j] = c * a.scale;
        cs[r * 2 * a.half + a.half + j] = s * a.scale;
    }
    if (tid < rows) {
        live[tid] = a.positions[row0 + tid] >= 0;
        if constexpr (APPEND) {
            const int slot = a.slots[row0 + tid];
            int64_t to = -1;
            if (live[tid] && slot >= 0 && slot < a.num_slots) {
                const int page = (int)fdiv((uint32_t)slot, a.fd_page);
                to = page * a.page_stride + (slot - page * a.page_size) * a.slot_stride;
            }
            to_slot[tid] = to;
        }
    }
    __syncthreads();

    for (int i0 = 0; i0 < total; i0 += kAtOnce * kThreads) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (!it[j].first) continue;
            const int r = it[j].row;
            if (it[j].turned) {
                const float* c = cs + r * 2 * a.half;
                const float* s = c + a.half;
                if constexpr (PAIRS) {
#pragma unroll
                    for (int n = 0; n < V / 2; ++n) {
                        const auto turn = [&](Piece<S, V>& p, int pair) {
                            if (pair >= a.half) return;
                            const float u = TR::to_f32(p.value[2 * n]);
                            const float v = TR::to_f32(p.value[2 * n + 1]);
                            p.value[2 * n] = TR::from_f32(u * c[pair] - v * s[pair]);
                            p.value[2 * n + 1] = TR::from_f32(v * c[pair] + u * s[pair]);
                        };
                        turn(p0[j], it[j].d0 / 2 + n);
                        if (it[j].second) turn(p1[j], it[j].d1 / 2 + n);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < V; ++n) {
                        const float u = TR::to_f32(p0[j].value[n]), v = TR::to_f32(p1[j].value[n]);
                        const float cn = c[it[j].d0 + n], sn = s[it[j].d0 + n];
                        p0[j].value[n] = TR::from_f32(u * cn - v * sn);
                        p1[j].value[n] = TR::from_f32(v * cn + u * sn);
                    }
                }
            }
            const int64_t row = row0 + r;
            S* to;
            bool write = live[r];
            if (it[j].kind == 0) {
                to = static_cast<S*>(a.q_out) + row * a.q_out_row + it[j].head * a.q_out_head;
            } else if constexpr (APPEND) {
                const int64_t at = to_slot[r];
                write = at >= 0;
                to = static_cast<S*>(it[j].kind == 1 ? a.k_out : a.v_out) + at +
                     it[j].head * a.k_out_head;
            } else {
                to = static_cast<S*>(a.k_out) + row * a.k_out_row + it[j].head * a.k_out_head;
            }
            if (!write) continue;
            p0[j].store(to + it[j].d0);
            if (it[j].second) p1[j].store(to + it[j].d1);
        }
    }
}

template <class TR, int V, bool PAIRS>
hipError_t rotary_v(RotaryArgs a, bool append, hipStream_t s) {
    const int rotated = PAIRS ? 0 : a.half / V;
    const int rest = PAIRS ? a.D : a.D - 2 * a.half;
    a.units = rotated + (rest + 2 * V - 1) / (2 * V);
    a.v_units = append ? (a.D + 2 * V - 1) / (2 * V) : 1;
    a.items = (a.Hq + a.Hk) * a.units + (append ? a.Hk * a.v_units : 0);
    a.fd_units = make_fastdiv((uint32_t)a.units);
    a.fd_v_units = make_fastdiv((uint32_t)a.v_units);
    a.fd_items = make_fastdiv((uint32_t)a.items);
    a.fd_half = make_fastdiv((uint32_t)a.half);
    // one round of every thread's pieces per workgroup, if the rows still
    // spread over the chip (40 heads of 64 channels, bf16, one row a workgroup |
    // two: 512 rows 7.0 | 7.3 us, 2048 8.4 | 7.2, 32768 92 | 66)
    int per = kAtOnce * kThreads / a.items;
    per = per < 1 ? 1 : per > kMostRows ? kMostRows : per;
    while (per > 1 && a.rows / per < 1024) per >>= 1;
    a.per = per;
    const dim3 grid = grid_of(((int64_t)a.rows + per - 1) / per);
    if (append)
        rotary_kernel<TR, V, PAIRS, true><<<grid, dim3(kThreads), 0, s>>>(a);
    else
        rotary_kernel<TR, V, PAIRS, false><<<grid, dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
}

template <class TR>
hipError_t rotary_t(const RotaryArgs& a, bool pairs, bool append, hipStream_t s) {
    constexpr int VEC = TR::kVec;
    if (pairs) return rotary_v<TR, VEC, true>(a, append, s);
    if (a.half % VEC == 0) return rotary_v<TR, VEC, false>(a, append, s);
    if constexpr (VEC == 8)
        if (a.half % 4 == 0) return rotary_v<TR, 4, false>(a, append, s);
    if (a.half % 2 == 0) return rotary_v<TR, 2, false>(a, append, s);
    return rotary_v<TR, 1, false>(a, append, s);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, ctconv_dtype dt, bool pairs, bool append,
                         hipStream_t s) {
    switch (dt) {
        case CTCONV_F32: return rotary_t<TF32>(a, pairs, append, s);
        case CTCONV_BF16: return rotary_t<TBF16>(a, pairs, append, s);
        case CTCONV_F16: return rotary_t<TF16>(a, pairs, append, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace block
}  // namespace ctconv
