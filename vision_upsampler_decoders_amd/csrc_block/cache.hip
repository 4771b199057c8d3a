// The paged cache's writers: append (rows in) and evict (rows out, by the
// attention weight they have drawn).

#include "block_internal.h"

namespace ctconv {
namespace block {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Append.  Pure copying: 16 bytes of K and of V per lane and step, four steps
// in flight.  A workgroup copies a run of new rows of one sequence.
// ---------------------------------------------------------------------------
template <class S>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
    constexpr int VEC = 16 / sizeof(S);
    constexpr int UNROLL = 4;
    const int b = (int)fdiv(blockIdx.x, a.fd_groups);
    const int first = (int)(blockIdx.x - (uint32_t)b * a.groups) * a.rows_per_group;
    const int len = a.lengths[b] < 0 ? 0 : a.lengths[b];
    int cnt = clamped(a.counts ? a.counts[b] : a.n, a.n);
    cnt = cnt < len ? cnt : len;
    int rows = cnt - first;
    if (rows <= 0) return;
    rows = rows < a.rows_per_group ? rows : a.rows_per_group;
    const int total = rows * a.Hkv * a.chunks;
    const int seen = a.now ? a.now[b] : a.lengths[b];
    const S* kn = static_cast<const S*>(a.k_new) + b * a.new_b;
    const S* vn = static_cast<const S*>(a.v_new) + b * a.new_b;
    S* kc = static_cast<S*>(a.k);
    S* vc = static_cast<S*>(a.v);
    for (int i0 = threadIdx.x; i0 < total; i0 += 256 * UNROLL) {
        u32x4 rk[UNROLL], rv[UNROLL];
        int64_t to[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            to[u] = -1;
            const int idx = i0 + u * 256;
            if (idx >= total) continue;
            const int row = (int)fdiv((uint32_t)idx, a.fd_chunks);
            const int c = idx - row * a.chunks;
            const int i = (int)fdiv((uint32_t)row, a.fd_heads);
            const int h = row - i * a.Hkv;
            const int t = len - cnt + first + i;  // the new row's slot
            if (t >= a.pages.slots) continue;
            const int64_t at = slot_offset(a.pages, b, t);
            if (c == 0) {
                const int64_t m = b * a.slot_b + h * a.slot_h + t;
                if (a.positions) a.positions[m] = seen - cnt + first + i;
                if (a.weight_sum) a.weight_sum[m] = 0.f;
            }
            if (at < 0) continue;
            to[u] = at + h * a.pages.head_stride + c * VEC;
            const int64_t from = (int64_t)(first + i) * a.new_row + h * a.new_head + c * VEC;
            rk[u] = *reinterpret_cast<const u32x4*>(kn + from);
            rv[u] = *reinterpret_cast<const u32x4*>(vn + from);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (to[u] < 0) continue;
            *reinterpret_cast<u32x4*>(kc + to[u]) = rk[u];
            *reinterpret_cast<u32x4*>(vc + to[u]) = rv[u];
        }
    }
}

// ---------------------------------------------------------------------------
// Evict, first kernel: which slots stay.  One workgroup per sequence and
// head.  A slot's rank is a 32-bit key that orders like (protected, weight);
// the m-th largest key is found digit by digit from the top (8 bits a pass,
// counted in LDS with one private column per lane so that equal digits do
// not collide), then one bit per slot says who stays, and prefix sums over
// the 64-slot words pair the holes below m with the kept slots from m on.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kDigits = 256, kColumns = 32;

__device__ inline uint32_t rank_key(float w, bool safe) {
    if (safe) return 0xFFFFFFFFu;
    // NaN below everything; above the largest finite number as that
    w = w != w ? -__builtin_huge_valf() : fminf(w, 3.402823466e38f);
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);  // -0 ranks like 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Exclusive prefix sums of v[0, n) in place; the total is returned to every
// thread.  All kSelThreads threads call it.
__device__ inline int scan_words(int* v, int n, int* wave_sums) {
    const int per = (n + kSelThreads - 1) / kSelThreads;
    const int lo = threadIdx.x * per, hi = lo + per < n ? lo + per : n;
    int sum = 0;
    for (int i = lo; i < hi; ++i) sum += v[i];
    int inc = sum;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 63) wave_sums[wave] = inc;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kSelWaves; ++w) {
        if (w < wave) base += wave_sums[w];
        total += wave_sums[w];
    }
    int run = base + inc - sum;
    for (int i = lo; i < hi; ++i) {
        const int t = v[i];
        v[i] = run;
        run += t;
    }
    __syncthreads();
    return total;
}

// Index of the n-th (from 0) set bit of w.
__device__ inline int nth_bit(uint64_t w, int n) {
    int at = 0;
#pragma unroll
    for (int half = 32; half > 0; half >>= 1) {
        const int c = __popcll(w & ((1ull << half) - 1));
        if (n >= c) {
            n -= c;
            at += half;
            w >>= half;
        }
    }
    return at;
}

// KEYS > 0: the keys of up to KEYS * kSelThreads slots stay in registers;
// KEYS = 0: computed again from memory for each pass.
template <int KEYS>
__global__ __launch_bounds__(kSelThreads) void select_kernel(EvictArgs a) {
    extern __shared__ __align__(16) uint32_t lds[];
    __shared__ int wave_sums[kSelWaves], found[4];
    uint32_t* hist = lds;                                // kDigits x kColumns, first
    uint64_t* bits = reinterpret_cast<uint64_t*>(lds);   // then a.words, and
    int* pre = reinterpret_cast<int*>(bits + a.words);   // a.words prefix sums
    const int bh = blockIdx.x, b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = clamped(a.lengths[b], a.pages.slots);
    const int m = n < a.keep ? n : a.keep;
    const float* weight = a.weight_sum + b * a.slot_b + h * a.slot_h;
    const int32_t* position = a.positions ? a.positions + b * a.slot_b + h * a.slot_h : nullptr;
    const int64_t seen = a.now ? a.now[b] : a.lengths[b];
    int32_t* source = a.source + (int64_t)bh * a.keep;
    float* weight_out = a.weight_out + b * a.out_b + h * a.out_h;
    int32_t* position_out = a.positions_out ? a.positions_out + b * a.out_b + h * a.out_h : nullptr;
    const bool all = n == m;

    const auto key_of = [&](int t) {
        const int64_t pos = position ? position[t] : t;
        return rank_key(weight[t], pos < a.sink || pos >= seen - a.recent);
    };
    uint32_t keys[KEYS > 0 ? KEYS : 1];
    const int rounds = (n + kSelThreads - 1) / kSelThreads;
    if (!all) {
        if constexpr (KEYS > 0) {
#pragma unroll
            for (int i = 0; i < KEYS; ++i) {
                const int t = i * kSelThreads + tid;
                keys[i] = t < n ? key_of(t) : 0;
            }
        }
        // f(slot, key, i) for every slot of this thread, whole waves at a time
        const auto each = [&](auto f) {
            if constexpr (KEYS > 0) {
#pragma unroll
                for (int i = 0; i < KEYS; ++i)
                    if (i < rounds) f(i * kSelThreads + tid, keys[i]);
            } else {
                for (int i = 0; i < rounds; ++i) {
                    const int t = i * kSelThreads + tid;
                    f(t, t < n ? key_of(t) : 0u);
                }
            }
        };
        // the m-th largest key
        uint32_t prefix = 0, mask = 0;
        int want = m;
        bool exact = false;  // every key with this prefix stays
        for (int shift = 24; shift >= 0 && !exact; shift -= 8) {
            for (int i = tid; i < kDigits * kColumns; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            each([&](int t, uint32_t key) {
                if (t < n && (key & mask) == prefix)
                    atomicAdd(&hist[((key >> shift) & 255) * kColumns + (tid & (kColumns - 1))], 1u);
            });
            __syncthreads();
            // four threads add up a digit's columns
            int c = 0;
            for (int i = 0; i < kColumns / 4; ++i)
                c += hist[(tid >> 2) * kColumns + (((tid & 3) + 4 * (i + (tid >> 2))) & (kColumns - 1))];
            c += __shfl_xor(c, 1);
            c += __shfl_xor(c, 2);
            __syncthreads();
            if ((tid & 3) == 0) hist[tid >> 2] = c;
            __syncthreads();
            if (wave == 0) {
                // lane l: digits 255 - 4l .. 252 - 4l, from the top
                int d[4], sum = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d[i] = hist[255 - 4 * lane - i];
                    sum += d[i];
                }
                int inc = sum;
#pragma unroll
                for (int o = 1; o < 64; o <<= 1) {
                    const int t = __shfl_up(inc, o);
                    if (lane >= o) inc += t;
                }
                int above = inc - sum;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (above < want && above + d[i] >= want) {
                        found[0] = 255 - 4 * lane - i;
                        found[1] = want - above;  // still wanted among this digit
                        found[2] = d[i];
                    }
                    above += d[i];
                }
            }
            __syncthreads();
            prefix |= (uint32_t)found[0] << shift;
            mask |= 255u << shift;
            want = found[1];
            exact = found[1] == found[2];
            __syncthreads();
        }
        // keys from `prefix` on stay; where not `exact`, only the first
        // `want` of those equal to it
        each([&](int t, uint32_t key) {
            const uint64_t w = __ballot(t < n && key >= prefix);
            if (lane == 0) bits[t >> 6] = w;
            if (!exact) {
                const uint64_t e = __ballot(t < n && key == prefix);
                if (lane == 0) pre[t >> 6] = __popcll(e);
            }
        });
        __syncthreads();
        const int words = (n + 63) >> 6;
        if (!exact) {
            scan_words(pre, words, wave_sums);
            each([&](int t, uint32_t key) {
                const bool level = t < n && key == prefix;
                const uint64_t e = __ballot(level);
                const int before = __popcll(e & ((1ull << lane) - 1));
                const uint64_t gone = __ballot(level && (t >> 6) < words &&
                                               pre[(t >> 6) < words ? t >> 6 : 0] + before >= want);
                if (lane == 0 && (t >> 6) < words) bits[t >> 6] &= ~gone;
            });
            __syncthreads();
        }
        // holes per word below m, kept slots per word from m on
        const int edge = m >> 6;
        const uint64_t below = (1ull << (m & 63)) - 1;
        for (int w = tid; w < words; w += kSelThreads)
            pre[w] = w < edge ? __popcll(~bits[w])
                              : __popcll(w == edge ? bits[w] & ~below : bits[w]);
        __syncthreads();
        scan_words(pre, words, wave_sums);
    }
    const int words = (n + 63) >> 6, edge = m >> 6;
    for (int j = tid; j < a.keep; j += kSelThreads) {
        int src = -1;
        if (j < m) {
            src = j;
            if (!all && !((bits[j >> 6] >> (j & 63)) & 1)) {
                const int r = pre[j >> 6] + __popcll(~bits[j >> 6] & ((1ull << (j & 63)) - 1));
                // the last word from `edge` on whose kept slots start at or before rank r
                const int base = pre[edge];
                int lo = edge, hi = words - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (pre[mid] - base <= r) lo = mid;
                    else hi = mid - 1;
                }
                uint64_t w = bits[lo];
                if (lo == edge) w &= ~((1ull << (m & 63)) - 1);
                src = lo * 64 + nth_bit(w, r - (pre[lo] - base));
            }
        }
        source[j] = src;
        const float wt = src >= 0 ? weight[src] : 0.f;
        const int pos = src < 0 ? -1 : position ? position[src] : src;
        weight_out[j] = wt;
        if (position_out) position_out[j] = pos;
    }
}

// Second kernel: the rows of the filled holes.  Sources are kept slots from m
// on and targets lie below m, so no copy reads what another one writes.
constexpr int kMoveSlots = 64;

template <class S>
__global__ __launch_bounds__(256) void move_kernel(EvictArgs a) {
    constexpr int VEC = 16 / sizeof(S);
    const int tiles = (a.keep + kMoveSlots - 1) / kMoveSlots;
    const int bh = blockIdx.x / tiles, first = (int)(blockIdx.x - (uint32_t)bh * tiles) * kMoveSlots;
    const int b = bh / a.Hkv, h = bh - b * a.Hkv;
    if (a.lengths_out && h == 0 && first == 0 && threadIdx.x == 0) {
        // the one place that reads lengths here: lengths_out may be lengths
        const int n = clamped(a.lengths[b], a.pages.slots);
        a.lengths_out[b] = n < a.keep ? n : a.keep;
    }
    const int32_t* source = a.source + (int64_t)bh * a.keep;
    const int slots = a.keep - first < kMoveSlots ? a.keep - first : kMoveSlots;
    S* k = static_cast<S*>(a.k) + h * a.pages.head_stride;
    S* v = static_cast<S*>(a.v) + h * a.pages.head_stride;
    for (int i = threadIdx.x; i < slots * a.chunks; i += 256) {
        const int row = (int)fdiv((uint32_t)i, a.fd_chunks);
        const int c = i - row * a.chunks;
        const int to = first + row, from = source[to];
        if (from < 0 || from == to) continue;
        const int64_t o1 = slot_offset(a.pages, b, to), o0 = slot_offset(a.pages, b, from);
        if (o0 < 0 || o1 < 0) continue;
        const u32x4 rk = *reinterpret_cast<const u32x4*>(k + o0 + c * VEC);
        const u32x4 rv = *reinterpret_cast<const u32x4*>(v + o0 + c * VEC);
        *reinterpret_cast<u32x4*>(k + o1 + c * VEC) = rk;
        *reinterpret_cast<u32x4*>(v + o1 + c * VEC) = rv;
    }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, ctconv_dtype dt, hipStream_t s) {
    const dim3 grid((unsigned)(a.B * a.groups));
    if (dt == CTCONV_F32)
        append_kernel<float><<<grid, dim3(256), 0, s>>>(a);
    else
        append_kernel<uint16_t><<<grid, dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_evict(const EvictArgs& a, ctconv_dtype dt, hipStream_t s) {
    const dim3 grid((unsigned)(a.B * a.Hkv));
    size_t lds = (size_t)a.words * 12;
    if (lds < kDigits * kColumns * 4) lds = kDigits * kColumns * 4;
    const int slots = a.words * 64;
    const void* fn = slots <= 8 * kSelThreads    ? reinterpret_cast<const void*>(&select_kernel<8>)
                     : slots <= 40 * kSelThreads ? reinterpret_cast<const void*>(&select_kernel<40>)
                                                 : reinterpret_cast<const void*>(&select_kernel<0>);
    if (lds > 64u << 10) {
        const hipError_t e =
            hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    EvictArgs args = a;
    void* params[] = {&args};
    hipError_t e = hipLaunchKernel(fn, grid, dim3(kSelThreads), params, lds, s);
    if (e != hipSuccess) return e;
    const int64_t tiles = ((int64_t)a.keep + kMoveSlots - 1) / kMoveSlots;
    const dim3 mgrid((unsigned)(a.B * a.Hkv * tiles));
    if (dt == CTCONV_F32)
        move_kernel<float><<<mgrid, dim3(256), 0, s>>>(a);
    else
        move_kernel<uint16_t><<<mgrid, dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace block
}  // namespace ctconv
