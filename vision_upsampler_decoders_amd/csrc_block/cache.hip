// The paged cache's writers: append (rows in) and evict (rows out, by the
// attention weight they have drawn).

#include "block_internal.h"

namespace ctconv {
namespace block {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// N slots' values at once; slot arrays are only aligned to one value
template <int N>
struct Slots {
    typedef float weights __attribute__((ext_vector_type(N), aligned(4)));
    typedef int numbers __attribute__((ext_vector_type(N), aligned(4)));
};

// ---------------------------------------------------------------------------
// Append.  Pure copying: 16 bytes of K and of V per lane and step, four steps
// in flight.  A workgroup copies a run of new rows of one sequence.  Bound by
// memory: 8 ragged prompts of up to 4099 rows (152 MB) take 30.5 us, 5 TB/s.
// More rows than the L2 caches hold together are written past them (35.8 us
// otherwise); a step's rows stay there for the attention that follows.
// ---------------------------------------------------------------------------
template <class S, bool STREAM>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
    constexpr int VEC = 16 / sizeof(S);
    constexpr int UNROLL = 4;
    const uint32_t item = block_number();
    if (item >= (uint32_t)(a.B * a.groups)) return;
    const int b = (int)fdiv(item, a.fd_groups);
    const int first = (int)(item - (uint32_t)b * a.groups) * a.rows_per_group;
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
            u32x4* const tk = reinterpret_cast<u32x4*>(kc + to[u]);
            u32x4* const tv = reinterpret_cast<u32x4*>(vc + to[u]);
            if constexpr (STREAM) {
                __builtin_nontemporal_store(rk[u], tk);
                __builtin_nontemporal_store(rv[u], tv);
            } else {
                *tk = rk[u];
                *tv = rv[u];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Evict, first kernel: which slots stay.  One workgroup per sequence and
// head.  A slot's rank is a 32-bit key that orders like (protected, weight);
// the m-th largest key is found digit by digit from the top (8 bits a pass,
// counted in LDS in 4 columns: lanes with equal digits then meet less, and more
// columns cost more to clear and to add than they save: with 32, 320 slots
// take 9.3 us instead of 8.3), then one bit per slot says who stays, and
// prefix sums over the 64-slot words pair the holes below m with the kept
// slots from m on.
// A slot without a page has no row that could move: below m it stays where it
// is, ranked above every other, so that it is neither a hole nor a source; from
// m on it is given up, ranked below every other (n - m slots lie there, so
// enough with a page remain).  Only sequences that have such a slot look up the
// page of each.
// Two passes over the slots as a rule: the first digit, then the keys that
// share it and the next are gathered in LDS.  Everything is counted in
// integers, so no order of the atomics changes a result.
// 64 heads of up to 40001 slots: 29 us, bound by one compute unit's vector
// instructions per head; then 36 us for the rows (below).  A few hundred slots
// are one kernel, select and fill together.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kDigits = 256, kColumns = 4;
constexpr int kBatch = 2;                    // rounds in flight
// Keys gathered in LDS (512 and 8192: no difference in any case measured).
constexpr int kNear = 2048;

// LDS words for the digits' counts, then for the ties' bit map.
__host__ __device__ inline int count_words(int map_words) {
    return 2 * map_words > kDigits * kColumns ? 2 * map_words : kDigits * kColumns;
}

// Orders like the weight: NaN like minus infinity, infinity like the largest
// finite number, -0 like 0.  No weight's key is as small as those of slots past
// the end (0) and of given up ones without a page, or as large as those of
// protected slots and of ones without a page that stay.
constexpr uint32_t kNoPageGone = 1u, kProtected = 0xFFFFFFFEu, kNoPageStays = 0xFFFFFFFFu;
__device__ inline uint32_t rank_key(float w) {
    w = fminf(fmaxf(w + 0.f, -__builtin_huge_valf()), 3.402823466e38f);
    const uint32_t u = __float_as_uint(w);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Bits t .. t + N - 1 of a bit map from N slots of each lane (t = N times the
// lane, from a multiple of 64 N).
template <int N>
__device__ inline void put_bits(uint64_t* map, int t, uint32_t mine) {
    if constexpr (N == 1) {
        const uint64_t w = __ballot(mine);
        if ((threadIdx.x & 63) == 0) map[t >> 6] = w;
    } else {
        // two lanes' bits make a byte
        const uint32_t next = __builtin_amdgcn_mov_dpp((int)mine, 0xF5, 0xF, 0xF, true);
        if (!(threadIdx.x & 1))
            reinterpret_cast<uint8_t*>(map)[t >> 3] = (uint8_t)(mine | next << 4);
    }
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

// What slots j (one per lane of a wave) become, once it is known that they
// take `src` (-1: empty): weight and position, and the rows of the holes.
// Sources are kept slots from m on and targets lie below m, so no copy reads
// what another one writes, in place or not.
struct MovedRow {
    int64_t from, to;
};

template <class S, int U>
__device__ inline void fill_slots(const EvictArgs& a, int b, int h, const int (&j)[U],
                                  const int (&src)[U], MovedRow* rows) {
    constexpr int VEC = 16 / sizeof(S);
    const int lane = threadIdx.x & 63;
    const int64_t in = b * a.slot_b + h * a.slot_h, out = b * a.out_b + h * a.out_h;
    float wt[U];
    int pos[U];
    int64_t from[U], to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = src[u] < 0 ? 0 : src[u];
        wt[u] = a.weight_sum[in + i];
        pos[u] = a.positions ? a.positions[in + i] : i;
        const bool hole = src[u] >= 0 && src[u] != j[u];
        from[u] = to[u] = -1;
        if (hole) {
            from[u] = slot_offset(a.pages, b, src[u]);
            to[u] = slot_offset(a.pages, b, j[u]);
        }
    }
    int count = 0;  // rows to move, listed in LDS
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (j[u] < a.keep) {
            a.weight_out[out + j[u]] = src[u] < 0 ? 0.f : wt[u];
            if (a.positions_out) a.positions_out[out + j[u]] = src[u] < 0 ? -1 : pos[u];
        }
        const bool moves = from[u] >= 0 && to[u] >= 0;
        const uint64_t mask = __ballot(moves);
        if (moves)
            rows[count + __popcll(mask & ((1ull << lane) - 1))] = MovedRow{from[u], to[u]};
        count += __popcll(mask);
    }
    if (count == 0) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // one wave's LDS, in order
    const int at_once = 64 / a.chunks;
    const int mine = (int)fdiv((uint32_t)lane, a.fd_chunks), c = lane - mine * a.chunks;
    S* k = static_cast<S*>(a.k) + h * a.pages.head_stride + c * VEC;
    S* v = static_cast<S*>(a.v) + h * a.pages.head_stride + c * VEC;
    if (mine < at_once) {
        constexpr int UNROLL = 4;
        for (int r0 = mine; r0 < count; r0 += UNROLL * at_once) {
            u32x4 rk[UNROLL], rv[UNROLL];
            int64_t dst[UNROLL];
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                const int r = r0 + i * at_once;
                const MovedRow row = rows[r < count ? r : r0];
                dst[i] = row.to;
                rk[i] = *reinterpret_cast<const u32x4*>(k + row.from);
                rv[i] = *reinterpret_cast<const u32x4*>(v + row.from);
            }
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                if (r0 + i * at_once >= count) continue;
                *reinterpret_cast<u32x4*>(k + dst[i]) = rk[i];
                *reinterpret_cast<u32x4*>(v + dst[i]) = rv[i];
            }
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// N slots per thread and round.  N = 1: one round, the keys stay in registers.
// N = 4: more than kSelThreads slots; the keys are computed again from memory
// for each pass, in a loop.  (All 40 keys of 40001 slots in registers took
// 37 us: every pass is then straight-line code that runs once, at the rate at
// which instructions are fetched.  One slot per thread and round took 39 us,
// four 29: with no conversion behind a branch and one address for four, a pass
// costs half the instructions, which bound it; more loads in flight change
// nothing.  320 slots: N = 1 takes
// 0.6 us of 9 less than N = 4.)
template <class S, int N>
__global__ __launch_bounds__(kSelThreads) void select_kernel(EvictArgs a) {
    extern __shared__ __align__(16) uint32_t lds[];
    __shared__ int wave_sums[kSelWaves], found[4];
    uint64_t* bits = reinterpret_cast<uint64_t*>(lds);   // a.words: who stays
    int* pre = reinterpret_cast<int*>(bits + a.words);   // a.words prefix sums
    uint32_t* work = reinterpret_cast<uint32_t*>(pre + a.words);
    uint32_t* hist = work;                               // kDigits x kColumns
    uint32_t* near = work + count_words(a.words);        // kNear keys and slots
    int* near_slot = reinterpret_cast<int*>(near + kNear);
    uint64_t* ties = reinterpret_cast<uint64_t*>(work);  // later: a.words
    int* spare = reinterpret_cast<int*>(work);           // last: a.list kept slots from m on
    if (block_number() >= (uint32_t)(a.B * a.Hkv)) return;
    const int bh = (int)block_number(), b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t* table = a.pages.table + b * a.pages.table_stride;
    const auto pages_of = [&](int slots) {
        return (int)fdiv((uint32_t)slots + (uint32_t)a.pages.page_size - 1, a.pages.fd_page);
    };
    // (asked for before the length has arrived)
    const int32_t page0 = tid < pages_of(a.pages.slots) ? table[tid] : 0;
    const int n = clamped(a.lengths[b], a.pages.slots);
    const int m = n < a.keep ? n : a.keep;
    const float* weight = a.weight_sum + b * a.slot_b + h * a.slot_h;
    const int32_t* position = a.positions ? a.positions + b * a.slot_b + h * a.slot_h : nullptr;
    const int64_t seen = a.now ? a.now[b] : a.lengths[b];
    int32_t* source = a.source + (int64_t)bh * a.keep;
    const bool all = n == m;
    int moves = 0;

    if (!all) {
        // protected: positions outside [sink, sink + open), one comparison
        const int64_t edge_pos = seen - a.recent;
        const uint32_t open = edge_pos > a.sink ? (uint32_t)(edge_pos - a.sink) : 0u;
        // Keys of slots t .. t + N - 1; 0 for those past n.  The last N slots
        // stand in for what would reach past them, then are shifted in place.
        // No load is behind a branch.
        typedef typename Slots<N>::weights Weights;
        typedef typename Slots<N>::numbers Numbers;
        const int last = n > N ? n - N : 0;
        // Does a slot lie in no page?  The waves' answers meet behind the barrier
        // that the cleared counts need.
        const auto missing = [&](int32_t page) {
            return (uint32_t)page >= (uint32_t)a.pages.num_pages;
        };
        const int pages = pages_of(n);
        bool gap = tid < pages && missing(page0);
#pragma unroll 8
        for (int i = tid + kSelThreads; i < pages; i += kSelThreads) gap |= missing(table[i]);
        gap = __any(gap);
        if (lane == 0) wave_sums[wave] = gap;
        const auto clear = [&]() {
            for (int i = tid; i < kDigits * kColumns; i += kSelThreads) hist[i] = 0;
            __syncthreads();
        };
        clear();
        gap = __any(wave_sums[lane % kSelWaves] != 0);
        const bool gaps = __builtin_amdgcn_readfirstlane(gap);
        const int32_t* position_or = position ? position : reinterpret_cast<const int32_t*>(weight);
        const auto load = [&](int t, Weights& w, Numbers& pos) {
            const int at = t < last ? t : last;
            w = *reinterpret_cast<const Weights*>(weight + at);
            pos = *reinterpret_cast<const Numbers*>(position_or + at);
        };
        const auto keys_of = [&](int t, const Weights& w, const Numbers& pos,
                                 uint32_t (&key)[N]) {
            const int at = t < last ? t : last;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const uint32_t k = rank_key(w[e]);
                const int q = position ? pos[e] : at + e;
                key[e] = (uint32_t)q - (uint32_t)a.sink < open ? k : kProtected;
            }
            if (gaps) {
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (missing(table[fdiv((uint32_t)(at + e), a.pages.fd_page)]))
                        key[e] = at + e < m ? kNoPageStays : kNoPageGone;
            }
            if (!__any(t + N > n)) return;
            const int shift = t - at;
            if constexpr (N == 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) key[e] = shift & 1 ? (e < 3 ? key[e + 1] : 0u) : key[e];
#pragma unroll
                for (int e = 0; e < 4; ++e) key[e] = shift & 2 ? (e < 2 ? key[e + 2] : 0u) : key[e];
            }
#pragma unroll
            for (int e = 0; e < N; ++e) key[e] = t + e < n ? key[e] : 0u;
        };
        uint32_t held[N];
        if constexpr (N == 1) {
            Weights w;
            Numbers pos;
            load(tid, w, pos);
            keys_of(tid, w, pos, held);
        }
        // f(t, keys of slots t .. t + N - 1), whole waves at a time
        const auto each = [&](auto f) {
            const int from = N * 64 * wave;
            if constexpr (N == 1) {
                if (from < n) f(tid, held);
            } else {
                constexpr int kRound = N * kSelThreads;
                for (int t0 = 0; t0 + from < n; t0 += kBatch * kRound) {
                    Weights w[kBatch];
                    Numbers pos[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) load(t0 + i * kRound + N * tid, w[i], pos[i]);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int t = t0 + i * kRound;
                        if (t + from >= n) break;
                        uint32_t key[N];
                        keys_of(t + N * tid, w[i], pos[i], key);
                        f(t + N * tid, key);
                    }
                }
            }
        };
        // The m-th largest key.  Once few enough keys share its digits, those
        // are gathered in LDS with their slots and only they are looked at;
        // the larger ones are marked as staying in the same pass.
        uint32_t prefix = 0, mask = 0;
        int want = m;
        bool exact = false;  // every key with this prefix stays
        int near_n = -1;
        if (tid == 0) found[3] = 0;
        for (int shift = 24; shift >= 0 && !exact; shift -= 8) {
            if (shift < 24) clear();
            uint32_t* column = hist + (tid & (kColumns - 1));
            const auto count = [&](uint32_t key) {
                atomicAdd(&column[__builtin_amdgcn_ubfe(key, shift, 8) * kColumns], 1u);
            };
            if (near_n >= 0) {
                for (int i = tid; i < near_n; i += kSelThreads)
                    if ((near[i] & mask) == prefix) count(near[i]);
            } else {
                // (slots past n count as key 0, below every other)
                each([&](int, const uint32_t (&key)[N]) {
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if ((key[e] & mask) == prefix) count(key[e]);
                });
            }
            __syncthreads();
            if (wave == 0) {
                // lane l: digits 255 - 4l .. 252 - 4l, from the top
                int d[4], sum = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x4 c = reinterpret_cast<const u32x4*>(hist)[255 - 4 * lane - i];
                    d[i] = (int)(c[0] + c[1] + c[2] + c[3]);
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
            if (near_n < 0 && !exact && found[2] <= kNear) {
                near_n = found[2];
                each([&](int t, const uint32_t (&key)[N]) {
                    uint32_t above = 0;
                    uint64_t equal[N];
                    int count = 0, at = 0;
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        above |= (key[e] & mask) > prefix ? 1u << e : 0u;
                        equal[e] = __ballot((key[e] & mask) == prefix);
                        count += __popcll(equal[e]);
                    }
                    put_bits<N>(bits, t, above);
                    if (count == 0) return;
                    // in any order: what follows does not depend on it
                    if (lane == 0) at = atomicAdd(&found[3], count);
                    at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        if ((equal[e] >> lane) & 1) {
                            const int i = at + __popcll(equal[e] & ((1ull << lane) - 1));
                            near[i] = key[e];
                            near_slot[i] = t + e;
                        }
                        at += __popcll(equal[e]);
                    }
                });
            }
            __syncthreads();
        }
        const int words = (n + 63) >> 6;
        // Keys from `prefix` on stay; where not `exact`, only the first `want`
        // of those equal to it, by their rank among the slots of `ties`.
        if (!exact)
            for (int w = tid; w < words; w += kSelThreads) ties[w] = 0;
        __syncthreads();
        const auto mark = [&](uint64_t* to, int t) {
            atomicOr(reinterpret_cast<unsigned long long*>(&to[t >> 6]), 1ull << (t & 63));
        };
        if (near_n >= 0) {
            for (int i = tid; i < near_n; i += kSelThreads) {
                const uint32_t key = near[i];
                if (key > prefix || (exact && key == prefix)) mark(bits, near_slot[i]);
                else if (key == prefix) mark(ties, near_slot[i]);
            }
        } else {
            each([&](int t, const uint32_t (&key)[N]) {
                uint32_t stay = 0, tie = 0;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    stay |= (exact ? key[e] >= prefix : key[e] > prefix) ? 1u << e : 0u;
                    tie |= key[e] == prefix ? 1u << e : 0u;
                }
                put_bits<N>(bits, t, stay);
                if (!exact) put_bits<N>(ties, t, tie);
            });
        }
        __syncthreads();
        if (!exact) {
            for (int w = tid; w < words; w += kSelThreads) pre[w] = __popcll(ties[w]);
            __syncthreads();
            scan_words(pre, words, wave_sums);
            for (int w = tid; w < words; w += kSelThreads) {
                // the first want - pre[w] ties of the word
                const int left = want - pre[w], all_of = __popcll(ties[w]);
                if (left <= 0 || all_of == 0) continue;
                bits[w] |= left >= all_of ? ties[w]
                                          : ties[w] & ((1ull << nth_bit(ties[w], left)) - 1);
            }
            __syncthreads();
        }
        // holes per word below m, kept slots per word from m on
        const int edge = m >> 6;
        const uint64_t below = (1ull << (m & 63)) - 1;
        for (int w = tid; w < words; w += kSelThreads)
            pre[w] = w < edge ? __popcll(~bits[w])
                              : __popcll(w == edge ? bits[w] & ~below : bits[w]);
        __syncthreads();
        moves = scan_words(pre, words, wave_sums) - pre[edge];
    }
    // the kept slots from m on, in order, where they fit
    const int words = (n + 63) >> 6, edge = m >> 6;
    const int base = all ? 0 : pre[edge];
    const uint64_t below = (1ull << (m & 63)) - 1;
    const bool listed = moves <= a.list;
    if (!all && listed) {
        for (int t = m + tid; t < n; t += kSelThreads) {
            const uint64_t w = (t >> 6) == edge ? bits[edge] & ~below : bits[t >> 6];
            const int at = t & 63;
            if ((w >> at) & 1)
                spare[pre[t >> 6] - base + __popcll(w & ((1ull << at) - 1))] = t;
        }
        __syncthreads();
    }
    const auto spare_at = [&](int r) {
        if (listed) return spare[r];
        // the last word from `edge` on whose kept slots start at or before rank r
        int lo = edge, hi = words - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] - base <= r) lo = mid;
            else hi = mid - 1;
        }
        const uint64_t w = lo == edge ? bits[lo] & ~below : bits[lo];
        return lo * 64 + nth_bit(w, r - (pre[lo] - base));
    };
    // sources of slots j .. j + M - 1 of one word
    const auto sources = [&](int j, auto& src) {
        constexpr int M = sizeof(src) / sizeof(src[0]);
        const bool some = !all && j < m;
        const uint64_t word = some ? bits[j >> 6] : ~0ull;
        int r = some ? pre[j >> 6] + __popcll(~word & ((1ull << (j & 63)) - 1)) : 0;
#pragma unroll
        for (int e = 0; e < M; ++e) {
            const bool hole = j + e < m && !((word >> ((j + e) & 63)) & 1);
            src[e] = j + e >= m ? -1 : j + e;
            if (hole) src[e] = spare_at(r++);
        }
    };
    if (!a.fused) {
        for (int j = 4 * tid; j < a.keep; j += 4 * kSelThreads) {
            int src[4];
            sources(j, src);
            if (j + 4 <= a.keep) {
                *reinterpret_cast<Slots<4>::numbers*>(source + j) =
                    Slots<4>::numbers{src[0], src[1], src[2], src[3]};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < a.keep) source[j + e] = src[e];
            }
        }
        return;
    }
    MovedRow* rows = reinterpret_cast<MovedRow*>(work + ((a.list + 3) & ~3)) + wave * 64;
    for (int j0 = 0; j0 < a.keep; j0 += kSelThreads) {
        const int js[1] = {j0 + tid};
        int srcs[1];
        sources(js[0], srcs);
        if (js[0] < a.keep) source[js[0]] = srcs[0];
        fill_slots<S, 1>(a, b, h, js, srcs, rows);
    }
    if (a.lengths_out && h == 0 && tid == 0) a.lengths_out[b] = m;
}

// Second kernel: every wave fills 64 slots kFill times.  Bound by memory: 64
// heads cut from up to 40001 to 32768 slots (rows of 256 bytes, moved one by
// one: about 130 MB with the slots' numbers) take 36 us, 3.7 TB/s.
constexpr int kFillThreads = 256, kFill = 4, kFillSlots = kFillThreads * kFill;

template <class S>
__global__ __launch_bounds__(kFillThreads) void fill_kernel(EvictArgs a) {
    __shared__ MovedRow rows[kFillThreads / 64][64 * kFill];
    const int tiles = (a.keep + kFillSlots - 1) / kFillSlots;
    if (block_number() >= (uint32_t)(a.B * a.Hkv * tiles)) return;
    const int item = (int)block_number(), bh = item / tiles, tile = item - bh * tiles;
    const int b = bh / a.Hkv, h = bh - b * a.Hkv;
    if (a.lengths_out && h == 0 && tile == 0 && threadIdx.x == 0) {
        // the one place that reads lengths here: lengths_out may be lengths
        const int n = clamped(a.lengths[b], a.pages.slots);
        a.lengths_out[b] = n < a.keep ? n : a.keep;
    }
    const int32_t* source = a.source + (int64_t)bh * a.keep;
    int j[kFill], src[kFill];
#pragma unroll
    for (int u = 0; u < kFill; ++u) {
        j[u] = tile * kFillSlots + u * kFillThreads + threadIdx.x;
        src[u] = source[j[u] < a.keep ? j[u] : a.keep - 1];
        if (j[u] >= a.keep) src[u] = -1;
    }
    fill_slots<S, kFill>(a, b, h, j, src, rows[threadIdx.x >> 6]);
}

constexpr int64_t kStreamBytes = 32 << 20;  // the XCDs' L2 caches together

template <class S>
hipError_t append_t(const AppendArgs& a, hipStream_t s) {
    const dim3 grid = grid_of((int64_t)a.B * a.groups);
    if ((int64_t)a.B * a.n * a.Hkv * a.D * 2 * (int64_t)sizeof(S) > kStreamBytes)
        append_kernel<S, true><<<grid, dim3(256), 0, s>>>(a);
    else
        append_kernel<S, false><<<grid, dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <class S>
hipError_t evict_t(const EvictArgs& a, hipStream_t s) {
    const size_t count = (size_t)(count_words(a.words) + 2 * kNear) * 4;
    size_t work = (size_t)((a.list + 3) & ~3) * 4 + (a.fused ? kSelThreads * sizeof(MovedRow) : 0);
    if (work < count) work = count;
    const size_t lds = (size_t)a.words * 12 + work;
    const int slots = a.words * 64;
    const void* fn = slots <= kSelThreads ? reinterpret_cast<const void*>(&select_kernel<S, 1>)
                                          : reinterpret_cast<const void*>(&select_kernel<S, 4>);
    if (lds > 48u << 10) {
        const hipError_t e =
            hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    EvictArgs args = a;
    void* params[] = {&args};
    const hipError_t e = hipLaunchKernel(fn, grid_of((int64_t)a.B * a.Hkv), dim3(kSelThreads),
                                         params, lds, s);
    if (e != hipSuccess || a.fused) return e;
    const int64_t tiles = ((int64_t)a.keep + kFillSlots - 1) / kFillSlots;
    fill_kernel<S><<<grid_of(a.B * a.Hkv * tiles), dim3(kFillThreads), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, ctconv_dtype dt, hipStream_t s) {
    return dt == CTCONV_F32 ? append_t<float>(a, s) : append_t<uint16_t>(a, s);
}

hipError_t launch_evict(const EvictArgs& a, ctconv_dtype dt, hipStream_t s) {
    return dt == CTCONV_F32 ? evict_t<float>(a, s) : evict_t<uint16_t>(a, s);
}

}  // namespace block
}  // namespace ctconv
