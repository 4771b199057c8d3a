// Page tables that follow the requests' lengths, and the maps of their new rows.
//
// One workgroup keeps the stack of free pages in order: it sums, over the
// sequences, the pages given back, the pages taken and the new rows (three
// inclusive sums in one scan), then moves the pages, an entry per thread that
// finds its sequence by bisection in those sums.  No atomics: the order on the
// stack is that of sequences and columns.  A step moves few pages, so its time
// is a chain of latencies: the lengths, the scan, the stack, the table (48
// sequences that go on by a row, with slot arrays of 8 heads: 4.9 us).  Where many
// pages move, four entries of a thread are on their way together: 96 sequences of
// which a third ends and a third is new, some 8000 pages: 11 us, and 15 one by one.
// The maps of few rows are written by the same workgroup, of many by a kernel of
// their own, a row per thread (61 k rows 4 us).

#include "block_internal.h"

namespace ctconv {
namespace block {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kAtOnce = 4;
constexpr int kRowThreads = 256;
constexpr uint32_t kMost = INT32_MAX;

// Sums of counts stop at the largest int32 (the order of additions does not
// matter to that).
__device__ inline uint32_t add(uint32_t a, uint32_t b) { return min(a + b, kMost); }

// The first of n entries of `ends` (ascending) above e.
__device__ inline int sequence_of(const uint32_t* ends, int n, uint32_t e) {
    int lo = 0;
    while (n > 0) {
        const int half = n >> 1;
        const bool right = ends[lo + half] <= e;
        lo = right ? lo + half + 1 : lo;
        n = right ? n - half - 1 : half;
    }
    return lo;
}

// The maps of row r; ends: the sums of the counts up to and with each sequence.
__device__ inline void map_row(const TablesArgs& a, const uint32_t* ends, int r) {
    int position = -1, slot = -1;
    if ((uint32_t)r < ends[a.B - 1]) {
        const int b = sequence_of(ends, a.B, (uint32_t)r);
        const int back = (int)(ends[b] - (uint32_t)r);
        const int t = a.lengths[b] - back;
        position = (a.now ? a.now[b] : a.lengths[b]) - back;
        if (t >= 0 && t < a.max_pages * a.page_size) {
            const int column = (int)fdiv((uint32_t)t, a.fd_page);
            const int page = a.table[b * a.table_stride + column];
            if (page >= 0 && page < a.num_pages)
                slot = page * a.page_size + (t - column * a.page_size);
            const int64_t at = b * a.slot_b + t;
            if (a.positions)
                for (int h = 0; h < a.Hkv; ++h) a.positions[at + h * a.slot_h] = position;
            if (a.weight_sum)
                for (int h = 0; h < a.Hkv; ++h) a.weight_sum[at + h * a.slot_h] = 0.f;
        }
    }
    a.row_positions[r] = position;
    a.row_slots[r] = slot;
}

__global__ __launch_bounds__(kThreads) void tables_kernel(TablesArgs a) {
    extern __shared__ __align__(16) uint32_t lds[];
    __shared__ uint32_t sums[3][kWaves], found[2][kAtOnce][kWaves];
    uint32_t *need = lds, *back = lds + a.B, *grow = back + a.B, *rows = grow + a.B;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int slots = a.max_pages * a.page_size;
    int top = clamped(*a.free_count, a.num_pages);

    uint32_t before[3] = {0, 0, 0};
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        uint32_t needed = 0, v[3] = {0, 0, 0};
        if (b < a.B) {
            const int length = a.lengths[b], has = clamped(a.held[b], a.max_pages);
            const uint32_t used = clamped(length, slots);
            needed = fdiv(used, a.fd_page);
            needed += used > needed * a.page_size;
            v[0] = has > (int)needed ? has - needed : 0;
            v[1] = has < (int)needed ? needed - has : 0;
            v[2] = a.counts ? clamped(a.counts[b], length > 0 ? length : 0) : 0;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1)
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const uint32_t w = __shfl_up(v[i], o);
                if (lane >= o) v[i] = add(v[i], w);
            }
        if (lane == 63)
#pragma unroll
            for (int i = 0; i < 3; ++i) sums[i][wave] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            uint32_t s = before[i];
            for (int w = 0; w < kWaves && b0 + 64 * w < a.B; ++w) {
                if (w == wave) v[i] = add(v[i], s);
                s = add(s, sums[i][w]);
            }
            before[i] = s;
        }
        if (b < a.B) {
            need[b] = needed;
            back[b] = v[0];
            grow[b] = v[1];
            rows[b] = v[2];
            if (a.counts) {
                a.row_starts[b + 1] = (int)v[2];
                if (b == 0) a.row_starts[0] = 0;
            }
        }
        __syncthreads();
    }

    // given back, pages only, in order: kAtOnce entries of a thread on their way together
    const uint32_t given = before[0], taken = before[1];
    for (uint32_t e0 = 0, turn = 0; e0 < given; e0 += kAtOnce * kThreads, turn ^= 1) {
        int page[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const uint32_t e = e0 + k * kThreads + tid;
            page[k] = -1;
            if (e < given) {
                const int b = sequence_of(back, a.B, e);
                page[k] = a.table[b * a.table_stride + need[b] + (e - (b > 0 ? back[b - 1] : 0))];
            }
        }
        uint64_t votes[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            votes[k] = __ballot(page[k] >= 0 && page[k] < a.num_pages);
            if (lane == 0) found[turn][k][wave] = __popcll(votes[k]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (e0 + k * kThreads >= given) break;
            int at = top;
            for (int w = 0; w < kWaves; ++w) {
                const int n = (int)found[turn][k][w];
                if (w < wave) at += n;
                top += n;
            }
            at += __popcll(votes[k] & ((1ull << lane) - 1));
            if ((votes[k] >> lane & 1) && at < a.num_pages) a.free_pages[at] = page[k];
            top = top < a.num_pages ? top : a.num_pages;
        }
    }
    if (given > 0) __syncthreads();
    for (uint32_t e0 = 0; e0 < taken; e0 += kAtOnce * kThreads) {
        int page[kAtOnce];
        int32_t* to[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const uint32_t e = e0 + k * kThreads + tid;
            page[k] = -1;
            to[k] = nullptr;
            if (e >= taken) continue;
            if (e < (uint32_t)top) page[k] = a.free_pages[top - 1 - (int)e];
            const int b = sequence_of(grow, a.B, e);
            to[k] = a.table + b * a.table_stride + (need[b] - (grow[b] - e));
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (to[k]) *to[k] = page[k];
    }
    for (int b = tid; b < a.B; b += kThreads) {
        const uint32_t first = b > 0 ? grow[b - 1] : 0, wanted = grow[b] - first;
        const int left = top - (int)first;
        a.held_out[b] = (int)(need[b] - wanted) + clamped(left, (int)wanted);
    }
    if (tid == 0) *a.free_count_out = (uint32_t)top > taken ? top - (int)taken : 0;
    if (!a.fused) return;
    __syncthreads();
    for (int r = tid; r < a.rows; r += kThreads) map_row(a, rows, r);
}

__global__ __launch_bounds__(kRowThreads) void rows_kernel(TablesArgs a) {
    extern __shared__ __align__(16) uint32_t ends[];
    for (int b = threadIdx.x; b < a.B; b += kRowThreads) ends[b] = (uint32_t)a.row_starts[b + 1];
    __syncthreads();
    const int64_t r = (int64_t)block_number() * kRowThreads + threadIdx.x;
    if (r < a.rows) map_row(a, ends, (int)r);
}

}  // namespace

hipError_t launch_tables(const TablesArgs& a, hipStream_t s) {
    const size_t lds = (size_t)a.B * 16;
    if (lds > 48u << 10) {
        const hipError_t e =
            hipFuncSetAttribute(reinterpret_cast<const void*>(&tables_kernel),
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    tables_kernel<<<dim3(1), dim3(kThreads), lds, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.fused || !a.counts || a.rows == 0) return e;
    rows_kernel<<<grid_of(((int64_t)a.rows + kRowThreads - 1) / kRowThreads), dim3(kRowThreads),
                  (size_t)a.B * 4, s>>>(a);
    return hipGetLastError();
}

}  // namespace block
}  // namespace ctconv
