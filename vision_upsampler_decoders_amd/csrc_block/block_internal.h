// Internal declarations of the decoder-block operators (not installed):
// kernel arguments, filled on the host by block_api.hip and request_api.hip, and
// launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ctconv.h"
#include "ctconv_internal.h"

namespace ctconv {
namespace block {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// The cache as a kernel addresses it: strides in elements.
struct Pages {
    const int32_t* table;
    int64_t table_stride;
    int64_t page_stride, slot_stride, head_stride;
    int num_pages, page_size;
    int slots;  // max_pages * page_size, also at most max_length where one is given
    FastDiv fd_page;
};

// Element offset (within a head) of slot t, which lies in `page`, or -1 where
// there is no such page.
__device__ inline int64_t offset_in_page(const Pages& p, int t, int32_t page) {
    if (page < 0 || page >= p.num_pages) return -1;
    const int at = t - (int)fdiv((uint32_t)t, p.fd_page) * p.page_size;
    return (int64_t)page * p.page_stride + (int64_t)at * p.slot_stride;
}
__device__ inline int64_t slot_offset(const Pages& p, int b, int t) {
    return offset_in_page(p, t, p.table[b * p.table_stride + (int)fdiv((uint32_t)t, p.fd_page)]);
}

__device__ inline int clamped(int v, int hi) { return v < 0 ? 0 : v > hi ? hi : v; }

// A launch holds fewer than 2^32 threads along x: past kGridRow workgroups (of up
// to 1024) they go to further rows of the grid, and those past the last one
// end at once.
constexpr int kGridRowBits = 20;
inline dim3 grid_of(int64_t blocks) {
    constexpr int64_t row = (int64_t)1 << kGridRowBits;
    return blocks <= row ? dim3((unsigned)blocks)
                         : dim3((unsigned)row, (unsigned)((blocks + row - 1) / row));
}
__device__ inline uint32_t block_number() { return blockIdx.y << kGridRowBits | blockIdx.x; }

struct AppendArgs {
    const void *k_new, *v_new;
    void *k, *v;
    const int32_t *lengths, *counts, *now;
    int32_t* positions;
    float* weight_sum;
    Pages pages;
    int64_t new_b, new_row, new_head, slot_b, slot_h;
    int B, n, Hkv, D;
    int chunks;         // 16-byte pieces of a row
    int rows_per_group; // new rows that one workgroup copies
    int groups;         // workgroups per sequence
    FastDiv fd_chunks, fd_heads, fd_groups;
};

struct EvictArgs {
    void *k, *v;
    const int32_t *lengths, *now;
    const float* weight_sum;
    const int32_t* positions;
    float* weight_out;
    int32_t *positions_out, *lengths_out, *source;
    Pages pages;
    int64_t slot_b, slot_h, out_b, out_h;
    int B, Hkv, D, keep, sink, recent;
    int words;  // 64-slot words of the longest sequence, a multiple of 16
    int list;   // kept slots past keep that select_kernel has room to list
    int fused;  // few slots: select_kernel fills them itself
    int chunks;
    FastDiv fd_chunks;
};

// Attention of R = Lq * G query rows per (sequence, cache head): row r is
// query position r / G, query head h * G + r % G.
struct AttnArgs {
    const void *q, *k, *v;
    void* out;
    float* lse;
    const int32_t* lengths;
    const uint8_t* mask;
    float* weight_sum;
    float *part_o, *part_ml, *scores;
    Pages pages;                 // paged calls
    int64_t q_b, q_row, q_head;
    int64_t k_b, k_row, k_head;  // dense calls
    int64_t v_b, v_row, v_head;
    int64_t o_b, o_row, o_head;
    int64_t mask_stride, slot_b, slot_h;
    int64_t score_stride;        // floats per query row of `scores`
    int B, Lq, Lk, Hq, Hkv, G, D, R;
    int window;
    int chunk, splits;           // keys per workgroup, workgroups per row tile
    int wide;                    // stream kernel: a workgroup of as many waves as it can have
    int direct;                  // one workgroup per row tile, and no weights: no join
    int row_tiles;
    FastDiv fd_G;
    float c;                     // |scale| * log2(e)
    int negate;                  // scale < 0: the queries change sign
    // Chunk calls: each sequence's own number of rows.
    const int32_t *row_starts, *counts;
    float* lse2;                 // log2 of the sums of weights, [rows, Hq] (weights)
    int most;                    // what row_starts' counts are clamped to
    int n, rows;                 // most rows of a sequence that exist, rows of the call
};

struct NormArgs {
    const void *x, *h, *post_w, *post_b, *scale, *gate, *pre_w, *pre_b;
    void *x_out, *y;
    int64_t xs, hs, gs, os, ys;
    int64_t rows, rows_per_gate;
    int C, post, pre, gate_fn;
    float eps, inv_C;
};

// ctconv_cache_pages.
struct TablesArgs {
    const int32_t *lengths, *counts, *now, *held, *free_count;
    int32_t *table, *free_pages, *held_out, *free_count_out;
    int32_t *row_starts, *row_positions, *row_slots, *positions;
    float* weight_sum;
    int64_t table_stride, slot_b, slot_h;
    int B, rows, Hkv, num_pages, page_size, max_pages;
    int fused;  // few rows: mapped by the workgroup that moves the pages
    FastDiv fd_page;
};

// ctconv_rotary and ctconv_rotary_append; strides in elements.
struct RotaryArgs {
    const void *q, *k, *v;
    const int32_t *positions, *slots;
    const double* frequencies;
    void *q_out, *k_out, *v_out;
    int64_t q_row, q_head, k_row, k_head;  // (of k and v)
    int64_t q_out_row, q_out_head, k_out_row, k_out_head;
    int64_t page_stride, slot_stride;
    int rows, Hq, Hk, D;
    int half;                    // pairs
    int page_size, num_slots;
    int units, v_units, items;   // pairs of pieces per head of q or k, of v, per row
    int per;                     // rows of a workgroup
    float scale;
    FastDiv fd_page, fd_units, fd_v_units, fd_items, fd_half;
};

hipError_t launch_append(const AppendArgs& a, ctconv_dtype dt, hipStream_t s);
hipError_t launch_evict(const EvictArgs& a, ctconv_dtype dt, hipStream_t s);
hipError_t launch_norm(const NormArgs& a, ctconv_dtype dt, bool vec, hipStream_t s);
// Few query rows (paged calls, single tokens): keys streamed from memory.
hipError_t launch_attn_stream(const AttnArgs& a, ctconv_dtype dt, bool paged, hipStream_t s);
// Many query rows: keys and values through LDS tiles.
hipError_t launch_attn_tile(const AttnArgs& a, ctconv_dtype dt, hipStream_t s);
// The partial results of `splits` workgroups joined, and the slots' weights.
hipError_t launch_attn_join(const AttnArgs& a, ctconv_dtype dt, bool paged, hipStream_t s);
// The chunk call with few query rows per key head and with many (row_tiles: of
// all sequences), the joins of their splits, and the weights.
hipError_t launch_chunk_stream(const AttnArgs& a, ctconv_dtype dt, hipStream_t s);
hipError_t launch_chunk_join(const AttnArgs& a, ctconv_dtype dt, hipStream_t s);
hipError_t launch_chunk_tile(const AttnArgs& a, ctconv_dtype dt, hipStream_t s);
hipError_t launch_chunk_tile_join(const AttnArgs& a, ctconv_dtype dt, hipStream_t s);
hipError_t launch_chunk_weights(const AttnArgs& a, ctconv_dtype dt, hipStream_t s);
hipError_t launch_tables(const TablesArgs& a, hipStream_t s);
hipError_t launch_rotary(const RotaryArgs& a, ctconv_dtype dt, bool pairs, bool append,
                         hipStream_t s);

}  // namespace block
}  // namespace ctconv
