// Host-side checks and rules that the entry points of csrc_block share.
#pragma once

#include <math.h>
#include <string.h>

#include <initializer_list>

#include "block_internal.h"

namespace ctconv {
namespace block {

constexpr int64_t kMaxInt = INT32_MAX;

inline size_t esize(ctconv_dtype dt) { return dt == CTCONV_F32 ? 4 : 2; }

inline bool dtype_ok(int dt) { return dt == CTCONV_F32 || dt == CTCONV_BF16 || dt == CTCONV_F16; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline ctconv_status to_status(hipError_t e) { return e == hipSuccess ? CTCONV_OK : CTCONV_ERR_HIP; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Strides of a tensor whose last dimension holds D values: not negative, the
// last element addressable.
inline ctconv_status strides_ok(const int64_t* strides, const int64_t* sizes, int n, int64_t D,
                         ctconv_dtype dt) {
    __int128 last = D;
    for (int i = 0; i < n; ++i) {
        if (strides[i] < 0) return CTCONV_ERR_SHAPE;
        if (sizes[i] > 0) last += (__int128)(sizes[i] - 1) * strides[i];
    }
    if (last * (int64_t)esize(dt) > INT64_MAX) return CTCONV_ERR_SHAPE;
    return CTCONV_OK;
}

// Every row starts on 16 bytes (strides of a dimension of one are not stepped).
inline bool rows_aligned(const int64_t* strides, const int64_t* sizes, int n, ctconv_dtype dt) {
    const int64_t step = 16 / (int64_t)esize(dt);
    for (int i = 0; i < n; ++i)
        if (sizes[i] > 1 && strides[i] % step != 0) return false;
    return true;
}

// What is written: rows of `row` values that lie apart.  From the smallest
// stride up, a step must pass everything below it.  (A layout whose dimensions
// interleave without meeting is not told from one where they meet.)
inline bool rows_apart(const int64_t* strides, std::initializer_list<int64_t> sizes, int64_t row) {
    constexpr int kDims = 3;
    int64_t step[kDims], size[kDims];
    int n = 0, dim = 0;
    for (const int64_t s : sizes) {
        const int64_t st = strides[dim++];
        if (s <= 1) continue;
        int at = n++;
        for (; at > 0 && step[at - 1] > st; --at) {
            step[at] = step[at - 1];
            size[at] = size[at - 1];
        }
        step[at] = st;
        size[at] = s;
    }
    __int128 extent = row;
    for (int i = 0; i < n; ++i) {
        if (step[i] < extent) return false;
        extent += (__int128)(size[i] - 1) * step[i];
    }
    return true;
}

struct Check {
    ctconv_status st = CTCONV_OK;
    bool align = true;
    void tensor(const void* p, const int64_t* strides, std::initializer_list<int64_t> sizes,
                int64_t D, ctconv_dtype dt) {
        const ctconv_status s = strides_ok(strides, sizes.begin(), (int)sizes.size(), D, dt);
        if (st == CTCONV_OK) st = s;
        if (p && !aligned16(p)) align = false;
        if (!rows_aligned(strides, sizes.begin(), (int)sizes.size(), dt)) align = false;
    }
    void pointer(const void* p) {
        if (p && !aligned16(p)) align = false;
    }
    ctconv_status status() const {
        return st != CTCONV_OK ? st : align ? CTCONV_OK : CTCONV_ERR_ALIGN;
    }
};

// Heads and row width of the attention and cache calls.
inline ctconv_status head_sizes(int64_t B, int64_t Hkv, int64_t D, ctconv_dtype dt) {
    if (!dtype_ok(dt)) return CTCONV_ERR_DTYPE;
    if (B < 0 || B > kMaxInt || Hkv < 1 || Hkv > 65535) return CTCONV_ERR_SHAPE;
    if (D < 8 || D > 256 || D % 8 != 0) return CTCONV_ERR_SHAPE;
    return CTCONV_OK;
}

inline ctconv_status page_sizes(int64_t num_pages, int64_t page_size, int64_t max_pages) {
    if (num_pages < 1 || num_pages > kMaxInt || page_size < 1 || page_size > kMaxInt ||
        max_pages < 1 || max_pages > kMaxInt)
        return CTCONV_ERR_SHAPE;
    // slot numbers, and what rounding up to whole workgroups adds, fit int32
    if ((__int128)page_size * max_pages > kMaxInt - (1 << 20)) return CTCONV_ERR_SHAPE;
    return CTCONV_OK;
}

inline Pages make_pages(const int32_t* table, int64_t table_stride, const int64_t* kv_strides,
                 int64_t num_pages, int64_t page_size, int64_t max_pages, int64_t max_length) {
    Pages p;
    p.table = table;
    p.table_stride = table_stride;
    p.page_stride = kv_strides[0];
    p.slot_stride = kv_strides[1];
    p.head_stride = kv_strides[2];
    p.num_pages = (int)num_pages;
    p.page_size = (int)page_size;
    const int64_t slots = page_size * max_pages;
    p.slots = (int)(slots < max_length ? slots : max_length);
    p.fd_page = make_fastdiv((uint32_t)page_size);
    return p;
}

// Slot arrays (positions, weights): one value per slot.
inline ctconv_status slot_strides_ok(const int64_t* strides, int64_t B, int64_t Hkv, int64_t slots) {
    const int64_t sizes[2] = {B, Hkv};
    return strides_ok(strides, sizes, 2, slots, CTCONV_F32);
}

inline int64_t round_up(int64_t v, int64_t to) { return ceil_div(v, to) * to; }

// |scale| log2(e), not zero: hidden scores are minus infinity times it.
// (Scores times 1e-30 weigh the same as scores times 0.)
inline float score_factor(float scale) {
    const float c = fabsf(scale) * kLog2e;
    return c > 1e-30f ? c : 1e-30f;
}

// Keys per workgroup of tile_kernel.  A workgroup costs about one tile on top
// of its own (its first loads, its last stores), and the compute units take
// the workgroups in rounds; splitting pays a join.
inline int64_t tile_chunk(int64_t tiles, int64_t keys) {
    const int64_t cus = 256, steps = ceil_div(keys, 64);
    int64_t best = 1, cost = INT64_MAX;
    for (int64_t s = 1; s <= 16 && s <= ceil_div(steps, 4); ++s) {
        const int64_t c =
            ceil_div(tiles * s, cus) * (ceil_div(steps, s) + 1) + (s > 1 ? 4 + s : 0);
        if (c < cost) {
            cost = c;
            best = s;
        }
    }
    return round_up(ceil_div(keys, best), 128);
}

// Keys per workgroup of stream_kernel, and its waves (figures: one query row,
// keys and values in memory, not in a cache).
//  - One workgroup per row tile and no join, where few keys or many row tiles
//    allow it: 500 keys on 8 tiles 9.8 us against 12.1 split, 1000 keys on 256
//    tiles 28 against 32; but 2000 keys on 64 tiles 25 against 20 (bf16, D =
//    128).  Rows of more than 128 values take a wave longer: up to 500 of 256
//    on 8 tiles 20.8 us against 19.4 split in bf16 (350: 17.2 against 19.3),
//    56.3 against 35.7 in fp32 (350: 43.3 against 35.5).
//  - Else chunks that give every compute unit one round of the workgroups its
//    registers hold (4, 3 or 1 of 4 waves for D up to 64, 128, 256): 30000
//    keys on 8 tiles take 33 us in 469 workgroups, 40 in 938.  At least 256
//    keys (a workgroup's start costs about as much as 128), at most 1024, so
//    that ragged sequences still spread.
//  - An undivided row tile takes as many waves as its registers allow (16 up to
//    D = 64, 8 up to 128) where 4 would have more than a block of keys each and
//    the tiles do not fill the chip by themselves, so that more loads are in
//    flight: 500 keys of 64 on 64 tiles 9.4 us against 10.3 (fp32 12.7 against
//    23.4), 2000 on 256 fp32 76 against 86.  More tiles bring loads enough, and
//    the merge of many waves costs most of a short call (16 keys on 1024 tiles
//    19.3 us against 6.7, 250 on 8192 198 against 136): there only where each
//    wave has two blocks (1000 of 128 on 1024, fp32, 229 against 265).
inline void stream_split(int64_t tiles, int64_t keys, int64_t D, ctconv_dtype dt, int64_t* chunk,
                  bool* wide) {
    const int64_t block = dt == CTCONV_F32 ? 16 : 32, waves = D <= 64 ? 16 : 8;
    const int64_t few = D <= 128 ? 512 : dt == CTCONV_F32 ? 256 : 384;
    const bool whole = keys <= few || (keys <= 1024 && tiles >= 128) ||
                       (keys <= 2048 && tiles >= 256);
    *wide = whole && D <= 128 && keys > (tiles <= 256 ? 4 : 2 * waves) * block;
    if (whole) {
        *chunk = round_up(keys, 128);
        return;
    }
    const int64_t room = D <= 64 ? 1024 : D <= 128 ? 768 : 256;
    const int64_t c = round_up(ceil_div(keys * tiles, room), 128);
    *chunk = c < 256 ? 256 : c > 1024 ? 1024 : c;
}

}  // namespace block
}  // namespace ctconv
