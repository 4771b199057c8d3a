// C ABI of the operators on requests of many lengths: argument validation,
// planning and launches.  No allocation, no synchronisation, no global state.

#include <math.h>
#include <string.h>

#include "block_check.h"
#include "block_internal.h"

using namespace ctconv;
using namespace ctconv::block;

namespace {

constexpr int64_t kMostSequences = 8192;  // tables_kernel keeps 16 bytes of each in LDS
// Up to here one workgroup maps the rows after it has moved the pages, and a second
// launch is saved: 64 sequences of 8 key heads, one workgroup | two launches, each
// with slots' statistics to clear: 2048 rows 8.8 | 11.8 us, 4096 10.8 | 12.1,
// 16384 30 | 11.7 (without statistics 8.6 | 12.0, 8.8 | 12.2, 20 | 11.6).
constexpr int64_t kFusedRows = 4096;
constexpr double kTwoPi = 6.283185307179586476925;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int as_int(const void* e) {  // a C caller may pass any int for an enumerator
    int v;
    memcpy(&v, e, sizeof v);
    return v;
}

ctconv_status rotary_sizes(int64_t rows, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int layout,
                           float scale, ctconv_dtype dt) {
    if (!dtype_ok(dt)) return CTCONV_ERR_DTYPE;
    if (layout != CTCONV_ROTARY_HALF && layout != CTCONV_ROTARY_PAIRS) return CTCONV_ERR_PARAM;
    if (rows < 0 || rows > kMaxInt || Hq < 0 || Hq > 65535 || Hk < 0 || Hk > 65535 || Hq + Hk < 1)
        return CTCONV_ERR_SHAPE;
    if (D < 8 || D > 256 || D % 8 != 0 || R < 2 || R > D || R % 2 != 0) return CTCONV_ERR_SHAPE;
    if (!isfinite(scale)) return CTCONV_ERR_PARAM;
    return CTCONV_OK;
}

void rotary_common(int64_t rows, int64_t Hq, int64_t Hk, int64_t D, int64_t R, float scale,
                   RotaryArgs* a) {
    memset(a, 0, sizeof(*a));
    a->rows = (int)rows;
    a->Hq = (int)Hq;
    a->Hk = (int)Hk;
    a->D = (int)D;
    a->half = (int)(R / 2);
    a->scale = scale;
    a->fd_half = make_fastdiv((uint32_t)a->half);
}

// The two kernels' times in ns, as far as the host can tell, for the choice between
// them and the splits.  `once`: all keys and values.  tile_kernel: rounds of the
// workgroups that the chip holds, a step per 64 keys, their start and end, at least
// the reading of `once`, and for split tiles the partial rows, written and read (19 k
// rows of 32 heads over up to 8192 keys take 1565 us whole and 2160 in chunks of
// 4096), and the join.  stream_kernel: `once` from memory, then again from the L2
// caches for every 16 rows past the first, and workgroups without work where
// sequences have fewer rows than n.  Measured (us, stream and tile; 32 heads on 8, D =
// 128): bf16, 24 sequences of 8192 keys, 32 rows per key head 201 and 180, 64 rows
// 307 and 187; one of 8192, 32 rows 20 and 28, 128 rows 38 and 32; one of 65536, 32
// rows 72 and 78.  fp32, 24 of 8192, 64 rows 688 and 985, 128 rows 1274 and 1000; one
// of 65536, 64 rows 239 and 338, 128 rows 430 and 345.
double tile_time(double tiles, double keys, double splits, double once, int64_t D,
                 ctconv_dtype dt) {
    const bool f32 = dt == CTCONV_F32;
    // two workgroups share a compute unit up to 256 bytes a row; a step of both
    const bool pair = D * (int64_t)esize(dt) <= 256;
    double step = f32 ? (D <= 32 ? 5400 : D <= 64 ? 9000 : D <= 96 ? 8000 : 9500)
                      : D <= 32 ? 1200 : D <= 64 ? 1500 : D <= 96 ? 2100 : D <= 128 ? 2400 : 3600;
    if (pair && tiles * splits <= 256) step *= 0.6;
    const double rounds = ceil(tiles * splits / (pair ? 512 : 256));
    double t = 8000 + fmax(rounds * (ceil(ceil(keys / 64) / splits) * step + 4500), once / 4800);
    if (splits > 1) t += 6000 + tiles * splits * 128 * (double)D * 8 / 5000;
    return t;
}
double stream_time(double tiles, double padded, double keys, double once, int64_t D,
                   ctconv_dtype dt) {
    const int64_t width = D <= 64 ? 64 : D <= 128 ? 128 : 256;  // as it computes
    const double all = tiles * keys * 2 * (double)(width * (int64_t)esize(dt));
    return 10000 + once / 5400 + fmax(all - once, 0) / (dt == CTCONV_F32 ? 12000 : 15000) +
           padded * ceil(keys / 512) * 2;
}

// Keys per workgroup of stream_kernel: `tiles` row tiles in a grid of `padded`, which a
// packed call does not fill where one sequence has most of its rows.  From 2048
// workgroups on
//  - without a split, if enough of them have rows (32 query heads over 8 of 128
//    channels, bf16, ragged lengths, whole | split: 512 tiles of 16 rows over at most
//    4000 keys 90 | 90 us, 1024 145 | 155, 2048 243 | 269; over 8000 167 | 144, 256 |
//    246, 447 | 450);
//  - else in no more splits than shorten a workgroup's walk over its keys, some 30
//    bytes a ns (a key of 64, 128, 256 values: f32 21, 30, 52 ns, bf16 11, 15, 32), by
//    more than the workgroups without a row take, 2 ns each.  19 sequences with one new
//    row and one with 101, 24 heads of 64 on 12, up to 23918 keys, fp32 (336 of 3120 have
//    rows): whole 803 us, in 9 splits 475.
void stream_chunk(int64_t tiles, int64_t padded, int64_t span, int64_t D, ctconv_dtype dt,
                  int64_t* chunk, bool* wide) {
    if (padded >= 2048 && tiles >= 1024) {
        *chunk = round_up(span, 128);
        return;
    }
    stream_split(padded, span, D, dt, chunk, wide);
    if (padded < 2048) return;
    const double walk = (double)span * 2 * (double)(D * (int64_t)esize(dt)) / 30;
    double most = sqrt(walk / (2 * (double)(padded - tiles)));
    most = fmax(fmin(most, (double)(kMaxInt / 2) / (double)padded), 1);
    const int64_t least = round_up((int64_t)ceil((double)span / most), 128);
    *chunk = *chunk > least ? *chunk : least;
}

// Splits of tile_kernel's row tiles, at least two steps of keys each.
//  - Of several sequences the lengths may differ, and the longest one's tiles are the
//    last to end.  Lengths spread evenly make (s + 1) / 2 workgroups of a tile in the
//    mean: as many as fill the chip, of 1024 keys at least.  24 x 8 rows of 32 heads
//    over up to 8192 keys: 99 us in chunks of 2048, 118 of 1664 (the second round of
//    a few), 121 of 4096.  Tiles over up to 4096 keys, bf16, D = 128, whole | 2 | 3 | 4
//    | 8 splits: 64 110 | 70 | 56 | 52 | 62 (the rule takes 4), 128 112 | 82 | 91 | 89 |
//    104 (4), 192 123 | 130 | 117 | 113 | 128 (4), 256 145 | 143 | 138 | 156 | 152 (3),
//    384 188 | 190 | 191 | 179 | 204 (1), 512 208 | 229 | 230 | 232 | 267 (1).
//  - So may their rows, where there are several tiles of the longest and in the mean
//    fewer than half of n: one that goes on by a row has the keys of a whole tile.
//    47 such and one of 2048 rows over up to 16384 keys: 411 us in chunks of 4096,
//    479 of 8192, 636 whole.  Means of five draws of their lengths, whole | 3 | 4 | 8
//    splits: the same 736 | 720 | 691 | 743 (the rule takes 4), 11 of 16384 624 | 496 |
//    457 | 517 (6), 95 of 8192 472 | 524 | 528 | 566 (3), 23 and 512 rows of 4096 126 |
//    124 | 127 | 145 (4), of 16384 and 47 490 | 469 | 478 | 490 (7).
int64_t tile_splits(int64_t tiles, int64_t keys, double once, int64_t D, ctconv_dtype dt,
                    bool several, bool uneven) {
    const int64_t n = tiles > 0 ? tiles : 1, steps = ceil_div(keys, 64);
    const int64_t slots = D * (int64_t)esize(dt) <= 256 ? 512 : 256;
    int64_t best = 1;
    double cost = HUGE_VAL;
    for (int64_t s = 1; s <= 64 && s <= ceil_div(steps, 2); ++s) {
        const double t = tile_time((double)n, (double)keys, (double)s, once, D, dt);
        if (t < cost) {
            cost = t;
            best = s;
        }
    }
    int64_t more = 1;
    if (several && n < slots) more = 2 * slots / n - 1;
    if (several && uneven) {
        const int64_t s = 8 * slots / n < 8 ? 8 * slots / n : 8;
        more = s > more ? s : more;
    }
    const int64_t most = ceil_div(keys, 1024);
    more = more < most ? more : most;
    return more > best ? more : best;
}

struct ChunkPlan {
    bool tile;  // many rows per key head: tile_kernel, else stream_kernel
    bool wide;
    int64_t n, row_tiles, chunk, splits;
    int64_t part_o_bytes, part_ml_bytes, lse_bytes, bytes;
};

ctconv_status chunk_plan(int64_t B, int64_t rows, int64_t n, int64_t Hq, int64_t Hkv, int64_t D,
                         int64_t max_length, int64_t window, bool weights, ctconv_dtype dt,
                         ChunkPlan* p) {
    memset(p, 0, sizeof(*p));
    const ctconv_status st = head_sizes(B, Hkv, D, dt);
    if (st != CTCONV_OK) return st;
    if (Hq < 1 || Hq > kMaxInt || Hq % Hkv != 0) return CTCONV_ERR_SHAPE;
    if (rows < 0 || rows > kMaxInt || n < 0 || n > kMaxInt) return CTCONV_ERR_SHAPE;
    if (max_length < 0 || max_length > kMaxInt - (1 << 20) || window < 0) return CTCONV_ERR_SHAPE;
    const int64_t G = Hq / Hkv;
    // (kernels step past the last row by less than that)
    if ((__int128)n * G > kMaxInt - (1 << 20)) return CTCONV_ERR_SHAPE;
    if ((__int128)B * Hkv * n * G > kMaxInt) return CTCONV_ERR_SHAPE;
    // rows of a sequence that exist: n may be any bound (of a packed call; else rows = B n)
    p->n = n < rows ? n : rows;
    const int64_t R = p->n * G;
    // row tiles of all sequences: each may end inside one
    const auto tiles_of = [&](int64_t height) {
        const __int128 all = (__int128)rows * G / height + B;
        const __int128 most = (__int128)B * ceil_div(R, height);
        return (all < most ? all : most) * Hkv;
    };
    // keys that the rows of one tile see together
    const auto span_of = [&](int64_t height) {
        const int64_t together = n < height ? n : height;
        const int64_t s = window > 0 && window + together < max_length ? window + together
                                                                       : max_length;
        return s > 0 ? s : 1;
    };
    const __int128 padded = (__int128)B * Hkv * ceil_div(R, 16);
    if (tiles_of(16) > kMaxInt) return CTCONV_ERR_SHAPE;
    const int64_t tiles = (int64_t)tiles_of(128);
    int64_t span = span_of(128);
    // (fp32 rows past 512 bytes are too long for the tile kernel's LDS)
    if (R > 16 && D * (int64_t)esize(dt) <= 512) {
        const double once =
            (double)B * (double)Hkv * (double)span * 2 * (double)(D * (int64_t)esize(dt));
        const bool uneven = R > 128 && rows * 2 <= B * p->n;
        const int64_t splits = tile_splits(tiles, span, once, D, dt, B > 1, uneven);
        p->tile = tile_time((double)tiles, (double)span, (double)splits, once, D, dt) <
                  stream_time((double)tiles_of(16), (double)padded, (double)span_of(16), once, D,
                              dt);
        p->chunk = round_up(ceil_div(span, splits), 128);
        p->row_tiles = tiles / Hkv;
    }
    if (!p->tile) {
        p->row_tiles = ceil_div(R, 16);
        span = span_of(16);
        stream_chunk((int64_t)tiles_of(16), (int64_t)padded, span, D, dt, &p->chunk, &p->wide);
    }
    p->splits = ceil_div(span, p->chunk);
    const __int128 values = (__int128)rows * Hq;
    const __int128 parts = p->splits > 1 ? values * p->splits : 0;
    const __int128 groups = (p->tile ? (__int128)tiles : padded) * p->splits;
    // workgroups of the join of tiles (8 each) and of the weights (32 keys at least)
    if (p->tile && p->splits > 1 && (__int128)tiles * 8 > kMaxInt) return CTCONV_ERR_SHAPE;
    if (weights && (__int128)B * Hkv * ceil_div(max_length, 32) > kMaxInt) return CTCONV_ERR_SHAPE;
    if (groups > kMaxInt - 8 || parts * D > ((__int128)1 << 59) ||
        values > ((__int128)1 << 59))
        return CTCONV_ERR_SHAPE;
    p->part_o_bytes = (int64_t)parts * D * 4;
    p->part_ml_bytes = round_up((int64_t)parts * 8, 16);
    p->lse_bytes = weights ? round_up((int64_t)values * 4, 16) : 0;
    p->bytes = p->part_o_bytes + p->part_ml_bytes + p->lse_bytes;
    return CTCONV_OK;
}

}  // namespace

extern "C" {

ctconv_status ctconv_cache_pages(const int32_t* lengths, const int32_t* counts,
                                 const int32_t* now, const int32_t* held,
                                 const int32_t* free_count, int32_t* page_table,
                                 int32_t* free_pages, int32_t* held_out, int32_t* free_count_out,
                                 int32_t* row_starts, int32_t* row_positions, int32_t* row_slots,
                                 int32_t* positions, float* weight_sum, int64_t B, int64_t rows,
                                 int64_t Hkv, int64_t num_pages, int64_t page_size,
                                 int64_t max_pages, int64_t table_stride,
                                 const int64_t* slot_strides, void* stream) {
    if (B < 0 || B > kMostSequences || rows < 0 || rows > kMaxInt || Hkv < 1 || Hkv > 65535 ||
        table_stride < 0)
        return CTCONV_ERR_SHAPE;
    ctconv_status st = page_sizes(num_pages, page_size, max_pages);
    if (st != CTCONV_OK) return st;
    if ((__int128)B * max_pages > kMaxInt || (__int128)num_pages * page_size > kMaxInt)
        return CTCONV_ERR_SHAPE;
    if (B == 0) return CTCONV_OK;
    const bool slots = counts && (positions || weight_sum);
    if (!lengths || !held || !free_count || !page_table || !free_pages || !held_out ||
        !free_count_out || (counts && !row_starts) ||
        (counts && rows > 0 && (!row_positions || !row_slots)) || (slots && !slot_strides))
        return CTCONV_ERR_NULL;
    const int64_t table_rows[1] = {table_stride}, sizes[1] = {B};
    st = strides_ok(table_rows, sizes, 1, max_pages, CTCONV_F32);
    if (st == CTCONV_OK && slots) st = slot_strides_ok(slot_strides, B, Hkv, page_size * max_pages);
    if (st != CTCONV_OK) return st;
    const void* const arrays[] = {lengths,    counts,        now,       held,      free_count,
                                  page_table, free_pages,    held_out,  free_count_out,
                                  row_starts, row_positions, row_slots, positions, weight_sum};
    for (const void* p : arrays)
        if (!aligned4(p)) return CTCONV_ERR_ALIGN;
    if (!rows_apart(table_rows, {B}, max_pages) ||
        (slots && !rows_apart(slot_strides, {B, Hkv}, page_size * max_pages)))
        return CTCONV_ERR_SHAPE;
    TablesArgs a;
    memset(&a, 0, sizeof(a));
    a.lengths = lengths;
    a.counts = counts;
    a.now = now;
    a.held = held;
    a.free_count = free_count;
    a.table = page_table;
    a.free_pages = free_pages;
    a.held_out = held_out;
    a.free_count_out = free_count_out;
    a.row_starts = row_starts;
    a.row_positions = row_positions;
    a.row_slots = row_slots;
    a.positions = slots ? positions : nullptr;
    a.weight_sum = slots ? weight_sum : nullptr;
    a.table_stride = table_stride;
    if (slots) {
        a.slot_b = slot_strides[0];
        a.slot_h = slot_strides[1];
    }
    a.B = (int)B;
    a.rows = counts ? (int)rows : 0;
    a.Hkv = (int)Hkv;
    a.num_pages = (int)num_pages;
    a.page_size = (int)page_size;
    a.max_pages = (int)max_pages;
    a.fused = counts && rows <= kFusedRows;
    a.fd_page = make_fastdiv((uint32_t)page_size);
    return to_status(launch_tables(a, static_cast<hipStream_t>(stream)));
}

ctconv_status ctconv_rotary(const void* q, const void* k, const int32_t* positions,
                            const double* frequencies, void* q_out, void* k_out, int64_t rows,
                            int64_t Hq, int64_t Hk, int64_t D, int64_t R,
                            const int64_t* q_strides, const int64_t* k_strides,
                            const int64_t* q_out_strides, const int64_t* k_out_strides,
                            ctconv_rotary_layout layout, float scale, ctconv_dtype dtype,
                            void* stream) {
    const int kind = as_int(&layout);
    ctconv_status st = rotary_sizes(rows, Hq, Hk, D, R, kind, scale, dtype);
    if (st != CTCONV_OK) return st;
    if (rows == 0) return CTCONV_OK;
    if (!positions || !frequencies || (Hq > 0 && (!q || !q_out || !q_strides || !q_out_strides)) ||
        (Hk > 0 && (!k || !k_out || !k_strides || !k_out_strides)))
        return CTCONV_ERR_NULL;
    RotaryArgs a;
    rotary_common(rows, Hq, Hk, D, R, scale, &a);
    Check c;
    c.pointer(frequencies);
    if (Hq > 0) {
        c.tensor(q, q_strides, {rows, Hq}, D, dtype);
        c.tensor(q_out, q_out_strides, {rows, Hq}, D, dtype);
        a.q = q;
        a.q_out = q_out;
        a.q_row = q_strides[0];
        a.q_head = q_strides[1];
        a.q_out_row = q_out_strides[0];
        a.q_out_head = q_out_strides[1];
    }
    if (Hk > 0) {
        c.tensor(k, k_strides, {rows, Hk}, D, dtype);
        c.tensor(k_out, k_out_strides, {rows, Hk}, D, dtype);
        a.k = k;
        a.k_out = k_out;
        a.k_row = k_strides[0];
        a.k_head = k_strides[1];
        a.k_out_row = k_out_strides[0];
        a.k_out_head = k_out_strides[1];
    }
    st = c.status();
    if (st == CTCONV_OK && !aligned4(positions)) st = CTCONV_ERR_ALIGN;
    if (st != CTCONV_OK) return st;
    if ((Hq > 0 && !rows_apart(q_out_strides, {rows, Hq}, D)) ||
        (Hk > 0 && !rows_apart(k_out_strides, {rows, Hk}, D)))
        return CTCONV_ERR_SHAPE;
    // in place: the same rows
    const auto moved = [](const void* in, const void* out, const int64_t* s, const int64_t* t) {
        return in == out && (s[0] != t[0] || s[1] != t[1]);
    };
    if ((Hq > 0 && moved(q, q_out, q_strides, q_out_strides)) ||
        (Hk > 0 && moved(k, k_out, k_strides, k_out_strides)))
        return CTCONV_ERR_PARAM;
    a.positions = positions;
    a.frequencies = frequencies;
    return to_status(launch_rotary(a, dtype, kind == CTCONV_ROTARY_PAIRS, false,
                                   static_cast<hipStream_t>(stream)));
}

ctconv_status ctconv_rotary_append(const void* q, const void* k_new, const void* v_new,
                                   const int32_t* positions, const int32_t* slots,
                                   const double* frequencies, void* q_out, void* k_cache,
                                   void* v_cache, int64_t rows, int64_t Hq, int64_t Hkv,
                                   int64_t D, int64_t R, int64_t num_pages, int64_t page_size,
                                   const int64_t* q_strides, const int64_t* new_strides,
                                   const int64_t* q_out_strides, const int64_t* kv_strides,
                                   ctconv_rotary_layout layout, float scale, ctconv_dtype dtype,
                                   void* stream) {
    const int kind = as_int(&layout);
    ctconv_status st = rotary_sizes(rows, Hq, Hkv, D, R, kind, scale, dtype);
    if (st != CTCONV_OK) return st;
    if (Hkv < 1) return CTCONV_ERR_SHAPE;
    st = page_sizes(num_pages, page_size, 1);
    if (st != CTCONV_OK) return st;
    if ((__int128)num_pages * page_size > kMaxInt) return CTCONV_ERR_SHAPE;
    if (rows == 0) return CTCONV_OK;
    if (!k_new || !v_new || !positions || !slots || !frequencies || !k_cache || !v_cache ||
        !new_strides || !kv_strides || (Hq > 0 && (!q || !q_out || !q_strides || !q_out_strides)))
        return CTCONV_ERR_NULL;
    RotaryArgs a;
    rotary_common(rows, Hq, Hkv, D, R, scale, &a);
    Check c;
    c.pointer(frequencies);
    if (Hq > 0) {
        c.tensor(q, q_strides, {rows, Hq}, D, dtype);
        c.tensor(q_out, q_out_strides, {rows, Hq}, D, dtype);
        a.q = q;
        a.q_out = q_out;
        a.q_row = q_strides[0];
        a.q_head = q_strides[1];
        a.q_out_row = q_out_strides[0];
        a.q_out_head = q_out_strides[1];
    }
    c.tensor(k_new, new_strides, {rows, Hkv}, D, dtype);
    c.tensor(k_cache, kv_strides, {num_pages, page_size, Hkv}, D, dtype);
    c.pointer(v_new);
    c.pointer(v_cache);
    st = c.status();
    if (st == CTCONV_OK && !(aligned4(positions) && aligned4(slots))) st = CTCONV_ERR_ALIGN;
    if (st != CTCONV_OK) return st;
    if ((Hq > 0 && !rows_apart(q_out_strides, {rows, Hq}, D)) ||
        !rows_apart(kv_strides, {num_pages, page_size, Hkv}, D))
        return CTCONV_ERR_SHAPE;
    if (Hq > 0 && q == q_out &&
        (q_strides[0] != q_out_strides[0] || q_strides[1] != q_out_strides[1]))
        return CTCONV_ERR_PARAM;
    a.k = k_new;
    a.v = v_new;
    a.k_out = k_cache;
    a.v_out = v_cache;
    a.k_row = new_strides[0];
    a.k_head = new_strides[1];
    a.page_stride = kv_strides[0];
    a.slot_stride = kv_strides[1];
    a.k_out_head = kv_strides[2];
    a.positions = positions;
    a.slots = slots;
    a.frequencies = frequencies;
    a.page_size = (int)page_size;
    a.num_slots = (int)(num_pages * page_size);
    a.fd_page = make_fastdiv((uint32_t)page_size);
    return to_status(launch_rotary(a, dtype, kind == CTCONV_ROTARY_PAIRS, true,
                                   static_cast<hipStream_t>(stream)));
}

ctconv_status ctconv_rotary_frequencies(int64_t R, double base, ctconv_rotary_scaling scaling,
                                        double factor, double original, double low, double high,
                                        double* frequencies) {
    const int kind = as_int(&scaling);
    if (R < 2 || R > 256 || R % 2 != 0) return CTCONV_ERR_SHAPE;
    if (kind < CTCONV_ROTARY_NONE || kind > CTCONV_ROTARY_RAMP_TURNS) return CTCONV_ERR_PARAM;
    const auto positive = [](double v) { return isfinite(v) && v > 0; };
    if (!positive(base) || !positive(factor)) return CTCONV_ERR_PARAM;
    const bool dims = kind == CTCONV_ROTARY_RAMP_DIMS, turns = kind == CTCONV_ROTARY_RAMP_TURNS;
    if ((dims || turns) &&
        (!positive(original) || !positive(low) || !isfinite(high) || high <= low))
        return CTCONV_ERR_PARAM;
    if (dims && base <= 1) return CTCONV_ERR_PARAM;
    if (!frequencies) return CTCONV_ERR_NULL;
    if (kind == CTCONV_ROTARY_BASE && R > 2) base *= pow(factor, (double)R / (double)(R - 2));
    double from = 0, to = 1;
    if (dims) {
        const auto pair = [&](double t) {
            return (double)R * log(original / (t * kTwoPi)) / (2 * log(base));
        };
        from = fmax(floor(pair(high)), 0);
        to = fmin(ceil(pair(low)), (double)(R - 1));
    }
    for (int64_t i = 0; i < R / 2; ++i) {
        const double f = pow(base, -2.0 * (double)i / (double)R);
        double keep = 1;
        if (kind == CTCONV_ROTARY_LINEAR) keep = 0;
        if (dims) keep = 1 - fmin(fmax(((double)i - from) / fmax(to - from, 0.001), 0), 1);
        if (turns) keep = fmin(fmax((original * f / kTwoPi - low) / (high - low), 0), 1);
        frequencies[i] = keep * f + (1 - keep) * f / factor;
    }
    return CTCONV_OK;
}

ctconv_status ctconv_chunk_attention_workspace_bytes(int64_t B, int64_t rows, int64_t n,
                                                     int64_t Hq, int64_t Hkv, int64_t D,
                                                     int64_t max_length, int64_t window,
                                                     int weights, ctconv_dtype dtype,
                                                     size_t* bytes) {
    if (!bytes) return CTCONV_ERR_NULL;
    ChunkPlan p;
    const ctconv_status st =
        chunk_plan(B, rows, n, Hq, Hkv, D, max_length, window, weights != 0, dtype, &p);
    if (st != CTCONV_OK) return st;
    *bytes = (size_t)p.bytes;
    return CTCONV_OK;
}

ctconv_status ctconv_chunk_attention(const void* q, const void* k_cache, const void* v_cache,
                                     const int32_t* page_table, const int32_t* lengths,
                                     const int32_t* row_starts, const int32_t* counts, void* out,
                                     float* lse, float* weight_sum, int64_t B, int64_t rows,
                                     int64_t n, int64_t Hq, int64_t Hkv, int64_t D,
                                     int64_t num_pages, int64_t page_size, int64_t max_pages,
                                     int64_t max_length, int64_t window, const int64_t* q_strides,
                                     const int64_t* kv_strides, const int64_t* out_strides,
                                     int64_t table_stride, const int64_t* slot_strides,
                                     float scale, ctconv_dtype dtype, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    ChunkPlan p;
    ctconv_status st = chunk_plan(B, rows, n, Hq, Hkv, D, max_length, window,
                                  weight_sum != nullptr, dtype, &p);
    if (st != CTCONV_OK) return st;
    st = page_sizes(num_pages, page_size, max_pages);
    if (st != CTCONV_OK) return st;
    if (max_length > page_size * max_pages || table_stride < 0) return CTCONV_ERR_SHAPE;
    if (!row_starts && (__int128)B * n != rows) return CTCONV_ERR_SHAPE;
    if (!isfinite(scale)) return CTCONV_ERR_PARAM;
    if (B == 0 || rows == 0 || n == 0) return CTCONV_OK;
    if (!q || !k_cache || !v_cache || !page_table || !lengths || !out || !q_strides ||
        !kv_strides || !out_strides || (weight_sum && !slot_strides))
        return CTCONV_ERR_NULL;
    const int64_t batch = row_starts ? 1 : B, in_batch = row_starts ? rows : n;
    Check c;
    c.tensor(q, q_strides, {batch, in_batch, Hq}, D, dtype);
    c.tensor(out, out_strides, {batch, in_batch, Hq}, D, dtype);
    c.tensor(k_cache, kv_strides, {num_pages, page_size, Hkv}, D, dtype);
    c.pointer(v_cache);
    c.pointer(workspace);
    if (weight_sum && c.st == CTCONV_OK)
        c.st = slot_strides_ok(slot_strides, B, Hkv, page_size * max_pages);
    st = c.status();
    for (const void* i : {(const void*)page_table, (const void*)lengths, (const void*)row_starts,
                          (const void*)counts, (const void*)lse, (const void*)weight_sum})
        if (st == CTCONV_OK && !aligned4(i)) st = CTCONV_ERR_ALIGN;
    if (st != CTCONV_OK) return st;
    if (!rows_apart(out_strides, {batch, in_batch, Hq}, D) ||
        (weight_sum && !rows_apart(slot_strides, {B, Hkv}, max_length)))
        return CTCONV_ERR_SHAPE;
    if (p.bytes > 0 && (!workspace || workspace_bytes < (size_t)p.bytes))
        return CTCONV_ERR_WORKSPACE;
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.out = out;
    a.lse = lse;
    a.lengths = lengths;
    a.weight_sum = weight_sum;
    a.row_starts = row_starts;
    a.counts = row_starts ? nullptr : counts;
    a.pages = make_pages(page_table, table_stride, kv_strides, num_pages, page_size, max_pages,
                         max_length);
    a.q_b = q_strides[0];
    a.q_row = q_strides[1];
    a.q_head = q_strides[2];
    a.o_b = out_strides[0];
    a.o_row = out_strides[1];
    a.o_head = out_strides[2];
    if (weight_sum) {
        a.slot_b = slot_strides[0];
        a.slot_h = slot_strides[1];
    }
    a.B = (int)B;
    a.n = (int)p.n;
    a.most = (int)n;
    a.rows = (int)rows;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.R = (int)(p.n * a.G);
    a.D = (int)D;
    a.window = (int)(window < max_length ? window : 0);
    a.fd_G = make_fastdiv((uint32_t)a.G);
    a.c = score_factor(scale);
    a.negate = scale < 0;
    a.row_tiles = (int)p.row_tiles;
    a.chunk = (int)p.chunk;
    a.splits = (int)p.splits;
    a.wide = p.wide;
    char* at = static_cast<char*>(workspace);
    a.part_o = reinterpret_cast<float*>(at);
    a.part_ml = reinterpret_cast<float*>(at + p.part_o_bytes);
    a.lse2 = weight_sum ? reinterpret_cast<float*>(at + p.part_o_bytes + p.part_ml_bytes) : nullptr;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    st = to_status(p.tile ? launch_chunk_tile(a, dtype, s) : launch_chunk_stream(a, dtype, s));
    if (st == CTCONV_OK && a.splits > 1)
        st = to_status(p.tile ? launch_chunk_tile_join(a, dtype, s)
                              : launch_chunk_join(a, dtype, s));
    if (st == CTCONV_OK && weight_sum) st = to_status(launch_chunk_weights(a, dtype, s));
    return st;
}

}  // extern "C"
