// C ABI of the decoder-block operators: argument validation, planning and
// launches.  No allocation, no synchronisation, no global state.

#include <math.h>
#include <string.h>

#include "block_internal.h"

using namespace ctconv;
using namespace ctconv::block;

namespace {

constexpr int64_t kMaxInt = INT32_MAX;
constexpr int64_t kMaxEvictSlots = 262144;  // select_kernel keeps a few bits per slot in LDS
constexpr int64_t kEvictLds = 128 << 10;     // of the 160 KB, with what it declares itself
// Up to this many kept slots eviction is one kernel: 8 heads cut to 256 slots
// take 8.9 us against 11.4 in two, to 1000 12.1 against 15.1, to 2000 15.7
// against 16.5, but to 3000 19.9 against 17.0, to 5000 25.8 against 17.8.
constexpr int64_t kFusedKeep = 2048;
constexpr int64_t kMaxRowValues = 16384;    // norm_kernel keeps a row in registers

size_t esize(ctconv_dtype dt) { return dt == CTCONV_F32 ? 4 : 2; }

bool dtype_ok(int dt) { return dt == CTCONV_F32 || dt == CTCONV_BF16 || dt == CTCONV_F16; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

ctconv_status to_status(hipError_t e) { return e == hipSuccess ? CTCONV_OK : CTCONV_ERR_HIP; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Strides of a tensor whose last dimension holds D values: not negative, the
// last element addressable.
ctconv_status strides_ok(const int64_t* strides, const int64_t* sizes, int n, int64_t D,
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
bool rows_aligned(const int64_t* strides, const int64_t* sizes, int n, ctconv_dtype dt) {
    const int64_t step = 16 / (int64_t)esize(dt);
    for (int i = 0; i < n; ++i)
        if (sizes[i] > 1 && strides[i] % step != 0) return false;
    return true;
}

// What is written: rows of `row` values that lie apart.  From the smallest
// stride up, a step must pass everything below it.  (A layout whose dimensions
// interleave without meeting is not told from one where they meet.)
bool rows_apart(const int64_t* strides, std::initializer_list<int64_t> sizes, int64_t row) {
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
ctconv_status head_sizes(int64_t B, int64_t Hkv, int64_t D, ctconv_dtype dt) {
    if (!dtype_ok(dt)) return CTCONV_ERR_DTYPE;
    if (B < 0 || B > kMaxInt || Hkv < 1 || Hkv > 65535) return CTCONV_ERR_SHAPE;
    if (D < 8 || D > 256 || D % 8 != 0) return CTCONV_ERR_SHAPE;
    return CTCONV_OK;
}

ctconv_status page_sizes(int64_t num_pages, int64_t page_size, int64_t max_pages) {
    if (num_pages < 1 || num_pages > kMaxInt || page_size < 1 || page_size > kMaxInt ||
        max_pages < 1 || max_pages > kMaxInt)
        return CTCONV_ERR_SHAPE;
    // slot numbers, and what rounding up to whole workgroups adds, fit int32
    if ((__int128)page_size * max_pages > kMaxInt - (1 << 20)) return CTCONV_ERR_SHAPE;
    return CTCONV_OK;
}

Pages make_pages(const int32_t* table, int64_t table_stride, const int64_t* kv_strides,
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
ctconv_status slot_strides_ok(const int64_t* strides, int64_t B, int64_t Hkv, int64_t slots) {
    const int64_t sizes[2] = {B, Hkv};
    return strides_ok(strides, sizes, 2, slots, CTCONV_F32);
}

// The split of one attention call: R query rows per (sequence, cache head),
// at most `span` visible keys.
struct Plan {
    bool tile;  // tile_kernel (many rows), else stream_kernel
    bool wide;
    int64_t row_tiles, chunk, splits;
    bool direct;
    int64_t score_stride;  // floats per query row (weights), else 0
    int64_t parts;         // partial rows
    int64_t score_bytes, part_o_bytes, part_ml_bytes, bytes;
};

constexpr int64_t kTileRows = 128;  // query rows per workgroup of tile_kernel
// More rows per cache head than this: tile_kernel.  No one limit is best for all.
// 64 or 65 rows in stream_kernel and in tile_kernel (from memory; heads x keys,
// us): bf16, D = 64: 8 x 2000 12.0 and 18.1, 64 x 500 11.0 and 13.3, 64 x 4000
// 51.9 and 26.1; fp32: 15.3 and 49.2, 15.2 and 45.1, 82.1 and 86.2.  96 rows:
// bf16 13.0 and 17.9, 12.3 and 14.2, 63.0 and 27.7; fp32 17.7 and 49.5, 20.6
// and 45.5, 113 and 87.5.
constexpr int64_t kTileFrom = 64;

int64_t round_up(int64_t v, int64_t to) { return ceil_div(v, to) * to; }

// Keys per workgroup of tile_kernel.  A workgroup costs about one tile on top
// of its own (its first loads, its last stores), and the compute units take
// the workgroups in rounds; splitting pays a join.
int64_t tile_chunk(int64_t tiles, int64_t keys) {
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
void stream_split(int64_t tiles, int64_t keys, int64_t D, ctconv_dtype dt, int64_t* chunk,
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

ctconv_status plan_attention(int64_t B, int64_t Hkv, int64_t R, int64_t D, int64_t span,
                             bool weights, bool tile, ctconv_dtype dt, Plan* p) {
    memset(p, 0, sizeof(*p));
    p->tile = tile;
    p->row_tiles = ceil_div(R, tile ? kTileRows : 16);
    const __int128 tiles = (__int128)B * Hkv * p->row_tiles;
    if (tiles > kMaxInt || (__int128)B * Hkv * R > kMaxInt) return CTCONV_ERR_SHAPE;
    const int64_t keys = span > 0 ? span : 1;
    int64_t chunk;
    if (tile) {
        chunk = tile_chunk((int64_t)tiles, keys);
    } else {
        stream_split((int64_t)tiles, keys, D, dt, &chunk, &p->wide);
    }
    p->chunk = chunk;
    p->splits = span > 0 ? ceil_div(span, chunk) : 1;
    p->direct = p->splits == 1 && !weights;
    __int128 score = 0, parts = 0;
    if (weights) {
        p->score_stride = round_up(span > 0 ? span : 1, 128);
        score = (__int128)B * Hkv * R * p->score_stride * 4;
    }
    if (!p->direct) parts = (__int128)B * Hkv * R * p->splits;
    const __int128 total = score + parts * (D + 2) * 4 + 64;
    if (tiles * p->splits > kMaxInt - 8 || parts * D > ((__int128)1 << 61) ||
        total > ((__int128)1 << 62))
        return CTCONV_ERR_SHAPE;
    if (weights && (__int128)B * Hkv * R + (__int128)B * Hkv * ceil_div(p->score_stride, 1024) >
                       kMaxInt)
        return CTCONV_ERR_SHAPE;
    p->parts = (int64_t)parts;
    p->score_bytes = (int64_t)score;
    p->part_o_bytes = (int64_t)parts * D * 4;
    p->part_ml_bytes = round_up((int64_t)parts * 8, 16);
    p->bytes = p->score_bytes + p->part_o_bytes + p->part_ml_bytes;
    return CTCONV_OK;
}

// |scale| log2(e), not zero: hidden scores are minus infinity times it.
// (Scores times 1e-30 weigh the same as scores times 0.)
float score_factor(float scale) {
    const float c = fabsf(scale) * kLog2e;
    return c > 1e-30f ? c : 1e-30f;
}

void apply_plan(const Plan& p, void* ws, AttnArgs* a) {
    a->row_tiles = (int)p.row_tiles;
    a->chunk = (int)p.chunk;
    a->splits = (int)p.splits;
    a->direct = p.direct;
    a->wide = p.wide;
    a->score_stride = p.score_stride;
    char* at = static_cast<char*>(ws);
    a->scores = p.score_bytes ? reinterpret_cast<float*>(at) : nullptr;
    a->part_o = reinterpret_cast<float*>(at + p.score_bytes);
    a->part_ml = reinterpret_cast<float*>(at + p.score_bytes + p.part_o_bytes);
}

ctconv_status paged_plan(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_length,
                         int64_t window, bool weights, ctconv_dtype dt, Plan* p) {
    const ctconv_status st = head_sizes(B, Hkv, D, dt);
    if (st != CTCONV_OK) return st;
    if (Hq < 1 || Hq > kMaxInt || Hq % Hkv != 0) return CTCONV_ERR_SHAPE;
    if (max_length < 0 || max_length > kMaxInt - (1 << 20) || window < 0) return CTCONV_ERR_SHAPE;
    const int64_t span = window > 0 && window < max_length ? window : max_length;
    return plan_attention(B, Hkv, Hq / Hkv, D, span, weights, false, dt, p);
}

ctconv_status cross_plan(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t D,
                         ctconv_dtype dt, Plan* p) {
    const ctconv_status st = head_sizes(B, Hkv, D, dt);
    if (st != CTCONV_OK) return st;
    if (Hq < 1 || Hq > kMaxInt || Hq % Hkv != 0) return CTCONV_ERR_SHAPE;
    if (Lq < 0 || Lq > kMaxInt || Lk < 0 || Lk > kMaxInt - (1 << 20)) return CTCONV_ERR_SHAPE;
    if ((__int128)Lq * (Hq / Hkv) > kMaxInt) return CTCONV_ERR_SHAPE;
    const int64_t R = Lq * (Hq / Hkv);
    // (fp32 rows past 512 bytes are too long for its LDS tiles)
    const bool tile = R > kTileFrom && D * (int64_t)esize(dt) <= 512;
    return plan_attention(B, Hkv, R, D, Lk, false, tile, dt, p);
}

}  // namespace

extern "C" {

ctconv_status ctconv_cache_append(const void* k_new, const void* v_new, void* k_cache,
                                  void* v_cache, const int32_t* page_table,
                                  const int32_t* lengths, const int32_t* counts,
                                  const int32_t* now, int32_t* positions, float* weight_sum,
                                  int64_t B, int64_t n, int64_t Hkv, int64_t D,
                                  int64_t num_pages, int64_t page_size, int64_t max_pages,
                                  const int64_t* new_strides, const int64_t* kv_strides,
                                  int64_t table_stride, const int64_t* slot_strides,
                                  ctconv_dtype dtype, void* stream) {
    ctconv_status st = head_sizes(B, Hkv, D, dtype);
    if (st != CTCONV_OK) return st;
    if (n < 0 || n > kMaxInt - (1 << 20) || table_stride < 0) return CTCONV_ERR_SHAPE;
    st = page_sizes(num_pages, page_size, max_pages);
    if (st != CTCONV_OK) return st;
    if (B == 0 || n == 0) return CTCONV_OK;
    const bool slots = positions || weight_sum;
    if (!k_new || !v_new || !k_cache || !v_cache || !page_table || !lengths || !new_strides ||
        !kv_strides || (slots && !slot_strides))
        return CTCONV_ERR_NULL;
    Check c;
    c.tensor(k_new, new_strides, {B, n, Hkv}, D, dtype);
    c.tensor(k_cache, kv_strides, {num_pages, page_size, Hkv}, D, dtype);
    c.pointer(v_new);
    c.pointer(v_cache);
    if (slots && c.st == CTCONV_OK)
        c.st = slot_strides_ok(slot_strides, B, Hkv, page_size * max_pages);
    st = c.status();
    if (st != CTCONV_OK) return st;
    if (!rows_apart(kv_strides, {num_pages, page_size, Hkv}, D) ||
        (slots && !rows_apart(slot_strides, {B, Hkv}, page_size * max_pages)))
        return CTCONV_ERR_SHAPE;
    AppendArgs a;
    memset(&a, 0, sizeof(a));
    a.k_new = k_new;
    a.v_new = v_new;
    a.k = k_cache;
    a.v = v_cache;
    a.lengths = lengths;
    a.counts = counts;
    a.now = now;
    a.positions = positions;
    a.weight_sum = weight_sum;
    a.pages = make_pages(page_table, table_stride, kv_strides, num_pages, page_size, max_pages,
                         kMaxInt);
    a.new_b = new_strides[0];
    a.new_row = new_strides[1];
    a.new_head = new_strides[2];
    if (slots) {
        a.slot_b = slot_strides[0];
        a.slot_h = slot_strides[1];
    }
    a.B = (int)B;
    a.n = (int)n;
    a.Hkv = (int)Hkv;
    a.D = (int)D;
    a.chunks = (int)(D * (int64_t)esize(dtype) / 16);
    // about 2048 pieces of K and of V per workgroup
    int64_t rows = 2048 / (Hkv * a.chunks);
    rows = rows < 1 ? 1 : rows > n ? n : rows;
    a.rows_per_group = (int)rows;
    const int64_t groups = ceil_div(n, rows);
    if ((__int128)groups * B > kMaxInt) return CTCONV_ERR_SHAPE;
    a.groups = (int)groups;
    a.fd_chunks = make_fastdiv((uint32_t)a.chunks);
    a.fd_heads = make_fastdiv((uint32_t)Hkv);
    a.fd_groups = make_fastdiv((uint32_t)groups);
    return to_status(launch_append(a, dtype, static_cast<hipStream_t>(stream)));
}

ctconv_status ctconv_paged_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                                                     int64_t max_length, int64_t window,
                                                     int weights, ctconv_dtype dtype,
                                                     size_t* bytes) {
    if (!bytes) return CTCONV_ERR_NULL;
    Plan p;
    const ctconv_status st =
        paged_plan(B, Hq, Hkv, D, max_length, window, weights != 0, dtype, &p);
    if (st != CTCONV_OK) return st;
    *bytes = (size_t)p.bytes;
    return CTCONV_OK;
}

ctconv_status ctconv_paged_attention(const void* q, const void* k_cache, const void* v_cache,
                                     const int32_t* page_table, const int32_t* lengths, void* out,
                                     float* lse, float* weight_sum, int64_t B, int64_t Hq,
                                     int64_t Hkv, int64_t D, int64_t num_pages, int64_t page_size,
                                     int64_t max_pages, int64_t max_length, int64_t window,
                                     const int64_t* q_strides, const int64_t* kv_strides,
                                     const int64_t* out_strides, int64_t table_stride,
                                     const int64_t* slot_strides, float scale, ctconv_dtype dtype,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    Plan p;
    ctconv_status st =
        paged_plan(B, Hq, Hkv, D, max_length, window, weight_sum != nullptr, dtype, &p);
    if (st != CTCONV_OK) return st;
    st = page_sizes(num_pages, page_size, max_pages);
    if (st != CTCONV_OK) return st;
    if (max_length > page_size * max_pages || table_stride < 0) return CTCONV_ERR_SHAPE;
    if (!isfinite(scale)) return CTCONV_ERR_PARAM;
    if (B == 0) return CTCONV_OK;
    if (!q || !k_cache || !v_cache || !page_table || !lengths || !out || !q_strides ||
        !kv_strides || !out_strides || (weight_sum && !slot_strides))
        return CTCONV_ERR_NULL;
    Check c;
    c.tensor(q, q_strides, {B, Hq}, D, dtype);
    c.tensor(out, out_strides, {B, Hq}, D, dtype);
    c.tensor(k_cache, kv_strides, {num_pages, page_size, Hkv}, D, dtype);
    c.pointer(v_cache);
    c.pointer(workspace);
    if (weight_sum && c.st == CTCONV_OK)
        c.st = slot_strides_ok(slot_strides, B, Hkv, page_size * max_pages);
    st = c.status();
    if (st != CTCONV_OK) return st;
    if (!rows_apart(out_strides, {B, Hq}, D) ||
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
    a.pages = make_pages(page_table, table_stride, kv_strides, num_pages, page_size, max_pages,
                         max_length);
    a.q_b = q_strides[0];
    a.q_head = q_strides[1];
    a.o_b = out_strides[0];
    a.o_head = out_strides[1];
    if (weight_sum) {
        a.slot_b = slot_strides[0];
        a.slot_h = slot_strides[1];
    }
    a.B = (int)B;
    a.Lq = 1;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.G = a.R = (int)(Hq / Hkv);
    a.D = (int)D;
    a.window = (int)(window < max_length ? window : 0);
    a.fd_G = make_fastdiv((uint32_t)a.G);
    a.c = score_factor(scale);
    a.negate = scale < 0;
    apply_plan(p, workspace, &a);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    st = to_status(launch_attn_stream(a, dtype, true, s));
    if (st != CTCONV_OK || a.direct) return st;
    return to_status(launch_attn_join(a, dtype, true, s));
}

ctconv_status ctconv_cache_evict(void* k_cache, void* v_cache, const int32_t* page_table,
                                 const int32_t* lengths, const int32_t* now,
                                 const float* weight_sum, const int32_t* positions,
                                 float* weight_out, int32_t* positions_out, int32_t* lengths_out,
                                 int32_t* source, int64_t B, int64_t Hkv, int64_t D,
                                 int64_t num_pages, int64_t page_size, int64_t max_pages,
                                 int64_t max_length, int64_t keep, int64_t sink, int64_t recent,
                                 const int64_t* kv_strides, int64_t table_stride,
                                 const int64_t* slot_strides, const int64_t* out_slot_strides,
                                 ctconv_dtype dtype, void* stream) {
    ctconv_status st = head_sizes(B, Hkv, D, dtype);
    if (st != CTCONV_OK) return st;
    st = page_sizes(num_pages, page_size, max_pages);
    if (st != CTCONV_OK) return st;
    if (max_length < 0 || max_length > page_size * max_pages || max_length > kMaxEvictSlots ||
        table_stride < 0)
        return CTCONV_ERR_SHAPE;
    if (keep < 1 || sink < 0 || recent < 0) return CTCONV_ERR_PARAM;
    if (keep > kMaxInt - (1 << 20)) return CTCONV_ERR_SHAPE;
    if (B == 0) return CTCONV_OK;
    if (!k_cache || !v_cache || !page_table || !lengths || !weight_sum || !weight_out || !source ||
        !kv_strides || !slot_strides || !out_slot_strides || (positions && !positions_out))
        return CTCONV_ERR_NULL;
    Check c;
    c.tensor(k_cache, kv_strides, {num_pages, page_size, Hkv}, D, dtype);
    c.pointer(v_cache);
    if (c.st == CTCONV_OK) c.st = slot_strides_ok(slot_strides, B, Hkv, page_size * max_pages);
    if (c.st == CTCONV_OK) c.st = slot_strides_ok(out_slot_strides, B, Hkv, keep);
    st = c.status();
    if (st != CTCONV_OK) return st;
    if (!rows_apart(kv_strides, {num_pages, page_size, Hkv}, D)) return CTCONV_ERR_SHAPE;
    // rows of `keep` results: a shorter one would run into the next head's, which another
    // workgroup may still be reading
    if (!rows_apart(out_slot_strides, {B, Hkv}, keep)) return CTCONV_ERR_SHAPE;
    // in place: the same slots, and no more of them than there are
    if (weight_out == weight_sum || (positions && positions_out == positions)) {
        if (keep > page_size * max_pages) return CTCONV_ERR_SHAPE;
        if (slot_strides[0] != out_slot_strides[0] || slot_strides[1] != out_slot_strides[1])
            return CTCONV_ERR_PARAM;
    }
    EvictArgs a;
    memset(&a, 0, sizeof(a));
    a.k = k_cache;
    a.v = v_cache;
    a.lengths = lengths;
    a.now = now;
    a.weight_sum = weight_sum;
    a.positions = positions;
    a.weight_out = weight_out;
    a.positions_out = positions_out;
    a.lengths_out = lengths_out;
    a.source = source;
    a.pages = make_pages(page_table, table_stride, kv_strides, num_pages, page_size, max_pages,
                         max_length);
    a.slot_b = slot_strides[0];
    a.slot_h = slot_strides[1];
    a.out_b = out_slot_strides[0];
    a.out_h = out_slot_strides[1];
    a.B = (int)B;
    a.Hkv = (int)Hkv;
    a.D = (int)D;
    a.keep = (int)keep;
    a.sink = (int)(sink < kMaxInt ? sink : kMaxInt);
    a.recent = (int)(recent < kMaxInt ? recent : kMaxInt);
    a.words = (int)(round_up(max_length > 0 ? max_length : 1, 1024) / 64);
    const int64_t excess = max_length > keep ? max_length - keep : 0;
    const int64_t moves = excess < keep ? excess : keep;
    const int64_t room = (kEvictLds - a.words * 12) / 4;
    a.list = (int)(moves < room ? moves : room);
    // (one kernel writes lengths_out while other heads may still read the counts)
    a.fused = keep <= kFusedKeep && lengths_out != lengths && lengths_out != now;
    a.chunks = (int)(D * (int64_t)esize(dtype) / 16);
    a.fd_chunks = make_fastdiv((uint32_t)a.chunks);
    if ((__int128)B * Hkv * ceil_div(keep, 64) > kMaxInt) return CTCONV_ERR_SHAPE;
    return to_status(launch_evict(a, dtype, static_cast<hipStream_t>(stream)));
}

ctconv_status ctconv_cross_attention_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq,
                                                     int64_t Hkv, int64_t D, ctconv_dtype dtype,
                                                     size_t* bytes) {
    if (!bytes) return CTCONV_ERR_NULL;
    Plan p;
    const ctconv_status st = cross_plan(B, Lq, Lk, Hq, Hkv, D, dtype, &p);
    if (st != CTCONV_OK) return st;
    *bytes = (size_t)p.bytes;
    return CTCONV_OK;
}

ctconv_status ctconv_cross_attention(const void* q, const void* k, const void* v,
                                     const int32_t* lengths, const uint8_t* mask, void* out,
                                     float* lse, int64_t B, int64_t Lq, int64_t Lk, int64_t Hq,
                                     int64_t Hkv, int64_t D, const int64_t* q_strides,
                                     const int64_t* k_strides, const int64_t* v_strides,
                                     const int64_t* out_strides, int64_t mask_stride, float scale,
                                     ctconv_dtype dtype, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    Plan p;
    ctconv_status st = cross_plan(B, Lq, Lk, Hq, Hkv, D, dtype, &p);
    if (st != CTCONV_OK) return st;
    if (!isfinite(scale)) return CTCONV_ERR_PARAM;
    if (mask && mask_stride < 0) return CTCONV_ERR_SHAPE;
    if (B == 0 || Lq == 0) return CTCONV_OK;
    if (!q || !out || ((!k || !v) && Lk > 0) || !q_strides || !k_strides || !v_strides ||
        !out_strides)
        return CTCONV_ERR_NULL;
    Check c;
    c.tensor(q, q_strides, {B, Lq, Hq}, D, dtype);
    c.tensor(out, out_strides, {B, Lq, Hq}, D, dtype);
    c.tensor(k, k_strides, {B, Lk, Hkv}, D, dtype);
    c.tensor(v, v_strides, {B, Lk, Hkv}, D, dtype);
    c.pointer(workspace);
    st = c.status();
    if (st != CTCONV_OK) return st;
    if (!rows_apart(out_strides, {B, Lq, Hq}, D)) return CTCONV_ERR_SHAPE;
    if (p.bytes > 0 && (!workspace || workspace_bytes < (size_t)p.bytes))
        return CTCONV_ERR_WORKSPACE;
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.lse = lse;
    a.lengths = lengths;
    a.mask = mask;
    a.q_b = q_strides[0];
    a.q_row = q_strides[1];
    a.q_head = q_strides[2];
    a.k_b = k_strides[0];
    a.k_row = k_strides[1];
    a.k_head = k_strides[2];
    a.v_b = v_strides[0];
    a.v_row = v_strides[1];
    a.v_head = v_strides[2];
    a.o_b = out_strides[0];
    a.o_row = out_strides[1];
    a.o_head = out_strides[2];
    a.mask_stride = mask_stride;
    a.B = (int)B;
    a.Lq = (int)Lq;
    a.Lk = (int)Lk;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.R = (int)(Lq * a.G);
    a.D = (int)D;
    a.fd_G = make_fastdiv((uint32_t)a.G);
    a.c = score_factor(scale);
    a.negate = scale < 0;
    apply_plan(p, workspace, &a);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    // tile_kernel holds offsets within a tile of 64 keys in 32 bits
    const int64_t reach = a.k_row > a.v_row ? a.k_row : a.v_row;
    const bool far = reach > (((int64_t)1 << 32) / (int64_t)esize(dtype) - D) / 64;
    if (p.tile && far) {
        // the same split by the other kernel, whose row tiles are smaller
        const int64_t tiles = ceil_div(a.R, 16);
        if ((__int128)B * Hkv * tiles * a.splits > kMaxInt) return CTCONV_ERR_SHAPE;
        a.row_tiles = (int)tiles;
    }
    st = to_status(p.tile && !far ? launch_attn_tile(a, dtype, s)
                                  : launch_attn_stream(a, dtype, false, s));
    if (st != CTCONV_OK || a.direct) return st;
    return to_status(launch_attn_join(a, dtype, false, s));
}

ctconv_status ctconv_norm_residual(const void* x, const void* h, const void* post_weight,
                                   const void* post_bias, const void* scale, const void* gate,
                                   const void* pre_weight, const void* pre_bias, void* x_out,
                                   void* y, int64_t rows, int64_t C, const int64_t* strides,
                                   int64_t rows_per_gate, ctconv_norm post, ctconv_norm pre,
                                   ctconv_gate gate_fn, float eps, ctconv_dtype dtype,
                                   void* stream) {
    int kinds[3];
    // a C caller may pass any int: read them as ints
    memcpy(&kinds[0], &post, sizeof(int));
    memcpy(&kinds[1], &pre, sizeof(int));
    memcpy(&kinds[2], &gate_fn, sizeof(int));
    if (!dtype_ok(dtype)) return CTCONV_ERR_DTYPE;
    if (kinds[0] < 0 || kinds[0] > CTCONV_NORM_LAYER || kinds[1] < 0 ||
        kinds[1] > CTCONV_NORM_LAYER || kinds[2] < 0 || kinds[2] > CTCONV_GATE_TANH)
        return CTCONV_ERR_PARAM;
    if (!isfinite(eps) || eps < 0) return CTCONV_ERR_PARAM;
    if (rows < 0 || rows > kMaxInt || C < 1 || C > kMaxRowValues) return CTCONV_ERR_SHAPE;
    const bool gated = kinds[2] != CTCONV_GATE_NONE, normed = kinds[1] != CTCONV_NORM_NONE;
    if (gated && rows_per_gate < 1) return CTCONV_ERR_SHAPE;
    if (rows == 0) return CTCONV_OK;
    if (!x || !h || !x_out || !strides || (gated && !gate) || (normed && !y))
        return CTCONV_ERR_NULL;
    const int64_t gate_rows = gated ? (rows - 1) / rows_per_gate + 1 : 1;
    Check c;
    bool vec = C % (16 / (int64_t)esize(dtype)) == 0;
    const struct {
        const void* p;
        int64_t stride, n;
        bool used, written;
    } row[5] = {{x, strides[0], rows, true, false},
                {h, strides[1], rows, true, false},
                {gate, strides[2], gate_rows, gated, false},
                {x_out, strides[3], rows, true, true},
                {y, strides[4], rows, normed, true}};
    for (const auto& r : row) {
        if (!r.used) continue;
        const ctconv_status s = strides_ok(&r.stride, &r.n, 1, C, dtype);
        if (s != CTCONV_OK) return s;
        if (r.written && r.n > 1 && r.stride < C) return CTCONV_ERR_SHAPE;
        if (!rows_aligned(&r.stride, &r.n, 1, dtype)) vec = false;
        c.pointer(r.p);
    }
    const bool posted = kinds[0] != CTCONV_NORM_NONE;
    if (posted) {
        c.pointer(post_weight);
        c.pointer(post_bias);
    }
    if (normed) {
        c.pointer(pre_weight);
        c.pointer(pre_bias);
    }
    c.pointer(scale);
    if (c.status() != CTCONV_OK) return c.status();
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.x = x;
    a.h = h;
    a.post_w = post_weight;
    a.post_b = post_bias;
    a.scale = scale;
    a.gate = gate;
    a.pre_w = pre_weight;
    a.pre_b = pre_bias;
    a.x_out = x_out;
    a.y = y;
    a.xs = strides[0];
    a.hs = strides[1];
    a.gs = strides[2];
    a.os = strides[3];
    a.ys = strides[4];
    a.rows = rows;
    a.rows_per_gate = gated ? rows_per_gate : 1;
    a.C = (int)C;
    a.post = kinds[0];
    a.pre = kinds[1];
    a.gate_fn = kinds[2];
    a.eps = eps;
    a.inv_C = (float)(1.0 / (double)C);
    return to_status(launch_norm(a, dtype, vec, static_cast<hipStream_t>(stream)));
}

ctconv_status ctconv_block_run(ctconv_block_op op, const int64_t* sizes, void* const* buffers,
                               void* workspace, size_t workspace_bytes, void* stream) {
    if (!sizes || !buffers) return CTCONV_ERR_NULL;
    int which;
    memcpy(&which, &op, sizeof which);  // a C caller may pass any int
    const int64_t* z = sizes;
    void* const* p = buffers;
    const auto f32 = [](int64_t bits) {
        double d;
        memcpy(&d, &bits, sizeof d);
        return (float)d;
    };
    const auto i32 = [&](int i) { return static_cast<int32_t*>(p[i]); };
    const auto fp = [&](int i) { return static_cast<float*>(p[i]); };
    // enumerators: any int64 outside them becomes one that the call refuses
    const auto code = [](int64_t v) { return v < 0 || v > 1000 ? -1 : (int)v; };
    const auto as_dtype = [&](int64_t v) {
        const int c = code(v);
        ctconv_dtype d;
        memcpy(&d, &c, sizeof d);
        return d;
    };
    switch (which) {
        case CTCONV_OP_CACHE_APPEND:
            return ctconv_cache_append(p[0], p[1], p[2], p[3], i32(4), i32(5), i32(6), i32(7),
                                       i32(8), fp(9), z[0], z[1], z[2], z[3], z[4], z[5], z[6],
                                       z + 7, z + 10, z[13], z + 14, as_dtype(z[16]), stream);
        case CTCONV_OP_PAGED_ATTENTION:
            return ctconv_paged_attention(p[0], p[1], p[2], i32(3), i32(4), p[5], fp(6), fp(7),
                                          z[0], z[1], z[2], z[3], z[4], z[5], z[6], z[7], z[8],
                                          z + 9, z + 11, z + 14, z[16], z + 17, f32(z[19]),
                                          as_dtype(z[20]), workspace, workspace_bytes, stream);
        case CTCONV_OP_CACHE_EVICT:
            return ctconv_cache_evict(p[0], p[1], i32(2), i32(3), i32(4), fp(5), i32(6), fp(7),
                                      i32(8), i32(9), i32(10), z[0], z[1], z[2], z[3], z[4], z[5],
                                      z[6], z[7], z[8], z[9], z + 10, z[13], z + 14, z + 16,
                                      as_dtype(z[18]), stream);
        case CTCONV_OP_CROSS_ATTENTION:
            return ctconv_cross_attention(p[0], p[1], p[2], i32(3),
                                          static_cast<const uint8_t*>(p[4]), p[5], fp(6), z[0],
                                          z[1], z[2], z[3], z[4], z[5], z + 6, z + 9, z + 12,
                                          z + 15, z[18], f32(z[19]), as_dtype(z[20]), workspace,
                                          workspace_bytes, stream);
        case CTCONV_OP_NORM_RESIDUAL: {
            const int kinds[3] = {code(z[8]), code(z[9]), code(z[10])};
            ctconv_norm post, pre;
            ctconv_gate gate;
            memcpy(&post, &kinds[0], sizeof(int));
            memcpy(&pre, &kinds[1], sizeof(int));
            memcpy(&gate, &kinds[2], sizeof(int));
            return ctconv_norm_residual(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9],
                                        z[0], z[1], z + 2, z[7], post, pre, gate, f32(z[11]),
                                        as_dtype(z[12]), stream);
        }
    }
    return CTCONV_ERR_PARAM;
}

}  // extern "C"
