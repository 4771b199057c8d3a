// Attention of many query rows per cache head to an encoder's states.
//
// A workgroup of 4 waves takes 128 query rows of one (sequence, cache head),
// a wave 32 of them, and walks the keys in tiles of 64.  Keys and values go
// through LDS (each is used by all four waves), queries and outputs stay in
// registers.
//  - S^T = K Q^T by 32x32 matrix instructions: a key per row, a query per
//    column, so lane (col = lane % 32, half = lane / 32) holds the scores of
//    query col for keys 8 (i / 4) + 4 half + i % 4, i < 16, of each 32.
//  - O^T = V^T P^T.  The k slots of a matrix instruction are summed in any
//    order, so slot j of a half in step s stands for key
//    16 s + 8 (j / 4) + 4 half + j % 4: the weights that the half already
//    holds.  P never leaves its lane.  V is turned while it is staged: a
//    thread loads the 8 keys of one such slot group for a few value columns,
//    transposes them in registers and writes 16-byte pieces of V^T.
//  - Two halves of 32 keys per tile make a pipeline: while the vector unit
//    turns one half's scores into weights, the matrix unit multiplies the
//    previous half's weights with its values and the queries with the next
//    half's keys.  The two kinds of instruction are interleaved in one block:
//    at D = 128 they cost about the same (16 matrix instructions of 32 cycles;
//    16 exponentials of 16 and some 45 others of 4 cycles).
//  - Weights are taken against a reference that is only moved when a half's
//    weights sum to more than 2^10 times the reference's own in some lane; the
//    sum is needed anyway, and a sum of positive numbers bounds each of them,
//    so the maximum of the scores is not computed otherwise.  The reference
//    starts at minus infinity, which makes the first sum infinite or NaN: not
//    below any bound.
//  - 16-bit weights are rounded to the element type for the product with V (a
//    matrix instruction takes both operands in one type): relative error up
//    to 2^-8 (bf16) or 2^-11 (f16) each, the size of the output's own rounding.
//    Their sum is taken before that, in fp32.  f16 ends at 2^-24: its weights
//    are 2^5 times larger (the reference lies that much below the maximum), up
//    to 2^15, so that what is dropped of a small one is 2^-30 of the largest:
//    many keys of small weight beside one of a large one still add up.
// LDS rows are spread over the banks by an exclusive-or of the 16-byte piece
// with row bits.  K and V have two buffers each; tiles travel through
// registers, from the moment that the tile before is written to LDS until a
// whole tile later.  One barrier per tile: K of tile t + 1 is written before
// it and read behind it, V is written behind it and read behind the next one.
//
// 64 heads of 4000 x 2000 positions, D = 128, bf16: 305 us, 860 TFLOP/s, and
// 4096 x 4096: 548 us, 1000 TFLOP/s (a plain library product of 8192^3 reaches
// 1200 on the same card).  The counters say 45 % matrix unit, 42 % vector unit,
// half of either beside the other; the rest is waves waiting for the two, and
// a tenth the starts and ends of workgroups.  Tried: loads behind conditions
// (the compiler then waits for all of them at every store, 333 us), operands
// read right before their use (350), 3 workgroups per compute unit at D = 64
// (spills: 243 against 174), wave priorities (no difference).
// The 16-bit kernels for D up to 128 and 256 need more registers than there are:
// 7 (bf16) and 8 (f16), 6 and 2, live in scratch memory.  At D = 128 bf16 touches
// them outside the loop only; f16 reads one back in it, behind loads that it
// then waits for: 331 us against 304 for the call above.
//
// Chunk calls (CHUNK: the new rows of sequences over the paged cache, in causal
// order) differ in three things.  A workgroup finds its sequence by a scan over
// their numbers of rows, so that ragged batches take as many workgroups as they
// have row tiles.  Rows of keys and values lie in pages: the offsets of a tile's
// keys go through LDS, one tile ahead of their loads.  And every row has its own
// last (and, in a window, first) key: tiles that some row does not see whole hide
// scores per lane.  Waves without a row only move tiles.
// Loads are of 64-bit addresses (a cache may be larger than 4 GB), and the offsets
// of K's pieces in LDS are turned on their way, so that as many registers are left
// as the other form has: what lies in scratch memory is not read in the loop (where
// it is, it waits behind the loads in flight: 1590 us against 1518 below).
// 8 ragged prompts of 19.4 k rows over up to 8192 slots, 32 heads on 8, D = 128, bf16:
// 1518 us, 855 TFLOP/s; 2 x 4096 rows over 32768, 24 heads on 4, f16: 3640 us, 850.
// 32 heads of 4 x 2048 rows over 8192, bf16: D = 32 450 TFLOP/s, 64 717, 96 770, 128
// 913, 256 615; one sequence in fp32: 100, 116, 99, 109.

#pragma once

#include "attn_chunk.h"
#include "attn_mma.h"
#include "block_internal.h"

namespace ctconv {
namespace block {

namespace {

using mfma::u32x2;
using mfma::u32x4;

constexpr int kThreads = 256;
constexpr float kMostSum = 1024.f;
// log2 of the weight that a maximum gets when the reference moves to it
template <class TR>
constexpr float kTopWeight = 0.f;
template <>
constexpr float kTopWeight<TF16> = 5.f;
constexpr int kAhead = 4;  // LDS operands read ahead of their instruction

// DP: values of a row in LDS; DU of them are used (a multiple of 32).
template <class TR, int DP, int DU = DP>
struct Shape {
    static constexpr int ES = sizeof(typename TR::storage);
    static constexpr int VEC = 16 / ES;
    static constexpr int KT = 64;                       // keys per tile
    static constexpr int ROW = DP * ES;                 // bytes of a K row in LDS
    static constexpr int BYTES = KT * ROW;              // of a tile of K, or of V
    static constexpr int LDS = 4 * BYTES;
    static constexpr int PER_CU = LDS > (80 << 10) ? 1 : 2;  // workgroups per compute unit
    static constexpr int NF = DU / (2 * VEC);           // 16-byte pieces of a key per half
    static constexpr int ND = DU / 32;                  // output tiles
    static constexpr int PIECES = DP / VEC;             // 16-byte pieces of a row
    static constexpr int LOADS = BYTES / (16 * kThreads);
    static constexpr int VD = ES == 2 ? DP / 32 : 1;    // 16-bit: value columns per thread
};

// f(i) for i in [FROM, TO), i a constant.
template <int FROM, int TO, class F>
__device__ __forceinline__ void unrolled(F f) {
    if constexpr (FROM < TO) {
        f(std::integral_constant<int, FROM>{});
        unrolled<FROM + 1, TO>(f);
    }
}

// A half's weights: packed pairs in 16 bits, or as they are.
template <class TR>
struct Weights {
    u32x4 v[2];
};
template <>
struct Weights<TF32> {
    f32x16 v;
};

// EXACT: D = DP (else K pieces past the row are zeroed on their way).
// CHUNK: the new rows of sequences over the paged cache (see above).
template <class TR, int DP, bool EXACT, bool CHUNK = false, int DU = DP>
__global__ __launch_bounds__(kThreads, (Shape<TR, DP>::PER_CU)) void tile_kernel(AttnArgs a) {
    using S = typename TR::storage;
    using Sh = Shape<TR, DP, DU>;
    constexpr int ES = Sh::ES, VEC = Sh::VEC, KT = Sh::KT, NF = Sh::NF, ND = Sh::ND;
    constexpr int PIECES = Sh::PIECES, LOADS = Sh::LOADS, VD = Sh::VD;
    extern __shared__ __align__(16) char lds[];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 31, half = lane >> 5;
    int split, tile, bh, b, h, start, n, rows = a.R;
    ChunkRows cr;
    int slot0 = 0;                     // CHUNK: slot of the first key
    int all_from = 0, all_to = 0;      // CHUNK: the keys that every row of the tile sees
    bool direct = a.direct;
    if constexpr (CHUNK) {
        if (!chunk_item(a, kThreads / 64, block_number(), true, b, h, tile, split)) return;
        bh = 0;
        cr = chunk_rows(a, b);
        rows = cr.live * a.G;
        const int last = tile * 128 + 127 < rows ? tile * 128 + 127 : rows - 1;
        const int i0 = (int)fdiv((uint32_t)(tile * 128), a.fd_G);
        const int i1 = (int)fdiv((uint32_t)last, a.fd_G);
        int first, span;
        chunk_span(a, cr, i0, i1, first, span);
        start = split * a.chunk;
        if (split > 0 && start >= span) return;
        direct = span <= a.chunk;
        n = span - start;
        slot0 = first + start;
        all_from = a.window > 0 ? cr.off + i1 + 1 - a.window - slot0 : 0;
        all_to = cr.off + i0 + 1 - slot0;
    } else {
        // (sequence, head) pairs stay on one XCD: their keys are read from its L2
        // by all of their row tiles.
        const uint32_t per = ((uint32_t)(a.B * a.Hkv * a.row_tiles * a.splits) + 7) >> 3;
        const uint32_t number = block_number();
        if (number >= 8 * per) return;
        int item = (int)((number & 7) * per + (number >> 3));
        split = item % a.splits;
        item /= a.splits;
        tile = item % a.row_tiles;
        bh = item / a.row_tiles;
        if (bh >= a.B * a.Hkv) return;
        b = bh / a.Hkv;
        h = bh - b * a.Hkv;

        const int len = a.lengths ? clamped(a.lengths[b], a.Lk) : a.Lk;
        start = split * a.chunk;
        if (a.splits > 1 && start >= len) return;
        n = len - start;
    }
    n = n < a.chunk ? n : a.chunk;

    int row = tile * 128 + wave * 32 + col;
    bool live = row < rows;
    int lq = live ? (int)fdiv((uint32_t)row, a.fd_G) : 0;
    int hq = h * a.G + (live ? row - lq * a.G : 0);
    // CHUNK: the keys that this lane's row sees; whether the wave has no row at all
    const int my_end = CHUNK ? cr.off + lq + 1 - slot0 : 0;
    const int my_begin = CHUNK && a.window > 0 ? my_end - a.window : 0;
    const bool idle = CHUNK && tile * 128 + wave * 32 >= rows;

    u32x4 qf[NF];
    {
        const int64_t from = CHUNK && a.row_starts ? cr.row0 * a.q_row : b * a.q_b;
        const S* qr = static_cast<const S*>(a.q) + from + lq * a.q_row + hq * a.q_head;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int d = (2 * f + half) * VEC;
            qf[f] = u32x4{0, 0, 0, 0};
            if (live && (EXACT || d < a.D)) {
                qf[f] = *reinterpret_cast<const u32x4*>(qr + d);
                const uint32_t flip = a.negate ? (ES == 2 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[f][i] ^= flip;
            }
        }
    }

    const S* kb = static_cast<const S*>(a.k) +
                  (CHUNK ? h * a.pages.head_stride
                         : b * a.k_b + h * a.k_head + (int64_t)start * a.k_row);
    const S* vb = static_cast<const S*>(a.v) +
                  (CHUNK ? h * a.pages.head_stride
                         : b * a.v_b + h * a.v_head + (int64_t)start * a.v_row);
    const uint8_t* mask = !CHUNK && a.mask ? a.mask + b * a.mask_stride + start : nullptr;
    // always read, so that every tile issues the same loads (see `step`)
    const uint8_t* seen_from = mask ? mask : reinterpret_cast<const uint8_t*>(a.q);

    // What of a tile this thread moves.  K (and fp32 V): piece k_c of keys
    // k_key + i * KSTEP.  16-bit V: columns v_d .. v_d + VD of the 8 keys of
    // slot group v_group (step v_group / 2, half v_group % 2).
    constexpr int KSTEP = kThreads / PIECES;
    const int k_key = tid / PIECES, k_c = tid % PIECES;
    const int k_d = k_c * VEC < a.D ? k_c * VEC : 0;  // pieces past the row: read, not used
    const bool k_past = k_c * VEC >= a.D;
    constexpr int VDW = ES == 2 ? VD / 2 : 1;
    constexpr int VCOLS = DP / VD;
    const int v_group = tid / VCOLS, v_d = (tid % VCOLS) * VD;
    const int v_from = v_d < a.D ? v_d : 0;
    const auto v_key = [&](int j) __attribute__((always_inline)) {
        return 16 * (v_group >> 1) + 4 * (v_group & 1) + 8 * (j >> 2) + (j & 3);
    };
    // Byte offsets of this thread's pieces from the tile's first key.  Tiles
    // start every 64 keys, the last one where it ends with the keys: the keys
    // that it repeats are not seen again.  Only a single short tile reads the
    // last key in the place of those behind it.
    uint32_t k_off[LOADS], v_off[ES == 2 ? 8 : LOADS];
#pragma unroll
    for (int i = 0; i < LOADS && !CHUNK; ++i) {
        const int key = k_key + i * KSTEP < n ? k_key + i * KSTEP : n - 1;
        k_off[i] = (uint32_t)((key * a.k_row + k_d) * ES);
        if (ES == 4) v_off[i] = (uint32_t)((key * a.v_row + k_d) * ES);
    }
    if constexpr (ES == 2 && !CHUNK) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int key = v_key(j) < n ? v_key(j) : n - 1;
            v_off[j] = (uint32_t)((key * a.v_row + v_from) * ES);
        }
    }
    u32x4 kr[LOADS];
    uint32_t vr[ES == 2 ? 8 * VDW : 1];
    u32x4 vr4[ES == 4 ? LOADS : 1];
    uint32_t seen_byte;

    const int tiles = n > 0 ? (n + KT - 1) / KT : 0;
    const int last_t0 = n > KT ? n - KT : 0;
    // first key of tile t; behind the last tile, the last one's
    const auto first_key = [&](int t) __attribute__((always_inline)) {
        return t * KT < last_t0 ? t * KT : last_t0;
    };
    // A tile as a buffer: uniform base, 32-bit offsets per lane, which are in
    // bounds by themselves.
    const auto tile_of = [](const S* base) __attribute__((always_inline)) {
        return __builtin_amdgcn_make_buffer_rsrc(mfma::uniform_ptr(base), 0, 0xFFFFFFFFu,
                                                 mfma::kBufferWord3);
    };
    // CHUNK: byte offsets of the rows of four tiles' keys, [tile % 4][key].
    // Tile t + 3's are written while tile t is worked on (each wave a quarter, from
    // the page that it asked for a tile before), before the barrier; what they
    // replace was read last two barriers ago.
    int64_t* const ring = reinterpret_cast<int64_t*>(lds + Sh::LDS);
    int32_t page = 0, place = -1;  // of this lane's key of the tile asked for; -1: no key
    uint64_t seen_next[3] = {0, 0, 0};  // of the tile after this one and the ones after that
    const uint64_t page_bytes = (uint64_t)a.pages.page_stride * ES;
    const uint64_t slot_bytes = (uint64_t)a.pages.slot_stride * ES;
    const int32_t* const table = a.pages.table + b * a.pages.table_stride;
    const auto ask_page = [&](int t) __attribute__((always_inline)) {
        const int key = t * KT + lane;
        const int slot = slot0 + (key < n ? key : n - 1);
        const int column = (int)fdiv((uint32_t)slot, a.pages.fd_page);
        place = key < n ? slot - column * a.pages.page_size : -1;
        page = table[column];
    };
    const auto put_offsets = [&](int t) __attribute__((always_inline)) {
        const bool is = place >= 0 && (uint32_t)page < (uint32_t)a.pages.num_pages;
        const uint32_t p = is ? page : 0, q = is ? place : 0;
        uint64_t at = (uint64_t)p * (uint32_t)page_bytes + (uint64_t)q * (uint32_t)slot_bytes;
        if ((page_bytes | slot_bytes) >> 32)
            at += (uint64_t)(p * (uint32_t)(page_bytes >> 32) + q * (uint32_t)(slot_bytes >> 32))
                  << 32;
        if (lane >> 4 == wave) ring[(t & 3) * KT + lane] = (int64_t)at;
        seen_next[0] = seen_next[1];
        seen_next[1] = seen_next[2];
        seen_next[2] = __ballot(is);
    };
    const char* const k_from = reinterpret_cast<const char*>(kb + k_d);
    const char* const v_from4 = reinterpret_cast<const char*>(vb + (ES == 2 ? v_from : k_d));
    const auto load_k = [&](int t) __attribute__((always_inline)) {
        if constexpr (CHUNK) {
            const int64_t* off = ring + (t & 3) * KT + k_key;
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                kr[i] = *reinterpret_cast<const u32x4*>(k_from + off[i * KSTEP]);
            return;
        }
        const auto from = tile_of(kb + first_key(t) * a.k_row);
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            kr[i] = __builtin_amdgcn_raw_buffer_load_b128(from, k_off[i], 0, 0);
    };
    const auto load_v = [&](int t) __attribute__((always_inline)) {
        if constexpr (CHUNK) {
            const int64_t* off = ring + (t & 3) * KT;
            if constexpr (ES == 2) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const char* from = v_from4 + off[v_key(j)];
                    if constexpr (VDW == 1) {
                        vr[j] = *reinterpret_cast<const uint32_t*>(from);
                    } else if constexpr (VDW == 2) {
                        const u32x2 w = *reinterpret_cast<const u32x2*>(from);
                        vr[2 * j] = w[0];
                        vr[2 * j + 1] = w[1];
                    } else {
                        const u32x4 w = *reinterpret_cast<const u32x4*>(from);
#pragma unroll
                        for (int q = 0; q < 4; ++q) vr[4 * j + q] = w[q];
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < LOADS; ++i)
                    vr4[i] = *reinterpret_cast<const u32x4*>(v_from4 + off[k_key + i * KSTEP]);
            }
            return;
        }
        const int t0 = first_key(t);
        const auto from = tile_of(vb + t0 * a.v_row);
        const int key = t0 + lane < n ? t0 + lane : n - 1;
        seen_byte = seen_from[mask ? key : 0];
        if constexpr (ES == 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (VDW == 1) {
                    vr[j] = __builtin_amdgcn_raw_buffer_load_b32(from, v_off[j], 0, 0);
                } else if constexpr (VDW == 2) {
                    const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(from, v_off[j], 0, 0);
                    vr[2 * j] = w[0];
                    vr[2 * j + 1] = w[1];
                } else {
                    const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(from, v_off[j], 0, 0);
#pragma unroll
                    for (int q = 0; q < 4; ++q) vr[4 * j + q] = w[q];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                vr4[i] = __builtin_amdgcn_raw_buffer_load_b128(from, v_off[i], 0, 0);
        }
    };
    // Which keys of tile t (loaded last) are seen: not in the tile before, not
    // past the end, not masked.
    const auto seen_keys = [&](int t) __attribute__((always_inline)) {
        const int key = first_key(t) + lane;
        return __ballot(key >= t * KT && key < n && (!mask || seen_byte != 0));
    };
    // K rows of DP values: piece c of row r at c ^ (r % 16)
    const uint32_t k_to = k_key * Sh::ROW + ((k_c ^ (k_key & 15 & (PIECES - 1))) << 4);
    static_assert(KSTEP % 16 == 0 || PIECES >= 32 || KSTEP * 2 == 16 || KSTEP == 4, "row bits");
    const auto store_k = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            if (!EXACT && k_past) kr[i] = u32x4{0, 0, 0, 0};
            const int key = k_key + i * KSTEP;
            const uint32_t to =
                KSTEP % 16 == 0 ? k_to + i * KSTEP * Sh::ROW
                                : key * Sh::ROW + ((k_c ^ (key & 15 & (PIECES - 1))) << 4);
            *reinterpret_cast<u32x4*>(lds + buf + to) = kr[i];
        }
    };
    // CHUNK: a hidden value's weight is 0, but 0 times an infinity or a NaN is NaN.
    // Tiles that not every row sees whole go without such values; they are added to
    // the rows that see them at the end.  (Keys that are not there read slot 0 of page
    // 0, another request's: they are zero before that, or its NaN would cost this call
    // the loop at the end.  Two sequences of 128 rows of 32 heads on 8 over 8000 keys,
    // bf16: 155 us with it, 65 without.)
    int* const odd_values = reinterpret_cast<int*>(ring + 4 * KT);
    const auto store_v = [&](int buf, uint64_t seen, int t) __attribute__((always_inline)) {
        if constexpr (ES == 2)
            if (seen != ~0ull) {
                // what an unseen key's row holds may be NaN: zero, not 0 * NaN
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (!((seen >> v_key(j)) & 1))
#pragma unroll
                        for (int w = 0; w < VDW; ++w) vr[VDW * j + w] = 0;
            }
        if constexpr (CHUNK)
            if (t * KT < all_from || t * KT + KT > all_to) {
                uint32_t odd = 0;
                if constexpr (ES == 2) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int w = 0; w < VDW; ++w) odd |= take_odd<TR>(vr[VDW * j + w]);
                } else {
#pragma unroll
                    for (int i = 0; i < LOADS; ++i)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            uint32_t u = (seen >> (k_key + i * KSTEP)) & 1 ? vr4[i][w] : 0;
                            odd |= take_odd<TR>(u);
                            vr4[i][w] = u;
                        }
                }
                if (odd) *odd_values = 1;
            }
        if constexpr (ES == 2) {
            // V^T rows of 64 keys: slot group c of row d at c ^ (d / 2) ^ (d / 16)
#pragma unroll
            for (int r = 0; r < VD; ++r) {
                const unsigned sel = (r & 1) ? 0x07060302u : 0x05040100u;
                u32x4 o;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    o[w] = __builtin_amdgcn_perm(vr[VDW * (2 * w + 1) + (r >> 1)],
                                                 vr[VDW * (2 * w) + (r >> 1)], sel);
                const int d = v_d + r;
                const int c = (v_group ^ (d >> 1) ^ (d >> 4)) & 7;
                *reinterpret_cast<u32x4*>(lds + buf + d * (KT * 2) + (c << 4)) = o;
            }
        } else {
            // V rows, the pieces of every other 4 keys moved by 32 values
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int key = k_key + i * KSTEP;
                const u32x4 w = (seen >> key) & 1 ? vr4[i] : u32x4{0, 0, 0, 0};
                *reinterpret_cast<u32x4*>(lds + buf + key * Sh::ROW +
                                          ((k_c ^ (((key >> 2) & 1) << 3)) << 4)) = w;
            }
        }
    };

    f32x16 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
    float m = -__builtin_huge_valf(), l = 0.f;

    // LDS offsets of this lane's operands; what else varies is constant.  Piece f of a
    // key lies at the first one's offset with bits of f turned, value tile i the
    // same: CHUNK, which is short of registers, keeps the first ones only.
    constexpr int KAT = CHUNK ? 1 : NF > 8 ? 8 : NF, VAT = CHUNK && ES == 2 ? 1 : 4;
    uint32_t k_at[KAT];
#pragma unroll
    for (int f = 0; f < KAT; ++f)
        k_at[f] = col * Sh::ROW + (((2 * f + half) ^ (col & 15 & (PIECES - 1))) << 4);
    uint32_t v_at[VAT];
#pragma unroll
    for (int i = 0; i < VAT; ++i)
        v_at[i] = ES == 2 ? col * (KT * 2) +
                                (((2 * i + half) ^ (((col >> 1) ^ (col >> 4)) & 7)) << 4)
                          : 4 * half * Sh::ROW + ((col + (((i ^ half) & 1) << 5)) << 2);
    // (volatile, or the turned ones are computed ahead of the loop and kept)
    const auto turned = [](uint32_t at, int f) __attribute__((always_inline)) {
        uint32_t to;
        asm volatile("v_xor_b32 %0, %1, %2" : "=v"(to) : "i"(f << 5), "v"(at));
        return to;
    };
    const auto k_piece_at = [&](int f) __attribute__((always_inline)) {
        if constexpr (CHUNK) return f == 0 ? k_at[0] : turned(k_at[0], f);
        else return k_at[f];
    };
    const auto v_piece_at = [&](int i) __attribute__((always_inline)) {
        if constexpr (VAT == 1) return i == 0 ? v_at[0] : turned(v_at[0], i);
        else return v_at[i];
    };

    // Operands and instructions of S_new = K Q^T, piece f of half kh.
    const auto k_piece = [&](int kbuf, int kh, int f) __attribute__((always_inline)) {
        // pieces 8 and up (rows of 512 bytes and more) repeat the pattern of
        // the low four bits 256 bytes on
        return *reinterpret_cast<const u32x4*>(lds + kbuf + kh * 32 * Sh::ROW + k_piece_at(f & 7) +
                                               (f >> 3) * 256);
    };
    // Of acc += V^T P^T, i of a half: 16-bit, step i / ND, output tile i % ND;
    // fp32, key i / ND, output tile i % ND.
    constexpr int PV = ES == 2 ? 2 * ND : 16 * ND;
    const auto v_piece = [&](int vbuf, int vh, int i) __attribute__((always_inline)) {
        // slot group 2 (2 vh + step) + half, row 32 d + col: the row bits
        // above col move it by 2 d
        const int d = i % ND, st = i / ND;
        return *reinterpret_cast<const u32x4*>(lds + vbuf + d * 32 * (KT * 2) +
                                               v_piece_at(((2 * vh + st) ^ d) & 3));
    };
    const auto v_value = [&](int vbuf, int vh, int i) __attribute__((always_inline)) {
        const int d = i % ND, st = i / ND;
        const int key = 32 * vh + 8 * (st >> 2) + (st & 3);
        return *reinterpret_cast<const float*>(lds + vbuf + key * Sh::ROW + v_at[d & 1] +
                                               (d >> 1) * 256);
    };
    const auto hide = [&](f32x16& s, uint32_t bits, int at) __attribute__((always_inline)) {
        if constexpr (CHUNK) {
            if (at < all_from || at + 32 > all_to)
                bits &= low_bits(my_end - at) & ~low_bits(my_begin - at);
            if (!__any(bits != 0xFFFFFFFFu)) return;
        } else {
            if (bits == 0xFFFFFFFFu) return;
        }
        const uint32_t w = bits >> (4 * half);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int at_bit = 8 * (i >> 2) + (i & 3);
            if constexpr (CHUNK) {
                // (bits that differ by lane: no compare masks, the scalar registers are full)
                const uint32_t keep = __builtin_amdgcn_sbfe((int)w, at_bit, 1);
                s[i] = __uint_as_float((__float_as_uint(s[i]) & keep) | (0xFF800000u & ~keep));
            } else {
                if (!((w >> at_bit) & 1)) s[i] = -__builtin_huge_valf();
            }
        }
    };
    // The weights of s against the reference m (slices of the pipeline below).
    const float c = a.c;
    const auto weigh = [&](const f32x16& s, int i, Weights<TR>& p, float (&sum)[2], float& prev) {
        // (the sum takes the weight before: an exponential is not ready at once)
        if (i > 0) sum[i & 1] += prev;
        const float e = exp2_fast(fmaf(s[i], c, -m));
        if constexpr (ES == 2) {
            if (i & 1) p.v[i >> 3][(i >> 1) & 3] = mfma::pack2<TR>(prev, e);
        } else {
            p.v[i] = e;
        }
        prev = e;
        if (i == 15) sum[0] += e;
    };
    // After a half's weights: keep them, or move the reference and repeat.
    const auto settle = [&](const f32x16& s, Weights<TR>& p, float (&sum)[2]) {
        float total = sum[0] + sum[1];
        if (__any(!(total <= kMostSum * (1 << (int)kTopWeight<TR>)))) {
            float top = -__builtin_huge_valf();
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[i]);
            top *= c;
            top = fmaxf(top, __shfl_xor(top, 32));
            const float up = fmaxf(m, top - kTopWeight<TR>);
            // nothing seen yet: weights and sum stay zero, or become NaN where a
            // score is
            const bool none = up == -__builtin_huge_valf();
            const float f = none || m == up ? 1.f : exp2_fast(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[d][i] *= f;
            total = 0.f;
            float prev = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e = exp2_fast(none ? s[i] : fmaf(s[i], c, -up));
                total += e;
                if constexpr (ES == 2) {
                    if (i & 1) p.v[i >> 3][(i >> 1) & 3] = mfma::pack2<TR>(prev, e);
                    prev = e;
                } else {
                    p.v[i] = e;
                }
            }
        }
        l += total;
    };
    const auto zero = [](f32x16& s) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.f;
    };
    // s_new = K Q^T of a half, acc += V^T P^T of another, p = weights of s.
    const auto stage = [&](int kbuf, int kh, f32x16& s_new, int vbuf, int vh,
                           const Weights<TR>& p_old, const f32x16& s, Weights<TR>& p) __attribute__((always_inline)) {
        if (CHUNK && idle) return;
        zero(s_new);
        float sum[2] = {0.f, 0.f}, prev = 0.f;
        if constexpr (ES == 2) {
            // Operand k (K and V in turn) is read AHEAD instructions before
            // its use: the compiler, left alone, reads each right before it
            // and waits for LDS every time.  Nothing moves across the barriers
            // between the steps.
            constexpr int MM = NF + PV, AHEAD = kAhead;
            static_assert(NF == PV, "K and V in turn");
            const auto piece = [&](auto k) __attribute__((always_inline)) {
                if constexpr (k % 2 == 0) return k_piece(kbuf, kh, k / 2);
                else return v_piece(vbuf, vh, k / 2);
            };
            u32x4 ring[AHEAD];
            unrolled<0, AHEAD>([&](auto k) __attribute__((always_inline)) { ring[k] = piece(k); });
            __builtin_amdgcn_sched_barrier(0);
            unrolled<0, MM>([&](auto k) __attribute__((always_inline)) {
                if constexpr (k % 2 == 0)
                    Mma32<TR>::step(s_new, ring[k % AHEAD], qf[k / 2]);
                else
                    Mma32<TR>::step(acc[(k / 2) % ND], ring[k % AHEAD], p_old.v[(k / 2) / ND]);
                if constexpr (k + AHEAD < MM)
                    ring[k % AHEAD] = piece(std::integral_constant<int, k + AHEAD>{});
                unrolled<k * 16 / MM, (k + 1) * 16 / MM>([&](auto i) __attribute__((always_inline)) {
                    weigh(s, i, p, sum, prev);
                });
                __builtin_amdgcn_sched_barrier(0);
            });
        } else {
            // the same with one value of a key piece and one of V per step
            constexpr int AHEAD = 2 * kAhead;
            static_assert(4 * NF == PV, "K and V in turn");
            u32x4 keys[2];
            float ring[AHEAD];
            keys[0] = k_piece(kbuf, kh, 0);
            unrolled<0, AHEAD>([&](auto k) __attribute__((always_inline)) {
                ring[k] = v_value(vbuf, vh, k);
            });
            __builtin_amdgcn_sched_barrier(0);
            unrolled<0, PV>([&](auto k) __attribute__((always_inline)) {
                if constexpr (k % 4 == 0 && k / 4 + 1 < NF)
                    keys[(k / 4 + 1) % 2] = k_piece(kbuf, kh, k / 4 + 1);
                s_new = __builtin_amdgcn_mfma_f32_32x32x2f32(
                    __uint_as_float(keys[k / 4 % 2][k % 4]), __uint_as_float(qf[k / 4][k % 4]), s_new,
                    0, 0, 0);
                acc[k % ND] = __builtin_amdgcn_mfma_f32_32x32x2f32(ring[k % AHEAD], p_old.v[k / ND],
                                                                   acc[k % ND], 0, 0, 0);
                if constexpr (k + AHEAD < PV) ring[k % AHEAD] = v_value(vbuf, vh, k + AHEAD);
                unrolled<k * 16 / PV, (k + 1) * 16 / PV>([&](auto i) __attribute__((always_inline)) {
                    weigh(s, i, p, sum, prev);
                });
                __builtin_amdgcn_sched_barrier(0);
            });
        }
        settle(s, p, sum);
    };

    const auto k_buf = [](int i) __attribute__((always_inline)) { return i * Sh::BYTES; };
    const auto v_buf = [](int i) __attribute__((always_inline)) { return (2 + i) * Sh::BYTES; };
    if (tiles > 0) {
        uint64_t bits;
        f32x16 sa, sb;
        Weights<TR> pa, pb;
        if constexpr (CHUNK) {
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                ask_page(t);
                put_offsets(t);
            }
            ask_page(3);
            if (tid == 0) *odd_values = 0;
            __syncthreads();
        }
        load_k(0);
        load_v(0);
        bits = CHUNK ? seen_next[0] : seen_keys(0);
        store_k(k_buf(0));
        store_v(v_buf(0), bits, 0);
        if constexpr (ES == 2) {
#pragma unroll
            for (int i = 0; i < 8 * VDW; ++i) vr[i] = 0;
            pb.v[0] = pb.v[1] = u32x4{0, 0, 0, 0};
        } else {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) vr4[i] = u32x4{0, 0, 0, 0};
            zero(pb.v);
        }
        store_v(v_buf(1), ~0ull, 0);  // "tile -1": zeros times zeros
        load_k(1);
        load_v(1);
        __syncthreads();
        zero(sa);
        unrolled<0, NF>([&](auto f) __attribute__((always_inline)) {
            Mma32<TR>::step(sa, k_piece(k_buf(0), 0, f), qf[f]);
        });
        const auto step = [&](int t, auto parity) __attribute__((always_inline)) {
            constexpr int P = decltype(parity)::value;
            // Loads and stores without a condition: behind the last tile they
            // repeat it.  (With one, the compiler cannot count the loads in
            // flight, and every store waits for all of them.)
            store_k(k_buf(P ^ 1));
            load_k(t + 2);
            if constexpr (CHUNK) {
                put_offsets(t + 3);
                ask_page(t + 4);
            }
            hide(sa, (uint32_t)bits, t * KT);
            stage(k_buf(P), 1, sb, v_buf(P ^ 1), 1, pb, sa, pa);
            __syncthreads();
            const uint32_t late = (uint32_t)(bits >> 32);
            bits = CHUNK ? seen_next[0] : seen_keys(t + 1);
            store_v(v_buf(P ^ 1), bits, t + 1);
            load_v(t + 2);
            hide(sb, late, t * KT + 32);
            // behind the last tile: scores that are not used
            stage(k_buf(P ^ 1), 0, sa, v_buf(P), 0, pa, sb, pb);
        };
        for (int t = 0; t < tiles; t += 2) {
            step(t, std::integral_constant<int, 0>{});
            if (t + 1 < tiles) step(t + 1, std::integral_constant<int, 1>{});
        }
        const int last = v_buf((tiles - 1) & 1);
        unrolled<0, PV>([&](auto i) __attribute__((always_inline)) {
            if constexpr (ES == 2)
                Mma32<TR>::step(acc[i % ND], v_piece(last, 1, i), pb.v[i / ND]);
            else
                acc[i % ND] = __builtin_amdgcn_mfma_f32_32x32x2f32(v_value(last, 1, i), pb.v[i / ND],
                                                                   acc[i % ND], 0, 0, 0);
        });
    }
    if constexpr (CHUNK) {
        // What was taken out of the values of tiles that not every row sees whole.
        __syncthreads();
        if (*odd_values) {
            // [0, whole_from) and [whole_to, n)
            const int whole_from = (all_from > 0 ? all_from + KT - 1 : 0) & ~(KT - 1);
            const int whole_to = all_to & ~(KT - 1);
            for (int key = 0; key < n; ++key) {
                if (key == whole_from && whole_to > key) key = whole_to;
                if (key >= n) break;
                const int64_t at = slot_offset(a.pages, b, slot0 + key);
                if (at < 0) continue;
                const bool sees = key >= my_begin && key < my_end;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // (what lies past a row's end goes to columns that are not written)
                        const int at_d = 32 * d + 8 * i + 4 * half;
                        S v[4];
                        const S* from = vb + at + (EXACT || at_d < a.D ? at_d : 0);
                        if constexpr (ES == 2)
                            *reinterpret_cast<u32x2*>(v) = *reinterpret_cast<const u32x2*>(from);
                        else
                            *reinterpret_cast<u32x4*>(v) = *reinterpret_cast<const u32x4*>(from);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = TR::to_f32(v[e]);
                            acc[d][4 * i + e] += sees && !(fabsf(x) <= __FLT_MAX__) ? x : 0.f;
                        }
                    }
            }
        }
    }
    l += __shfl_xor(l, 32);
    // CHUNK: the row's numbers again (kept, they would hold registers in the loop)
    if constexpr (CHUNK) {
        int here = tile * 128 + (int)threadIdx.x / 64 * 32 + ((int)threadIdx.x & 31);
        asm volatile("" : "+v"(here));
        row = here;
        live = row < rows;
        lq = live ? (int)fdiv((uint32_t)row, a.fd_G) : 0;
        hq = h * a.G + (live ? row - lq * a.G : 0);
    }
    if (!live) return;
    if (direct) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t o_from = CHUNK && a.row_starts ? cr.row0 * a.o_row : b * a.o_b;
        S* to = static_cast<S*>(a.out) + o_from + lq * a.o_row + hq * a.o_head;
        if constexpr (CHUNK) {
            if (half == 0) write_lse(a, (cr.row0 + lq) * a.Hq + hq, m, l);
        } else if (a.lse && half == 0)
            a.lse[((int64_t)b * a.Hq + hq) * a.Lq + lq] = m * kLn2 + logf(l);
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at_d = 32 * d + 8 * i + 4 * half;
                if (at_d >= a.D) continue;
                if constexpr (ES == 2) {
                    u32x2 w{mfma::pack2<TR>(acc[d][4 * i] * inv, acc[d][4 * i + 1] * inv),
                            mfma::pack2<TR>(acc[d][4 * i + 2] * inv, acc[d][4 * i + 3] * inv)};
                    *reinterpret_cast<u32x2*>(to + at_d) = w;
                } else {
                    *reinterpret_cast<f32x4*>(to + at_d) =
                        f32x4{acc[d][4 * i] * inv, acc[d][4 * i + 1] * inv, acc[d][4 * i + 2] * inv,
                              acc[d][4 * i + 3] * inv};
                }
            }
    } else {
        const int64_t part = CHUNK ? ((cr.row0 + lq) * a.Hq + hq) * a.splits + split
                                   : ((int64_t)bh * a.splits + split) * a.R + row;
        if (half == 0) {
            a.part_ml[2 * part] = m;
            a.part_ml[2 * part + 1] = l;
        }
        float* to = a.part_o + part * a.D;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at_d = 32 * d + 8 * i + 4 * half;
                if (at_d < a.D)
                    *reinterpret_cast<f32x4*>(to + at_d) =
                        f32x4{acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2],
                              acc[d][4 * i + 3]};
            }
    }
}

}  // namespace
}  // namespace block
}  // namespace ctconv
