// Host program for the sanitizer tier of the decoder-block operators: the C
// entry points (validation, plans, workspace sizes) over seeded shapes, valid
// and invalid, with the launchers replaced by checks of what the planners
// hand to the kernels.  No GPU call is made.  Prints "ok <launches>".
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "block_internal.h"

using namespace ctconv;
using namespace ctconv::block;

static long launches = 0;
static const char* ws_lo = nullptr;
static size_t ws_size = 0;
static int64_t span_bound = 0;

#define EXPECT(cond)                                                 \
    do {                                                             \
        if (!(cond)) {                                               \
            std::printf("failed at line %d: %s\n", __LINE__, #cond); \
            std::exit(1);                                            \
        }                                                            \
    } while (0)

static bool inside(const void* p, int64_t bytes) {
    const char* c = static_cast<const char*>(p);
    return c >= ws_lo && bytes >= 0 && c + bytes <= ws_lo + ws_size;
}

static void check_attention(const AttnArgs& a, int row_tile) {
    ++launches;
    EXPECT(a.B > 0 && a.G >= 1 && a.R == a.Lq * a.G && a.Hq == a.G * a.Hkv);
    EXPECT(a.splits >= 1 && a.chunk >= 128 && a.chunk % 128 == 0);
    EXPECT((int64_t)a.chunk * a.splits >= span_bound);
    EXPECT((int64_t)a.row_tiles * row_tile >= a.R);
    EXPECT((int64_t)a.B * a.Hkv * a.row_tiles * a.splits <= INT32_MAX - 8);
    EXPECT(a.c > 0.f && std::isfinite(a.c));
    if (!a.direct) {
        const int64_t parts = (int64_t)a.B * a.Hkv * a.R * a.splits;
        EXPECT(inside(a.part_o, parts * a.D * 4));
        EXPECT(inside(a.part_ml, parts * 8));
    }
    if (a.weight_sum) {
        EXPECT(!a.direct && a.score_stride % 128 == 0 && a.score_stride >= span_bound);
        EXPECT(inside(a.scores, (int64_t)a.B * a.Hkv * a.R * a.score_stride * 4));
    }
}

namespace ctconv {
namespace block {
hipError_t launch_append(const AppendArgs& a, ctconv_dtype, hipStream_t) {
    ++launches;
    EXPECT((int64_t)a.groups * a.rows_per_group >= a.n);
    EXPECT((int64_t)a.rows_per_group * a.Hkv * a.chunks <= INT32_MAX / 2);
    EXPECT(fdiv((uint32_t)(a.B * a.groups - 1), a.fd_groups) == (uint32_t)a.B - 1);
    return hipSuccess;
}
hipError_t launch_evict(const EvictArgs& a, ctconv_dtype dt, hipStream_t) {
    ++launches;
    EXPECT(a.words % 16 == 0 && (int64_t)a.words * 64 >= a.pages.slots);
    EXPECT(a.list >= 0 && a.list <= a.keep);
    EXPECT(a.chunks == a.D * (dt == CTCONV_F32 ? 4 : 2) / 16 && 64 / a.chunks >= 1);
    // the selection's LDS: words, then what it works on, and its static arrays
    const int64_t work = (int64_t)((a.list + 3) & ~3) * 4 + (a.fused ? 1024 * 16 : 0);
    EXPECT((int64_t)a.words * 12 + (work > 49152 ? work : 49152) + 2048 <= 160 << 10);
    EXPECT(a.words * 8 <= 32768);  // the ties' bit map lies where the digits were counted
    return hipSuccess;
}
hipError_t launch_norm(const NormArgs& a, ctconv_dtype, bool, hipStream_t) {
    ++launches;
    EXPECT(a.C >= 1 && a.C <= 16384 && a.rows >= 1 && a.rows_per_gate >= 1);
    return hipSuccess;
}
hipError_t launch_attn_stream(const AttnArgs& a, ctconv_dtype, bool paged, hipStream_t) {
    check_attention(a, 16);
    // row offsets (8 bytes a key) and visibility of a paged chunk lie in LDS
    if (paged) EXPECT((int64_t)a.chunk * 8 + a.chunk / 8 <= 64 << 10);
    return hipSuccess;
}
hipError_t launch_attn_tile(const AttnArgs& a, ctconv_dtype dt, hipStream_t) {
    check_attention(a, 128);
    const int64_t es = dt == CTCONV_F32 ? 4 : 2;
    EXPECT(a.D * es <= 512);
    EXPECT((63 * a.k_row + a.D) * es <= (int64_t)UINT32_MAX);
    EXPECT((63 * a.v_row + a.D) * es <= (int64_t)UINT32_MAX);
    return hipSuccess;
}
hipError_t launch_attn_join(const AttnArgs& a, ctconv_dtype, bool, hipStream_t) {
    EXPECT(!a.direct);
    return hipSuccess;
}
}  // namespace block
}  // namespace ctconv

static uint64_t st = 0x9E3779B97F4A7C15ull;
static int64_t rnd(int64_t lo, int64_t hi) {
    st ^= st << 13;
    st ^= st >> 7;
    st ^= st << 17;
    return lo + (int64_t)(st % (uint64_t)(hi - lo + 1));
}
static int64_t wide(int64_t hi) { return rnd(0, 9) ? rnd(0, hi) : rnd(0, 5) ? rnd(0, 1ll << 40) : rnd(-3, 1); }

int main() {
    int32_t table[4] = {0};
    alignas(16) static char buf[64];
    float* f = reinterpret_cast<float*>(buf);
    ws_lo = reinterpret_cast<const char*>(uintptr_t(1) << 40);  // never dereferenced
    for (int it = 0; it < 200000; ++it) {
        const ctconv_dtype dt = (ctconv_dtype)rnd(0, 2);
        const int64_t H = wide(16), G = rnd(1, 20), D = rnd(0, 9) ? 8 * rnd(1, 32) : wide(300);
        const int64_t B = wide(100), page = rnd(0, 9) ? rnd(1, 300) : wide(1 << 20);
        const int64_t cols = wide(3000), pool = wide(100000), ts = wide(4000);
        const int64_t slots = cols > 0 && page > 0 && cols < (1 << 20) && page < (1 << 20) ? cols * page : 0;
        const int64_t len = rnd(0, 9) ? rnd(0, slots > 0 ? slots : 1) : wide(1 << 20);
        int64_t kv[3] = {wide(1 << 20) * 8, wide(4096) * 8, wide(1 << 16) * 8};
        int64_t row[3] = {wide(1 << 24) * 8, wide(1 << 16) * 8, wide(4096) * 8};
        int64_t sl[2] = {wide(1 << 24), wide(1 << 20)};
        const float scale = rnd(0, 20) ? (float)rnd(-4, 4) : INFINITY;
        switch (rnd(0, 4)) {
            case 0:
                ctconv_cache_append(buf, buf, buf, buf, table, table, nullptr, nullptr, table, f, B,
                                    wide(5000), H, D, pool, page, cols, row, kv, ts, sl, dt, nullptr);
                break;
            case 1: {
                const int64_t window = rnd(0, 1) ? 0 : wide(5000);
                const bool w = rnd(0, 1);
                size_t nb = 0;
                if (ctconv_paged_attention_workspace_bytes(B, H * G, H, D, len, window, w, dt, &nb) !=
                    CTCONV_OK)
                    nb = 0;
                ws_size = nb;
                span_bound = window > 0 && window < len ? window : len;
                ctconv_paged_attention(buf, buf, buf, table, table, buf, f, w ? f : nullptr, B, H * G,
                                       H, D, pool, page, cols, len, window, row, kv, row, ts, sl,
                                       scale, dt, const_cast<char*>(ws_lo), nb, nullptr);
                break;
            }
            case 2:
                ctconv_cache_evict(buf, buf, table, table, nullptr, f, table, f + 4, table + 1,
                                   rnd(0, 1) ? table : nullptr, table, B, H, D, pool, page, cols, len,
                                   wide(60000), wide(9), wide(5000), kv, ts, sl, sl, dt, nullptr);
                break;
            case 3: {
                const int64_t Lq = wide(5000), Lk = wide(9000);
                size_t nb = 0;
                if (ctconv_cross_attention_workspace_bytes(B, Lq, Lk, H * G, H, D, dt, &nb) != CTCONV_OK)
                    nb = 0;
                ws_size = nb;
                span_bound = Lk;
                int64_t far[3] = {0, wide(1 << 28) * 8, 8 * wide(64)};
                ctconv_cross_attention(buf, buf, buf, rnd(0, 1) ? table : nullptr, nullptr, buf, f, B,
                                       Lq, Lk, H * G, H, D, row, rnd(0, 1) ? far : row, row, row, 0,
                                       scale, dt, const_cast<char*>(ws_lo), nb, nullptr);
                break;
            }
            case 4: {
                int64_t s5[5] = {wide(20000), wide(20000), wide(20000), wide(40000), wide(40000)};
                ctconv_norm_residual(buf, buf, buf, nullptr, buf, buf, buf, buf, buf, buf, wide(1 << 30),
                                     wide(20000), s5, wide(100), (ctconv_norm)rnd(0, 2),
                                     (ctconv_norm)rnd(0, 2), (ctconv_gate)rnd(0, 3), 1e-5f, dt,
                                     nullptr);
                break;
            }
        }
    }
    std::printf("ok %ld\n", launches);
    return 0;
}
