// Host program for the sanitizer tier of the operators on requests of many
// lengths: the C entry points (validation, plans, workspace sizes) over seeded
// shapes, valid and invalid, with the launchers replaced by checks of what the
// planners hand to the kernels.  No GPU call is made.  Prints "ok <launches>".
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "block_internal.h"

using namespace ctconv;
using namespace ctconv::block;

static long launches = 0, tiles = 0, streams = 0, joins = 0;
static const char* ws_lo = nullptr;
static size_t ws_size = 0;
static int64_t call_rows = 0, call_span16 = 0, call_span128 = 0;
static bool call_weights = false;

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

static void check_chunk(const AttnArgs& a, int64_t span) {
    ++launches;
    EXPECT(a.B > 0 && a.G >= 1 && a.Hq == a.G * a.Hkv && a.R == a.n * a.G && a.rows == call_rows);
    EXPECT(a.splits >= 1 && a.chunk >= 128 && a.chunk % 128 == 0);
    EXPECT((int64_t)a.chunk * a.splits >= span);
    EXPECT(a.c > 0.f && std::isfinite(a.c));
    EXPECT(a.window == 0 || a.window < a.pages.slots || a.pages.slots == 0);
    const int64_t values = (int64_t)a.rows * a.Hq;
    if (a.splits > 1) {
        EXPECT(inside(a.part_o, values * a.splits * a.D * 4));
        EXPECT(inside(a.part_ml, values * a.splits * 8));
    }
    EXPECT((a.lse2 != nullptr) == call_weights);
    if (a.lse2) EXPECT(inside(a.lse2, values * 4));
}

namespace ctconv {
namespace block {
hipError_t launch_tables(const TablesArgs& a, hipStream_t) {
    ++launches;
    EXPECT(a.B >= 1 && (int64_t)a.B * 16 + 1024 <= 160 << 10);
    EXPECT((int64_t)a.B * a.max_pages <= INT32_MAX);
    EXPECT((int64_t)a.max_pages * a.page_size <= INT32_MAX);
    EXPECT((int64_t)a.num_pages * a.page_size <= INT32_MAX);
    EXPECT(a.counts || (a.rows == 0 && !a.positions && !a.weight_sum));
    return hipSuccess;
}
hipError_t launch_rotary(const RotaryArgs& a, ctconv_dtype, bool, bool append, hipStream_t) {
    ++launches;
    EXPECT(a.rows >= 1 && a.half >= 1 && 2 * a.half <= a.D && a.D <= 256);
    EXPECT((int64_t)(a.Hq + 2 * a.Hk) * a.D <= INT32_MAX);
    EXPECT(!append || (a.num_slots >= a.page_size && a.Hk >= 1));
    return hipSuccess;
}
hipError_t launch_chunk_stream(const AttnArgs& a, ctconv_dtype, hipStream_t) {
    ++streams;
    check_chunk(a, call_span16);
    EXPECT((int64_t)a.row_tiles * 16 >= a.R);
    EXPECT((int64_t)a.B * a.Hkv * a.row_tiles * a.splits <= INT32_MAX);
    return hipSuccess;
}
hipError_t launch_chunk_join(const AttnArgs& a, ctconv_dtype, hipStream_t) {
    EXPECT(a.splits > 1 && (int64_t)a.B * a.Hkv * a.R <= INT32_MAX);
    return hipSuccess;
}
hipError_t launch_chunk_tile(const AttnArgs& a, ctconv_dtype dt, hipStream_t) {
    ++tiles;
    check_chunk(a, call_span128);
    EXPECT(a.D * (dt == CTCONV_F32 ? 4 : 2) <= 512);
    // the row tiles that `rows` rows of at most n per sequence can make
    const int64_t all = (int64_t)a.rows * a.G / 128 + a.B, most = (int64_t)a.B * ((a.R + 127) / 128);
    EXPECT(a.row_tiles >= (all < most ? all : most));
    EXPECT((int64_t)a.row_tiles * a.splits * a.Hkv <= INT32_MAX);
    return hipSuccess;
}
hipError_t launch_chunk_tile_join(const AttnArgs& a, ctconv_dtype, hipStream_t) {
    ++joins;
    EXPECT(a.splits > 1 && (int64_t)a.row_tiles * a.Hkv * 8 <= INT32_MAX);
    return hipSuccess;
}
hipError_t launch_chunk_weights(const AttnArgs& a, ctconv_dtype, hipStream_t) {
    EXPECT(a.lse2 && (int64_t)a.B * a.Hkv * ((a.pages.slots + 31) / 32) <= INT32_MAX);
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

static int64_t mul(int64_t a, int64_t b) {
    int64_t v;
    return __builtin_mul_overflow(a, b, &v) ? (int64_t)1 << 62 : v;
}

int main() {
    alignas(16) static int32_t ints[16];
    alignas(16) static char buf[64];
    alignas(16) static char other[64];
    float* f = reinterpret_cast<float*>(buf);
    double* d = reinterpret_cast<double*>(buf);
    ws_lo = reinterpret_cast<const char*>(uintptr_t(1) << 40);  // never dereferenced
    for (int it = 0; it < 200000; ++it) {
        const ctconv_dtype dt = (ctconv_dtype)rnd(0, 2);
        const int64_t H = wide(16), G = rnd(1, 20), D = rnd(0, 9) ? 8 * rnd(1, 32) : wide(300);
        const int64_t B = wide(100), page = rnd(0, 9) ? rnd(1, 300) : wide(1 << 20);
        const int64_t cols = wide(3000), pool = wide(100000);
        const int64_t slots = cols > 0 && page > 0 && cols < (1 << 20) && page < (1 << 20) ? cols * page : 0;
        const int64_t kv0 = mul(mul(H, page), D);
        int64_t kv[3] = {rnd(0, 9) ? kv0 : wide(1 << 20) * 8, D, mul(page, D)};
        const int64_t Hq = rnd(0, 20) ? mul(H, G) : wide(300);
        int64_t row[3] = {wide(1 << 24) * 8, rnd(0, 9) ? mul(Hq, D) : wide(1 << 16) * 8, rnd(0, 9) ? D : wide(4096) * 8};
        int64_t krow[2] = {rnd(0, 9) ? mul(H, D) : wide(1 << 16) * 8, D};
        int64_t sl[2] = {rnd(0, 5) ? mul(H, slots) : wide(1 << 24), rnd(0, 5) ? slots : wide(1 << 20)};
        const float scale = rnd(0, 20) ? (float)rnd(-4, 4) : INFINITY;
        const int64_t R = rnd(0, 9) ? 2 * rnd(1, D / 2 > 0 && D < 300 ? D / 2 : 1) : wide(300);
        const ctconv_rotary_layout layout = (ctconv_rotary_layout)rnd(0, 1);
        switch (rnd(0, 5)) {
            case 0:
                ctconv_cache_pages(ints, rnd(0, 3) ? ints : nullptr, nullptr, ints, ints, ints, ints,
                                   ints, ints, ints, ints, ints, rnd(0, 1) ? ints : nullptr,
                                   rnd(0, 1) ? f : nullptr, rnd(0, 9) ? B : wide(20000), wide(100000),
                                   H, pool, page, cols, rnd(0, 9) ? cols : wide(5000), sl, nullptr);
                break;
            case 1:
                ctconv_rotary(buf, buf, ints, d, buf, buf, wide(1 << 20), Hq, H, D, R, row + 1, krow,
                              row + 1, krow, layout, scale, dt, nullptr);
                break;
            case 2:
                ctconv_rotary_append(buf, buf, buf, ints, ints, d, buf, other, other, wide(1 << 20),
                                     rnd(0, 5) ? Hq : 0, H, D, R, pool, page, row + 1, krow, row + 1,
                                     kv, layout, scale, dt, nullptr);
                break;
            case 3: {
                double out[128];
                const auto v = [] { return rnd(0, 9) ? (double)rnd(1, 100000) / 7 : rnd(0, 1) ? -1.0 : INFINITY; };
                const int64_t n = rnd(0, 9) ? 2 * rnd(1, 128) : wide(300);
                if (ctconv_rotary_frequencies(n, v(), (ctconv_rotary_scaling)rnd(0, 4), v(), v(), v(), v(),
                                              out) == CTCONV_OK) {
                    ++launches;
                    for (int64_t i = 0; i < n / 2; ++i) EXPECT(!std::isnan(out[i]));
                }
                break;
            }
            default: {
                const bool packed = rnd(0, 1);
                const int64_t n = wide(3000), len = rnd(0, 9) ? rnd(0, slots > 0 ? slots : 1) : wide(1 << 20);
                const int64_t rows = packed ? wide(40000) : rnd(0, 20) ? (n > (1 << 24) || B > (1 << 24) ? 0 : B * n) : wide(9);
                const int64_t window = rnd(0, 1) ? 0 : wide(5000);
                const bool w = rnd(0, 2) == 0;
                if (!packed && rnd(0, 9)) row[0] = mul(mul(n, Hq), D);
                size_t nb = 0;
                if (ctconv_chunk_attention_workspace_bytes(B, rows, n, Hq, H, D, len, window, w, dt, &nb) !=
                    CTCONV_OK)
                    nb = 0;
                ws_size = nb;
                call_rows = rows;
                call_weights = w;
                const auto span = [&](int64_t height) {
                    const int64_t s = window + (n < height ? n : height) - 1;
                    return window > 0 && s < len ? s : len;
                };
                call_span16 = span(16);
                call_span128 = span(128);
                ctconv_chunk_attention(buf, other, other, ints, ints, packed ? ints : nullptr,
                                       rnd(0, 1) ? ints : nullptr, buf, f, w ? f : nullptr, B, rows, n, Hq,
                                       H, D, pool, page, cols, len, window, row, kv, row, cols, sl, scale,
                                       dt, const_cast<char*>(ws_lo), nb, nullptr);
                break;
            }
        }
    }
    EXPECT(tiles > 1000 && streams > 1000 && joins > 100);
    std::printf("ok %ld\n", launches);
    return 0;
}
