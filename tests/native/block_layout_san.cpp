// Host program for the sanitizer tier of the decoder-block operators: seeded
// calls whose tensors lie apart in memory, dimensions in any order and with
// gaps.  All of them reach their launcher, which checks what it is handed, the
// rows that are written among it; and launch grids hold what they should.
// No GPU call is made.  Prints "ok <launches>".
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "block_internal.h"

using namespace ctconv;
using namespace ctconv::block;

static long launches = 0;

#define EXPECT(cond)                                                 \
    do {                                                             \
        if (!(cond)) {                                               \
            std::printf("failed at line %d: %s\n", __LINE__, #cond); \
            std::exit(1);                                            \
        }                                                            \
    } while (0)

static void check_grid(int64_t blocks) {
    const dim3 g = grid_of(blocks);
    EXPECT(g.z == 1 && g.y >= 1 && g.y <= 65535 && (int64_t)g.x * g.y >= blocks);
    EXPECT((int64_t)g.x * 1024 < (int64_t)1 << 32);
    EXPECT(g.y == 1 || (int64_t)g.x * (g.y - 1) < blocks);
    EXPECT(g.y == 1 || g.x == 1u << kGridRowBits);
    EXPECT((int64_t)g.x * g.y <= UINT32_MAX);
}

static void check_attention(const AttnArgs& a) {
    ++launches;
    EXPECT(a.splits >= 1 && a.chunk % 128 == 0 && a.row_tiles >= 1);
    check_grid((int64_t)a.B * a.Hkv * a.row_tiles * a.splits);
}

namespace ctconv {
namespace block {
hipError_t launch_append(const AppendArgs& a, ctconv_dtype, hipStream_t) {
    ++launches;
    check_grid((int64_t)a.B * a.groups);
    return hipSuccess;
}
hipError_t launch_evict(const EvictArgs& a, ctconv_dtype, hipStream_t) {
    ++launches;
    // a row of results ends before the next one starts, and in place inside its own slots
    if (a.Hkv > 1) EXPECT(a.out_h >= a.keep);
    if (a.B > 1) EXPECT(a.out_b >= a.keep);
    if (a.weight_out == a.weight_sum) {
        EXPECT(a.out_b == a.slot_b && a.out_h == a.slot_h);
        EXPECT(a.keep <= 1600);  // the tables below hold no more slots
    }
    check_grid((int64_t)a.B * a.Hkv * ((a.keep + 63) / 64));
    return hipSuccess;
}
hipError_t launch_norm(const NormArgs& a, ctconv_dtype, bool, hipStream_t) {
    ++launches;
    EXPECT(a.rows >= 1 && a.rows_per_gate >= 1);
    check_grid(a.rows);
    return hipSuccess;
}
hipError_t launch_attn_stream(const AttnArgs& a, ctconv_dtype, bool, hipStream_t) {
    check_attention(a);
    return hipSuccess;
}
hipError_t launch_attn_tile(const AttnArgs& a, ctconv_dtype, hipStream_t) {
    check_attention(a);
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

// Strides (multiples of `step`) of n dimensions in some order, rows of `row` values apart.
static void lay(int64_t* strides, const int64_t* sizes, int n, int64_t row, int64_t step) {
    int order[3] = {0, 1, 2};
    for (int i = n - 1; i > 0; --i) std::swap(order[i], order[rnd(0, i)]);
    int64_t extent = row;
    for (int i = 0; i < n; ++i) {
        const int d = order[i];
        strides[d] = (extent + step - 1) / step * step + (rnd(0, 1) ? 0 : step * rnd(0, 9));
        extent += (sizes[d] - 1) * strides[d];
        if (sizes[d] == 1) strides[d] = rnd(0, 1) ? 0 : strides[d];  // not stepped
    }
}

int main() {
    int32_t table[4] = {0};
    alignas(16) static char buf[64];
    float* f = reinterpret_cast<float*>(buf);
    char* ws = reinterpret_cast<char*>(uintptr_t(1) << 40);  // never dereferenced
    for (int64_t b : {int64_t(1), int64_t(255), (int64_t(1) << 20) - 1, int64_t(1) << 20,
                      (int64_t(1) << 20) + 1, (int64_t(1) << 24) + 5, (int64_t(1) << 31) - 8})
        check_grid(b);
    for (int it = 0; it < 20000; ++it)
        check_grid(std::min<int64_t>(rnd(1, (int64_t)1 << rnd(1, 31)), INT32_MAX - 7));
    long calls = 0;
    for (int it = 0; it < 100000; ++it) {
        const ctconv_dtype dt = (ctconv_dtype)rnd(0, 2);
        const int64_t H = rnd(1, 9), G = rnd(1, 9), D = 8 * rnd(1, 32), Hq = H * G;
        const int64_t B = rnd(1, 40), page = rnd(1, 100), cols = rnd(1, 16), pool = rnd(1, 2000);
        const int64_t slots = page * cols, len = rnd(0, slots);
        int64_t kv[3], row[3], sl[2], out[2];
        const int64_t kv_n[3] = {pool, page, H}, sl_n[2] = {B, H}, q_n[2] = {B, Hq};
        lay(kv, kv_n, 3, D, 8);
        lay(sl, sl_n, 2, slots, 1);
        ctconv_status s;
        switch (rnd(0, 4)) {
            case 0: {
                const int64_t n = rnd(1, 500), new_n[3] = {B, n, H};
                lay(row, new_n, 3, D, 8);
                s = ctconv_cache_append(buf, buf, buf, buf, table, table, nullptr, nullptr,
                                        rnd(0, 1) ? table : nullptr, rnd(0, 1) ? f : nullptr, B, n,
                                        H, D, pool, page, cols, row, kv, 16, sl, dt, nullptr);
                break;
            }
            case 1: {
                const bool w = rnd(0, 1);
                lay(row, q_n, 2, D, 8);
                lay(out, q_n, 2, D, 8);
                s = ctconv_paged_attention(buf, buf, buf, table, table, buf, f, w ? f : nullptr, B,
                                           Hq, H, D, pool, page, cols, len, rnd(0, 1) ? 0 : rnd(1, 300),
                                           row, kv, out, 16, sl, 0.1f, dt, ws, SIZE_MAX / 2, nullptr);
                break;
            }
            case 2: {
                const bool place = rnd(0, 1);
                const int64_t keep = rnd(1, place ? slots : 2 * slots);
                lay(out, sl_n, 2, keep, 1);
                s = ctconv_cache_evict(buf, buf, table, table, nullptr, f, table, place ? f : f + 4,
                                       place ? table : table + 1, nullptr, table, B, H, D, pool,
                                       page, cols, len, keep, rnd(0, 9), rnd(0, 99), kv, 16, sl,
                                       place ? sl : out, dt, nullptr);
                break;
            }
            case 3: {
                const int64_t Lq = rnd(1, 300), Lk = rnd(0, 3000), o_n[3] = {B, Lq, Hq};
                lay(row, o_n, 3, D, 8);
                const int64_t k_st[3] = {8 * rnd(0, 999), 8 * rnd(0, 999), 8 * rnd(0, 99)};
                s = ctconv_cross_attention(buf, buf, buf, nullptr, nullptr, buf, f, B, Lq, Lk, Hq, H,
                                           D, row, k_st, k_st, row, 0, 0.1f, dt, ws, SIZE_MAX / 2,
                                           nullptr);
                break;
            }
            default: {
                const int64_t C = rnd(1, 16384), rows = rnd(0, 3) ? rnd(1, 5000) : rnd(1, INT32_MAX);
                const int64_t s5[5] = {C, rnd(0, 2 * C), C + rnd(0, 9), C + rnd(0, 99), C};
                s = ctconv_norm_residual(buf, buf, buf, nullptr, buf, buf, buf, buf, buf, buf, rows, C,
                                         s5, rnd(0, 3) ? rnd(1, 100) : INT64_MAX - rnd(0, 9),
                                         (ctconv_norm)rnd(0, 2), (ctconv_norm)rnd(0, 2),
                                         (ctconv_gate)rnd(0, 3), 1e-5f, dt, nullptr);
                break;
            }
        }
        if (s != CTCONV_OK) {
            std::printf("call %d refused with %d\n", it, (int)s);
            return 1;
        }
        ++calls;
    }
    EXPECT(launches == calls);
    std::printf("ok %ld\n", launches);
    return 0;
}
