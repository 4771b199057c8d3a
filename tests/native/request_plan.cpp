// Host program: which kernel, in how many splits, a chunk call with these sizes
// takes.  The C entry point is called with the launchers replaced; no GPU call is
// made.  Reads lines "B rows n Hq Hkv D max_length window weights dtype packed",
// prints "<kernel> <splits> <keys per split> <workgroups>" for each.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "block_internal.h"

using namespace ctconv;
using namespace ctconv::block;

static void say(const char* kernel, const AttnArgs& a, int64_t groups) {
    std::printf("%s %d %d %lld\n", kernel, a.splits, a.chunk, (long long)groups);
}

namespace ctconv {
namespace block {
hipError_t launch_tables(const TablesArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_rotary(const RotaryArgs&, ctconv_dtype, bool, bool, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_chunk_stream(const AttnArgs& a, ctconv_dtype, hipStream_t) {
    say("stream", a, (int64_t)a.B * a.Hkv * a.row_tiles * a.splits);
    return hipSuccess;
}
hipError_t launch_chunk_tile(const AttnArgs& a, ctconv_dtype, hipStream_t) {
    say("tile", a, (int64_t)a.row_tiles * a.Hkv * a.splits);
    return hipSuccess;
}
hipError_t launch_chunk_join(const AttnArgs&, ctconv_dtype, hipStream_t) { return hipSuccess; }
hipError_t launch_chunk_tile_join(const AttnArgs&, ctconv_dtype, hipStream_t) { return hipSuccess; }
hipError_t launch_chunk_weights(const AttnArgs&, ctconv_dtype, hipStream_t) { return hipSuccess; }
}  // namespace block
}  // namespace ctconv

int main() {
    alignas(16) static int32_t ints[16];
    alignas(16) static char buf[16];
    long long v[11];
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2,
                      v + 3, v + 4, v + 5, v + 6, v + 7, v + 8, v + 9, v + 10) == 11) {
        const int64_t B = v[0], rows = v[1], n = v[2], Hq = v[3], H = v[4], D = v[5], len = v[6];
        const bool weights = v[8] != 0, packed = v[10] != 0;
        const int64_t row[3] = {n * Hq * D, Hq * D, D}, kv[3] = {H * D * 16, D, 16 * D};
        const int64_t cols = (len + 15) / 16 + 1, slot[2] = {H * cols * 16, cols * 16};
        const auto dt = static_cast<ctconv_dtype>(v[9]);
        size_t bytes = 0;
        ctconv_status st = ctconv_chunk_attention_workspace_bytes(B, rows, n, Hq, H, D, len, v[7],
                                                                  weights, dt, &bytes);
        if (st == CTCONV_OK)
            st = ctconv_chunk_attention(
                buf, buf, buf, ints, ints, packed ? ints : nullptr, nullptr, buf, nullptr,
                weights ? reinterpret_cast<float*>(buf) : nullptr, B, rows, n, Hq, H, D, 1 << 16,
                16, cols, len, v[7], row, kv, row, cols, slot, 0.1f, dt, buf, bytes, nullptr);
        if (st != CTCONV_OK) std::printf("refused %d\n", (int)st);
    }
    return 0;
}
