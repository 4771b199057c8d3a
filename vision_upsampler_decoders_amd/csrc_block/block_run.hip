// ctconv_block_run: the decoder-block functions with their arguments in tables.

#include <string.h>

#include "block_internal.h"

extern "C" {

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
        case CTCONV_OP_CACHE_PAGES:
            return ctconv_cache_pages(i32(0), i32(1), i32(2), i32(3), i32(4), i32(5), i32(6),
                                      i32(7), i32(8), i32(9), i32(10), i32(11), i32(12), fp(13),
                                      z[0], z[1], z[2], z[3], z[4], z[5], z[6], z + 7, stream);
        case CTCONV_OP_ROTARY: {
            const int kind = code(z[13]);
            ctconv_rotary_layout layout;
            memcpy(&layout, &kind, sizeof(int));
            return ctconv_rotary(p[0], p[1], i32(2), static_cast<double*>(p[3]), p[4], p[5], z[0],
                                 z[1], z[2], z[3], z[4], z + 5, z + 7, z + 9, z + 11, layout,
                                 f32(z[14]), as_dtype(z[15]), stream);
        }
        case CTCONV_OP_ROTARY_APPEND: {
            const int kind = code(z[16]);
            ctconv_rotary_layout layout;
            memcpy(&layout, &kind, sizeof(int));
            return ctconv_rotary_append(p[0], p[1], p[2], i32(3), i32(4),
                                        static_cast<double*>(p[5]), p[6], p[7], p[8], z[0], z[1],
                                        z[2], z[3], z[4], z[5], z[6], z + 7, z + 9, z + 11, z + 13,
                                        layout, f32(z[17]), as_dtype(z[18]), stream);
        }
        case CTCONV_OP_CHUNK_ATTENTION:
            return ctconv_chunk_attention(p[0], p[1], p[2], i32(3), i32(4), i32(5), i32(6), p[7],
                                          fp(8), fp(9), z[0], z[1], z[2], z[3], z[4], z[5], z[6],
                                          z[7], z[8], z[9], z[10], z + 11, z + 14, z + 17, z[20],
                                          z + 21, f32(z[23]), as_dtype(z[24]), workspace,
                                          workspace_bytes, stream);
    }
    return CTCONV_ERR_PARAM;
}

}  // extern "C"
