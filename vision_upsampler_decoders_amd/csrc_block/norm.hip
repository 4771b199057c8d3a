// The seam between two blocks: x_out = x + scale * g(gate) * post(h) and
// y = pre(x_out), one pass over each row.
//
// A row lives in the registers of one group of lanes from its first load to
// its last store, so x, h and the gate are read once and x_out and y written
// once: 5 row-sized transfers where separate steps take 12.  The statistics
// are the two-pass ones (mean, then the mean square of the deviations) over
// the registers, in fp32.  A row of up to 256 16-byte pieces belongs to one
// wave, which needs no barrier; longer rows to a workgroup of 256 or 1024.
// Bound by memory: 32768 rows of 2048 bf16 with a gate take 148 us, 4.5 TB/s
// (a copy reaches 5.15); one frame's rows take a launch.

#include "block_internal.h"

namespace ctconv {
namespace block {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// VEC consecutive values of a row (VEC = 1, or 16 bytes of them).
template <class TR, int VEC>
struct Piece {
    using S = typename TR::storage;
    u32x4 raw;
    template <bool STREAM = false>
    __device__ void load(const S* p) {
        if constexpr (VEC == 1)
            raw[0] = __float_as_uint(TR::to_f32(*p));
        else if constexpr (STREAM)
            raw = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
        else
            raw = *reinterpret_cast<const u32x4*>(p);
    }
    __device__ float get(int i) const {
        if constexpr (VEC == 1 || sizeof(S) == 4)
            return __uint_as_float(raw[i]);
        else
            return TR::to_f32((uint16_t)(raw[i >> 1] >> ((i & 1) * 16)));
    }
};

template <class TR, int VEC, bool STREAM>
__device__ inline void store_piece(typename TR::storage* p, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        *p = TR::from_f32(f[0]);
    } else {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (VEC == 4)
                r[i] = __float_as_uint(f[i]);
            else
                r[i] = (uint32_t)TR::from_f32(f[2 * i]) |
                       ((uint32_t)TR::from_f32(f[2 * i + 1]) << 16);
        }
        if constexpr (STREAM)
            __builtin_nontemporal_store(r, reinterpret_cast<u32x4*>(p));
        else
            *reinterpret_cast<u32x4*>(p) = r;
    }
}

// Sum over the NT lanes of a row, the same bits in every lane.
template <int NT>
__device__ inline float row_sum(float v, float* red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if constexpr (NT > 64) {
        __syncthreads();  // the last sum's readers are done with red
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) v += red[w];
    }
    return v;
}

// u := norm(u) * w + b over a row of C values, of which this lane holds
// pieces p0 + i * NT.
template <class TR, int VEC, int NT, int PIECES>
__device__ inline void normalise(float (&u)[PIECES][VEC], int kind, const void* w, const void* b,
                                 const NormArgs& a, int p0, int n_pieces, float* red) {
    using S = typename TR::storage;
    if (kind == CTCONV_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += u[i][e];
        const float mean = row_sum<NT>(s, red) * a.inv_C;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                u[i][e] = p0 + i * NT < n_pieces ? u[i][e] - mean : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s = fmaf(u[i][e], u[i][e], s);
    const float r = 1.f / sqrtf(row_sum<NT>(s, red) * a.inv_C + a.eps);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int p = p0 + i * NT;
        if (p >= n_pieces) continue;
        Piece<TR, VEC> pw, pb;
        if (w) pw.load(static_cast<const S*>(w) + (int64_t)p * VEC);
        if (b) pb.load(static_cast<const S*>(b) + (int64_t)p * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float v = u[i][e] * r;
            if (w) v *= pw.get(e);
            if (b) v += pb.get(e);
            u[i][e] = v;
        }
    }
}

__device__ inline float gated(float g, int fn) {
    if (fn == CTCONV_GATE_SIGMOID) return 1.f / (1.f + expf(-g));
    if (fn == CTCONV_GATE_TANH) return tanhf(g);
    return g;
}

// NT lanes per row, 256 / NT rows per workgroup of 256 lanes (one row where
// NT > 256); PIECES pieces of a row per lane.  STREAM: rows pass the caches by.
template <class TR, int VEC, int NT, int PIECES, bool STREAM>
__global__ __launch_bounds__(NT > 256 ? NT : 256) void norm_kernel(NormArgs a) {
    using S = typename TR::storage;
    constexpr int ROWS = NT > 256 ? 1 : 256 / NT;
    __shared__ float red_all[NT > 64 ? 16 : 1];
    static_assert(ROWS == 1 || NT == 64, "rows of a workgroup share no reduction buffer");
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / NT;
    if (row >= a.rows) return;  // NT = 64: whole waves; else the grid is exact
    const int p0 = threadIdx.x % NT;
    const int n_pieces = a.C / VEC;
    const S* xr = static_cast<const S*>(a.x) + row * a.xs;
    const S* hr = static_cast<const S*>(a.h) + row * a.hs;
    const S* gr = a.gate_fn != CTCONV_GATE_NONE
                      ? static_cast<const S*>(a.gate) + (row / a.rows_per_gate) * a.gs
                      : nullptr;
    Piece<TR, VEC> px[PIECES], ph[PIECES], pg[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int p = p0 + i * NT;
        if (p >= n_pieces) continue;
        ph[i].template load<STREAM>(hr + (int64_t)p * VEC);
        px[i].template load<STREAM>(xr + (int64_t)p * VEC);
        if (gr) pg[i].template load<STREAM>(gr + (int64_t)p * VEC);
    }
    float u[PIECES][VEC];
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[i][e] = p0 + i * NT < n_pieces ? ph[i].get(e) : 0.f;
    if (a.post != CTCONV_NORM_NONE)
        normalise<TR, VEC, NT, PIECES>(u, a.post, a.post_w, a.post_b, a, p0, n_pieces, red_all);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int p = p0 + i * NT;
        if (p >= n_pieces) continue;
        Piece<TR, VEC> ps;
        if (a.scale) ps.load(static_cast<const S*>(a.scale) + (int64_t)p * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float v = u[i][e];
            if (a.scale) v *= ps.get(e);
            if (gr) v *= gated(pg[i].get(e), a.gate_fn);
            u[i][e] = px[i].get(e) + v;
        }
        store_piece<TR, VEC, STREAM>(static_cast<S*>(a.x_out) + row * a.os + (int64_t)p * VEC, u[i]);
    }
    if (a.pre == CTCONV_NORM_NONE) return;
    normalise<TR, VEC, NT, PIECES>(u, a.pre, a.pre_w, a.pre_b, a, p0, n_pieces, red_all);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int p = p0 + i * NT;
        if (p < n_pieces)
            store_piece<TR, VEC, STREAM>(static_cast<S*>(a.y) + row * a.ys + (int64_t)p * VEC, u[i]);
    }
}

// More than the XCDs' L2 caches hold together: what is written is not there any
// more when its reader comes, and rows read and written past the caches go
// faster (32768 rows of 2048 bf16, 671 MB: 148 us against 155).
constexpr int64_t kStreamBytes = 32 << 20;

template <class TR, int VEC, int NT, int PIECES>
hipError_t run(const NormArgs& a, hipStream_t s) {
    constexpr int ROWS = NT > 256 ? 1 : 256 / NT;
    const dim3 grid((unsigned)((a.rows + ROWS - 1) / ROWS)), block(NT > 256 ? NT : 256);
    if constexpr (VEC > 1) {
        if (a.rows * a.C * (int64_t)sizeof(typename TR::storage) > kStreamBytes) {
            norm_kernel<TR, VEC, NT, PIECES, true><<<grid, block, 0, s>>>(a);
            return hipGetLastError();
        }
    }
    norm_kernel<TR, VEC, NT, PIECES, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

template <class TR>
hipError_t norm_t(const NormArgs& a, bool vec, hipStream_t s) {
    constexpr int V = 16 / sizeof(typename TR::storage);
    if (!vec) {
        if (a.C <= 512) return run<TR, 1, 64, 8>(a, s);
        if (a.C <= 4096) return run<TR, 1, 256, 16>(a, s);
        return run<TR, 1, 1024, 16>(a, s);
    }
    const int n = a.C / V;
    if (n <= 64) return run<TR, V, 64, 1>(a, s);
    if (n <= 128) return run<TR, V, 64, 2>(a, s);
    if (n <= 256) return run<TR, V, 64, 4>(a, s);
    if (n <= 512) return run<TR, V, 256, 2>(a, s);
    if (n <= 1024) return run<TR, V, 256, 4>(a, s);
    if (n <= 2048) return run<TR, V, 1024, 2>(a, s);
    return run<TR, V, 1024, 4>(a, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, ctconv_dtype dt, bool vec, hipStream_t s) {
    switch (dt) {
        case CTCONV_F32: return norm_t<TF32>(a, vec, s);
        case CTCONV_BF16: return norm_t<TBF16>(a, vec, s);
        case CTCONV_F16: return norm_t<TF16>(a, vec, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace block
}  // namespace ctconv
