// The seam between two blocks: x_out = x + scale * g(gate) * post(h) and
// y = pre(x_out), one pass over each row.
//
// A row lives in the registers of one group of lanes from its first load to
// its last store, so x, h and the gate are read once and x_out and y written
// once: 5 row-sized transfers where separate steps take 12.  The statistics
// are the two-pass ones (mean, then the mean square of the deviations) over
// the registers, in fp32.  A row of up to 256 16-byte pieces belongs to one
// wave, which needs no barrier; longer rows to a workgroup of 256 or 1024.
// Bound by memory: 32768 rows of 2048 bf16 with a gate take 115 us, 5.8 TB/s
// (a copy, half of it writes, reaches 5.15); one frame's rows take a launch.

#include "block_internal.h"
#include "mfma_common.h"

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
                r[i] = mfma::pack2<TR>(f[2 * i], f[2 * i + 1]);
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

// u := u - mean, and the factor of the norm over a row of C values, of which
// this lane holds pieces p0 + i * NT (the rest of u is 0).  No branch writes u:
// a row held twice where two branches meet costs registers and with them waves
// (up to 178 registers against 88: 163 us against 115 for the rows above).
template <int VEC, int NT, int PIECES>
__device__ inline float centre(float (&u)[PIECES][VEC], int kind, const NormArgs& a, int p0,
                               int n_pieces, float* red) {
    float mean = 0.f;
    if (kind == CTCONV_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += u[i][e];
        mean = row_sum<NT>(s, red) * a.inv_C;
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const float m = p0 + i * NT < n_pieces ? mean : 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[i][e] -= m;
    }
    if (kind == CTCONV_NORM_NONE) return 1.f;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s = fmaf(u[i][e], u[i][e], s);
    return 1.f / sqrtf(row_sum<NT>(s, red) * a.inv_C + a.eps);
}

// v := v * r * w + b for the piece at element `at`.
template <class TR, int VEC>
__device__ inline void apply(float (&v)[VEC], float r, const void* w, const void* b, int64_t at) {
    using S = typename TR::storage;
    Piece<TR, VEC> pw, pb;
    if (w) pw.load(static_cast<const S*>(w) + at);
    if (b) pb.load(static_cast<const S*>(b) + at);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] *= r;
    if (w)
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] *= pw.get(e);
    if (b)
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] += pb.get(e);
}

// The 16-bit types take the hardware's exponential and reciprocal (relative
// error below 2^-16, beside the types' own 2^-8 and 2^-11; the outputs' error
// against 64 bits is the same to two digits): with the exact ones the gate
// was half of the kernel's instructions, 138 us against 115 for the rows above.
template <class TR, int VEC>
__device__ inline void gate_values(const Piece<TR, VEC>& p, int fn, float (&g)[VEC]) {
    constexpr bool SHORT = sizeof(typename TR::storage) == 2;
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] = p.get(e);
    if (fn == CTCONV_GATE_SIGMOID) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            g[e] = SHORT ? __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g[e] * -kLog2e))
                         : 1.f / (1.f + expf(-g[e]));
    } else if (fn == CTCONV_GATE_TANH) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float x = g[e];
            if constexpr (SHORT) {
                // 1 - 2 / (1 + e^2x); near 0, where that cancels, x - x^3 / 3
                const float y = 1.f + __builtin_amdgcn_exp2f(x * (2.f * kLog2e));
                const float far = fmaf(-2.f, __builtin_amdgcn_rcpf(y), 1.f);
                g[e] = fabsf(x) < 0.03125f ? fmaf(x * x * x, -1.f / 3.f, x) : far;
            } else {
                g[e] = tanhf(x);
            }
        }
    }
}

// NT lanes per row, 256 / NT rows per workgroup of 256 lanes (one row where
// NT > 256); PIECES pieces of a row per lane.  STREAM: rows pass the caches by.
template <class TR, int VEC, int NT, int PIECES, bool STREAM>
__global__ __launch_bounds__(NT > 256 ? NT : 256) void norm_kernel(NormArgs a) {
    using S = typename TR::storage;
    constexpr int ROWS = NT > 256 ? 1 : 256 / NT;
    __shared__ float red_all[NT > 64 ? 16 : 1];
    static_assert(ROWS == 1 || NT == 64, "rows of a workgroup share no reduction buffer");
    const int64_t row = (int64_t)block_number() * ROWS + threadIdx.x / NT;
    if (row >= a.rows) return;  // NT = 64: whole waves; else whole workgroups
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
        ph[i].raw = u32x4{0, 0, 0, 0};
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
        for (int e = 0; e < VEC; ++e) u[i][e] = ph[i].get(e);
    const bool post = a.post != CTCONV_NORM_NONE;
    const float rp = centre<VEC, NT, PIECES>(u, a.post, a, p0, n_pieces, red_all);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int p = p0 + i * NT;
        if (p >= n_pieces) continue;
        const int64_t at = (int64_t)p * VEC;
        apply<TR, VEC>(u[i], rp, post ? a.post_w : nullptr, post ? a.post_b : nullptr, at);
        if (a.scale) {
            Piece<TR, VEC> ps;
            ps.load(static_cast<const S*>(a.scale) + at);
#pragma unroll
            for (int e = 0; e < VEC; ++e) u[i][e] *= ps.get(e);
        }
        if (gr) {
            float g[VEC];
            gate_values<TR, VEC>(pg[i], a.gate_fn, g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) u[i][e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[i][e] += px[i].get(e);
        store_piece<TR, VEC, STREAM>(static_cast<S*>(a.x_out) + row * a.os + at, u[i]);
    }
    if (a.pre == CTCONV_NORM_NONE) return;
    const float r = centre<VEC, NT, PIECES>(u, a.pre, a, p0, n_pieces, red_all);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int p = p0 + i * NT;
        if (p >= n_pieces) continue;
        const int64_t at = (int64_t)p * VEC;
        apply<TR, VEC>(u[i], r, a.pre_w, a.pre_b, at);
        store_piece<TR, VEC, STREAM>(static_cast<S*>(a.y) + row * a.ys + at, u[i]);
    }
}

// More than the XCDs' L2 caches hold together: what is written is not there any
// more when its reader comes, and rows read and written past the caches go
// faster (32768 rows of 2048 bf16, 671 MB: 115 us against 127).
constexpr int64_t kStreamBytes = 32 << 20;

template <class TR, int VEC, int NT, int PIECES>
hipError_t run(const NormArgs& a, hipStream_t s) {
    constexpr int ROWS = NT > 256 ? 1 : 256 / NT;
    const dim3 grid = grid_of((a.rows + ROWS - 1) / ROWS), block(NT > 256 ? NT : 256);
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
