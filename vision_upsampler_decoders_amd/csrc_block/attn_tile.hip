// Attention of many query rows per cache head to an encoder's states.
//
// A workgroup of 4 waves takes 128 query rows of one (sequence, cache head),
// a wave 32 of them, and walks the keys in tiles of KT.  Keys and values go
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
//  - Softmax is the one-pass one, base 2, the running maximum raised only
//    when a score passes it by 2^8 (see attn_stream.hip).
// LDS rows are spread over the banks by an exclusive-or of the 16-byte piece
// with row bits.  Two buffers: the next tile is loaded into registers while
// the current one is used, and one barrier per tile separates them.

#include "block_internal.h"
#include "mfma_common.h"

namespace ctconv {
namespace block {

namespace {

using mfma::u32x2;
using mfma::u32x4;

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr float kRaise = 8.f;

template <class TR>
struct Mma32;
template <>
struct Mma32<TBF16> {
    __device__ static inline void step(f32x16& acc, const u32x4 a, const u32x4 b) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                      __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
    }
};
template <>
struct Mma32<TF16> {
    __device__ static inline void step(f32x16& acc, const u32x4 a, const u32x4 b) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                     __builtin_bit_cast(f16x8, b), acc, 0, 0, 0);
    }
};
template <>
struct Mma32<TF32> {
    // a half holds values 4 half .. 4 half + 3 of 8; instruction e consumes
    // value e of both halves
    __device__ static inline void step(f32x16& acc, const u32x4 a, const u32x4 b) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]),
                                                       __uint_as_float(b[e]), acc, 0, 0, 0);
    }
};

template <class TR, int DP>
struct Shape {
    static constexpr int ES = sizeof(typename TR::storage);
    static constexpr int VEC = 16 / ES;
    // keys per tile: at most 16 KB of K and of V, at least one score tile
    static constexpr int KT = DP * ES <= 256 ? 64 : 32;
    static constexpr int ROW = DP * ES;                 // bytes of a K row in LDS
    static constexpr int KBYTES = KT * ROW;
    static constexpr int BUF = 2 * KBYTES;              // K, then V
    static constexpr int NF = DP / (2 * VEC);           // 16-byte pieces of a key per half
    static constexpr int NU = KT / 32;                  // score tiles
    static constexpr int ND = DP / 32;                  // output tiles
    static constexpr int KLOADS = KBYTES / (16 * kThreads);
    // V staging, 16-bit: 8 keys x VD value columns per thread
    static constexpr int VD = ES == 2 ? KT * DP / (8 * kThreads) : 0;
};

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

template <class TR, int DP>
__global__ __launch_bounds__(kThreads, DP == 256 ? 1 : 2) void tile_kernel(AttnArgs a) {
    using S = typename TR::storage;
    using Sh = Shape<TR, DP>;
    constexpr int ES = Sh::ES, VEC = Sh::VEC, KT = Sh::KT, NF = Sh::NF, NU = Sh::NU, ND = Sh::ND;
    extern __shared__ __align__(16) char lds[];

    // (sequence, head) pairs stay on one XCD: their keys are read from its L2
    // by all of their row tiles.
    const uint32_t per = gridDim.x >> 3;
    int item = (int)((blockIdx.x & 7) * per + (blockIdx.x >> 3));
    const int split = item % a.splits;
    item /= a.splits;
    const int tile = item % a.row_tiles;
    const int bh = item / a.row_tiles;
    if (bh >= a.B * a.Hkv) return;
    const int b = bh / a.Hkv, h = bh - b * a.Hkv;

    const int len = a.lengths ? clamped(a.lengths[b], a.Lk) : a.Lk;
    const int start = split * a.chunk;
    if (a.splits > 1 && start >= len) return;
    int n = len - start;
    n = n < a.chunk ? n : a.chunk;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 31, half = lane >> 5;
    const int row = tile * 128 + wave * 32 + col;
    const bool live = row < a.R;
    const int lq = live ? (int)fdiv((uint32_t)row, a.fd_G) : 0;
    const int hq = h * a.G + (live ? row - lq * a.G : 0);

    u32x4 qf[NF];
    {
        const S* qr = static_cast<const S*>(a.q) + b * a.q_b + lq * a.q_row + hq * a.q_head;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int d = (2 * f + half) * VEC;
            qf[f] = u32x4{0, 0, 0, 0};
            if (live && d < a.D) {
                qf[f] = *reinterpret_cast<const u32x4*>(qr + d);
                const uint32_t flip = a.negate ? (ES == 2 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[f][i] ^= flip;
            }
        }
    }

    const S* kb = static_cast<const S*>(a.k) + b * a.k_b + h * a.k_head + (int64_t)start * a.k_row;
    const S* vb = static_cast<const S*>(a.v) + b * a.v_b + h * a.v_head + (int64_t)start * a.v_row;
    const uint8_t* mask = a.mask ? a.mask + b * a.mask_stride + start : nullptr;

    // Staging registers and what of a tile this thread moves.
    constexpr int KL = Sh::KLOADS;
    constexpr int PIECES = DP / VEC;  // 16-byte pieces of a row
    u32x4 kr[KL];
    constexpr int VDW = ES == 2 ? Sh::VD / 2 : 1;  // dwords per key (16-bit)
    uint32_t vr[ES == 2 ? 8 * VDW : 1];
    u32x4 vr4[ES == 4 ? KL : 1];
    constexpr int VCOLS = ES == 2 ? DP / (ES == 2 ? Sh::VD : 1) : 1;
    const int v_group = ES == 2 ? tid / VCOLS : 0;        // slot group: step v_group / 2, half & 1
    const int v_d = ES == 2 ? (tid % VCOLS) * Sh::VD : 0;
    uint64_t seen = 0;  // visibility of the tile in the registers, then in LDS

    const auto load = [&](int t0) {
        bool ok = lane < KT && t0 + lane < n;
        if (ok && mask) ok = mask[t0 + lane] != 0;
        seen = __ballot(ok);
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const int id = tid + i * kThreads;
            const int key = id / PIECES, d = (id % PIECES) * VEC;
            const int t = t0 + key < n ? t0 + key : 0;
            kr[i] = *reinterpret_cast<const u32x4*>(kb + (int64_t)t * a.k_row + (d < a.D ? d : 0));
            if (d >= a.D) kr[i] = u32x4{0, 0, 0, 0};
        }
        if constexpr (ES == 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int key = 16 * (v_group >> 1) + 8 * (j >> 2) + 4 * (v_group & 1) + (j & 3);
                const int t = t0 + key < n ? t0 + key : 0;
                const S* p = vb + (int64_t)t * a.v_row + (v_d < a.D ? v_d : 0);
                if constexpr (VDW == 2) {
                    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
                    vr[2 * j] = w[0];
                    vr[2 * j + 1] = w[1];
                } else {
                    vr[j] = *reinterpret_cast<const uint32_t*>(p);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                const int id = tid + i * kThreads;
                const int key = id / PIECES, d = (id % PIECES) * VEC;
                const int t = t0 + key < n ? t0 + key : 0;
                vr4[i] = *reinterpret_cast<const u32x4*>(vb + (int64_t)t * a.v_row +
                                                         (d < a.D ? d : 0));
            }
        }
    };
    constexpr uint64_t kAll = KT == 64 ? ~0ull : (1ull << 32) - 1;
    const auto store = [&](char* buf) {
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const int id = tid + i * kThreads;
            const int key = id / PIECES, c = id % PIECES;
            *reinterpret_cast<u32x4*>(buf + key * Sh::ROW + ((c ^ (key & 15 & (PIECES - 1))) << 4)) =
                kr[i];
        }
        char* vt = buf + Sh::KBYTES;
        if constexpr (ES == 2) {
            if (seen != kAll) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int key = 16 * (v_group >> 1) + 8 * (j >> 2) + 4 * (v_group & 1) + (j & 3);
                    if (!((seen >> key) & 1))
#pragma unroll
                        for (int w = 0; w < VDW; ++w) vr[VDW * j + w] = 0;
                }
            }
            // V^T rows of KT keys, KT / 8 pieces
#pragma unroll
            for (int r = 0; r < Sh::VD; ++r) {
                const unsigned sel = (r & 1) ? 0x07060302u : 0x05040100u;
                u32x4 o;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    o[w] = __builtin_amdgcn_perm(vr[VDW * (2 * w + 1) + (r >> 1)],
                                                 vr[VDW * (2 * w) + (r >> 1)], sel);
                const int d = v_d + r;
                const int c = (v_group ^ (d >> 1) ^ (d >> 4)) & (KT / 8 - 1);
                *reinterpret_cast<u32x4*>(vt + d * (KT * 2) + (c << 4)) = o;
            }
        } else {
            // V rows, the pieces of every other 4 keys moved by 32 values
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                const int id = tid + i * kThreads;
                const int key = id / PIECES, c = id % PIECES;
                if (!((seen >> key) & 1)) vr4[i] = u32x4{0, 0, 0, 0};
                *reinterpret_cast<u32x4*>(vt + key * Sh::ROW + ((c ^ (((key >> 2) & 1) << 3)) << 4)) =
                    vr4[i];
            }
        }
    };

    f32x16 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
    float m = -__builtin_huge_valf(), l = 0.f;

    if (n > 0) {
        load(0);
        store(lds);
    }
    int at = 0;
    for (int t0 = 0; t0 < n; t0 += KT, at ^= 1) {
        const uint64_t bits = seen;
        const bool more = t0 + KT < n;
        if (more) load(t0 + KT);
        __syncthreads();
        const char* buf = lds + at * Sh::BUF;
        const char* vt = buf + Sh::KBYTES;
        if (bits != 0) {
            f32x16 s[NU];
#pragma unroll
            for (int u = 0; u < NU; ++u) {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[u][i] = 0.f;
                const char* krow = buf + (32 * u + col) * Sh::ROW;
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    const int c = (2 * f + half) ^ (col & 15 & (PIECES - 1));
                    Mma32<TR>::step(s[u], *reinterpret_cast<const u32x4*>(krow + (c << 4)), qf[f]);
                }
            }
            float c = a.c;
            if (bits != kAll) {
                c = 1.f;
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    const uint32_t w = (uint32_t)(bits >> (32 * u)) >> (4 * half);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[u][i] = (w >> (8 * (i >> 2) + (i & 3))) & 1 ? s[u][i] * a.c
                                                                      : -__builtin_huge_valf();
                }
            }
            float top = s[0][0];
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
            top *= c;
            if (__any(top > m + kRaise)) {
                top = fmaxf(top, __shfl_xor(top, 32));
                const float up = fmaxf(m, top);
                const float f = m == up ? 1.f : exp2_fast(m - up);
                m = up;
                l *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[d][i] *= f;
            }
            const float ref = m == -__builtin_huge_valf() ? 0.f : m;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[u][i] = exp2_fast(fmaf(s[u][i], c, -ref));
                    l += s[u][i];
                }
            if constexpr (ES == 2) {
#pragma unroll
                for (int st = 0; st < KT / 16; ++st) {
                    u32x4 pf;
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        pf[w] = mfma::pack2<TR>(s[st >> 1][8 * (st & 1) + 2 * w],
                                                s[st >> 1][8 * (st & 1) + 2 * w + 1]);
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        const int dr = 32 * d + col;
                        const int cc = ((2 * st + half) ^ (dr >> 1) ^ (dr >> 4)) & (KT / 8 - 1);
                        Mma32<TR>::step(
                            acc[d],
                            *reinterpret_cast<const u32x4*>(vt + dr * (KT * 2) + (cc << 4)), pf);
                    }
                }
            } else {
#pragma unroll
                for (int u = 0; u < NU; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int key = 32 * u + 8 * (i >> 2) + 4 * half + (i & 3);
                        const float* vrow = reinterpret_cast<const float*>(vt + key * Sh::ROW);
#pragma unroll
                        for (int d = 0; d < ND; ++d)
                            acc[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                                vrow[(32 * d + col) ^ (half << 5)], s[u][i], acc[d], 0, 0, 0);
                    }
            }
        }
        if (more) store(lds + (at ^ 1) * Sh::BUF);
    }
    l += __shfl_xor(l, 32);
    if (!live) return;
    if (a.direct) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        S* to = static_cast<S*>(a.out) + b * a.o_b + lq * a.o_row + hq * a.o_head;
        if (a.lse && half == 0)
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
        const int64_t part = ((int64_t)bh * a.splits + split) * a.R + row;
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

template <class TR, int DP>
hipError_t tile_d(const AttnArgs& a, hipStream_t s) {
    const int64_t items = (int64_t)a.B * a.Hkv * a.row_tiles * a.splits;
    const size_t lds = 2 * Shape<TR, DP>::BUF;
    const void* fn = reinterpret_cast<const void*>(&tile_kernel<TR, DP>);
    if (lds > 64u << 10) {
        const hipError_t e =
            hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    AttnArgs args = a;
    void* params[] = {&args};
    return hipLaunchKernel(fn, dim3((unsigned)((items + 7) / 8 * 8)), dim3(kThreads), params, lds, s);
}

template <class TR>
hipError_t tile_t(const AttnArgs& a, hipStream_t s) {
    if (a.D <= 64) return tile_d<TR, 64>(a, s);
    if (a.D <= 128) return tile_d<TR, 128>(a, s);
    return tile_d<TR, 256>(a, s);
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs& a, ctconv_dtype dt, hipStream_t s) {
    switch (dt) {
        case CTCONV_F32: return tile_t<TF32>(a, s);
        case CTCONV_BF16: return tile_t<TBF16>(a, s);
        case CTCONV_F16: return tile_t<TF16>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace block
}  // namespace ctconv
