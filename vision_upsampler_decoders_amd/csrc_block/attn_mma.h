// The 32x32 matrix step of the attention kernels, per element type.
#pragma once

#include "mfma_common.h"

namespace ctconv {
namespace block {

namespace {

using mfma::u32x4;

typedef float f32x16 __attribute__((ext_vector_type(16)));

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

}  // namespace
}  // namespace block
}  // namespace ctconv
