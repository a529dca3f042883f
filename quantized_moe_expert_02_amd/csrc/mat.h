// Matrix instructions of the two 16-bit row types, and what the translation
// units that use them share.
#pragma once

#include "rows.h"

namespace moe {

template <int V>
struct Const {
  static constexpr int value = V;
};

// Matrix instructions of the two row types.
template <int DT>
struct Mat;
template <>
struct Mat<MOE_T_F16> {
  typedef _Float16 elem;
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mma(v8 a, v8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mat<MOE_T_BF16> {
  typedef __bf16 elem;
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mma(v8 a, v8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

template <int DT>
using v8_t = typename Mat<DT>::v8;

// Row strides are whole 16-byte vectors.
inline bool bad_ld(int64_t ld, int width) { return ld < width || ld % 8; }
inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

constexpr int64_t kMaxElems = (int64_t)1 << 35;  // rows times width of one operand

}  // namespace moe
