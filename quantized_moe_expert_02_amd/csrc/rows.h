// Rows of binary16, bfloat16 or fp32 moved and summed as 16-byte vectors, and
// the argument checks that the entry points of moe_dispatch.h and
// moe_adapter.h share.
#pragma once

#include "moe_adapter.h"
#include "wave.h"

namespace moe {

// One 16-byte vector of a row.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int DT>
struct RowType;
template <>
struct RowType<MOE_T_F16> {
  typedef _Float16 elem;
};
template <>
struct RowType<MOE_T_BF16> {
  typedef __bf16 elem;
};
template <>
struct RowType<MOE_T_F32> {
  typedef float elem;
};

// Elements of one vector.
template <int DT>
constexpr int kVec = 16 / (int)sizeof(typename RowType<DT>::elem);

template <int DT>
struct alignas(16) RowVec {
  typename RowType<DT>::elem e[kVec<DT>];
};

template <int DT>
__device__ __forceinline__ void unpack_vec(u32x4 v, float (&f)[kVec<DT>]) {
  const RowVec<DT> r = __builtin_bit_cast(RowVec<DT>, v);
#pragma unroll
  for (int i = 0; i < kVec<DT>; ++i) f[i] = (float)r.e[i];
}

// Rounds to the rows' type (to nearest, ties to even).
template <int DT>
__device__ __forceinline__ u32x4 pack_vec(const float (&f)[kVec<DT>]) {
  RowVec<DT> r;
#pragma unroll
  for (int i = 0; i < kVec<DT>; ++i) r.e[i] = (typename RowType<DT>::elem)f[i];
  return __builtin_bit_cast(u32x4, r);
}

// Lanes of m below this one.
__device__ __forceinline__ int lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

inline bool aligned_to(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool bad(const void* p, unsigned align) { return !p || !aligned_to(p, align); }
inline size_t round256(size_t v) { return (v + 255) & ~(size_t)255; }
inline size_t elem_bytes(int dtype) { return dtype == MOE_T_F32 ? 4 : 2; }

// Limits of one call, which keep every launch below 2^32 threads.
constexpr int32_t kMaxRows = 1 << 20;   // T
constexpr int32_t kMaxWidth = 1 << 16;  // H, K, N
// Rows of sorted buffers that a call writes by or walks: no sort gives more, and
// with more the kernels' 32-bit row and item numbers could wrap.
constexpr int32_t kMaxSorted = (1 << 25) + (1 << 20);

// Shape of a sort: MOE_OK, MOE_E_INVAL or MOE_E_UNSUPPORTED.
int check_sort_shape(int32_t T, int32_t k, int32_t E, int32_t align);

// Sorts on `s` (arguments already checked, T * k > 0).
hipError_t launch_sort(const int32_t* idx, int T, int k, int E, int align, int rows, int32_t* offsets,
                       int32_t* pairs, int32_t* pos, void* ws, hipStream_t s);

}  // namespace moe
