// What the kernels of include/moe_w4.h share: products of rows with frozen 4-bit weights
// that have group scales (w4_few.hip, w4_rows.hip) and the gradient of the rows
// (w4_grad.hip).
//
// Packed matrix: blocks of 16 rows x 128 columns, 1 KiB each, [row block][column
// block].  Lane l = 16 g + r of a wavefront owns 16 bytes: dword j holds row r,
// columns 32 j + 8 g .. + 7, one nibble each (column p in nibble p), offset
// binary (u = q + 8).  So one 128-bit load per lane reads a whole block, and dword j
// of all lanes is one operand of a 16x16x32 matrix instruction whose contraction
// runs along the columns.  Rows and columns past the matrix hold q = 0 with scale 0.
// Scales (and zero points) follow, [row block][column block][16 rows][SG], with SG =
// 4, 2 or 1 groups per 128 columns (wider groups are repeated in every block).
//
// Masking a dword with 0x000F000F leaves the codes of two neighbouring columns in its
// halves: what a 16-bit operand holds, but for the number format.
#pragma once

#include <algorithm>

#include "mat.h"
#include "moe_w4.h"

namespace moe {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));

constexpr int kCUs = 256;
constexpr int kBlockRows = 16, kBlockCols = 128, kBlockBytes = 1024;
constexpr int kGradCols = 256, kStepRows = 64;  // columns of a gradient workgroup, matrix rows of its step

struct W4Args {
  const uint8_t* w;   // packed matrices
  size_t stride;      // bytes from matrix to matrix
  size_t soff, zoff;  // scales, zero points
  int n, N, K, NB, KB;  // NB x KB blocks
  const void* x;      // rows of the product (x, or dy in the gradient)
  int64_t ldx;
  int T;
  const int32_t* offsets;
  const void* add;
  int64_t ldadd;
  void* y;
  int64_t ldy;
  float* part;  // [split][T][width], or NULL
  int split;
};

// A tile of up to BM rows of one matrix; e < 0: rows outside the groups; rows == 0: none.
struct RowTile {
  int e, r0, rows;
};

// A barrier for LDS alone: __syncthreads also waits for the loads from memory that are
// still under way.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Tiles in their order: the full ones of all groups, their rests, then those of the rows
// outside (workgroups start in that order, the ones with most to do first).  Called by
// whole wavefronts; every lane gets the same.
template <int BM>
struct Tiles {
  const int32_t* offsets;
  int n, T;
  int e0, e1;              // this lane's experts
  int full, rest;          // their tiles,
  int full_at, rest_at;    // and the number of their first ones
  int head, end, grouped;  // the rows outside are [0, head) and [end, T); tiles of all groups

  __device__ __forceinline__ int at(int i) const { return min(max(offsets[i], 0), T); }
  // f(expert, first row, end) for this lane's experts, four offsets on their way at a time
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    int lo = 0;
    for (int e = e0; e < e1; e += 4) {
      int b[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) b[i] = at(min(e + i, e1));
      if (e == e0) lo = b[0];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int hi = max(lo, b[i + 1]);
        if (e + i < e1) f(e + i, lo, hi);
        lo = hi;
      }
    }
  }
  __device__ __forceinline__ Tiles(const int32_t* o, int n_, int T_) : offsets(o), n(n_), T(T_) {
    if (!offsets) return;
    const int per = (n + 63) / 64;
    e0 = min((int)(threadIdx.x & 63) * per, n);
    e1 = min(e0 + per, n);
    full = rest = 0;
    each([&](int, int lo, int hi) {
      full += (hi - lo) / BM;
      rest += (hi - lo) % BM != 0;
    });
    const int f = wave_inclusive_scan(full), r = wave_inclusive_scan(rest);
    full_at = f - full;
    rest_at = __builtin_amdgcn_readlane(f, 63) + r - rest;
    grouped = __builtin_amdgcn_readlane(f, 63) + __builtin_amdgcn_readlane(r, 63);
    head = __builtin_amdgcn_readfirstlane(at(0));
    end = __builtin_amdgcn_readfirstlane(max(head, at(n)));
  }
  __device__ __forceinline__ int total() const {
    return offsets ? grouped + (head + BM - 1) / BM + (T - end + BM - 1) / BM : (T + BM - 1) / BM;
  }
  __device__ __forceinline__ RowTile find(int tile) const {
    if (!offsets) return RowTile{0, tile * BM, min(BM, T - tile * BM)};
    RowTile r{-1, 0, 0};
    if (tile < grouped) {
      const int nth_full = tile - full_at, nth_rest = tile - rest_at;
      const bool in_full = nth_full >= 0 && nth_full < full, mine = in_full || (nth_rest >= 0 && nth_rest < rest);
      const int l = __ffsll((unsigned long long)__ballot(mine)) - 1;
      int left = in_full ? nth_full : nth_rest;
      each([&](int e, int lo, int hi) {
        const int f = (hi - lo) / BM, k = (hi - lo) % BM, c = in_full ? f : (k != 0);
        if (left >= 0 && left < c) r = in_full ? RowTile{e, lo + left * BM, BM} : RowTile{e, hi - k, k};
        left -= c;
      });
      return RowTile{__builtin_amdgcn_readlane(r.e, l), __builtin_amdgcn_readlane(r.r0, l),
                     __builtin_amdgcn_readlane(r.rows, l)};
    }
    int t = tile - grouped;
    const int heads = (head + BM - 1) / BM;
    if (t < heads) return RowTile{-1, t * BM, min(BM, head - t * BM)};
    t -= heads;
    if (t < (T - end + BM - 1) / BM) r = RowTile{-1, end + t * BM, min(BM, T - end - t * BM)};
    return r;
  }
};

// Upper bound on the tiles above.
inline int64_t max_tiles(int n, int T, int BM, bool grouped) {
  return grouped ? (int64_t)T / BM + std::min(n, T) + 2 : ceil_div(T, BM);
}

// Tile and run of columns of workgroup b, of `groups` runs per tile.  Workgroups go to the
// 8 dies in turn.  Tiles of groups: all runs of a tile on one die, whose L2 then holds
// its rows (16,384 rows of 64 experts, 6144 x 2048: 500 -> 475 us; of 256, 2048 x
// 1024: 151 -> 144).  One matrix: neither order was faster.
struct Place {
  int tile, run;
};
__device__ __forceinline__ Place place_of(int b, int groups, bool grouped) {
  if (!grouped) return Place{b / groups, b % groups};
  const int loc = b / 8;
  return Place{loc / groups * 8 + b % 8, loc % groups};
}
inline int64_t places(int64_t tiles, int groups, bool grouped) {
  return (grouped ? (tiles + 7) / 8 * 8 : tiles) * groups;
}

// ---------------------------------------------------------------------------
// Codes into operands.
// ---------------------------------------------------------------------------
__device__ __forceinline__ half2_t as_half2(uint32_t v) { return __builtin_bit_cast(half2_t, v); }
__device__ __forceinline__ uint32_t bits_of(half2_t v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ half2_t both(_Float16 v) { return half2_t{v, v}; }

// (d & mask) | bits, one instruction.
__device__ __forceinline__ uint32_t masked(uint32_t d, uint32_t mask, uint32_t bits) {
  return (uint32_t)__builtin_amdgcn_bitop3_b32(d, mask, bits, 0xEA);
}

// The codes of a dword as four pairs of binary16 numbers: 1024 + u, or, where the
// field sits at bit 4, 1024 + 16 u.
__device__ __forceinline__ void code_pairs(uint32_t d, half2_t (&v)[4]) {
  const uint32_t e = d >> 8;
  v[0] = as_half2(masked(d, 0x000F000Fu, 0x64006400u));
  v[1] = as_half2(masked(d, 0x00F000F0u, 0x64006400u));
  v[2] = as_half2(masked(e, 0x000F000Fu, 0x64006400u));
  v[3] = as_half2(masked(e, 0x00F000F0u, 0x64006400u));
}

// binary16: one packed subtraction or multiply-add leaves q - z exactly.  c = -(1032 + z).
__device__ __forceinline__ void codes_f16(uint32_t d, half2_t c, half2_t (&v)[4]) {
  const half2_t c16 = c + both((_Float16)960.0f);  // -(72 + z)
  const half2_t sixteenth = both((_Float16)0.0625f);
  code_pairs(d, v);
  v[0] += c;
  v[1] = v[1] * sixteenth + c16;
  v[2] += c;
  v[3] = v[3] * sixteenth + c16;
}

// Two values rounded to bfloat16, in one instruction.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, bf2_t));
}

// Scales and zero points as the packed matrix holds them, and what the operands
// need of them.
template <int DT>
__device__ __forceinline__ float scale_value(uint16_t s) {
  if constexpr (DT == MOE_T_F16) return (float)__builtin_bit_cast(_Float16, s);
  else return __builtin_bit_cast(float, (uint32_t)s << 16);
}

template <int SG>
struct ScaleVec;
template <>
struct ScaleVec<1> {
  typedef uint16_t s;
  typedef int8_t z;
};
template <>
struct ScaleVec<2> {
  typedef uint32_t s;
  typedef uint16_t z;
};
template <>
struct ScaleVec<4> {
  typedef uint64_t s;
  typedef uint32_t z;
};

// ---------------------------------------------------------------------------
// Many rows: tiles of BM = 16 MT rows, which pass through two LDS buffers.
// ---------------------------------------------------------------------------
constexpr int kTileThreads = 256;

// A workgroup's rows of one step of CS columns (64 or 128), from memory to registers
// to LDS, 16-byte pieces.  Pieces are swizzled so that an operand's 16 rows cover all
// banks (a line of 64 banks holds 16 pieces: one row of 128 columns or two of 64).  Rows
// past the tile repeat its last (their sums are not stored); of the last step's
// columns those past the width are zeros.
template <int CS>
__device__ __forceinline__ int piece_at(int row, int c) {
  return CS == 128 ? row * 16 + (c ^ (row & 15)) : row * 8 + (c ^ (row >> 1 & 7));
}

template <int DT, int MT, int CS>
struct Stage {
  static constexpr int PR = CS / 8, RP = kTileThreads / PR;  // pieces per row, rows per pass
  static constexpr int P = (16 * MT + RP - 1) / RP;
  struct Pieces {
    u32x4 v[P];
  };
  const char* base;
  uint32_t at[P];
  int width, c;
  __device__ __forceinline__ Stage(const W4Args& a, const RowTile& t, int w) {
    base = (const char*)a.x + (int64_t)t.r0 * a.ldx * 2;
    width = w;
    c = threadIdx.x % PR;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int row = min((int)threadIdx.x / PR + RP * p, t.rows - 1);
      at[p] = (uint32_t)row * (uint32_t)(a.ldx * 2) + c * 16;
    }
  }
  // pieces P0 .. P1 - 1
  template <int P0 = 0, int P1 = P>
  __device__ __forceinline__ void load(Pieces& v, int c0) const {
    const char* b = base + (size_t)c0 * 2;
    const uint32_t back = max(0, c - (min(width - c0, CS) / 8 - 1)) * 16;  // to the last piece of the row
#pragma unroll
    for (int p = P0; p < P1; ++p) v.v[p] = *(const u32x4*)(b + (at[p] - back));
  }
  template <int P0 = 0, int P1 = P>
  __device__ __forceinline__ void store(const Pieces& v, u32x4* lds, int c0) const {
#pragma unroll
    for (int p = P0; p < P1; ++p) lds[piece_at<CS>(threadIdx.x / PR + RP * p, c)] = v.v[p];
    if (c0 + CS > width && c0 + c * 8 >= width) {
#pragma unroll
      for (int p = P0; p < P1; ++p) lds[piece_at<CS>(threadIdx.x / PR + RP * p, c)] = u32x4{};
    }
  }
};

// Steps that are loaded ahead: tiles of few rows have little to do between loads, and
// registers to spare.
constexpr int steps_ahead(int M) { return M <= 2 ? 3 : M <= 4 ? 2 : 1; }

// Weights rounded to the rows' type as operands.  binary16: the exact code times the
// scale, a packed product.  bfloat16: (1024 + u) s - (1032 + z) s in one fp32
// multiply-add, whose result is exact (at most 8 + 8 bits; the addend is finite up to s =
// 2^117), then rounded.  One scale for all eight.
//
// That rounding is a choice: it is the one that a 16-bit model's weights have, and gives
// outputs 0.0022 to 0.0024 (bfloat16) or 0.00023 to 0.00030 (binary16) of their norm from
// the exact ones, where their own rounding alone gives 0.0017 or 0.0002.  What it takes off a
// weight fits the same type, and a second product with that gives 0.0017 and 0.0002, but
// (us, one and two products) 2,048 rows of 6144 x 6144 bfloat16 149 and 236, 16,384 rows of 256
// experts of 1024 x 2048 136 and 211; gradients, 2,048 rows of 2048 x 6144 binary16 65 and
// 96, 16,384 rows of 256 experts of 2048 x 512 bfloat16 92 and 135.  Group sums of exact
// codes times their scales in fp32, as few rows have them, need a second set of sums, for which
// there are no registers; a gradient has a scale for every term.
template <int DT, bool ZP>
struct GroupScale;
template <bool ZP>
struct GroupScale<MOE_T_F16, ZP> {
  half2_t s, c;
  __device__ __forceinline__ void set(uint16_t sv, int z) {
    s = both(__builtin_bit_cast(_Float16, sv));
    c = both((_Float16)(float)(-1032 - z));
  }
  __device__ __forceinline__ v8_t<MOE_T_F16> weights(uint32_t d) const {
    half2_t v[4];
    codes_f16(d, ZP ? c : both((_Float16)-1032.0f), v);
    return __builtin_bit_cast(v8_t<MOE_T_F16>,
                              u32x4{bits_of(v[0] * s), bits_of(v[1] * s), bits_of(v[2] * s), bits_of(v[3] * s)});
  }
};
template <bool ZP>
struct GroupScale<MOE_T_BF16, ZP> {
  float s, s16, c, c16;
  __device__ __forceinline__ void set(uint16_t sv, int z) {
    s = scale_value<MOE_T_BF16>(sv);
    s16 = s * 0.0625f;
    const float minus_z = (float)-z;  // (each addend is exact: at most 11 + 8 bits)
    c = fmaf(minus_z, s, -1032.0f * s);
    c16 = fmaf(minus_z, s, -72.0f * s);
  }
  __device__ __forceinline__ v8_t<MOE_T_BF16> weights(uint32_t d) const {
    half2_t v[4];
    code_pairs(d, v);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = i & 1 ? s16 : s, o = i & 1 ? c16 : c;
      r[i] = pack_bf16(fmaf((float)v[i][0], f, o), fmaf((float)v[i][1], f, o));
    }
    return __builtin_bit_cast(v8_t<MOE_T_BF16>, r);
  }
};

// f(Const<M>) with the smallest M of 1, 2, 4, .., MT groups of 16 that hold `rows`; or, for
// tiles that only large single matrices take, MT.
template <int MT, bool ONE, typename F>
__device__ __forceinline__ void by_height(int rows, F f) {
  if constexpr (MT > 1 && !ONE) {
    constexpr int HALF = MT > 4 ? 4 : MT / 2;
    if (rows <= 16 * HALF) return by_height<HALF, false>(rows, f);
  }
  f(Const<MT>{});
}

// Four consecutive sums of a row, from column c: to the split's partial sums, or with add, rounded.
template <int DT>
__device__ __forceinline__ void put4(const W4Args& a, int width, int split, int64_t row, int c, f32x4 v) {
  typedef typename Mat<DT>::elem elem;
  struct alignas(8) E4 {
    elem e[4];
  };
  if (a.part) {
    *(f32x4*)(a.part + ((int64_t)split * a.T + row) * width + c) = v;
    return;
  }
  if (a.add) {
    const E4 o = *(const E4*)((const elem*)a.add + row * a.ldadd + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += (float)o.e[i];
  }
  E4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.e[i] = (elem)v[i];
  *(E4*)((elem*)a.y + row * a.ldy + c) = o;
}

struct W4Layout {
  int NB, KB, SG;
  size_t soff, zoff, stride;
};

// Tiles of a call with many rows: MT groups of 16 rows by 64 R weight rows (forward) or
// 256 columns (gradient), and parts that a tile's sums are split into.
struct TilePlan {
  int MT, R, groups, split;
};

template <typename F>
inline void by_format(const moe_w4_dims_t& d, int SG, F f) {
  const auto zeros = [&](auto dt, auto sg) {
    if (d.zeros) f(dt, sg, Const<1>{});
    else f(dt, sg, Const<0>{});
  };
  const auto groups = [&](auto dt) {
    if (SG == 4) zeros(dt, Const<4>{});
    else if (SG == 2) zeros(dt, Const<2>{});
    else zeros(dt, Const<1>{});
  };
  if (d.dtype == MOE_T_F16) groups(Const<MOE_T_F16>{});
  else groups(Const<MOE_T_BF16>{});
}

// Launches of forward calls of few and of many rows, and of the gradient of few (tiles of 16 M) and of many.
void launch_w4_few(const W4Args& a, const moe_w4_dims_t& d, const W4Layout& l, hipStream_t s);
void launch_w4_rows(const W4Args& a, const moe_w4_dims_t& d, const W4Layout& l, const TilePlan& p, hipStream_t s);
void launch_w4_grad_few(const W4Args& a, const moe_w4_dims_t& d, const W4Layout& l, int M, hipStream_t s);
void launch_w4_grad(const W4Args& a, const moe_w4_dims_t& d, const W4Layout& l, const TilePlan& p, hipStream_t s);

}  // namespace moe
