// Products of rows with frozen 4-bit weights that have group scales
// (include/moe_w4.h): forward for few and for many rows, and the gradient of the
// rows.
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
// Masking a dword with 0x000F000F leaves the codes of columns p and p + 4 in the
// two halves: operands hold eight columns in the order 0 4 1 5 2 6 3 7, and the
// rows' operands are put in that order too.
#include <algorithm>

#include "mat.h"
#include "moe_w4.h"

namespace moe {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));

constexpr int kBlockRows = 16, kBlockCols = 128, kBlockBytes = 1024;

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
  __device__ __forceinline__ Tiles(const int32_t* o, int n_, int T_) : offsets(o), n(n_), T(T_) {
    if (!offsets) return;
    const int per = (n + 63) / 64;
    e0 = min((int)(threadIdx.x & 63) * per, n);
    e1 = min(e0 + per, n);
    full = rest = 0;
    for (int e = e0, lo = at(e0); e < e1; ++e) {
      const int hi = max(lo, at(e + 1));
      full += (hi - lo) / BM;
      rest += (hi - lo) % BM != 0;
      lo = hi;
    }
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
      for (int e = e0, lo = at(e0); e < e1; ++e) {
        const int hi = max(lo, at(e + 1)), f = (hi - lo) / BM, k = (hi - lo) % BM, c = in_full ? f : (k != 0);
        if (left >= 0 && left < c) r = in_full ? RowTile{e, lo + left * BM, BM} : RowTile{e, hi - k, k};
        left -= c;
        lo = hi;
      }
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

// ---------------------------------------------------------------------------
// Few rows: an item is 16 rows and one row block of a matrix; the W wavefronts of a
// workgroup split its columns, KPW column blocks each, and add their sums through LDS.
// A workgroup takes a run of items and keeps its rows in registers from item to item
// while the next item's blocks are under way.  The rows are the first operand (index l
// % 16: the row; rows past the tile are zeros) and a block the second (index l %
// 16: its row), so that a lane's four sums belong to one weight row and are
// multiplied by its scale.  binary16 factors are the codes q - z themselves;
// bfloat16 holds 128 + u exactly, and (136 + z) times the sum of the rows' elements
// is taken off each group's sum.
// ---------------------------------------------------------------------------
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

// The product of one output element in fp32, term by term as the formula has it.
template <int DT, int SG, bool ZP>
__device__ __forceinline__ float slow_dot(const uint8_t* w, size_t soff, size_t zoff, int K, int KB, int n,
                                                    const void* xrow) {
  typedef typename Mat<DT>::elem elem;
  const elem* x = (const elem*)xrow;
  const int nb = n / kBlockRows, r = n % kBlockRows;
  float acc = 0.f;
#pragma unroll 1
  for (int k = 0; k < K; ++k) {
    const int kb = k / kBlockCols, c = k % kBlockCols;
    const size_t block = (size_t)nb * KB + kb;
    const uint8_t byte = w[block * kBlockBytes + ((c / 8 % 4) * 16 + r) * 16 + c / 32 * 4 + c % 8 / 2];
    const int q = (int)(c & 1 ? byte >> 4 : byte & 15) - 8;
    const size_t at = (block * 16 + r) * SG + c / (kBlockCols / SG);
    const int z = ZP ? (int)((const int8_t*)(w + zoff))[at] : 0;
    acc = fmaf((float)(q - z) * scale_value<DT>(((const uint16_t*)(w + soff))[at]), (float)x[k], acc);
  }
  return acc;
}

// Eight elements of a row in the operands' order.
__device__ __forceinline__ u32x4 operand_order(u32x4 v) {
  return u32x4{__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
               __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
}

template <int DT, int SG, bool ZP, int W, int KPW>
__global__ __launch_bounds__(64 * W) void k_w4_few(W4Args a) {
  typedef typename Mat<DT>::elem elem;
  constexpr int GS = 4 / SG;  // matrix instructions per group
  typedef typename ScaleVec<SG>::s svec;
  typedef typename ScaleVec<SG>::z zvec;
  __shared__ f32x4 red[2][W][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, g = lane >> 4;
  const Tiles<16> tiles(a.offsets, a.n, a.T);
  const int64_t items = (int64_t)tiles.total() * a.NB;
  const int i0 = (int)(items * blockIdx.x / gridDim.x), i1 = (int)(items * (blockIdx.x + 1) / gridDim.x);
  if (i0 >= i1) return;
  const int passes = (a.KB + W * KPW - 1) / (W * KPW);  // over the columns (one up to 128 W KPW of them)
  u32x4 xv[KPW][4], wv[KPW], wn[KPW];
  svec sv[KPW], sn[KPW];
  zvec zv[KPW], zn[KPW];
  int tile = i0 / a.NB, nb = i0 % a.NB;
  RowTile t = tiles.find(tile), tn = t;
  const auto block_of = [&](int pass, int u) { return (pass * W + wave) * KPW + u; };
  const auto load_w = [&](const RowTile& rt, int b, int pass) {
    if (rt.e < 0) return;
    const uint8_t* w = a.w + (size_t)rt.e * a.stride;
#pragma unroll
    for (int u = 0; u < KPW; ++u) {
      const int kb = block_of(pass, u);
      if (kb >= a.KB) break;
      const size_t block = (size_t)b * a.KB + kb;
      wn[u] = __builtin_nontemporal_load((const u32x4*)(w + block * kBlockBytes) + lane);
      sn[u] = ((const svec*)(w + a.soff))[block * 16 + li];
      if (ZP) zn[u] = ((const zvec*)(w + a.zoff))[block * 16 + li];
    }
  };
  const auto load_x = [&](const RowTile& rt, int pass) {
    if (rt.e < 0) return;
    const elem* row = (const elem*)a.x + (int64_t)(rt.r0 + min(li, rt.rows - 1)) * a.ldx + 8 * g;
#pragma unroll
    for (int u = 0; u < KPW; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = block_of(pass, u) * kBlockCols + 32 * j;
        xv[u][j] = u32x4{};
        if (k < a.K && li < rt.rows) xv[u][j] = *(const u32x4*)(row + k);
      }
#pragma unroll
    for (int u = 0; u < KPW; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) xv[u][j] = operand_order(xv[u][j]);
  };
  f32x4 acc;
  const auto multiply = [&](int u) {
    v8_t<DT> ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = (elem)1.0f;
#pragma unroll
    for (int s = 0; s < SG; ++s) {
      f32x4 sum{}, xsum{};
      const int z = ZP ? (int)(int8_t)((uint32_t)zv[u] >> (8 * s)) : 0;
#pragma unroll
      for (int j = s * GS; j < (s + 1) * GS; ++j) {
        const v8_t<DT> xf = __builtin_bit_cast(v8_t<DT>, xv[u][j]);
        if (DT == MOE_T_BF16) xsum = Mat<DT>::mma(xf, ones, xsum);
        const uint32_t c = wv[u][j];
        u32x4 b;
        if constexpr (DT == MOE_T_F16) {
          half2_t v[4];
          codes_f16(c, both((_Float16)(float)(-1032 - z)), v);
          b = u32x4{bits_of(v[0]), bits_of(v[1]), bits_of(v[2]), bits_of(v[3])};
        } else {
          b = u32x4{masked(c, 0x000F000Fu, 0x43004300u),
                    masked(c >> 4, 0x000F000Fu, 0x43004300u),
                    masked(c >> 8, 0x000F000Fu, 0x43004300u),
                    masked(c >> 12, 0x000F000Fu, 0x43004300u)};
        }
        sum = Mat<DT>::mma(xf, __builtin_bit_cast(v8_t<DT>, b), sum);
      }
      const float f = scale_value<DT>((uint16_t)((uint64_t)sv[u] >> (16 * s)));
      if constexpr (DT == MOE_T_BF16) {
        const float off = (float)(-136 - z);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = fmaf(off, xsum[i], sum[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(f, sum[i], acc[i]);
    }
  };
  load_w(t, nb, 0);
  load_x(t, 0);
  for (int i = i0; i < i1; ++i) {
    const int nb_now = nb;
    acc = f32x4{};
    for (int pass = 0; pass < passes; ++pass) {
#pragma unroll
      for (int u = 0; u < KPW; ++u) {
        wv[u] = wn[u];
        sv[u] = sn[u];
        zv[u] = zn[u];
      }
      if (pass + 1 < passes) {
        load_w(t, nb_now, pass + 1);
      } else if (i + 1 < i1) {
        if (++nb == a.NB) {
          nb = 0;
          tn = tiles.find(++tile);
        }
        load_w(tn, nb, 0);
      }
      if (t.e >= 0) {
#pragma unroll
        for (int u = 0; u < KPW; ++u)
          if (block_of(pass, u) < a.KB) multiply(u);
      }
      if (passes > 1) load_x(pass + 1 < passes ? t : tn, (pass + 1) % passes);
    }
    const int p = i & 1;
    red[p][wave][lane] = acc;
    lds_barrier();
    const int n = nb_now * kBlockRows + li;
    if (wave == i % W && n < a.N && 4 * g < t.rows) {
      f32x4 v = red[p][0][lane];
#pragma unroll 3
      for (int u = 1; u < W; ++u) v += red[p][u][lane];
      const int live = min(4, t.rows - 4 * g);
      const int64_t row = t.r0 + 4 * g;
      if (DT == MOE_T_BF16 && t.e >= 0) {
        // the terms 128 + u and 136 + z beside an infinity, or past fp32's range, need
        // not cancel to the formula's value
        bool finite = true;
#pragma unroll
        for (int q = 0; q < 4; ++q) finite &= fabsf(v[q]) < INFINITY;
        if (!finite) {
#pragma unroll 1
          for (int q = 0; q < live; ++q) {
            const float o = slow_dot<DT, SG, ZP>(a.w + (size_t)t.e * a.stride, a.soff, a.zoff, a.K, a.KB, n,
                                                 (const elem*)a.x + (row + q) * a.ldx);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k == q && !(fabsf(v[k]) < INFINITY)) v[k] = o;
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q >= live) break;
        float o = v[q];
        if (a.add) o += (float)((const elem*)a.add)[(row + q) * a.ldadd + n];
        ((elem*)a.y)[(row + q) * a.ldy + n] = (elem)o;
      }
    }
    if (nb == 0 && i + 1 < i1) {
      t = tn;
      if (passes == 1) load_x(t, 0);
    }
  }
}

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

template <int DT, int MT, int CS, bool ORDER>
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
  __device__ __forceinline__ void load(Pieces& v, int c0) const {
    const char* b = base + (size_t)c0 * 2;
    const uint32_t back = max(0, c - (min(width - c0, CS) / 8 - 1)) * 16;  // to the last piece of the row
#pragma unroll
    for (int p = 0; p < P; ++p) v.v[p] = *(const u32x4*)(b + (at[p] - back));
  }
  __device__ __forceinline__ void store(const Pieces& v, u32x4* lds, int c0) const {
    const bool in = c0 + c * 8 < width;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      u32x4 o = ORDER ? operand_order(v.v[p]) : v.v[p];
      if (c0 + CS > width) o = in ? o : u32x4{};
      lds[piece_at<CS>(threadIdx.x / PR + RP * p, c)] = o;
    }
  }
};

// Steps that are loaded ahead: tiles of few rows have little to do between loads, and
// registers to spare.
constexpr int steps_ahead(int M) { return M <= 2 ? 3 : M <= 4 ? 2 : 1; }

// Weights rounded to the rows' type as operands.  binary16: the exact code times the
// scale, a packed product.  bfloat16: (1024 + u) s - (1032 + z) s in one fp32
// multiply-add, whose result is exact (at most 8 + 9 bits), then rounded.  One scale
// for all eight.
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
    return __builtin_bit_cast(v8_t<MOE_T_F16>, u32x4{bits_of(v[0] * s), bits_of(v[1] * s), bits_of(v[2] * s), bits_of(v[3] * s)});
  }
};
template <bool ZP>
struct GroupScale<MOE_T_BF16, ZP> {
  float s, s16, c, c16;
  __device__ __forceinline__ void set(uint16_t sv, int z) {
    s = scale_value<MOE_T_BF16>(sv);
    s16 = s * 0.0625f;
    c = (float)(-1032 - z) * s;
    c16 = (float)(-72 - z) * s;
  }
  __device__ __forceinline__ v8_t<MOE_T_BF16> weights(uint32_t d) const {
    half2_t v[4];
    code_pairs(d, v);
    return __builtin_bit_cast(v8_t<MOE_T_BF16>, u32x4{pack_bf16(fmaf((float)v[0][0], s, c), fmaf((float)v[0][1], s, c)),
                                                      pack_bf16(fmaf((float)v[1][0], s16, c16), fmaf((float)v[1][1], s16, c16)),
                                                      pack_bf16(fmaf((float)v[2][0], s, c), fmaf((float)v[2][1], s, c)),
                                                      pack_bf16(fmaf((float)v[3][0], s16, c16), fmaf((float)v[3][1], s16, c16))});
  }
};

// f(Const<M>) with the smallest M of 1, 2, 4, .., MT groups of 16 that hold `rows`.
template <int MT, typename F>
__device__ __forceinline__ void by_height(int rows, F f) {
  if constexpr (MT > 1) {
    constexpr int HALF = MT > 4 ? 4 : MT / 2;
    if (rows <= 16 * HALF) return by_height<HALF>(rows, f);
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

// Forward: each of four wavefronts takes R row blocks of the matrix, straight from
// memory into operands, and all rows of the tile.
template <int DT, int SG, bool ZP, int MT, int R>
__global__ __launch_bounds__(kTileThreads, 2) void k_w4_rows(W4Args a, int groups) {
  constexpr int BM = 16 * MT;
  typedef typename ScaleVec<SG>::s svec;
  typedef typename ScaleVec<SG>::z zvec;
  __shared__ u32x4 sx[2][BM * 16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, g = lane >> 4;
  const int split = blockIdx.x % a.split;
  const Place at = place_of(blockIdx.x / a.split, groups, a.offsets);
  const RowTile t = Tiles<BM>(a.offsets, a.n, a.T).find(at.tile);
  if (t.rows <= 0) return;
  const int nb0 = (at.run * 4 + wave) * R;
  const uint8_t* w = a.w + (size_t)max(t.e, 0) * a.stride;
  const int kb0 = (int)((int64_t)a.KB * split / a.split), kb1 = (int)((int64_t)a.KB * (split + 1) / a.split);
  by_height<MT>(t.rows, [&](auto mt) {
    constexpr int M = decltype(mt)::value;  // groups of 16 rows that hold rows
    f32x4 acc[M][R];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int r = 0; r < R; ++r) acc[m][r] = f32x4{};
    if (t.e >= 0 && kb0 < kb1) {
      typedef Stage<DT, M, kBlockCols, true> St;
      constexpr int D = steps_ahead(M);
      const St st(a, t, a.K);
      struct Step {
        typename St::Pieces x;
        u32x4 w[R];
        svec s[R];
        zvec z[R];
      } step[D];
      // (steps past the last read it again and go unused: without branches around loads
      // the waits for them are exact)
      const auto load = [&](Step& u, int kb) {
        kb = min(kb, kb1 - 1);
        st.load(u.x, kb * kBlockCols);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const size_t block = (size_t)min(nb0 + r, a.NB - 1) * a.KB + kb;
          u.w[r] = ((const u32x4*)(w + block * kBlockBytes))[lane];
          u.s[r] = ((const svec*)(w + a.soff))[block * 16 + li];
          if (ZP) u.z[r] = ((const zvec*)(w + a.zoff))[block * 16 + li];
        }
      };
#pragma unroll
      for (int d = 0; d < D; ++d) load(step[d], kb0 + d);
      st.store(step[0].x, sx[0], kb0 * kBlockCols);
      lds_barrier();
      int buf = 0;
      for (int k0 = kb0; k0 < kb1; k0 += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          const int kb = k0 + d;
          if (kb >= kb1) break;
          u32x4 wv[R];
          svec sv[R];
          zvec zv[R];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            wv[r] = step[d].w[r];
            sv[r] = step[d].s[r];
            zv[r] = step[d].z[r];
          }
          load(step[d], kb + D);
          const u32x4* x = sx[buf];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            constexpr int GS = 4 / SG;
            v8_t<DT> wf[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
              GroupScale<DT, ZP> s;
              s.set((uint16_t)((uint64_t)sv[r] >> (16 * (j / GS))), ZP ? (int)(int8_t)((uint32_t)zv[r] >> (8 * (j / GS))) : 0);
              wf[r] = s.weights(wv[r][j]);
            }
#pragma unroll
            for (int m = 0; m < M; ++m) {
              const v8_t<DT> xf = __builtin_bit_cast(v8_t<DT>, x[piece_at<kBlockCols>(16 * m + li, 4 * j + g)]);
#pragma unroll
              for (int r = 0; r < R; ++r) acc[m][r] = Mat<DT>::mma(wf[r], xf, acc[m][r]);
            }
          }
          buf ^= 1;
          st.store(step[(d + 1) % D].x, sx[buf], min(kb + 1, kb1 - 1) * kBlockCols);
          lds_barrier();
        }
      }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = 16 * m + li, n = (nb0 + r) * kBlockRows + 4 * g;
        if (row < t.rows && n < a.N) put4<DT>(a, a.N, split, t.r0 + row, n, acc[m][r]);
      }
  });
}

// ---------------------------------------------------------------------------
// Gradient of the rows: the contraction runs across the matrix' rows.  A step takes
// 64 of them: the packed blocks pass through LDS as they are, and
// ds_read_b64_tr_b4 hands lane j of 16 the nibble j of 16 rows' eight bytes, so that
// a lane holds 16 rows of one column.  The rows' addresses are given in the order
// that puts neighbouring rows into the operands' halves.  A wavefront takes 64
// columns (eight bytes of each lane's sixteen) and all rows of the tile.
// ---------------------------------------------------------------------------
constexpr int kStepRows = 64;
constexpr int kGradCols = 256;

// As GroupScale, with a scale for each of the eight.
template <int DT, bool ZP>
struct RowScales;
template <bool ZP>
struct RowScales<MOE_T_F16, ZP> {
  half2_t s[4], c[4];
  // sv: eight scales; cv: eight values -(1032 + z)
  __device__ __forceinline__ void set(u32x4 sv, u32x4 cv) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = as_half2(sv[i]);
      c[i] = ZP ? as_half2(cv[i]) : both((_Float16)-1032.0f);
    }
  }
  __device__ __forceinline__ v8_t<MOE_T_F16> weights(uint32_t d) const {
    const half2_t k = both((_Float16)960.0f), sixteenth = both((_Float16)0.0625f);
    half2_t v[4];
    code_pairs(d, v);
    v[0] = (v[0] + c[0]) * s[0];
    v[1] = (v[1] * sixteenth + (c[1] + k)) * s[1];
    v[2] = (v[2] + c[2]) * s[2];
    v[3] = (v[3] * sixteenth + (c[3] + k)) * s[3];
    return __builtin_bit_cast(v8_t<MOE_T_F16>, u32x4{bits_of(v[0]), bits_of(v[1]), bits_of(v[2]), bits_of(v[3])});
  }
};
template <bool ZP>
struct RowScales<MOE_T_BF16, ZP> {
  float s[8], c[8];  // of pairs 1 and 3: for 1024 + 16 u
  // cv: eight values -(8 + z)
  __device__ __forceinline__ void set(u32x4 sv, u32x4 cv) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool high = i / 2 & 1;
      const float f = scale_value<MOE_T_BF16>((uint16_t)(sv[i / 2] >> (16 * (i & 1))));
      c[i] = ((ZP ? scale_value<MOE_T_BF16>((uint16_t)(cv[i / 2] >> (16 * (i & 1)))) : -8.0f) - (high ? 64.0f : 1024.0f)) * f;
      s[i] = high ? f * 0.0625f : f;
    }
  }
  __device__ __forceinline__ v8_t<MOE_T_BF16> weights(uint32_t d) const {
    half2_t v[4];
    code_pairs(d, v);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = pack_bf16(fmaf((float)v[i][0], s[2 * i], c[2 * i]), fmaf((float)v[i][1], s[2 * i + 1], c[2 * i + 1]));
    return __builtin_bit_cast(v8_t<MOE_T_BF16>, r);
  }
};

template <int DT, int SG, bool ZP, int MT>
__global__ __launch_bounds__(kTileThreads, 2) void k_w4_grad(W4Args a, int groups) {
  constexpr int BM = 16 * MT;
  constexpr int CB = kGradCols / kBlockCols, SB = kStepRows / kBlockRows;  // blocks of a step: SB x CB
  constexpr int NS = SB * CB * 16 * SG, SP = (NS + kTileThreads - 1) / kTileThreads;
  typedef int v2i __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  __shared__ u32x4 sx[2][BM * 8];
  __shared__ u32x4 sw[2][SB * CB * 64];
  __shared__ __attribute__((aligned(16))) uint16_t ss[2][CB * SG][kStepRows], sz[ZP ? 2 : 1][CB * SG][kStepRows];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, g = lane >> 4;
  const int split = blockIdx.x % a.split;
  const Place at = place_of(blockIdx.x / a.split, groups, a.offsets);
  const RowTile t = Tiles<BM>(a.offsets, a.n, a.T).find(at.tile);
  if (t.rows <= 0) return;
  const int kb0 = at.run * CB;
  const uint8_t* w = a.w + (size_t)max(t.e, 0) * a.stride;
  const int steps = (a.NB + SB - 1) / SB;
  const int s0 = (int)((int64_t)steps * split / a.split), s1 = (int)((int64_t)steps * (split + 1) / a.split);
  const int kbi = wave >> 1, jj = wave & 1;
  // group of this lane's columns among the step's
  const int cg = kbi * SG + (SG == 4 ? 2 * jj + (li >> 3) : SG == 2 ? jj : 0);
  const int rho = (li & 8) + ((li & 7) < 4 ? 2 * (li & 7) : 2 * (li & 7) - 7);  // the row whose eight bytes this lane points at
  by_height<MT>(t.rows, [&](auto mt) {
    constexpr int M = decltype(mt)::value;
    f32x4 acc[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[m][f] = f32x4{};
    if (t.e >= 0 && s0 < s1) {
      typedef Stage<DT, M, kStepRows, false> St;
      constexpr int D = steps_ahead(M);
      const St st(a, t, a.N);
      struct Step {
        typename St::Pieces x;
        u32x4 w[2];
        uint16_t s[SP];
        int8_t z[SP];
      } step[D];
      // this thread's pieces of a step: blocks past the matrix repeat its last with scale 0
      const int wi = threadIdx.x & 63, wk = min(kb0 + (int)(threadIdx.x >> 6 & 1), a.KB - 1);
      const auto load = [&](Step& u, int s) {
        s = min(s, s1 - 1);
        st.load(u.x, s * kStepRows);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int rb = min(s * SB + (int)(threadIdx.x >> 7) + 2 * p, a.NB - 1);
          u.w[p] = ((const u32x4*)(w + ((size_t)rb * a.KB + wk) * kBlockBytes))[wi];
        }
#pragma unroll
        for (int p = 0; p < SP; ++p) {
          const int i = min((int)threadIdx.x + p * kTileThreads, NS - 1);
          const int rb = s * SB + i / (CB * 16 * SG), kb = kb0 + i / (16 * SG) % CB;
          const size_t at = ((size_t)min(rb, a.NB - 1) * a.KB + min(kb, a.KB - 1)) * 16 * SG + i % (16 * SG);
          u.s[p] = ((const uint16_t*)(w + a.soff))[at];
          if (ZP) u.z[p] = ((const int8_t*)(w + a.zoff))[at];
        }
      };
      const auto store = [&](const Step& u, int buf, int s) {
        s = min(s, s1 - 1);
        st.store(u.x, sx[buf], s * kStepRows);
#pragma unroll
        for (int p = 0; p < 2; ++p) sw[buf][threadIdx.x + p * kTileThreads] = u.w[p];
#pragma unroll
        for (int p = 0; p < SP; ++p) {
          const int i = threadIdx.x + p * kTileThreads;
          if (NS % kTileThreads && i >= NS) break;
          const int rb = s * SB + i / (CB * 16 * SG), kb = kb0 + i / (16 * SG) % CB;
          const int row = i / (CB * 16 * SG) * 16 + i / SG % 16, col = i / (16 * SG) % CB * SG + i % SG;
          ss[buf][col][row] = rb < a.NB && kb < a.KB ? u.s[p] : 0;
          if (ZP)
            sz[buf][col][row] = DT == MOE_T_F16 ? __builtin_bit_cast(uint16_t, (_Float16)(float)(-1032 - u.z[p]))
                                                : __builtin_bit_cast(uint16_t, (__bf16)(float)(-8 - u.z[p]));
        }
      };
#pragma unroll
      for (int d = 0; d < D; ++d) load(step[d], s0 + d);
      store(step[0], 0, s0);
      lds_barrier();
      int buf = 0;
      for (int k0 = s0; k0 < s1; k0 += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          const int s = k0 + d;
          if (s >= s1) break;
          load(step[d], s + D);
          v2i code[4];
#pragma unroll
          for (int f = 0; f < 4; ++f)
            code[f] = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                (lds_v2i*)((char*)&sw[buf][(g * CB + kbi) * 64 + f * 16 + rho] + 8 * jj));
#pragma unroll
          for (int q = 0; q < 2; ++q) {  // rows 16 g + 8 q .. + 7 of the step
            RowScales<DT, ZP> rs;
            rs.set(*(const u32x4*)&ss[buf][cg][16 * g + 8 * q], *(const u32x4*)&sz[ZP ? buf : 0][cg][16 * g + 8 * q]);
            v8_t<DT> wf[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) wf[f] = rs.weights((uint32_t)code[f][q]);
#pragma unroll
            for (int m = 0; m < M; ++m) {
              const v8_t<DT> xf = __builtin_bit_cast(v8_t<DT>, sx[buf][piece_at<kStepRows>(16 * m + li, 2 * g + q)]);
#pragma unroll
              for (int f = 0; f < 4; ++f) acc[m][f] = Mat<DT>::mma(wf[f], xf, acc[m][f]);
            }
          }
          buf ^= 1;
          store(step[(d + 1) % D], buf, s + 1);
          lds_barrier();
        }
      }
    }
    // lane's sums 4 g .. + 3 of fragment f: nibbles 4 g .. + 3 of the eight bytes
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int row = 16 * m + li;
        const int c = (kb0 + kbi) * kBlockCols + 32 * (2 * jj + (g >> 1)) + 8 * f + 4 * (g & 1);
        if (row < t.rows && c < a.K) put4<DT>(a, a.K, split, t.r0 + row, c, acc[m][f]);
      }
  });
}

// The splits' partial sums added in their order.
template <int DT>
__global__ __launch_bounds__(256) void k_w4_sum(W4Args a, int width) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = width / 4, row = i / per;
  if (row >= a.T) return;
  const int c = (int)(i % per) * 4;
  f32x4 v{};
  for (int s = 0; s < a.split; ++s) v += *(const f32x4*)(a.part + ((int64_t)s * a.T + row) * width + c);
  W4Args o = a;
  o.part = nullptr;
  put4<DT>(o, width, 0, row, c, v);
}

// ---------------------------------------------------------------------------
// Packing.
// ---------------------------------------------------------------------------
struct PackArgs {
  uint8_t* packed;
  size_t stride, soff, zoff;
  int N, K, NB, KB, group, SG, dtype;
  uint8_t* q;
  uint16_t* scales;
  int8_t* zeros;
};

// One workgroup per block and matrix.
template <bool PACK>
__global__ __launch_bounds__(64) void k_w4_pack(PackArgs a) {
  const int lane = threadIdx.x, li = lane & 15, g = lane >> 4;
  const size_t block = blockIdx.x;
  const int nb = (int)(block / a.KB), kb = (int)(block % a.KB), e = blockIdx.y, row = nb * kBlockRows + li;
  uint8_t* w = a.packed + (size_t)e * a.stride;
  const bool in = row < a.N;
  const size_t r = (size_t)e * a.N + row;
  u32x4* mine = (u32x4*)(w + block * kBlockBytes) + lane;
  u32x4 d{0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
  if (!PACK) d = *mine;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = kb * kBlockCols + 32 * j + 8 * g;
    if (!in || c >= a.K) continue;
    // (K is a multiple of 32: a dword of canonical codes is aligned)
    uint32_t* at = (uint32_t*)(a.q + (r * a.K + c) / 2);
    if (PACK) d[j] = *at ^ 0x88888888u;
    else *at = d[j] ^ 0x88888888u;
  }
  if (PACK) *mine = d;
  const int width = kBlockCols / a.SG, groups = a.K / a.group;
  for (int i = lane; i < 16 * a.SG; i += 64) {
    const int rr = nb * kBlockRows + i / a.SG, c = kb * kBlockCols + i % a.SG * width;
    const bool have = rr < a.N && c < a.K;
    uint16_t* s = (uint16_t*)(w + a.soff) + block * 16 * a.SG + i;
    int8_t* z = (int8_t*)(w + a.zoff) + block * 16 * a.SG + i;
    const size_t from = ((size_t)e * a.N + rr) * groups + c / a.group;
    if (PACK) {
      *s = have ? a.scales[from] : 0;
      if (a.zeros) *z = have ? a.zeros[from] : 0;
    } else if (have && c % a.group == 0) {
      a.scales[from] = *s;
      if (a.zeros) a.zeros[from] = *z;
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr int64_t kMaxLd = 1 << 22;
constexpr int kFewRows = 16;
constexpr int kCUs = 256;

struct W4Layout {
  int NB, KB, SG;
  size_t soff, zoff, stride;
};

W4Layout w4_layout(const moe_w4_dims_t& d) {
  W4Layout l;
  l.NB = ceil_div(d.N, kBlockRows);
  l.KB = ceil_div(d.K, kBlockCols);
  l.SG = d.group == 32 ? 4 : d.group == 64 ? 2 : 1;
  const size_t blocks = (size_t)l.NB * l.KB;
  l.soff = blocks * kBlockBytes;
  l.zoff = l.soff + round256(blocks * 16 * l.SG * 2);
  l.stride = l.zoff + (d.zeros ? round256(blocks * 16 * l.SG) : 0);
  return l;
}

int check_w4(const moe_w4_dims_t* d) {
  if (!d || d->n < 1 || d->N <= 0 || d->K <= 0 || d->group <= 0 || (d->zeros != 0 && d->zeros != 1)) return MOE_E_INVAL;
  if (d->dtype != MOE_T_F16 && d->dtype != MOE_T_BF16) return MOE_E_INVAL;
  if (d->K % d->group) return MOE_E_INVAL;
  if (d->K % 32 || d->K > kMaxWidth || d->N % 8 || d->N > (1 << 20) || d->n > kMaxExperts ||
      (int64_t)d->n * d->N > (1 << 24))
    return MOE_E_UNSUPPORTED;
  if (d->group != 32 && d->group != 64 && d->group % 128 && d->group != d->K) return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

int check_w4_rows(const moe_w4_dims_t* d, int32_t T) {
  const int st = check_w4(d);
  if (st != MOE_OK) return st;
  if (T < 0) return MOE_E_INVAL;
  return T > kMaxRows || (int64_t)T * std::max(d->N, d->K) > kMaxElems ? MOE_E_UNSUPPORTED : MOE_OK;
}

bool few_rows(const moe_w4_dims_t& d, int T) { return T <= (int64_t)kFewRows * d.n; }

// Tiles of a call with many rows: MT groups of 16 rows by 64 R weight rows (forward) or
// 256 columns (gradient), and parts that a tile's sums are split into.
struct TilePlan {
  int MT, R, groups, split;
};

// Measured in us; 6144 x 6144 unless said.  One matrix: the largest tiles that still give
// nearly two workgroups per CU (8,192 rows of 8192 x 8192: forward 128 x 256 1,033, 64 x
// 256 1,223, gradient 128 rows 1,112, 96 1,161, 64 1,290; 2,048 rows: forward 128 x 256 185
// (384 workgroups), 128 x 192 163 (512), gradient 128 rows 203, 96 183), else 64 rows
// (2,048 rows of 2048 x 6144: 128 x 256 115, 64 x 256 69).  Experts: 128 (gradient 96) rows
// only where they have that many on average (256 experts, 2048 x 1024, of 128 rows 180,
// in tiles of 64 238; 16,384 rows by Zipf's law 167 and 153; their gradient 88 and 89).
// The sums are split while all workgroups are resident at once (64 rows: 4 parts 19.7, 8
// 13.8, 12 17.1, with 24 tiles).
constexpr int kTwoPerCU = 460, kOnePerCU = 256, kStepsPerPart = 3;

TilePlan plan_tiles(const moe_w4_dims_t& d, int T, bool grad) {
  TilePlan p;
  const int avg = ceil_div(T, d.n);
  const auto blocks = [&](int MT, int R) {
    return (int64_t)ceil_div(T, 16 * MT) * (grad ? ceil_div(d.K, kGradCols) : ceil_div(d.N, 64 * R));
  };
  p.R = 4;
  if (avg <= 32) {
    p.MT = 2;
  } else if (d.n > 1) {
    p.MT = avg <= 96 ? 4 : grad ? 6 : 8;
  } else if (blocks(8, 4) >= kTwoPerCU) {
    p.MT = 8;
  } else if (grad) {
    p.MT = blocks(6, 4) >= kTwoPerCU ? 6 : 4;
  } else {
    p.R = blocks(8, 3) >= kTwoPerCU ? 3 : 4;
    p.MT = p.R == 3 ? 8 : 4;
  }
  p.groups = grad ? ceil_div(d.K, kGradCols) : ceil_div(d.N, 64 * p.R);
  const int steps = grad ? ceil_div(d.N, kStepRows) : ceil_div(d.K, kBlockCols);
  p.split = (int)std::max<int64_t>(1, std::min<int64_t>(kOnePerCU / blocks(p.MT, p.R), steps / kStepsPerPart));
  return p;
}

size_t part_bytes(const moe_w4_dims_t& d, int T, const TilePlan& p, bool grad) {
  return p.split > 1 ? (size_t)p.split * T * (grad ? d.K : d.N) * 4 : 0;
}

template <typename F>
void by_format(const moe_w4_dims_t& d, int SG, F f) {
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

int check_call(const moe_w4_dims_t* d, const void* packed, const void* x, int64_t ldx, int into, int32_t T,
               const int32_t* offsets, const void* add, int64_t ldadd, const void* y, int64_t ldy, int out) {
  if (bad(packed, 256)) return MOE_E_INVAL;
  if (offsets ? !aligned_to(offsets, 4) : d->n != 1) return MOE_E_INVAL;
  if (T == 0) return MOE_OK;
  if (bad(x, 16) || bad_ld(ldx, into) || bad(y, 16) || bad_ld(ldy, out)) return MOE_E_INVAL;
  if (add && (!aligned_to(add, 16) || bad_ld(ldadd, out))) return MOE_E_INVAL;
  return ldx > kMaxLd || ldy > kMaxLd || (add && ldadd > kMaxLd) ? MOE_E_UNSUPPORTED : MOE_OK;
}

template <int DT>
void launch_sum(const W4Args& a, int width, hipStream_t s) {
  k_w4_sum<DT><<<ceil_div((int64_t)a.T * (width / 4), 256), 256, 0, s>>>(a, width);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_w4_packed_bytes(const moe_w4_dims_t* d) {
  return check_w4(d) == MOE_OK ? (size_t)d->n * w4_layout(*d).stride : 0;
}

static int pack_call(const moe_w4_dims_t* d, const void* q, const void* scales, const void* zeros, const void* packed,
                     bool pack, void* stream) {
  const int st = check_w4(d);
  if (st != MOE_OK) return st;
  if (bad(q, 16) || bad(scales, 2) || bad(packed, 256) || (d->zeros != 0) != (zeros != nullptr)) return MOE_E_INVAL;
  const W4Layout l = w4_layout(*d);
  const PackArgs a{(uint8_t*)packed, l.stride, l.soff, l.zoff, d->N, d->K, l.NB, l.KB, d->group, l.SG, d->dtype,
                   (uint8_t*)q, (uint16_t*)scales, (int8_t*)zeros};
  const dim3 grid((unsigned)(l.NB * l.KB), (unsigned)d->n);
  if (pack) k_w4_pack<true><<<grid, 64, 0, (hipStream_t)stream>>>(a);
  else k_w4_pack<false><<<grid, 64, 0, (hipStream_t)stream>>>(a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

int moe_w4_pack(const moe_w4_dims_t* d, const void* q, const void* scales, const void* zeros, void* packed,
                void* stream) {
  return pack_call(d, q, scales, zeros, packed, true, stream);
}

int moe_w4_unpack(const moe_w4_dims_t* d, const void* packed, void* q, void* scales, void* zeros, void* stream) {
  return pack_call(d, q, scales, zeros, packed, false, stream);
}

int32_t moe_w4_few_rows(const moe_w4_dims_t* d, int32_t T) {
  return check_w4_rows(d, T) == MOE_OK && few_rows(*d, T) ? 1 : 0;
}

size_t moe_w4_workspace_bytes(const moe_w4_dims_t* d, int32_t T) {
  if (check_w4_rows(d, T) != MOE_OK || T == 0) return 0;
  const size_t f = few_rows(*d, T) ? 0 : part_bytes(*d, T, plan_tiles(*d, T, false), false);
  return std::max(f, part_bytes(*d, T, plan_tiles(*d, T, true), true));
}

int moe_w4_forward(const moe_w4_dims_t* d, const void* packed, const void* x, int64_t ldx, int32_t T,
                   const int32_t* offsets, const void* add, int64_t ldadd, void* y, int64_t ldy, void* ws,
                   size_t ws_bytes, void* stream) {
  int st = check_w4_rows(d, T);
  if (st == MOE_OK) st = check_call(d, packed, x, ldx, d->K, T, offsets, add, ldadd, y, ldy, d->N);
  if (st != MOE_OK || T == 0) return st;
  const W4Layout l = w4_layout(*d);
  const hipStream_t s = (hipStream_t)stream;
  W4Args a{(const uint8_t*)packed, l.stride, l.soff, l.zoff, d->n, d->N, d->K, l.NB, l.KB, x, ldx, T, offsets, add,
           ldadd, y, ldy, nullptr, 1};
  if (few_rows(*d, T)) {
    const int64_t items = max_tiles(d->n, T, 16, offsets != nullptr) * l.NB;
    by_format(*d, l.SG, [&](auto dt, auto sg, auto zp) {
      constexpr int DT = decltype(dt)::value, SG = decltype(sg)::value;
      constexpr bool ZP = decltype(zp)::value;
      const auto launch = [&](auto kernel, int W, int per_cu) {
        kernel<<<(unsigned)std::min<int64_t>(items, kCUs * per_cu), 64 * W, 0, s>>>(a);
      };
      if (l.KB <= 4) launch(k_w4_few<DT, SG, ZP, 4, 1>, 4, 6);
      else if (l.KB <= 8) launch(k_w4_few<DT, SG, ZP, 4, 2>, 4, 5);
      else if (l.KB <= 16) launch(k_w4_few<DT, SG, ZP, 8, 2>, 8, 2);
      else launch(k_w4_few<DT, SG, ZP, 16, 3>, 16, 1);
    });
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
  }
  const TilePlan p = plan_tiles(*d, T, false);
  const size_t need = part_bytes(*d, T, p, false);
  if (need) {
    if (bad(ws, 16)) return MOE_E_INVAL;
    if (ws_bytes < need) return MOE_E_WORKSPACE;
    a.part = (float*)ws;
    a.split = p.split;
  }
  by_format(*d, l.SG, [&](auto dt, auto sg, auto zp) {
    constexpr int DT = decltype(dt)::value, SG = decltype(sg)::value;
    constexpr bool ZP = decltype(zp)::value;
    const unsigned blocks =
        (unsigned)(places(max_tiles(d->n, T, 16 * p.MT, offsets != nullptr), p.groups, offsets != nullptr) * p.split);
    if (p.MT == 2) k_w4_rows<DT, SG, ZP, 2, 4><<<blocks, kTileThreads, 0, s>>>(a, p.groups);
    else if (p.MT == 4) k_w4_rows<DT, SG, ZP, 4, 4><<<blocks, kTileThreads, 0, s>>>(a, p.groups);
    else if (p.R == 3) k_w4_rows<DT, SG, ZP, 8, 3><<<blocks, kTileThreads, 0, s>>>(a, p.groups);
    else k_w4_rows<DT, SG, ZP, 8, 4><<<blocks, kTileThreads, 0, s>>>(a, p.groups);
    if (need) launch_sum<DT>(a, d->N, s);
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

int moe_w4_backward(const moe_w4_dims_t* d, const void* packed, const void* dy, int64_t lddy, int32_t T,
                    const int32_t* offsets, const void* add, int64_t ldadd, void* dx, int64_t lddx, void* ws,
                    size_t ws_bytes, void* stream) {
  int st = check_w4_rows(d, T);
  if (st == MOE_OK) st = check_call(d, packed, dy, lddy, d->N, T, offsets, add, ldadd, dx, lddx, d->K);
  if (st != MOE_OK || T == 0) return st;
  const W4Layout l = w4_layout(*d);
  const hipStream_t s = (hipStream_t)stream;
  const TilePlan p = plan_tiles(*d, T, true);
  const size_t need = part_bytes(*d, T, p, true);
  if (need && bad(ws, 16)) return MOE_E_INVAL;
  if (ws_bytes < need) return MOE_E_WORKSPACE;
  const W4Args a{(const uint8_t*)packed, l.stride, l.soff, l.zoff, d->n, d->N, d->K, l.NB, l.KB, dy, lddy, T, offsets,
                 add, ldadd, dx, lddx, need ? (float*)ws : nullptr, p.split};
  by_format(*d, l.SG, [&](auto dt, auto sg, auto zp) {
    constexpr int DT = decltype(dt)::value, SG = decltype(sg)::value;
    constexpr bool ZP = decltype(zp)::value;
    const unsigned blocks =
        (unsigned)(places(max_tiles(d->n, T, 16 * p.MT, offsets != nullptr), p.groups, offsets != nullptr) * p.split);
    if (p.MT == 2) k_w4_grad<DT, SG, ZP, 2><<<blocks, kTileThreads, 0, s>>>(a, p.groups);
    else if (p.MT == 4) k_w4_grad<DT, SG, ZP, 4><<<blocks, kTileThreads, 0, s>>>(a, p.groups);
    else if (p.MT == 6) k_w4_grad<DT, SG, ZP, 6><<<blocks, kTileThreads, 0, s>>>(a, p.groups);
    else k_w4_grad<DT, SG, ZP, 8><<<blocks, kTileThreads, 0, s>>>(a, p.groups);
    if (need) launch_sum<DT>(a, d->K, s);
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // extern "C"
