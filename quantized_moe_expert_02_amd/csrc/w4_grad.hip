// The gradient of rows multiplied by 4-bit weights (include/moe_w4.h, layout in w4.h).
#include "w4.h"

namespace moe {

namespace {

// ---------------------------------------------------------------------------
// Gradient of the rows: the contraction runs across the matrix' rows.  A step takes
// 64 of them: the packed blocks pass through LDS as they are, and
// ds_read_b64_tr_b4 hands lane j of 16 the nibble j of 16 rows' eight bytes, so that
// a lane holds 16 rows of one column.  The rows' addresses are given in the order
// that puts neighbouring rows into the operands' halves.  A wavefront takes 64
// columns (eight bytes of each lane's sixteen) and all rows of the tile.
// Turned are codes, a quarter of what turning decoded weights would move.  Bound, as the
// forward product, by decoding and matrix instructions, which take turns: 2,048 rows of
// 2048 x 6144 binary16 64 us (0.81 PFLOP/s; vector instructions 56% and matrix instructions
// 37% of a busy CU's cycles), 16,384 rows of 256 experts of 2048 x 512 bfloat16, laid out by
// Zipf's law, 90 us (64% and 25%, and a third of the CUs' time without a workgroup: some 840
// of unlike length on 512 places).
// ---------------------------------------------------------------------------
// As GroupScale (w4.h, also on why weights are rounded), with a scale for each of the eight.
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
// bfloat16: the factor s and the addend c of (1024 + u) s + c, or (1024 + 16 u) s + c for
// pairs 1 and 3, are made once for all wavefronts, where the scales are staged.
template <bool ZP>
struct RowScales<MOE_T_BF16, ZP> {
  float2 f[8];
  __device__ __forceinline__ void set(const float2* p) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const f32x4 v = *(const f32x4*)(p + i);
      f[i] = make_float2(v[0], v[1]);
      f[i + 1] = make_float2(v[2], v[3]);
    }
  }
  // for row `row` of a step
  static __device__ __forceinline__ float2 of(uint16_t scale, int z, int row) {
    const float v = scale_value<MOE_T_BF16>(scale);
    return row & 2 ? make_float2(v * 0.0625f, (float)(-72 - z) * v) : make_float2(v, (float)(-1032 - z) * v);
  }
  __device__ __forceinline__ v8_t<MOE_T_BF16> weights(uint32_t d) const {
    half2_t v[4];
    code_pairs(d, v);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = pack_bf16(fmaf((float)v[i][0], f[2 * i].x, f[2 * i].y),
                       fmaf((float)v[i][1], f[2 * i + 1].x, f[2 * i + 1].y));
    return __builtin_bit_cast(v8_t<MOE_T_BF16>, r);
  }
};

__device__ __forceinline__ uint32_t bits(float v) { return __builtin_bit_cast(uint32_t, v); }

template <int DT, int SG, bool ZP, int MT>
__global__ __launch_bounds__(kTileThreads, 2) void k_w4_grad(W4Args a, int groups) {
  constexpr int BM = 16 * MT;
  constexpr int CB = kGradCols / kBlockCols, SB = kStepRows / kBlockRows;  // blocks of a step: SB x CB
  constexpr int NS = SB * CB * 16 * SG, SP = (NS + kTileThreads - 1) / kTileThreads;
  typedef int v2i __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  __shared__ u32x4 sx[2][BM * 8];
  __shared__ u32x4 sw[2][SB * CB * 64];
  // scales by group and row: as they are with the zero points' -(1032 + z), or as RowScales has them
  constexpr bool F16 = DT == MOE_T_F16;
  __shared__ __attribute__((aligned(16))) uint16_t ss[F16 ? 2 : 1][CB * SG][F16 ? kStepRows : 8],
      sz[F16 && ZP ? 2 : 1][CB * SG][F16 ? kStepRows : 8];
  __shared__ __attribute__((aligned(16))) float2 sf[F16 ? 1 : 2][CB * SG][F16 ? 2 : kStepRows];
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
  // the row whose eight bytes this lane points at
  const int rho = (li & 8) + ((li & 7) < 4 ? 2 * (li & 7) : 2 * (li & 7) - 7);
  by_height<MT, false>(t.rows, [&](auto mt) {
    constexpr int M = decltype(mt)::value;
    f32x4 acc[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[m][f] = f32x4{};
    if (t.e >= 0 && s0 < s1) {
      typedef Stage<DT, M, kStepRows> St;
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
          const uint16_t sc = rb < a.NB && kb < a.KB ? u.s[p] : 0;
          const int z = ZP ? u.z[p] : 0;
          if constexpr (F16) {
            ss[buf][col][row] = sc;
            if (ZP) sz[buf][col][row] = __builtin_bit_cast(uint16_t, (_Float16)(float)(-1032 - z));
          } else {
            sf[buf][col][row] = RowScales<DT, ZP>::of(sc, z, row);
          }
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
          __builtin_amdgcn_sched_barrier(0);  // (or the loads sink to where their results are used)
          v2i code[4];
#pragma unroll
          for (int f = 0; f < 4; ++f)
            code[f] = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                (lds_v2i*)((char*)&sw[buf][(g * CB + kbi) * 64 + f * 16 + rho] + 8 * jj));
#pragma unroll
          for (int q = 0; q < 2; ++q) {  // rows 16 g + 8 q .. + 7 of the step
            RowScales<DT, ZP> rs;
            const int r0 = 16 * g + 8 * q;
            if constexpr (F16) {
              u32x4 zs{};
              if constexpr (ZP) zs = *(const u32x4*)&sz[buf][cg][r0];
              rs.set(*(const u32x4*)&ss[buf][cg][r0], zs);
            } else {
              rs.set(&sf[buf][cg][r0]);
            }
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
    // A lane's sums of fragment f belong to nibbles 4 g .. + 3 of the eight bytes: the even
    // columns of eight where g is even, else the odd ones.  Two exchanges between
    // neighbouring g give each four columns in a row.
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const auto lo = __builtin_amdgcn_permlane16_swap(bits(acc[m][f][0]), bits(acc[m][f][2]), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(bits(acc[m][f][1]), bits(acc[m][f][3]), false, false);
        const f32x4 v = __builtin_bit_cast(f32x4, u32x4{lo[0], lo[1], hi[0], hi[1]});
        const int row = 16 * m + li;
        const int c = (kb0 + kbi) * kBlockCols + 32 * (2 * jj + (g >> 1)) + 8 * f + 4 * (g & 1);
        if (row < t.rows && c < a.K) put4<DT>(a, a.K, split, t.r0 + row, c, v);
      }
  });
}

// ---------------------------------------------------------------------------
// Few rows: a workgroup takes 64 columns (eight bytes of each lane's sixteen of a block); its W
// wavefronts take the steps of 64 matrix rows in turn and add their sums through LDS, so
// that no partial sums go through memory and one launch does.  A wavefront has its own
// LDS and no barriers until the end; rows and scales come from memory straight into operands.
// Bound by its chain of loads, codes' turn and sum: 45 rows of 1000 x 2080 binary16, groups
// of 32 with zero points, 5.8 us (split over workgroups and summed 11.3).
// ---------------------------------------------------------------------------
// The scales and zero points of eight rows, as memory holds them, for a lane's group `in` of SG.
template <int DT, int SG, bool ZP>
struct EightRows {
  u32x4 s[SG];
  uint32_t z[ZP ? 2 * SG : 1];
  __device__ __forceinline__ void load(const uint8_t* scales, const uint8_t* zeros, size_t at) {
#pragma unroll
    for (int i = 0; i < SG; ++i) s[i] = ((const u32x4*)(scales + at * 2))[i];
    if constexpr (ZP) {
#pragma unroll
      for (int i = 0; i < 2 * SG; ++i) z[i] = ((const uint32_t*)(zeros + at))[i];
    }
  }
  // scales of rows 2 i and 2 i + 1
  __device__ __forceinline__ uint32_t pair(int i, int in) const {
    if constexpr (SG == 1) return s[0][i];
    const auto word = [&](int r) -> uint32_t {
      if constexpr (SG == 2) return s[r / 4][r % 4];
      const uint32_t lo = s[r * SG / 8][r % 2 * 2], hi = s[r * SG / 8][r % 2 * 2 + 1];
      return in & 2 ? hi : lo;
    };
    return __builtin_amdgcn_perm(word(2 * i + 1), word(2 * i), in & 1 ? 0x07060302u : 0x05040100u);
  }
  __device__ __forceinline__ int zero(int r, int in) const {
    return ZP ? (int)(int8_t)(z[ZP ? r * SG / 4 : 0] >> (8 * (r * SG % 4 + in))) : 0;
  }
  __device__ __forceinline__ RowScales<DT, ZP> get(int in, bool none) const {
    RowScales<DT, ZP> rs;
    u32x4 sv{}, cv{};
#pragma unroll
    for (int i = 0; i < 4; ++i) sv[i] = none ? 0u : pair(i, in);
    if constexpr (DT == MOE_T_F16) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        cv[i] = bits_of(half2_t{(_Float16)(float)(-1032 - zero(2 * i, in)), (_Float16)(float)(-1032 - zero(2 * i + 1, in))});
      rs.set(sv, cv);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) rs.f[i] = RowScales<DT, ZP>::of((uint16_t)(sv[i / 2] >> (16 * (i & 1))), zero(i, in), i);
    }
    return rs;
  }
};

template <int DT, int SG, bool ZP, int M, int W>
__global__ __launch_bounds__(64 * W) void k_w4_grad_few(W4Args a, int groups) {
  constexpr int BM = 16 * M, SB = kStepRows / kBlockRows;
  typedef typename Mat<DT>::elem elem;
  typedef int v2i __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  __shared__ uint64_t sw[W][SB * 64];
  __shared__ f32x4 red[W][4][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, g = lane >> 4;
  const Place at = place_of(blockIdx.x, groups, a.offsets);
  const RowTile t = Tiles<BM>(a.offsets, a.n, a.T).find(at.tile);
  if (t.rows <= 0) return;
  const int h = at.run, kb = h >> 1;  // half block
  const int in = SG == 4 ? 2 * (h & 1) + (li >> 3) : SG == 2 ? h & 1 : 0;
  const int rho = (li & 8) + ((li & 7) < 4 ? 2 * (li & 7) : 2 * (li & 7) - 7);  // as above
  const uint8_t* w = a.w + (size_t)max(t.e, 0) * a.stride;
  const int steps = t.e < 0 ? 0 : (a.NB + SB - 1) / SB;
  f32x4 acc[M][4];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[m][f] = f32x4{};
  struct Step {
    uint64_t w[SB];
    u32x4 x[M][2];
    EightRows<DT, SG, ZP> s[2];
  };
  // (blocks past the matrix repeat its last, with scale 0 and rows of zeros)
  const auto load = [&](Step& u, int s) {
#pragma unroll
    for (int p = 0; p < SB; ++p) {
      const size_t block = (size_t)min(s * SB + p, a.NB - 1) * a.KB + kb;
      u.w[p] = *(const uint64_t*)(w + block * kBlockBytes + lane * 16 + 8 * (h & 1));
    }
    const size_t scales = ((size_t)min(s * SB + g, a.NB - 1) * a.KB + kb) * 16 * SG;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      u.s[q].load(w + a.soff, w + a.zoff, scales + 8 * q * SG);
      const int c = s * kStepRows + 16 * g + 8 * q;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int64_t row = t.r0 + min(16 * m + li, t.rows - 1);
        u.x[m][q] = *(const u32x4*)((const elem*)a.x + row * a.ldx + min(c, a.N - 8));
        if (c >= a.N) u.x[m][q] = u32x4{};
      }
    }
  };
  Step now, next;
  if (wave < steps) load(now, wave);
  for (int s = wave; s < steps; s += W) {
    if (s + W < steps) load(next, s + W);
#pragma unroll
    for (int p = 0; p < SB; ++p) sw[wave][p * 64 + (lane ^ (p & 1) * 16)] = now.w[p];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    v2i code[4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
      code[f] = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
          (lds_v2i*)&sw[wave][g * 64 + ((f * 16 + rho) ^ (g & 1) * 16)]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    const bool none = s * SB + g >= a.NB;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const RowScales<DT, ZP> rs = now.s[q].get(in, none);
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const v8_t<DT> wf = rs.weights((uint32_t)code[f][q]);
#pragma unroll
        for (int m = 0; m < M; ++m) acc[m][f] = Mat<DT>::mma(wf, __builtin_bit_cast(v8_t<DT>, now.x[m][q]), acc[m][f]);
      }
    }
    now = next;
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
#pragma unroll
    for (int f = 0; f < 4; ++f) red[wave][f][lane] = acc[m][f];
    __syncthreads();
    if (wave < 4) {
      f32x4 v = red[0][wave][lane];
#pragma unroll
      for (int u = 1; u < W; ++u) v += red[u][wave][lane];
      const auto lo = __builtin_amdgcn_permlane16_swap(bits(v[0]), bits(v[2]), false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap(bits(v[1]), bits(v[3]), false, false);
      v = __builtin_bit_cast(f32x4, u32x4{lo[0], lo[1], hi[0], hi[1]});
      const int row = 16 * m + li, c = h * 64 + 32 * (g >> 1) + 8 * wave + 4 * (g & 1);
      if (row < t.rows && c < a.K) put4<DT>(a, a.K, 0, t.r0 + row, c, v);
    }
    if (m + 1 < M) __syncthreads();
  }
}

}  // namespace

void launch_w4_grad_few(const W4Args& a, const moe_w4_dims_t& d, const W4Layout& l, int M, hipStream_t s) {
  by_format(d, l.SG, [&](auto dt, auto sg, auto zp) {
    constexpr int DT = decltype(dt)::value, SG = decltype(sg)::value;
    constexpr bool ZP = decltype(zp)::value;
    const int groups = ceil_div(d.K, 64);
    const int64_t tiles = max_tiles(d.n, a.T, 16 * M, a.offsets != nullptr);
    const unsigned grid = (unsigned)places(tiles, groups, a.offsets != nullptr);
    if (M == 1) k_w4_grad_few<DT, SG, ZP, 1, 8><<<grid, 512, 0, s>>>(a, groups);
    else k_w4_grad_few<DT, SG, ZP, 2, 8><<<grid, 512, 0, s>>>(a, groups);
  });
}

void launch_w4_grad(const W4Args& a, const moe_w4_dims_t& d, const W4Layout& l, const TilePlan& p, hipStream_t s) {
  by_format(d, l.SG, [&](auto dt, auto sg, auto zp) {
    constexpr int DT = decltype(dt)::value, SG = decltype(sg)::value;
    constexpr bool ZP = decltype(zp)::value;
    const auto launch = [&](auto kernel) {
      const int64_t tiles = max_tiles(d.n, a.T, 16 * p.MT, a.offsets != nullptr);
      kernel<<<(unsigned)(places(tiles, p.groups, a.offsets != nullptr) * p.split), kTileThreads, 0, s>>>(a, p.groups);
    };
    if (p.MT == 2) launch(k_w4_grad<DT, SG, ZP, 2>);
    else if (p.MT == 4) launch(k_w4_grad<DT, SG, ZP, 4>);
    else launch(k_w4_grad<DT, SG, ZP, 8>);
  });
}

}  // namespace moe
