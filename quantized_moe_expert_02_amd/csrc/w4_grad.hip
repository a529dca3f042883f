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
// 2048 x 6144 binary16 64 us (0.81 PFLOP/s), 16,384 rows of 256 experts of 2048 x 512
// bfloat16, laid out by Zipf's law, 90 us.
// ---------------------------------------------------------------------------
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

}  // namespace

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
