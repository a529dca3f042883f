// Products of few rows with 4-bit weights (include/moe_w4.h, layout in w4.h).
#include "w4.h"

namespace moe {

namespace {

// ---------------------------------------------------------------------------
// Few rows: an item is 16 rows and one row block of a matrix; the W wavefronts of a
// workgroup split its columns, KPW column blocks each, and add their sums through LDS.
// A workgroup takes a run of items and keeps its rows in registers from item to item
// while the next item's blocks are under way.  The rows are the first operand (index l
// % 16: the row; rows past the tile are zeros) and a block the second (index l %
// 16: its row), so that a lane's four sums belong to one weight row and are
// multiplied by its scale.  The factors are the codes q - z themselves, in bfloat16 2^-15 of
// them (exact too: |q - z| <= 136), so that a group's sum, of up to 128 terms, stays in fp32's
// range whatever the rows hold; the result is multiplied by 2^15.  (Offset codes, 128 + u,
// with (136 + z) times the sum of the row taken off again, take 7 instead of 17 instructions
// per dword, 40.2 us instead of 42.8 below, but lose what stands beside a large element.)
// Bound by memory where there is much to read (64 rows of 256 experts of 2048 x 6144
// binary16, 369 MB: 73 us, 5.1 TB/s).  With groups of 32 and zero points a block of four
// dwords takes 105 vector and 4 matrix instructions beside it, 22 and 3 us of 8 rows of
// 128,000 x 2048 bfloat16, which hide only in part behind its 158 MB: 42.8 us, 3.7 TB/s.  Short
// calls (one row of 6144 x 6144: 9 us): the start, and 384 items on 256 workgroups.  An item
// per workgroup instead of runs: 136 and 61 us for the first two.
// ---------------------------------------------------------------------------
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
  const auto block_of = [&](int pass, int u) { return (pass * KPW + u) * W + wave; };
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
    // (the rows are awaited here: in the loop, where it is not known whether they are still
    // under way, the wait would be for the blocks requested after them too)
#pragma unroll
    for (int u = 0; u < KPW; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(xv[u][j]));
  };
  f32x4 acc;
  const auto multiply = [&](int u) {
#pragma unroll
    for (int s = 0; s < SG; ++s) {
      f32x4 sum{};
      const int z = ZP ? (int)(int8_t)((uint32_t)zv[u] >> (8 * s)) : 0;
      GroupScale<MOE_T_BF16, ZP> small;
      small.set(0x3800, z);  // 2^-15
#pragma unroll
      for (int j = s * GS; j < (s + 1) * GS; ++j) {
        v8_t<DT> b;
        if constexpr (DT == MOE_T_F16) {
          half2_t v[4];
          codes_f16(wv[u][j], both((_Float16)(float)(-1032 - z)), v);
          b = __builtin_bit_cast(v8_t<DT>, u32x4{bits_of(v[0]), bits_of(v[1]), bits_of(v[2]), bits_of(v[3])});
        } else {
          b = small.weights(wv[u][j]);
        }
        sum = Mat<DT>::mma(__builtin_bit_cast(v8_t<DT>, xv[u][j]), b, sum);
      }
      const float f = scale_value<DT>((uint16_t)((uint64_t)sv[u] >> (16 * s)));
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
      if (DT == MOE_T_BF16) v *= 0x1p15f;
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

}  // namespace

void launch_w4_few(const W4Args& a, const moe_w4_dims_t& d, const W4Layout& l, hipStream_t s) {
  const int64_t items = max_tiles(d.n, a.T, 16, a.offsets != nullptr) * l.NB;
  by_format(d, l.SG, [&](auto dt, auto sg, auto zp) {
    constexpr int DT = decltype(dt)::value, SG = decltype(sg)::value;
    constexpr bool ZP = decltype(zp)::value;
    const auto launch = [&](auto kernel, int W, int per_cu) {
      kernel<<<(unsigned)std::min<int64_t>(items, kCUs * per_cu), 64 * W, 0, s>>>(a);
    };
    // Wavefronts and column blocks of each so that W KPW fits the columns, and workgroups as
    // registers allow (us; 128,000 rows, K 2048, T 1, binary16, groups of 128: 4 x 4 28.2, 8 x 2
    // 32.9; T 8, bfloat16, groups of 32 with zero points, which need more registers: 47.6 and
    // 42.8; 24,576 rows, K 2560: 8 x 3 11.7, 16 x 3 14.3; K 5120: 16 x 3 17.7, 8 x 6 19.4;
    // 60,000 rows, K 512: 2 x 2 7.8, 4 x 1 9.8).
    if (l.KB <= 4) launch(k_w4_few<DT, SG, ZP, 2, 2>, 2, 8);
    else if (l.KB <= 8) launch(k_w4_few<DT, SG, ZP, 4, 2>, 4, 5);
    else if (l.KB <= 16 && SG == 1) launch(k_w4_few<DT, SG, ZP, 4, 4>, 4, 3);
    else if (l.KB <= 16) launch(k_w4_few<DT, SG, ZP, 8, 2>, 8, 2);
    else if (l.KB <= 24) launch(k_w4_few<DT, SG, ZP, 8, 3>, 8, 2);
    else launch(k_w4_few<DT, SG, ZP, 16, 3>, 16, 1);
  });
}

}  // namespace moe
