// Products of many rows with 4-bit weights (include/moe_w4.h, layout in w4.h).
#include "w4.h"

namespace moe {

namespace {

// Forward: each of four wavefronts takes R row blocks of the matrix, straight from
// memory into operands, and all rows of the tile, which pass through LDS.  So a block is
// decoded once per tile and by one wavefront.  Bound by decoding and matrix instructions, which
// hardly overlap: a 16x16x32 instruction takes 16 cycles, with 2, 3, 4 and 6 vector
// instructions beside it 18.8, 21.8, 25.0 and 31.0; the more rows a tile has the less
// decoding weighs.  2,048 rows of 6144 x 6144 bfloat16 147 us (1.05 PFLOP/s; vector
// instructions 48% and matrix instructions 50% of a busy CU's cycles); 16,384 rows of 256
// experts of 1024 x 2048, laid out by Zipf's law, 137 us (64% and 29%, and a fifth of the
// CUs' time without a workgroup, most of it at the end); 512 and 4,096 rows of 256 experts of
// 2048 x 1024 binary16 42 and 83 us (51% and 11%, 55% and 18%: waits for a tile's first steps).
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
  by_height<MT, R == 3>(t.rows, [&](auto mt) {
    constexpr int M = decltype(mt)::value;  // groups of 16 rows that hold rows
    f32x4 acc[M][R];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int r = 0; r < R; ++r) acc[m][r] = f32x4{};
    if (t.e >= 0 && kb0 < kb1) {
      typedef Stage<DT, M, kBlockCols> St;
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
      const auto load_w = [&](Step& u, int kb) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const size_t block = (size_t)min(nb0 + r, a.NB - 1) * a.KB + kb;
          u.w[r] = ((const u32x4*)(w + block * kBlockBytes))[lane];
          u.s[r] = ((const svec*)(w + a.soff))[block * 16 + li];
          if (ZP) u.z[r] = ((const zvec*)(w + a.zoff))[block * 16 + li];
        }
      };
      const auto last = [&](int kb) { return min(kb, kb1 - 1); };
      // with a single step ahead its rows come in two parts, one after the other through
      // the same registers
      constexpr bool PARTS = D == 1;
      constexpr int PH = PARTS ? St::P / 2 : St::P;
#pragma unroll
      for (int d = 0; d < D; ++d) {
        st.load(step[d].x, last(kb0 + d) * kBlockCols);
        load_w(step[d], last(kb0 + d));
      }
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
          const int c_far = last(kb + D) * kBlockCols, c_next = last(kb + 1) * kBlockCols;
          st.template load<0, PH>(step[d].x, c_far);
          load_w(step[d], last(kb + D));
          __builtin_amdgcn_sched_barrier(0);  // (or the loads sink to where their results are used)
          const u32x4* x = sx[buf];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            constexpr int GS = 4 / SG;
            if (PARTS && j == 2) {
              st.template store<0, PH>(step[0].x, sx[buf ^ 1], c_next);
              st.template load<PH, St::P>(step[0].x, c_far);
              __builtin_amdgcn_sched_barrier(0);
            }
            v8_t<DT> wf[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
              GroupScale<DT, ZP> s;
              s.set((uint16_t)((uint64_t)sv[r] >> (16 * (j / GS))),
                    ZP ? (int)(int8_t)((uint32_t)zv[r] >> (8 * (j / GS))) : 0);
              wf[r] = s.weights(wv[r][j]);
            }
#pragma unroll
            for (int m = 0; m < M; ++m) {
              const v8_t<DT> xf = __builtin_bit_cast(v8_t<DT>, x[piece_at<kBlockCols>(16 * m + li, 4 * j + g)]);
#pragma unroll
              for (int r = 0; r < R; ++r) acc[m][r] = Mat<DT>::mma(wf[r], xf, acc[m][r]);
            }
          }
          if (PARTS) st.template store<PH, St::P>(step[0].x, sx[buf ^ 1], c_next);
          else st.store(step[(d + 1) % D].x, sx[buf ^ 1], c_next);
          buf ^= 1;
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

}  // namespace

void launch_w4_rows(const W4Args& a, const moe_w4_dims_t& d, const W4Layout& l, const TilePlan& p, hipStream_t s) {
  by_format(d, l.SG, [&](auto dt, auto sg, auto zp) {
    constexpr int DT = decltype(dt)::value, SG = decltype(sg)::value;
    constexpr bool ZP = decltype(zp)::value;
    const auto launch = [&](auto kernel) {
      const int64_t tiles = max_tiles(d.n, a.T, 16 * p.MT, a.offsets != nullptr);
      kernel<<<(unsigned)(places(tiles, p.groups, a.offsets != nullptr) * p.split), kTileThreads, 0, s>>>(a, p.groups);
    };
    if (p.MT == 2) launch(k_w4_rows<DT, SG, ZP, 2, 4>);
    else if (p.MT == 4) launch(k_w4_rows<DT, SG, ZP, 4, 4>);
    else if (p.MT == 6) launch(k_w4_rows<DT, SG, ZP, 6, 4>);
    else launch(k_w4_rows<DT, SG, ZP, 8, 3>);
  });
}

}  // namespace moe
