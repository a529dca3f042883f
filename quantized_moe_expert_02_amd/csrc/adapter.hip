// Low-rank adapters of many requests beside a shared projection
// (include/moe_adapter.h), on the matrix cores.
//
// Rows are taken in tiles of one adapter (16 rows for small batches, 32
// otherwise).  Every product is a 16x16x32 matrix instruction with fp32
// accumulators whose operand fragments hold, in lane l, 8 consecutive terms
// (l / 16) * 8 .. + 7 of the contraction for index l % 16; its result holds
// index l % 16 of the second operand and (l / 16) * 4 .. + 3 of the first.
// Where the contraction runs along a tensor's rows (x, B) fragments come
// straight from memory; where it runs across them (B and A in the input's
// gradient, x and dy in the weights') the rows pass through LDS and are read
// back transposed (ds_read_b64_tr_b16).
#include <algorithm>

#include "rows.h"

namespace moe {

namespace {

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

// ---------------------------------------------------------------------------
// fp32 factors on 16-bit matrix instructions.  u and v are sums and are not
// rounded to 16 bits: a value is carried as a sum of 16-bit pieces, each the
// rounded rest of the ones before (two binary16 pieces hold 22 bits, two
// bfloat16 16 bits, three 24).  binary16 lacks fp32's range, so values are
// first scaled by a power of two per row (or per tile, where the contraction
// runs over rows) that brings the largest finite one to 2^13.
// ---------------------------------------------------------------------------
constexpr int kTopExp = 13;

// Power of two that scales a largest magnitude `top` as above (0 for 0).
template <int DT>
__device__ __forceinline__ int scale_exp(float top) {
  if (DT == MOE_T_BF16 || top == 0.0f) return 0;
  return kTopExp + 1 - __builtin_amdgcn_frexp_expf(top);
}

__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.0f;  // NaN too
}

template <int DT, int NP>
__device__ __forceinline__ void split_pieces(const float (&v)[8], int e, v8_t<DT> (&p)[NP]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float rest = DT == MOE_T_F16 ? __builtin_amdgcn_ldexpf(v[i], e) : v[i];
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const typename Mat<DT>::elem h = (typename Mat<DT>::elem)rest;
      p[q][i] = h;
      const float f = (float)h;
      rest = fabsf(f) < INFINITY ? rest - f : 0.0f;  // an infinity or NaN stays in the first piece
    }
  }
}

struct AdapterArgs {
  const void *a, *b;
  const float* scale;
  const int32_t* ranks;
  int n, K, N, R;
};

__device__ __forceinline__ int rank_of(const AdapterArgs& d, int a) {
  return d.ranks ? min(max(d.ranks[a], 0), d.R) : d.R;
}

// ---------------------------------------------------------------------------
// Tiles: up to M rows of one adapter.
// ---------------------------------------------------------------------------
// Which rows a call has and how they are grouped.  offsets == NULL: at most
// 64 rows, grouped by each workgroup itself from ids.
struct SharedTile;
struct RowSet {
  const int32_t *ids, *offsets, *pairs;
  SharedTile* kept;  // [tiles and those that follow]
  int T;
  int tiles;  // upper bound on tiles of adapters; with offsets, tiles of M rows in order of arrival follow, of
              // which each stands for its rows without an adapter
};

// a: adapter, or n for rows without one; cnt: rows (0: no such tile); first:
// place of its rows in the sorted order; this lane's row for lane < M, -1 past
// cnt.
struct Tile {
  int a, cnt, first, row;
  int rank;
  float scale;  // both 0 without an adapter
};

__device__ __forceinline__ int lanes_under(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// Inclusive sum over the wavefront's lanes (all active): row shifts, then the
// rows' ends broadcast on.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_shifted(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_prefix(int v) {
  v = add_shifted<0x111, 0xF>(v);  // row_shr:1
  v = add_shifted<0x112, 0xF>(v);  // row_shr:2
  v = add_shifted<0x114, 0xF>(v);  // row_shr:4
  v = add_shifted<0x118, 0xF>(v);  // row_shr:8
  v = add_shifted<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  return add_shifted<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
}

__device__ __forceinline__ int at_lane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float at_lane_f(float v, int lane) {
  return __builtin_bit_cast(float, at_lane(__builtin_bit_cast(int, v), lane));
}

// One adapter's group of rows, bounds checked.
__device__ __forceinline__ void group_of(const RowSet& rs, int a, int n, int* first, int* count) {
  const int i = min(a, n - 1);
  const int o0 = min(max(rs.offsets[i], 0), rs.T), o1 = min(max(rs.offsets[i + 1], 0), rs.T);
  *first = o0;
  *count = a < n ? max(0, o1 - o0) : 0;
}

// The lane-th set bit of m for lanes below its count.
__device__ __forceinline__ int nth_bit(uint64_t m, int most) {
  const int lane = threadIdx.x & 63;
  for (int i = 0; i < most - 1; ++i)
    if (i < lane) m &= m - 1;
  return m ? (int)__builtin_ctzll(m) : 0;
}

// Called by one whole wavefront; `tile` is uniform.
template <int M>
__device__ __forceinline__ Tile find_tile(const AdapterArgs& d, const RowSet& rs, int tile) {
  const int n = d.n;
  const int lane = threadIdx.x & 63;
  if (!rs.offsets) {
    int id = rs.ids[min(lane, rs.T - 1)];
    if ((unsigned)id >= (unsigned)n) id = n;
    const int rank = id < n ? rank_of(d, id) : 0;
    const float scale = id < n ? d.scale[id] : 0.0f;
    if (rs.T == 1) return {at_lane(id, 0), tile == 0, 0, lane == 0 ? 0 : -1, at_lane(rank, 0), at_lane_f(scale, 0)};
    uint64_t same = __ballot(lane < rs.T);
    for (int b = 0; b < 11; ++b) {
      const bool one = (id >> b) & 1;
      const uint64_t v = __ballot(one);
      same &= one ? v : ~v;
    }
    const int nth = lanes_under(same);
    uint64_t lead = __ballot(lane < rs.T && nth % M == 0);
    for (int i = 0; i < tile; ++i) lead &= lead - 1;
    if (!lead) return {n, 0, 0, -1, 0, 0.0f};
    const int at = __builtin_ctzll(lead);
    const int a = at_lane(id, at), n0 = at_lane(nth, at);
    const uint64_t mine = __ballot(lane < rs.T && id == a && nth >= n0 && nth < n0 + M);
    const int cnt = __popcll(mine), bit = nth_bit(mine, M);
    return {a, cnt, 0, lane < cnt ? bit : -1, at_lane(rank, at), at_lane_f(scale, at)};
  }
  if (tile >= rs.tiles) {
    const int t0 = (tile - rs.tiles) * M, t = t0 + lane;
    const int id = rs.ids[min(t, rs.T - 1)];
    const uint64_t mine = __ballot(lane < M && t < rs.T && (unsigned)id >= (unsigned)n);
    const int cnt = __popcll(mine), bit = nth_bit(mine, M);
    return {n, cnt, 0, lane < cnt ? t0 + bit : -1, 0, 0.0f};
  }
  for (int a0 = 0, done = 0; a0 < n; a0 += 64) {
    int first, count;
    group_of(rs, a0 + lane, n, &first, &count);
    const int rank = rank_of(d, min(a0 + lane, n - 1));
    const float scale = d.scale[min(a0 + lane, n - 1)];
    const int nt = (count + M - 1) / M, incl = wave_prefix(nt);
    const uint64_t past = __ballot(incl > tile - done);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int j = tile - done - at_lane(incl - nt, at);
      const int i0 = at_lane(first, at) + j * M, cnt = min(M, at_lane(count, at) - j * M);
      int row = rs.pairs[min(i0 + lane, rs.T - 1)];
      if (lane >= cnt || (unsigned)row >= (unsigned)rs.T) row = -1;
      return {a0 + at, cnt, i0, row, at_lane(rank, at), at_lane_f(scale, at)};
    }
    done += at_lane(incl, 63);
  }
  return {n, 0, 0, -1, 0, 0.0f};
}

// A tile as a workgroup holds it in LDS, and as the first launch of a pass
// leaves it in workspace for the second.
struct SharedTile {
  int a, cnt, first, rank;
  float scale;
  int pad[3];
  int row[32];
};
constexpr int kTileWords = sizeof(SharedTile) / 4;

// find_tile by the first wavefront; stored to *keep where given.  Ends with a
// barrier.
template <int M>
__device__ __forceinline__ void share_tile(SharedTile* s, const AdapterArgs& d, const RowSet& rs, int tile,
                                           SharedTile* keep) {
  if (threadIdx.x < 64) {
    const Tile t = find_tile<M>(d, rs, tile);
    const auto put = [&](SharedTile* o) {
      if (threadIdx.x < 32) o->row[threadIdx.x] = t.row;
      if (threadIdx.x == 0) {
        o->a = t.a;
        o->cnt = t.cnt;
        o->first = t.first;
        o->rank = t.rank;
        o->scale = t.scale;
      }
    };
    put(s);
    if (keep) put(keep);
  }
  __syncthreads();
}

// The same from workspace.
__device__ __forceinline__ void take_tile(SharedTile* s, const SharedTile* kept) {
  if (threadIdx.x < kTileWords) ((int*)s)[threadIdx.x] = ((const int*)kept)[threadIdx.x];
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Loads.  A lane whose vector lies outside what it may read or use loads
// another, valid one (the caller bends the address) and drops it where the
// value is used: no branch stands between loads, and none waits for another.
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ u32x4 load8(const void* base, uint32_t i) {
  return *(const u32x4*)((const typename Mat<DT>::elem*)base + i);
}

__device__ __forceinline__ u32x4 keep(u32x4 v, bool ok) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = ok ? v[i] : 0u;
  return v;
}

// The first `valid` of 8 columns (any value; whole: no vector is cut).
__device__ __forceinline__ u32x4 keep_upto(u32x4 v, int valid, bool whole) {
  v = keep(v, valid > 0);
  if (!whole) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] &= (valid > 2 * i ? 0xFFFFu : 0u) | (valid > 2 * i + 1 ? 0xFFFF0000u : 0u);
  }
  return v;
}

template <int DT>
__device__ __forceinline__ v8_t<DT> as_frag(u32x4 v) {
  return __builtin_bit_cast(v8_t<DT>, v);
}

// Between a wavefront's writes of its LDS rows and its reads of them by other
// lanes, and back: LDS keeps one wavefront's accesses in order, so only the
// compiler has to.
__device__ __forceinline__ void lds_order() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_wave_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// Fragment whose contraction runs across rows in LDS: each 16 lanes read 4
// rows of 16 columns (lane i: row i / 4, 4 columns at its address) and lane i
// receives column i of the 4 rows; lo and hi are this lane's addresses for
// terms 0..3 and 4..7.
template <int DT>
__device__ __forceinline__ v8_t<DT> read_across(const typename Mat<DT>::elem* lo, const typename Mat<DT>::elem* hi) {
  typedef __attribute__((address_space(3))) s16x4* lds_p;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)lo);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)hi);
  const s16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(v8_t<DT>, v);
}

// Sums acc over the workgroup's W wavefronts into wavefront 0, pairwise.
// red: W / 2 * NF fragments.
template <int W, int NF>
__device__ __forceinline__ void reduce_waves(f32x4 (&acc)[NF], f32x4* red, int wave, int lane) {
#pragma unroll
  for (int h = W / 2; h >= 1; h /= 2) {
    if (wave >= h && wave < 2 * h) {
#pragma unroll
      for (int f = 0; f < NF; ++f) red[((wave - h) * NF + f) * 64 + lane] = acc[f];
    }
    __syncthreads();
    if (wave < h) {
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[f] += red[(wave * NF + f) * 64 + lane];
    }
    __syncthreads();
  }
}

constexpr int cmax(int a, int b) { return a > b ? a : b; }

constexpr int kRowThreads = 512;
constexpr int kRowWaves = kRowThreads / kWave;

// The long sums over a tile's rows: u[t][r] = <A_a[r], x[t]> (ACROSS false), or
// v[t][r] = s_a sum_c dy[t][c] B_a[c][r] (ACROSS), of one segment of the columns
// (blockIdx.y of gridDim.y), split again over the wavefronts.  u: [S][T][R] by
// row; v: the same in the sorted order, and a copy of the forward pass's u in
// that order.
// Memory is read 128 contiguous bytes per row (8 lanes side by side: lanes that
// follow the fragments' layout, each in a row of its own, cost the address unit
// four times as many cycles); a wavefront's own LDS turns that into fragments,
// the next step's loads in flight meanwhile.
template <int DT, int MT, int RT, bool ACROSS>
__global__ __launch_bounds__(kRowThreads) void k_rows(AdapterArgs d, RowSet rs, const void* x, int64_t ldx, float* out,
                                                     bool zero_none, const float* u, float* u_sorted) {
  typedef typename Mat<DT>::elem E;
  constexpr int M = MT * 16, W = RT * 16;
  constexpr int KS = RT == 8 ? 32 : 64, NH = KS / 32;  // columns per step
  constexpr int XV = KS / 8, XS = KS + 8;              // x's rows in LDS: vectors, stride
  constexpr int FR = ACROSS ? KS : W, FV = ACROSS ? W / 8 : XV, FS = ACROSS ? W + 8 : XS;  // the factor's
  constexpr int XL = M * XV / 64, FL = FR * FV / 64;   // loads per lane
  constexpr int kStage = (M * XS + FR * FS) * 2;
  __shared__ SharedTile st;
  __shared__ __align__(16) char lds[cmax(kRowWaves * kStage, kRowWaves / 2 * MT * RT * 1024)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  if ((int)blockIdx.x >= rs.tiles && blockIdx.y) return;
  share_tile<M>(&st, d, rs, blockIdx.x, blockIdx.y ? nullptr : rs.kept + blockIdx.x);
  const int a = __builtin_amdgcn_readfirstlane(st.a), cnt = __builtin_amdgcn_readfirstlane(st.cnt);
  if (!cnt) return;
  float* o = out + (size_t)blockIdx.y * rs.T * d.R;
  if (a == d.n) {
    if (zero_none)
      for (int i = threadIdx.x; i < cnt * d.R; i += kRowThreads) o[(size_t)st.row[i / d.R] * d.R + i % d.R] = 0.0f;
    return;
  }
  const int rk = __builtin_amdgcn_readfirstlane(st.rank), C = ACROSS ? d.N : d.K;
  const bool whole = rk % 8 == 0;
  if (ACROSS && blockIdx.y == 0)
    for (int i = threadIdx.x; i < cnt * (d.R / 4); i += kRowThreads) {
      const int t = i / (d.R / 4), r = i % (d.R / 4) * 4;
      f32x4 v = *(const f32x4*)(u + (size_t)max(st.row[t], 0) * d.R + r);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = r + c < rk && st.row[t] >= 0 ? v[c] : 0.0f;
      *(f32x4*)(u_sorted + (size_t)(st.first + t) * d.R + r) = v;
    }
  const int steps = (C + KS - 1) / KS, parts = gridDim.y * kRowWaves, part = blockIdx.y * kRowWaves + wave;
  const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
  E* xs = (E*)(lds + wave * kStage);
  E* fs = xs + M * XS;
  const int xc = lane % XV * 8;
  const E* xrow[XL];
  bool xok[XL];
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int r = st.row[(lane + 64 * i) / XV];
    xok[i] = r >= 0;
    xrow[i] = (const E*)x + (size_t)max(r, 0) * ldx;
  }
  const E* fbase = (const E*)(ACROSS ? d.b : d.a) + (size_t)a * d.R * C;
  u32x4 xn[2][XL], fn[2][FL];  // the next two steps
  const auto fetch = [&](int s, u32x4 (&xn)[XL], u32x4 (&fn)[FL]) {
    const int c = s * KS + xc < C ? s * KS + xc : 0;
#pragma unroll
    for (int i = 0; i < FL; ++i) {
      const int row = (lane + 64 * i) / FV, fc = (lane + 64 * i) % FV * 8;
      const uint32_t at = ACROSS ? (uint32_t)min(s * KS + row, C - 1) * d.R + (fc < rk ? fc : 0)
                                 : (uint32_t)(row < rk ? row : 0) * C + c;
      fn[i] = load8<DT>(fbase, at);
    }
#pragma unroll
    for (int i = 0; i < XL; ++i) xn[i] = load8<DT>(xrow[i], c);
  };
  f32x4 acc[MT * RT] = {};
  const auto step = [&](int s, u32x4 (&xn)[XL], u32x4 (&fn)[FL]) {
    const bool cok = s * KS + xc < C;
#pragma unroll
    for (int i = 0; i < XL; ++i) *(u32x4*)(xs + (lane + 64 * i) / XV * XS + xc) = keep(xn[i], xok[i] && cok);
#pragma unroll
    for (int i = 0; i < FL; ++i) {
      const int row = (lane + 64 * i) / FV, fc = (lane + 64 * i) % FV * 8;
      const u32x4 v = ACROSS ? keep_upto(fn[i], s * KS + row < C ? rk - fc : 0, whole) : keep(fn[i], row < rk && cok);
      *(u32x4*)(fs + row * FS + fc) = v;
    }
    if (s + 2 < s1) fetch(s + 2, xn, fn);
    lds_order();
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      v8_t<DT> xf[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) xf[m] = *(const v8_t<DT>*)(xs + (m * 16 + li) * XS + h * 32 + g * 8);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        v8_t<DT> ff;
        if (ACROSS) {
          const E* p = fs + (h * 32 + g * 8 + (li >> 2)) * FS + r * 16 + (li & 3) * 4;
          ff = read_across<DT>(p, p + 4 * FS);
        } else {
          ff = *(const v8_t<DT>*)(fs + (r * 16 + li) * FS + h * 32 + g * 8);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m * RT + r] = Mat<DT>::mma(ff, xf[m], acc[m * RT + r]);
      }
    }
    lds_order();
  };
  if (s0 < s1) fetch(s0, xn[0], fn[0]);
  if (s0 + 1 < s1) fetch(s0 + 1, xn[1], fn[1]);
  for (int s = s0; s < s1; s += 2) {
    step(s, xn[0], fn[0]);
    if (s + 1 < s1) step(s + 1, xn[1], fn[1]);
  }
  __syncthreads();
  reduce_waves<kRowWaves, MT * RT>(acc, (f32x4*)lds, wave, lane);
  if (wave == 0) {
    const float f = st.scale;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int t = m * 16 + li, row = ACROSS ? (t < cnt ? st.first + t : -1) : st.row[t];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int c = r * 16 + g * 4;
        if (row >= 0 && c < d.R) *(f32x4*)(o + (size_t)row * d.R + c) = ACROSS ? acc[m * RT + r] * f : acc[m * RT + r];
      }
    }
  }
}

constexpr int kOutThreads = 256;
constexpr int kOutWaves = kOutThreads / kWave;

// LDS of a tile's u or v on its way to fragments.
template <int M, int RB>
struct RowPack {
  float v[M][RB * 32 + 4];
  alignas(16) float scale[M];      // what the products are multiplied by
  u32x4 frag[M / 16 * RB][2][64];  // contraction over r, two pieces
};

// p[0] + p[stride] + ... (S of them), in that order, four loads in flight.
__device__ __forceinline__ f32x4 sum_segments(const float* p, size_t stride, int S) {
  f32x4 v = *(const f32x4*)p;
  for (int s = 1; s < S; s += 4) {
    f32x4 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = *(const f32x4*)(p + min(s + k, S - 1) * stride);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s + k < S) v += w[k];
  }
  return v;
}

// Sums the S segments of a tile's rows (also written to u, where given), and
// splits them into fragments: a wavefront per fragment.  SORTED: part is in the
// sorted order.  Ends with a barrier.
template <int DT, int M, int RB, bool SORTED>
__device__ __forceinline__ void pack_rows(RowPack<M, RB>* p, const SharedTile& st, const float* part, int S, int T, int R,
                                          float f, float* u) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  const int rk = st.rank;
#pragma unroll
  for (int i0 = 0; i0 < M * RB * 8; i0 += kOutThreads) {
    const int i = i0 + tid, t = i / (RB * 8), r = i % (RB * 8) * 4;
    if (M * RB * 8 % kOutThreads && i >= M * RB * 8) break;
    const int row = SORTED ? (t < st.cnt ? st.first + t : -1) : st.row[t];
    f32x4 v = {0, 0, 0, 0};
    if (row >= 0 && r < rk) v = sum_segments(part + (size_t)row * R + r, (size_t)T * R, S);
    *(f32x4*)&p->v[t][r] = v;
    if (u && row >= 0 && r < R) *(f32x4*)(u + (size_t)row * R + r) = v;
  }
  __syncthreads();
#pragma unroll
  for (int unit0 = 0; unit0 < M / 16 * RB; unit0 += kOutWaves) {
    const int unit = unit0 + wave;
    if (M / 16 * RB % kOutWaves && unit >= M / 16 * RB) break;
    const int t = unit / RB * 16 + li, b = unit % RB;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p->v[t][b * 32 + g * 8 + i];
    int e = 0;
    if (DT == MOE_T_F16) {
      float top = 0.0f;
#pragma unroll
      for (int c = 0; c < RB * 8; c += 4) {  // a quarter of the row per lane group
        const f32x4 w = *(const f32x4*)&p->v[t][g * RB * 8 + c];
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, finite_abs(w[i]));
      }
      top = fmaxf(top, __builtin_bit_cast(float, partner<16>(__builtin_bit_cast(int, top))));
      top = fmaxf(top, __builtin_bit_cast(float, partner<32>(__builtin_bit_cast(int, top))));
      e = scale_exp<DT>(top);
    }
    v8_t<DT> h[2];
    split_pieces<DT, 2>(v, e, h);
    p->frag[unit][0][lane] = __builtin_bit_cast(u32x4, h[0]);
    p->frag[unit][1][lane] = __builtin_bit_cast(u32x4, h[1]);
    // below 2^-126 this factor loses bits of results that are far below the
    // 16-bit types' smallest step
    if (b == 0 && g == 0) p->scale[t] = __builtin_amdgcn_ldexpf(f, -e);
  }
  __syncthreads();
}

constexpr int kExpandCols = kOutWaves * 128;  // columns of a workgroup's pass

// y[t] = add[t] + s_a B_a u[t] for a tile's rows and a run of columns, 128
// columns at a time per wavefront.  Column 8 i + q of the 128 is lane i's
// column of product q, so that a lane ends with 8 consecutive columns and 16
// lanes with 256 contiguous bytes of a row.  B's rows pass through LDS, row
// 8 i + q at place 16 q + i (fragment reads then meet no bank conflict).
template <int DT, int MT, int RT>
__global__ __launch_bounds__(kOutThreads) void k_expand(AdapterArgs d, RowSet rs, const float* part, int S, float* u,
                                                       const void* add, int64_t ldadd, void* y, int64_t ldy, int passes) {
  typedef typename Mat<DT>::elem E;
  constexpr int M = MT * 16, RB = (RT + 1) / 2, VR = RT == 1 ? 2 : 4, BL = 128 * VR / 64, BS = VR * 8 + 8;
  __shared__ SharedTile st;
  __shared__ RowPack<M, RB> pk;
  __shared__ __align__(16) E lds[kOutWaves][128 * BS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  if ((int)blockIdx.x >= rs.tiles) {  // rows without an adapter: one workgroup takes all columns
    if (blockIdx.y) return;
    passes = (d.N + kExpandCols - 1) / kExpandCols;
  }
  take_tile(&st, rs.kept + blockIdx.x);
  if (!__builtin_amdgcn_readfirstlane(st.cnt)) return;
  const int rk = __builtin_amdgcn_readfirstlane(st.rank), a = min(__builtin_amdgcn_readfirstlane(st.a), d.n - 1);
  const bool whole = rk % 8 == 0;
  E* bs = lds[wave];
  const E* bbase = (const E*)d.b + (size_t)a * d.N * d.R;
  if (RT == 1) {  // rank 16 fills half of the contraction; the other half reads zeros
#pragma unroll
    for (int i = 0; i < 2; ++i) *(u32x4*)(bs + (lane + 64 * i) * BS + 16) = u32x4{0, 0, 0, 0};
  }
  u32x4 bn[BL];
  const auto fetch = [&](int n0, int b) {
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int v = lane + 64 * i, r = b * 32 + v % VR * 8;
      bn[i] = load8<DT>(bbase, (uint32_t)min(n0 + v / VR, d.N - 1) * d.R + (r < rk ? r : 0));
    }
  };
  const int first = (blockIdx.y * passes * kOutWaves + wave) * 128;
  fetch(first, 0);
  const E* addrow[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) addrow[m][i] = (const E*)add + (size_t)max(st.row[m * 16 + g * 4 + i], 0) * ldadd;
  u32x4 av[MT][4] = {};
  const auto fetch_add = [&](int n0) {
    const int c = n0 + li * 8 < d.N ? n0 + li * 8 : 0;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) av[m][i] = load8<DT>(addrow[m][i], c);
  };
  if (add) fetch_add(first);
  pack_rows<DT, M, RB, false>(&pk, st, part, S, rs.T, d.R, st.scale, blockIdx.y == 0 ? u : nullptr);
  for (int q0 = 0; q0 < passes; ++q0) {
    const int n0 = first + q0 * kExpandCols, c = n0 + li * 8;
    if (n0 >= d.N) break;
    f32x4 acc[MT][8] = {};
#pragma unroll
    for (int b = 0; b < RB; ++b) {
#pragma unroll
      for (int i = 0; i < BL; ++i) {
        const int v = lane + 64 * i, n = v / VR, r = b * 32 + v % VR * 8;
        *(u32x4*)(bs + (n % 8 * 16 + n / 8) * BS + v % VR * 8) = keep_upto(bn[i], rk - r, whole);
      }
      lds_order();
      if (b + 1 < RB) fetch(n0, b + 1);
      else if (q0 + 1 < passes) fetch(n0 + kExpandCols, 0);
      v8_t<DT> uf[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) uf[m][h] = as_frag<DT>(pk.frag[m * RB + b][h][lane]);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const v8_t<DT> bf = *(const v8_t<DT>*)(bs + (q * 16 + li) * BS + (RT == 1 ? min(g, 2) : g) * 8);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[m][q] = Mat<DT>::mma(uf[m][0], bf, acc[m][q]);
          acc[m][q] = Mat<DT>::mma(uf[m][1], bf, acc[m][q]);
        }
      }
      lds_order();
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const f32x4 f = *(const f32x4*)&pk.scale[m * 16 + g * 4];
      int row[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) row[i] = st.row[m * 16 + g * 4 + i];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float o[8];
        unpack_vec<DT>(av[m][i], o);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = fmaf(acc[m][q][i], f[i], o[q]);
        if (row[i] >= 0 && c < d.N) *(u32x4*)((E*)y + (size_t)row[i] * ldy + c) = pack_vec<DT>(o);
      }
    }
    if (add && q0 + 1 < passes) fetch_add(n0 + kExpandCols);
  }
}

// ---------------------------------------------------------------------------
// Backward pass: k_rows<ACROSS> forms v, k_grad_out dx, dA and dB, and
// k_grad_sum adds the partial dA and dB of adapters whose rows several
// workgroups took.
// ---------------------------------------------------------------------------
constexpr int kGradM = 32;  // rows per tile

// Pieces of a factor of a weight gradient (an fp32 output).
template <int DT>
constexpr int kGradPieces = DT == MOE_T_F16 ? 2 : 3;

// Work items of the weight gradients: up to G rows (a multiple of 32) of one
// adapter; an adapter without rows has one, which writes zeros.
struct Item {
  int a, first, cnt;  // adapter (n: no such item), place in pairs, rows
  int slot;           // partial sum it writes, or -1: the result itself
};

__device__ __forceinline__ Item find_item(const RowSet& rs, int n, int item, int G) {
  const int lane = threadIdx.x & 63;
  int slots = 0;
  for (int a0 = 0, done = 0; a0 < n; a0 += 64) {
    int first, count;
    group_of(rs, a0 + lane, n, &first, &count);
    const int parts = (count + G - 1) / G, ni = a0 + lane < n ? max(1, parts) : 0;
    const int ns = parts > 1 ? parts : 0;
    const int incl = wave_prefix(ni), is = wave_prefix(ns);
    const uint64_t past = __ballot(incl > item - done);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int j = item - done - at_lane(incl - ni, at), c = at_lane(count, at);
      const int slot = slots + at_lane(is - ns, at) + j;
      return {a0 + at, at_lane(first, at) + j * G, max(0, min(G, c - j * G)), at_lane(ns, at) ? slot : -1};
    }
    done += at_lane(incl, 63);
    slots += at_lane(is, 63);
  }
  return {n, 0, 0, -1};
}

constexpr int kStride = 72;                  // elements of an LDS row of 64 columns
constexpr int kOutCols = kOutWaves * 64;     // columns of a workgroup
constexpr int kDxStride = 68;                // floats of an LDS row of 64 results

// Rows of the weight gradients' factor held as fragments at a time.
template <int DT, int RT>
constexpr int kChunkTiles = RT == 1 ? 8 : RT == 2 ? 4 : RT == 4 ? 2 : 1;

template <int DT, int RT>
struct GradLds {
  static constexpr int RB = (RT + 1) / 2;
  struct Dx {
    SharedTile st;
    RowPack<kGradM, RB> pk;
    union {
      typename Mat<DT>::elem rows[32 * kStride];
      float out[kGradM * kDxStride];
    } w[kOutWaves];
  };
  struct Outer {
    float top[kOutWaves];
    u32x4 frag[kChunkTiles<DT, RT>][RT][kGradPieces<DT>][64];
    typename Mat<DT>::elem rows[kOutWaves][kGradM * kStride];
  };
  union {
    Dx dx;
    Outer o;
  };
  __device__ GradLds() {}
};

// dx of a tile's rows, 64 columns at a time per wavefront: rows of A through
// LDS, 32 at a time; the results go back through LDS so that 8 lanes finish
// 128 contiguous bytes of a row.
template <int DT, int RT>
__device__ __forceinline__ void grad_dx(GradLds<DT, RT>& lds, const AdapterArgs& d, const RowSet& rs, const float* v, int S,
                                        int tile, int chunk, int passes, const void* add, int64_t ldadd, void* dx,
                                        int64_t lddx) {
  typedef typename Mat<DT>::elem E;
  constexpr int RB = (RT + 1) / 2, MT = kGradM / 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  auto& L = lds.dx;
  if (tile >= rs.tiles) {  // rows without an adapter: one workgroup takes all columns
    if (chunk) return;
    passes = (d.K + kOutCols - 1) / kOutCols;
    share_tile<kGradM>(&L.st, d, rs, tile, nullptr);
  } else {
    take_tile(&L.st, rs.kept + tile);
  }
  if (!__builtin_amdgcn_readfirstlane(L.st.cnt)) return;
  const int rk = __builtin_amdgcn_readfirstlane(L.st.rank), a = min(__builtin_amdgcn_readfirstlane(L.st.a), d.n - 1);
  E* stage = L.w[wave].rows;
  float* out = L.w[wave].out;
  const E* abase = (const E*)d.a + (size_t)a * d.R * d.K;
  u32x4 an[4];
  const auto fetch = [&](int k0, int b) {
    const int k = k0 + lane % 8 * 8 < d.K ? k0 + lane % 8 * 8 : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = b * 32 + lane / 8 + 8 * i;
      an[i] = load8<DT>(abase, (uint32_t)(r < rk ? r : 0) * d.K + k);
    }
  };
  const int first = (chunk * passes * kOutWaves + wave) * 64;
  fetch(first, 0);
  int row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = L.st.row[lane / 8 + 8 * i];
  u32x4 av[4] = {};
  const auto fetch_add = [&](int k0) {
    const int k = k0 + lane % 8 * 8 < d.K ? k0 + lane % 8 * 8 : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) av[i] = load8<DT>((const E*)add + (size_t)max(row[i], 0) * ldadd, k);
  };
  if (add) fetch_add(first);
  pack_rows<DT, kGradM, RB, true>(&L.pk, L.st, v, S, rs.T, d.R, 1.0f, nullptr);
  for (int q0 = 0; q0 < passes; ++q0) {
    const int k0 = first + q0 * kOutCols, c = k0 + lane % 8 * 8;
    if (k0 >= d.K) break;
    f32x4 acc[MT][4] = {};
#pragma unroll
    for (int b = 0; b < RB; ++b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = lane / 8 + 8 * i;
        *(u32x4*)(stage + r * kStride + lane % 8 * 8) = keep(an[i], b * 32 + r < rk && c < d.K);
      }
      lds_order();
      if (b + 1 < RB) fetch(k0, b + 1);
      else if (q0 + 1 < passes) fetch(k0 + kOutCols, 0);
      v8_t<DT> vf[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) vf[m][h] = as_frag<DT>(L.pk.frag[m * RB + b][h][lane]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const E* p = stage + (g * 8 + (li >> 2)) * kStride + q * 16 + (li & 3) * 4;
        const v8_t<DT> af = read_across<DT>(p, p + 4 * kStride);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[m][q] = Mat<DT>::mma(af, vf[m][0], acc[m][q]);
          acc[m][q] = Mat<DT>::mma(af, vf[m][1], acc[m][q]);
        }
      }
      lds_order();
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q) *(f32x4*)(out + (m * 16 + li) * kDxStride + q * 16 + g * 4) = acc[m][q];
    lds_order();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = lane / 8 + 8 * i;
      const f32x4* r = (const f32x4*)(out + t * kDxStride + lane % 8 * 8);
      const f32x4 lo = r[0], hi = r[1];
      float o[8];
      unpack_vec<DT>(av[i], o);
      const float f = L.pk.scale[t];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        o[q] = fmaf(lo[q], f, o[q]);
        o[4 + q] = fmaf(hi[q], f, o[4 + q]);
      }
      if (row[i] >= 0 && c < d.K) *(u32x4*)((E*)dx + (size_t)row[i] * lddx + c) = pack_vec<DT>(o);
    }
    lds_order();
    if (add && q0 + 1 < passes) fetch_add(k0 + kOutCols);
  }
}

// A weight gradient's 64 columns per wavefront over an item's rows: the rows
// of x (dA = sum_t v x^T) or dy (TR: dB = s_a sum_t dy u^T) pass through LDS, 32
// at a time, against v or u (in the sorted order), which the workgroup holds as
// fragments for a few tiles at a time.  In binary16 those share one power of
// two, the smallest so far; where a chunk brings a smaller one, the sums are
// rescaled.
template <int DT, int RT, bool TR>
__device__ __forceinline__ void grad_outer(GradLds<DT, RT>& lds, const AdapterArgs& d, const RowSet& rs, const float* v,
                                           int S, int item, int G, int chunk, const void* x, int64_t ldx, float* out,
                                           float* sums, int slots) {
  typedef typename Mat<DT>::elem E;
  constexpr int NP = kGradPieces<DT>, CT = kChunkTiles<DT, RT>, UW = (CT * RT + kOutWaves - 1) / kOutWaves;
  auto& L = lds.o;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  const int C = TR ? d.N : d.K, c0 = chunk * kOutCols + wave * 64;
  const Item it = find_item(rs, d.n, item, G);  // by every wavefront: no barrier
  if (it.a >= d.n || it.slot >= slots) return;  // (past the slots: only for groups that overlap)
  const int rk = rank_of(d, it.a), tiles = rk ? (it.cnt + kGradM - 1) / kGradM : 0;
  E* stage = L.rows[wave];
  const int col = c0 + lane % 8 * 8, colc = col < C ? col : 0;
  int ids[4], next[4];  // rows of the tile in `rows`, and of the one after it
  const auto fetch_ids = [&](int j) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = j * kGradM + lane / 8 + 8 * q;
      const int r = rs.pairs[min(it.first + i, rs.T - 1)];
      next[q] = i < it.cnt && (unsigned)r < (unsigned)rs.T ? r : -1;
    }
  };
  u32x4 rows[4];
  const auto fetch = [&](int j) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      ids[q] = next[q];
      rows[q] = load8<DT>((const E*)x + (size_t)max(ids[q], 0) * ldx, colc);
    }
    if (j + 1 < tiles) fetch_ids(j + 1);
  };
  // this wavefront's part of a chunk of v: unit -> tile unit / RT, r tile unit % RT
  float w[UW][8];
  const auto fetch_v = [&](int j0) {
#pragma unroll
    for (int k = 0; k < UW; ++k) {
      const int unit = min(wave + k * kOutWaves, CT * RT - 1), r = min(unit % RT * 16 + li, d.R - 1);
      const int i = (j0 + unit / RT) * kGradM + g * 8;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float* p = v + (size_t)(it.first + min(i + q, it.cnt - 1)) * d.R + r;
        float s = p[0];
        for (int k2 = 1; k2 < S; ++k2) s += p[(size_t)k2 * rs.T * d.R];
        w[k][q] = s;
      }
    }
  };
  f32x4 acc[4][RT] = {};
  int e = 0;
  bool any = false;
  if (tiles) {
    fetch_ids(0);
    fetch_v(0);
    fetch(0);
  }
  for (int j0 = 0; j0 < tiles; j0 += CT) {
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < UW; ++k) {
      const int unit = wave + k * kOutWaves, r = unit % RT * 16 + li, i = (j0 + unit / RT) * kGradM + g * 8;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        w[k][q] = unit < CT * RT && r < rk && i + q < it.cnt ? w[k][q] : 0.0f;
        top = fmaxf(top, finite_abs(w[k][q]));
      }
    }
    if (DT == MOE_T_F16) {
      top = __builtin_bit_cast(float, wave_max_u32(__builtin_bit_cast(uint32_t, top)));
      if (lane == 0) L.top[wave] = top;
      __syncthreads();  // also: the last chunk's fragments have been read
#pragma unroll
      for (int q = 0; q < kOutWaves; ++q) top = fmaxf(top, L.top[q]);
      if (top > 0.0f) {
        const int en = any ? min(e, scale_exp<DT>(top)) : scale_exp<DT>(top);
        if (any && en < e) {
          const float f = __builtin_amdgcn_ldexpf(1.0f, en - e);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[q][r] *= f;
        }
        e = en;
        any = true;
      }
    } else {
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < UW; ++k) {
      const int unit = wave + k * kOutWaves;
      if (unit < CT * RT) {
        v8_t<DT> p[NP];
        split_pieces<DT, NP>(w[k], e, p);
#pragma unroll
        for (int q = 0; q < NP; ++q) L.frag[unit / RT][unit % RT][q][lane] = __builtin_bit_cast(u32x4, p[q]);
      }
    }
    __syncthreads();
    if (j0 + CT < tiles) fetch_v(j0 + CT);
    for (int j = j0; j < min(j0 + CT, tiles); ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(u32x4*)(stage + (lane / 8 + 8 * q) * kStride + lane % 8 * 8) = keep(rows[q], ids[q] >= 0 && col < C);
      if (j + 1 < tiles) fetch(j + 1);
      lds_order();
      v8_t<DT> xf[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const E* p = stage + (g * 8 + (li >> 2)) * kStride + (TR ? q * 16 + (li & 3) * 4 : (li & 3) * 16 + q * 4);
        xf[q] = read_across<DT>(p, p + 4 * kStride);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const v8_t<DT> vf = as_frag<DT>(L.frag[j - j0][r][p][lane]);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q][r] = TR ? Mat<DT>::mma(vf, xf[q], acc[q][r]) : Mat<DT>::mma(xf[q], vf, acc[q][r]);
        }
      lds_order();
    }
  }
  if (c0 >= C) return;
  const size_t per = (size_t)d.R * (d.K + d.N);
  float* o = it.slot >= 0 ? sums + it.slot * per + (TR ? (size_t)d.R * d.K : 0) : out + (size_t)it.a * d.R * C;
  const float f = __builtin_amdgcn_ldexpf(TR ? d.scale[it.a] : 1.0f, -e);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (TR) {  // [N][R]: a lane holds 4 consecutive r of one column
        const int n = c0 + q * 16 + li, rr = r * 16 + g * 4;
        if (n < C && rr < d.R) *(f32x4*)(o + (size_t)n * d.R + rr) = acc[q][r] * f;
      } else {  // [R][K]: 4 consecutive columns of one r
        const int k = c0 + g * 16 + q * 4, rr = r * 16 + li;
        if (k < C && rr < d.R) *(f32x4*)(o + (size_t)rr * C + k) = acc[q][r] * f;
      }
    }
}

struct GradArgs {
  const float *u, *v;  // [T][R], [S][T][R], in the sorted order
  int S, items, G, slots, dx_passes;
  const void *x, *dy, *add;
  int64_t ldx, lddy, ldadd, lddx;
  void* dx;
  float *d_a, *d_b, *sums;
};

// Workgroups [0, nA) take dA, [nA, nA + nB) dB, the rest dx.
template <int DT, int RT>
__global__ __launch_bounds__(kOutThreads) void k_grad_out(AdapterArgs d, RowSet rs, GradArgs ga) {
  __shared__ GradLds<DT, RT> lds;
  const int ka = (d.K + kOutCols - 1) / kOutCols, kb = (d.N + kOutCols - 1) / kOutCols;
  int b = blockIdx.x;
  if (b < ga.items * ka)
    return grad_outer<DT, RT, false>(lds, d, rs, ga.v, ga.S, b / ka, ga.G, b % ka, ga.x, ga.ldx, ga.d_a, ga.sums, ga.slots);
  b -= ga.items * ka;
  if (b < ga.items * kb)
    return grad_outer<DT, RT, true>(lds, d, rs, ga.u, 1, b / kb, ga.G, b % kb, ga.dy, ga.lddy, ga.d_b, ga.sums, ga.slots);
  b -= ga.items * kb;
  const int kx = (ka + ga.dx_passes - 1) / ga.dx_passes;
  const bool none = b >= rs.tiles * kx;
  grad_dx<DT, RT>(lds, d, rs, ga.v, ga.S, none ? b - rs.tiles * (kx - 1) : b / kx, none ? 0 : b % kx, ga.dx_passes, ga.add,
                  ga.ldadd, ga.dx, ga.lddx);
}

// Sums the partial gradients of adapters that have several.
__global__ __launch_bounds__(256) void k_grad_sum(AdapterArgs d, RowSet rs, const float* part, int slots, int G,
                                                  float* d_a, float* d_b) {
  const int a = blockIdx.x, lane = threadIdx.x & 63;
  int slot = 0, mine = 0;
  for (int a0 = 0; a0 <= a; a0 += 64) {
    int first, count;
    group_of(rs, a0 + lane, d.n, &first, &count);
    const int parts = (count + G - 1) / G, ns = parts > 1 ? parts : 0;
    const int incl = wave_prefix(ns);
    if (a - a0 < 64) {
      slot += at_lane(incl - ns, a - a0);
      mine = at_lane(ns, a - a0);
    } else {
      slot += at_lane(incl, 63);
    }
  }
  mine = min(mine, slots - slot);
  if (mine <= 0) return;
  const size_t na = (size_t)d.R * d.K / 4, nb = (size_t)d.R * d.N / 4;
  for (size_t i = (size_t)blockIdx.y * 256 + threadIdx.x; i < na + nb; i += (size_t)gridDim.y * 256) {
    f32x4 s = {0, 0, 0, 0};
    for (int j = 0; j < mine; ++j) s += ((const f32x4*)part)[(size_t)(slot + j) * (na + nb) + i];
    if (i < na) ((f32x4*)d_a)[(size_t)a * na + i] = s;
    else ((f32x4*)d_b)[(size_t)a * nb + i - na] = s;
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
inline bool bad(const void* p, unsigned align) { return !p || !aligned_to(p, align); }
inline bool bad_ld(int64_t ld, int width) { return ld < width || ld % 8; }
inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

constexpr int64_t kMaxElems = (int64_t)1 << 35;  // of x or dy

int check_adapters(const moe_adapters_t* d, int32_t T) {
  if (!d || T < 0 || d->n < 1 || d->K <= 0 || d->N <= 0 || d->R <= 0) return MOE_E_INVAL;
  if (d->dtype != MOE_T_F16 && d->dtype != MOE_T_BF16) return MOE_E_INVAL;
  if (d->K % 8 || d->N % 8 || d->R % 8 || d->R > 128 || d->n > kMaxExperts || T > kMaxRows || d->K > kMaxWidth ||
      d->N > kMaxWidth || (int64_t)T * std::max(d->K, d->N) > kMaxElems)
    return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

int check_adapter_ptrs(const moe_adapters_t* d) {
  if (bad(d->a, 16) || bad(d->b, 16) || bad(d->scale, 4) || (d->ranks && !aligned_to(d->ranks, 4))) return MOE_E_INVAL;
  return MOE_OK;
}

constexpr int kSmallRows = 64;      // rows that a workgroup groups by itself
constexpr int kSegment = 512;       // columns per K-segment of a small batch
constexpr int kWanted = 256;        // workgroups of k_rows that run at once
constexpr int kWantedOut = 512;     // workgroups of the second launch that do

// Matrix fragments of a rank: 1, 2, 4 or 8 of 16.
int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

struct AdapterPlan {
  bool small;         // forward: grouped by the workgroups, 16-row tiles
  int M, tiles, all;  // forward: rows per tile, bound on tiles of adapters, and with the others
  int S;              // forward: K-segments
  int gtiles, gS, G, items, slots;  // backward
  size_t kept, part, v, u, sums;    // partial u; partial v, sorted u, partial dA and dB
  size_t offsets, pairs, pos, sort, total;
};

AdapterPlan adapter_plan(const moe_adapters_t& d, int T) {
  AdapterPlan p{};
  p.small = T <= kSmallRows;
  p.M = p.small ? 16 : 32;
  p.tiles = (int)std::min<int64_t>(T, (int64_t)T / p.M + d.n + p.small);
  p.all = p.tiles + (p.small ? 0 : ceil_div(T, p.M));
  const auto segments = [](int width, int tiles) {
    return std::max(1, std::min(ceil_div(width, kSegment), kWanted / std::max(1, tiles)));
  };
  p.S = p.small ? ceil_div(d.K, kSegment) : segments(d.K, ceil_div(T, p.M) + d.n / 2);
  p.gS = segments(d.N, ceil_div(T, kGradM) + d.n / 2);
  p.gtiles = (int)std::min<int64_t>(T, (int64_t)T / kGradM + d.n);
  p.G = std::max(256, ceil_div(T, 32 * kGradM) * kGradM);
  p.items = T / p.G + d.n;
  p.slots = T > p.G ? 2 * (T / p.G) : 0;
  size_t o = 0;
  const auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += round256(bytes);
    return at;
  };
  p.offsets = take((size_t)(d.n + 1) * 4);
  p.pairs = take((size_t)T * 4);
  p.pos = take((size_t)T * 4);
  p.sort = take(moe_sort_workspace_bytes(T, 1, d.n));
  p.kept = take((size_t)std::max(p.all, p.gtiles) * sizeof(SharedTile));
  const size_t common = o;
  p.part = take((size_t)p.S * T * d.R * 4);
  const size_t forward = o;
  o = common;
  p.v = take((size_t)p.gS * T * d.R * 4);
  p.u = take((size_t)T * d.R * 4);
  p.sums = take((size_t)p.slots * d.R * ((size_t)d.K + d.N) * 4);
  p.total = std::max(forward, o);
  return p;
}

// Calls f with the type and the number of rank fragments as constants.
template <int V>
struct Const {
  static constexpr int value = V;
};
template <typename F>
void by_shape(const moe_adapters_t& d, F f) {
  const auto ranks = [&](auto dt) {
    switch (rank_tiles(d.R)) {
      case 1: return f(dt, Const<1>{});
      case 2: return f(dt, Const<2>{});
      case 4: return f(dt, Const<4>{});
      default: return f(dt, Const<8>{});
    }
  };
  if (d.dtype == MOE_T_F16) ranks(Const<MOE_T_F16>{});
  else ranks(Const<MOE_T_BF16>{});
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_adapter_workspace_bytes(const moe_adapters_t* d, int32_t T) {
  if (check_adapters(d, T) != MOE_OK) return 0;
  return adapter_plan(*d, T).total;
}

int moe_adapter_forward(const moe_adapters_t* d, const void* x, int64_t ldx, int32_t T, const int32_t* ids,
                        const int32_t* offsets, const int32_t* pairs, const void* add, int64_t ldadd, void* y,
                        int64_t ldy, float* u, void* ws, size_t ws_bytes, void* stream) {
  int st = check_adapters(d, T);
  if (st == MOE_OK) st = check_adapter_ptrs(d);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (bad(x, 16) || bad_ld(ldx, d->K) || bad(ids, 4) || bad(y, 16) || bad_ld(ldy, d->N)) return MOE_E_INVAL;
  if (add && (!aligned_to(add, 16) || bad_ld(ldadd, d->N))) return MOE_E_INVAL;
  if ((offsets == nullptr) != (pairs == nullptr) || (offsets && (bad(offsets, 4) || bad(pairs, 4)))) return MOE_E_INVAL;
  if ((u && !aligned_to(u, 16)) || bad(ws, 16)) return MOE_E_INVAL;
  const AdapterPlan p = adapter_plan(*d, T);
  if (ws_bytes < p.total) return MOE_E_WORKSPACE;
  const hipStream_t s = (hipStream_t)stream;
  const AdapterArgs g{d->a, d->b, d->scale, d->ranks, d->n, d->K, d->N, d->R};
  char* w = (char*)ws;
  RowSet rs{ids, nullptr, nullptr, (SharedTile*)(w + p.kept), T, p.tiles};
  if (!p.small) {
    if (!offsets) {
      int32_t *o = (int32_t*)(w + p.offsets), *q = (int32_t*)(w + p.pairs);
      if (launch_sort(ids, T, 1, d->n, 1, T, o, q, (int32_t*)(w + p.pos), w + p.sort, s) != hipSuccess) return MOE_E_HIP;
      offsets = o;
      pairs = q;
    }
    rs.offsets = offsets;
    rs.pairs = pairs;
  }
  const bool direct = p.S == 1 && u;  // the only segment is u itself
  float* part = direct ? u : (float*)(w + p.part);
  const int cols = ceil_div(d->N, kExpandCols);
  const int passes = std::min(cols, ceil_div((int64_t)p.tiles * cols, kWantedOut));
  by_shape(*d, [&](auto dt, auto rt) {
    constexpr int DT = decltype(dt)::value, RT = decltype(rt)::value;
    const dim3 g1(p.all, p.S), g2(p.all, ceil_div(cols, passes));
    float* uo = direct ? nullptr : u;
    if (p.small) {
      k_rows<DT, 1, RT, false><<<g1, kRowThreads, 0, s>>>(g, rs, x, ldx, part, direct, nullptr, nullptr);
      k_expand<DT, 1, RT><<<g2, kOutThreads, 0, s>>>(g, rs, part, p.S, uo, add, ldadd, y, ldy, passes);
    } else {
      k_rows<DT, 2, RT, false><<<g1, kRowThreads, 0, s>>>(g, rs, x, ldx, part, direct, nullptr, nullptr);
      k_expand<DT, 2, RT><<<g2, kOutThreads, 0, s>>>(g, rs, part, p.S, uo, add, ldadd, y, ldy, passes);
    }
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

int moe_adapter_backward(const moe_adapters_t* d, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                         const float* u, int32_t T, const int32_t* ids, const int32_t* offsets,
                         const int32_t* pairs, const void* add, int64_t ldadd, void* dx, int64_t lddx, float* d_a,
                         float* d_b, void* ws, size_t ws_bytes, void* stream) {
  int st = check_adapters(d, T);
  if (st == MOE_OK) st = check_adapter_ptrs(d);
  if (st != MOE_OK) return st;
  if (bad(d_a, 16) || bad(d_b, 16) || bad(ws, 16)) return MOE_E_INVAL;
  if (T && (bad(dy, 16) || bad_ld(lddy, d->N) || bad(x, 16) || bad_ld(ldx, d->K) || bad(u, 16) || bad(ids, 4)))
    return MOE_E_INVAL;
  if (dx && (!aligned_to(dx, 16) || bad_ld(lddx, d->K))) return MOE_E_INVAL;
  if (add && (!dx || !aligned_to(add, 16) || bad_ld(ldadd, d->K))) return MOE_E_INVAL;
  if (T && (offsets == nullptr) != (pairs == nullptr)) return MOE_E_INVAL;
  if ((offsets && !aligned_to(offsets, 4)) || (pairs && !aligned_to(pairs, 4))) return MOE_E_INVAL;
  const AdapterPlan p = adapter_plan(*d, T);
  if (ws_bytes < p.total) return MOE_E_WORKSPACE;
  const hipStream_t s = (hipStream_t)stream;
  const AdapterArgs g{d->a, d->b, d->scale, d->ranks, d->n, d->K, d->N, d->R};
  char* w = (char*)ws;
  if (!offsets) {
    int32_t *o = (int32_t*)(w + p.offsets), *q = (int32_t*)(w + p.pairs);
    if (launch_sort(ids, T, 1, d->n, 1, T, o, q, (int32_t*)(w + p.pos), w + p.sort, s) != hipSuccess) return MOE_E_HIP;
    offsets = o;
    pairs = q;
  }
  const RowSet rs{ids, offsets, pairs, (SharedTile*)(w + p.kept), T, p.gtiles};
  const int ka = ceil_div(d->K, kOutCols), kb = ceil_div(d->N, kOutCols);
  const int passes = std::min(ka, std::max(1, ceil_div((int64_t)p.gtiles * ka, kWantedOut)));
  float *v = (float*)(w + p.v), *us = (float*)(w + p.u), *sums = (float*)(w + p.sums);
  const GradArgs ga{us, v,   p.gS, p.items, p.G,  p.slots, passes, x,   dy,
                    add, ldx, lddy, ldadd,   lddx, dx,      d_a,    d_b, sums};
  const int dx_groups = dx && T ? p.gtiles * ceil_div(ka, passes) + ceil_div(T, kGradM) : 0;
  by_shape(*d, [&](auto dt, auto rt) {
    constexpr int DT = decltype(dt)::value, RT = decltype(rt)::value;
    if (T) k_rows<DT, 2, RT, true><<<dim3(p.gtiles, p.gS), kRowThreads, 0, s>>>(g, rs, dy, lddy, v, false, u, us);
    k_grad_out<DT, RT><<<p.items * (ka + kb) + dx_groups, kOutThreads, 0, s>>>(g, rs, ga);
  });
  if (p.slots) k_grad_sum<<<dim3(d->n, 64), 256, 0, s>>>(g, rs, sums, p.slots, p.G, d_a, d_b);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // extern "C"
