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
struct RowSet {
  const int32_t *ids, *offsets, *pairs;
  int T;
  int tiles;  // upper bound on tiles of adapters; with offsets, tiles of M rows in order of arrival follow, of
              // which each stands for its rows without an adapter
};

// a: adapter, or n for rows without one; cnt: rows (0: no such tile); this
// lane's row for lane < M, -1 past cnt.
struct Tile {
  int a, cnt, row;
};

__device__ __forceinline__ int lanes_under(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// Inclusive sum over the wavefront's lanes.
__device__ __forceinline__ int wave_prefix(int v, int lane) {
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    v += lane >= d ? o : 0;
  }
  return v;
}

// One adapter's group of rows, bounds checked.
__device__ __forceinline__ void group_of(const RowSet& rs, int a, int n, int* first, int* count) {
  int o0 = 0, o1 = 0;
  if (a < n) {
    o0 = min(max(rs.offsets[a], 0), rs.T);
    o1 = min(max(rs.offsets[a + 1], 0), rs.T);
  }
  *first = o0;
  *count = max(0, o1 - o0);
}

// Called by one whole wavefront.
template <int M>
__device__ __forceinline__ Tile find_tile(const RowSet& rs, int n, int tile) {
  const int lane = threadIdx.x & 63;
  if (!rs.offsets) {
    int id = lane < rs.T ? rs.ids[lane] : 0;
    if ((unsigned)id >= (unsigned)n) id = n;
    uint64_t same = __ballot(lane < rs.T);
    for (int b = 0; b < 11; ++b) {
      const bool one = (id >> b) & 1;
      const uint64_t v = __ballot(one);
      same &= one ? v : ~v;
    }
    const int rank = lanes_under(same);
    uint64_t lead = __ballot(lane < rs.T && rank % M == 0);
    for (int i = 0; i < tile; ++i) lead &= lead - 1;
    if (!lead) return {n, 0, -1};
    const int at = __builtin_ctzll(lead);
    const int a = __shfl(id, at), r0 = __shfl(rank, at);
    const uint64_t mine = __ballot(lane < rs.T && id == a && rank >= r0 && rank < r0 + M);
    const int cnt = __popcll(mine);
    uint64_t m = mine;
    for (int i = 0; i < M - 1; ++i)
      if (i < lane) m &= m - 1;  // this lane's row is the lane-th set bit
    return {a, cnt, lane < cnt ? (int)__builtin_ctzll(m) : -1};
  }
  if (tile >= rs.tiles) {
    const int t = (tile - rs.tiles) * M + lane;
    const bool none = lane < M && t < rs.T && (unsigned)rs.ids[t] >= (unsigned)n;
    const uint64_t mine = __ballot(none);
    uint64_t m = mine;
    for (int i = 0; i < M - 1; ++i)
      if (i < lane) m &= m - 1;
    const int cnt = __popcll(mine);
    return {n, cnt, lane < cnt ? (tile - rs.tiles) * M + (int)__builtin_ctzll(m) : -1};
  }
  for (int a0 = 0, done = 0; a0 < n; a0 += 64) {
    int first, count;
    group_of(rs, a0 + lane, n, &first, &count);
    const int nt = (count + M - 1) / M, incl = wave_prefix(nt, lane);
    const uint64_t past = __ballot(incl > tile - done);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int j = tile - done - __shfl(incl - nt, at);
      const int i0 = __shfl(first, at) + j * M, cnt = min(M, __shfl(count, at) - j * M);
      int row = -1;
      if (lane < cnt) {
        row = rs.pairs[i0 + lane];
        if ((unsigned)row >= (unsigned)rs.T) row = -1;
      }
      return {a0 + at, cnt, row};
    }
    done += __shfl(incl, 63);
  }
  return {n, 0, -1};
}

// find_tile by the first wavefront, handed to the workgroup.
struct SharedTile {
  int a, cnt, row[32];
};
template <int M>
__device__ __forceinline__ void share_tile(SharedTile* s, const RowSet& rs, int n, int tile) {
  if (threadIdx.x < 64) {
    const Tile t = find_tile<M>(rs, n, tile);
    if (threadIdx.x == 0) {
      s->a = t.a;
      s->cnt = t.cnt;
    }
    if (threadIdx.x < 32) s->row[threadIdx.x] = t.row;
  }
  __syncthreads();
}

template <int DT>
__device__ __forceinline__ v8_t<DT> load8(const void* base, size_t i, bool ok) {
  u32x4 v = {0, 0, 0, 0};
  if (ok) v = *(const u32x4*)((const typename Mat<DT>::elem*)base + i);
  return __builtin_bit_cast(v8_t<DT>, v);
}

// load8 of 8 columns of a row of which the first `valid` count.
template <int DT>
__device__ __forceinline__ v8_t<DT> load8_upto(const void* base, size_t i, int valid) {
  v8_t<DT> v = load8<DT>(base, i, valid > 0);
  if (valid > 0 && valid < 8) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c >= valid) v[c] = (typename Mat<DT>::elem)0.0f;
  }
  return v;
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

constexpr int kShrinkThreads = 512;
constexpr int kShrinkWaves = kShrinkThreads / kWave;

// u[t][r] = <A_a[r], x[t]> for a tile's rows and a K-segment per workgroup
// (segment blockIdx.y of S), split again over the wavefronts.  out: [S][T][R].
// Columns are taken 64 at a time: lane group g holds columns 16 g .. + 15.
template <int DT, int MT, int RT>
__global__ __launch_bounds__(kShrinkThreads) void k_shrink(AdapterArgs d, RowSet rs, const void* x, int64_t ldx,
                                                          float* out, bool zero_none) {
  __shared__ SharedTile st;
  __shared__ f32x4 red[kShrinkWaves / 2 * MT * RT * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  share_tile<MT * 16>(&st, rs, d.n, blockIdx.x);
  const int a = st.a, cnt = st.cnt;
  if (!cnt) return;
  float* o = out + (size_t)blockIdx.y * rs.T * d.R;
  if (a == d.n) {
    if (zero_none)
      for (int i = threadIdx.x; i < cnt * d.R; i += kShrinkThreads)
        o[(size_t)st.row[i / d.R] * d.R + i % d.R] = 0.0f;
    return;
  }
  const int rk = rank_of(d, a);
  const int steps = (d.K + 63) / 64, parts = gridDim.y * kShrinkWaves, part = blockIdx.y * kShrinkWaves + wave;
  const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
  size_t xrow[MT], arow[RT];
  bool xok[MT], aok[RT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = st.row[m * 16 + li];
    xok[m] = r >= 0;
    xrow[m] = (size_t)max(r, 0) * ldx;
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    aok[r] = r * 16 + li < rk;
    arow[r] = ((size_t)a * d.R + r * 16 + li) * d.K;
  }
  v8_t<DT> xn[2][MT], an[2][RT];
  const auto fetch = [&](int s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = s * 64 + g * 16 + h * 8;
#pragma unroll
      for (int r = 0; r < RT; ++r) an[h][r] = load8<DT>(d.a, arow[r] + c, aok[r] && c < d.K);
#pragma unroll
      for (int m = 0; m < MT; ++m) xn[h][m] = load8<DT>(x, xrow[m] + c, xok[m] && c < d.K);
    }
  };
  f32x4 acc[MT * RT] = {};
  if (s0 < s1) fetch(s0);
  for (int s = s0; s < s1; ++s) {
    v8_t<DT> xf[2][MT], af[2][RT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int r = 0; r < RT; ++r) af[h][r] = an[h][r];
#pragma unroll
      for (int m = 0; m < MT; ++m) xf[h][m] = xn[h][m];
    }
    if (s + 1 < s1) fetch(s + 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[m * RT + r] = Mat<DT>::mma(af[h][r], xf[h][m], acc[m * RT + r]);
  }
  reduce_waves<kShrinkWaves, MT * RT>(acc, red, wave, lane);
  if (wave == 0) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = st.row[m * 16 + li];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int c = r * 16 + g * 4;
        if (row >= 0 && c < d.R) *(f32x4*)(o + (size_t)row * d.R + c) = acc[m * RT + r];
      }
    }
  }
}

constexpr int kExpandThreads = 256;
constexpr int kExpandWaves = kExpandThreads / kWave;

// Two output vectors (16 columns) of a row: add + f * 2^e * acc.  acc[q]
// holds columns 4 q .. + 3 of the 16.
template <int DT>
__device__ __forceinline__ void finish16(const f32x4 (&acc)[4], float f, int e, const u32x4 (&addv)[2], bool has_add,
                                         void* out, size_t at, int c, int C) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (c + h * 8 >= C) continue;
    float o[8] = {};
    if (has_add) unpack_vec<DT>(addv[h], o);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] += __builtin_amdgcn_ldexpf(acc[h * 2 + i / 4][i % 4] * f, e);
    *(u32x4*)((typename Mat<DT>::elem*)out + at + h * 8) = pack_vec<DT>(o);
  }
}

// y[t] = add[t] + s_a B_a u[t] for a tile's rows and a run of columns, 64
// columns at a time per wavefront.  part: [S][T][R], summed here in order
// (and written to u by the first column run, where S > 1 and u is wanted).
// Matrix row m of fragment q is column 16 (m / 4) + 4 q + m % 4 of the 64, so
// that a lane ends with 16 consecutive columns of one row.
template <int DT, int MT, int RB>
__global__ __launch_bounds__(kExpandThreads) void k_expand(AdapterArgs d, RowSet rs, const float* part, int S, float* u,
                                                          const void* add, int64_t ldadd, void* y, int64_t ldy,
                                                          int groups) {
  constexpr int M = MT * 16, RW = RB * 32;
  __shared__ SharedTile st;
  __shared__ float us[M][RW + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  share_tile<M>(&st, rs, d.n, blockIdx.x);
  const int a = st.a, cnt = st.cnt;
  if (!cnt) return;
  const bool none = a == d.n;
  const int rk = none ? 0 : rank_of(d, a);
  for (int i = tid; i < M * (RW / 4); i += kExpandThreads) {
    const int t = i / (RW / 4), r = i % (RW / 4) * 4, row = st.row[t];
    f32x4 v = {0, 0, 0, 0};
    if (row >= 0 && r < rk)
      for (int s = 0; s < S; ++s) v += *(const f32x4*)(part + ((size_t)s * rs.T + row) * d.R + r);
    *(f32x4*)&us[t][r] = v;
    if (u && blockIdx.y == 0 && row >= 0 && r < d.R) *(f32x4*)(u + (size_t)row * d.R + r) = v;
  }
  __syncthreads();
  v8_t<DT> uf[MT][RB][2];
  int ex[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float v[RB][8], top = 0.0f;
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[b][i] = us[m * 16 + li][b * 32 + g * 8 + i];
        top = fmaxf(top, finite_abs(v[b][i]));
      }
    top = fmaxf(top, __builtin_bit_cast(float, partner<16>(__builtin_bit_cast(int, top))));
    top = fmaxf(top, __builtin_bit_cast(float, partner<32>(__builtin_bit_cast(int, top))));
    ex[m] = scale_exp<DT>(top);
#pragma unroll
    for (int b = 0; b < RB; ++b) split_pieces<DT, 2>(v[b], ex[m], uf[m][b]);
  }
  const float f = none ? 0.0f : d.scale[a];
  for (int q0 = 0; q0 < groups; ++q0) {
    const int n0 = ((blockIdx.y * groups + q0) * kExpandWaves + wave) * 64;
    if (n0 >= d.N) break;
    f32x4 acc[MT][4] = {};
    u32x4 av[MT][2] = {};
    const int c = n0 + g * 16;
    if (add) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = st.row[m * 16 + li];
        const typename Mat<DT>::elem* p = (const typename Mat<DT>::elem*)add + (size_t)max(row, 0) * ldadd + c;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (row >= 0 && c + h * 8 < d.N) av[m][h] = *(const u32x4*)(p + h * 8);
      }
    }
    if (!none) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + (li >> 2) * 16 + q * 4 + (li & 3);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const int r = b * 32 + g * 8;
          const v8_t<DT> bf = load8_upto<DT>(d.b, ((size_t)a * d.N + n) * d.R + r, n < d.N ? rk - r : 0);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            acc[m][q] = Mat<DT>::mma(bf, uf[m][b][0], acc[m][q]);
            acc[m][q] = Mat<DT>::mma(bf, uf[m][b][1], acc[m][q]);
          }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = st.row[m * 16 + li];
      if (row >= 0) finish16<DT>(acc[m], f, -ex[m], av[m], add != nullptr, y, (size_t)row * ldy + c, c, d.N);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward pass: k_grad_rows forms v of every tile and packs v and u as
// fragments; k_grad_out turns them into dx, dA and dB; k_grad_sum adds the
// partial dA and dB of adapters whose rows several workgroups took.
// ---------------------------------------------------------------------------
constexpr int kGradM = 32;  // rows per tile

// What k_grad_rows leaves per tile, in workspace.
struct GradPack {
  u32x4* v1;       // [tiles][2][RB][2 pieces][64]: v, contraction over r
  u32x4 *v2, *u2;  // [tiles][RT][pieces][64]: v and u, contraction over the tile's rows
  int32_t* e;      // [tiles][34]: the rows' powers of two in v1, then v2's and u2's
  float* part;     // [slots][R K + R N]: partial dA and dB
  int slots;
};

// Pieces of a factor of a weight gradient (an fp32 output).
template <int DT>
constexpr int kGradPieces = DT == MOE_T_F16 ? 2 : 3;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// Between a wavefront's writes of its LDS rows and its reads of them by other
// lanes, and back: LDS keeps one wavefront's accesses in order, so only the
// compiler has to.
__device__ __forceinline__ void lds_order() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_wave_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Fragment of 8 contraction terms per lane from rows in LDS: each 16 lanes
// read 4 rows of 16 columns (lane i: row i / 4, 4 columns at its address) and
// lane i receives column i of the 4 rows; lo and hi are this lane's addresses
// for terms 0..3 and 4..7.
template <int DT>
__device__ __forceinline__ v8_t<DT> read_across(const typename Mat<DT>::elem* lo, const typename Mat<DT>::elem* hi) {
  typedef __attribute__((address_space(3))) s16x4* lds_p;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)lo);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)hi);
  const s16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(v8_t<DT>, v);
}

// v[t][r] = s_a sum_n dy[t][n] B_a[n][r] for a tile's rows, N split over the
// wavefronts.  Rows of B pass through LDS (each wavefront its own) and come
// back transposed, NB at a time; the next ones load meanwhile.
template <int DT, int RT>
__global__ __launch_bounds__(kShrinkThreads) void k_grad_rows(AdapterArgs d, RowSet rs, const void* dy, int64_t lddy,
                                                             const float* u, GradPack gp) {
  typedef typename Mat<DT>::elem E;
  constexpr int W = RT * 16, RB = (RT + 1) / 2, RW = RB * 32, MT = kGradM / 16, NP = kGradPieces<DT>;
  constexpr int NB = RT == 8 ? 32 : 64, NH = NB / 32, LS = W + 8, VP = NB * W / 8 / 64, US = RW + 4;
  constexpr int kStage = kShrinkWaves * NB * LS * 2, kRed = kShrinkWaves / 2 * MT * RT * 64 * 16;
  constexpr int kRows = 2 * kGradM * US * 4;
  constexpr int kLds = kStage > kRed ? (kStage > kRows ? kStage : kRows) : (kRed > kRows ? kRed : kRows);
  __shared__ SharedTile st;
  __shared__ float tops[2][kGradM];
  __shared__ __align__(16) char lds[kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4, tile = blockIdx.x;
  share_tile<kGradM>(&st, rs, d.n, tile);
  const int a = st.a;
  if (!st.cnt) return;
  const int rk = rank_of(d, a);
  const int steps = (d.N + NB - 1) / NB;
  const int s0 = steps * wave / kShrinkWaves, s1 = steps * (wave + 1) / kShrinkWaves;
  E* stage = (E*)lds + wave * NB * LS;
  size_t grow[MT];
  bool gok[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = st.row[m * 16 + li];
    gok[m] = r >= 0;
    grow[m] = (size_t)max(r, 0) * lddy;
  }
  v8_t<DT> bv[VP], gv[MT][NH];
  const auto fetch = [&](int s) {
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int v = lane + 64 * i, n = s * NB + v / (W / 8), r = v % (W / 8) * 8;
      bv[i] = load8_upto<DT>(d.b, ((size_t)a * d.N + n) * d.R + r, n < d.N ? rk - r : 0);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const int c = s * NB + g * (NB / 4) + h * 8;
        gv[m][h] = load8<DT>(dy, grow[m] + c, gok[m] && c < d.N);
      }
  };
  f32x4 acc[MT * RT] = {};
  if (s0 < s1) fetch(s0);
  for (int s = s0; s < s1; ++s) {
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int v = lane + 64 * i;
      *(v8_t<DT>*)(stage + v / (W / 8) * LS + v % (W / 8) * 8) = bv[i];
    }
    v8_t<DT> gf[MT][NH];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < NH; ++h) gf[m][h] = gv[m][h];
    if (s + 1 < s1) fetch(s + 1);
    lds_order();
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const E* p = stage + (g * (NB / 4) + h * 8 + (li >> 2)) * LS + r * 16 + (li & 3) * 4;
        const v8_t<DT> bf = read_across<DT>(p, p + 4 * LS);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m * RT + r] = Mat<DT>::mma(bf, gf[m][h], acc[m * RT + r]);
      }
    lds_order();
  }
  __syncthreads();
  reduce_waves<kShrinkWaves, MT * RT>(acc, (f32x4*)lds, wave, lane);

  float* vs = (float*)lds;  // [32][US], then u's
  float* us = vs + kGradM * US;
  if (wave == 0) {
    const float f = d.scale[a];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < RT; ++r) *(f32x4*)(vs + (m * 16 + li) * US + r * 16 + g * 4) = acc[m * RT + r] * f;
  }
  for (int i = tid; i < kGradM * (RW / 4); i += kShrinkThreads) {
    const int t = i / (RW / 4), r = i % (RW / 4) * 4, row = st.row[t];
    f32x4 v = {0, 0, 0, 0};
    if (row >= 0 && r < rk) {
      v = *(const f32x4*)(u + (size_t)row * d.R + r);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (r + c >= rk) v[c] = 0.0f;
    }
    *(f32x4*)(us + t * US + r) = v;
    if (r >= W) *(f32x4*)(vs + t * US + r) = f32x4{0, 0, 0, 0};
  }
  __syncthreads();
  {
    const int t = tid >> 4;  // 16 lanes per row
    float tv = 0.0f, tu = 0.0f;
    for (int r = tid & 15; r < RW; r += 16) {
      tv = fmaxf(tv, finite_abs(vs[t * US + r]));
      tu = fmaxf(tu, finite_abs(us[t * US + r]));
    }
    const auto most = [](float v) {
      v = fmaxf(v, __builtin_bit_cast(float, partner<1>(__builtin_bit_cast(int, v))));
      v = fmaxf(v, __builtin_bit_cast(float, partner<2>(__builtin_bit_cast(int, v))));
      v = fmaxf(v, __builtin_bit_cast(float, partner<4>(__builtin_bit_cast(int, v))));
      return fmaxf(v, __builtin_bit_cast(float, partner<8>(__builtin_bit_cast(int, v))));
    };
    tv = most(tv);
    tu = most(tu);
    if ((tid & 15) == 0) {
      tops[0][t] = tv;
      tops[1][t] = tu;
    }
  }
  __syncthreads();
  float topv = 0.0f, topu = 0.0f;
  for (int t = 0; t < kGradM; ++t) {
    topv = fmaxf(topv, tops[0][t]);
    topu = fmaxf(topu, tops[1][t]);
  }
  const int ev = scale_exp<DT>(topv), eu = scale_exp<DT>(topu);
  if (tid < kGradM) gp.e[tile * 34 + tid] = scale_exp<DT>(tops[0][tid]);
  if (tid == kGradM) gp.e[tile * 34 + kGradM] = ev;
  if (tid == kGradM + 1) gp.e[tile * 34 + kGradM + 1] = eu;
  for (int unit = wave; unit < MT * RB + 2 * RT; unit += kShrinkWaves) {
    float v[8];
    if (unit < MT * RB) {
      const int m = unit / RB, b = unit % RB;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = vs[(m * 16 + li) * US + b * 32 + g * 8 + i];
      v8_t<DT> p[2];
      split_pieces<DT, 2>(v, scale_exp<DT>(tops[0][m * 16 + li]), p);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        gp.v1[((size_t)tile * MT * RB * 2 + unit * 2 + q) * 64 + lane] = __builtin_bit_cast(u32x4, p[q]);
    } else {
      const bool is_u = unit >= MT * RB + RT;
      const int r = unit - MT * RB - (is_u ? RT : 0);
      const float* src = is_u ? us : vs;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = src[(g * 8 + i) * US + r * 16 + li];
      v8_t<DT> p[NP];
      split_pieces<DT, NP>(v, is_u ? eu : ev, p);
      u32x4* out = is_u ? gp.u2 : gp.v2;
#pragma unroll
      for (int q = 0; q < NP; ++q)
        out[((size_t)tile * RT * NP + r * NP + q) * 64 + lane] = __builtin_bit_cast(u32x4, p[q]);
    }
  }
}

// Work items of the weight gradients: up to G rows (a multiple of 32) of one
// adapter; an adapter without rows has one, which writes zeros.
struct Item {
  int a, first, cnt;  // adapter (n: no such item), place in pairs, rows
  int tile;           // of its first row
  int slot;           // partial sum it writes, or -1: the result itself
};

__device__ __forceinline__ Item find_item(const RowSet& rs, int n, int item, int G) {
  const int lane = threadIdx.x & 63;
  int tiles = 0, slots = 0;
  for (int a0 = 0, done = 0; a0 < n; a0 += 64) {
    int first, count;
    group_of(rs, a0 + lane, n, &first, &count);
    const int parts = (count + G - 1) / G, ni = a0 + lane < n ? max(1, parts) : 0;
    const int ns = parts > 1 ? parts : 0, nt = (count + kGradM - 1) / kGradM;
    const int incl = wave_prefix(ni, lane), it = wave_prefix(nt, lane), is = wave_prefix(ns, lane);
    const uint64_t past = __ballot(incl > item - done);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int j = item - done - __shfl(incl - ni, at), c = __shfl(count, at);
      const int slot = slots + __shfl(is - ns, at) + j;
      return {a0 + at, __shfl(first, at) + j * G, max(0, min(G, c - j * G)),
              tiles + __shfl(it - nt, at) + j * (G / kGradM), __shfl(ns, at) ? slot : -1};
    }
    done += __shfl(incl, 63);
    tiles += __shfl(it, 63);
    slots += __shfl(is, 63);
  }
  return {n, 0, 0, 0, -1};
}

constexpr int kOutStride = 72;  // elements of an LDS row of 64 columns
constexpr int kOutCols = kExpandWaves * 64;

// dx of a tile's rows, 64 columns per wavefront: rows of A through LDS, 32 at a time.
template <int DT, int RT>
__device__ __forceinline__ void grad_dx(const AdapterArgs& d, const RowSet& rs, const GradPack& gp, SharedTile* st,
                                        typename Mat<DT>::elem* stage, int tile, int chunk, const void* add,
                                        int64_t ldadd, void* dx, int64_t lddx) {
  typedef typename Mat<DT>::elem E;
  constexpr int RB = (RT + 1) / 2, MT = kGradM / 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  share_tile<kGradM>(st, rs, d.n, tile);
  const int a = st->a, k0 = chunk * kOutCols + wave * 64;
  if (!st->cnt || k0 >= d.K) return;
  const int rk = a == d.n ? 0 : rank_of(d, a);
  f32x4 acc[MT][4] = {};
  u32x4 av[MT][2] = {};
  const int c = k0 + g * 16;
  if (add) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = st->row[m * 16 + li];
      const E* p = (const E*)add + (size_t)max(row, 0) * ldadd + c;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (row >= 0 && c + h * 8 < d.K) av[m][h] = *(const u32x4*)(p + h * 8);
    }
  }
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    if (b * 32 >= rk) break;
    v8_t<DT> rows[4], vf[MT][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = b * 32 + lane / 8 + 8 * i, k = k0 + lane % 8 * 8;
      rows[i] = load8<DT>(d.a, ((size_t)a * d.R + r) * d.K + k, r < rk && k < d.K);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        vf[m][q] = __builtin_bit_cast(v8_t<DT>, gp.v1[((((size_t)tile * MT + m) * RB + b) * 2 + q) * 64 + lane]);
#pragma unroll
    for (int i = 0; i < 4; ++i) *(v8_t<DT>*)(stage + (lane / 8 + 8 * i) * kOutStride + lane % 8 * 8) = rows[i];
    lds_order();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const E* p = stage + (g * 8 + (li >> 2)) * kOutStride + (li & 3) * 16 + q * 4;
      const v8_t<DT> af = read_across<DT>(p, p + 4 * kOutStride);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[m][q] = Mat<DT>::mma(af, vf[m][0], acc[m][q]);
        acc[m][q] = Mat<DT>::mma(af, vf[m][1], acc[m][q]);
      }
    }
    lds_order();
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = st->row[m * 16 + li];
    const int e = rk ? -gp.e[tile * 34 + m * 16 + li] : 0;
    if (row >= 0) finish16<DT>(acc[m], 1.0f, e, av[m], add != nullptr, dx, (size_t)row * lddx + c, c, d.K);
  }
}

// A weight gradient's 64 columns per wavefront over an item's rows: the rows
// of x (dA) or dy (TR: dB) pass through LDS, 32 at a time, against the packed
// v or u.
template <int DT, int RT, bool TR>
__device__ __forceinline__ void grad_outer(const AdapterArgs& d, const RowSet& rs, const GradPack& gp,
                                           typename Mat<DT>::elem* stage, int item, int G, int chunk, const void* x,
                                           int64_t ldx, float* out) {
  typedef typename Mat<DT>::elem E;
  constexpr int NP = kGradPieces<DT>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  const int C = TR ? d.N : d.K, c0 = chunk * kOutCols + wave * 64;
  if (c0 >= C) return;
  const Item it = find_item(rs, d.n, item, G);
  if (it.a >= d.n || it.slot >= gp.slots) return;  // (slots: only for groups that overlap)
  const int tiles = rank_of(d, it.a) ? min((it.cnt + kGradM - 1) / kGradM, rs.tiles - it.tile) : 0;
  const u32x4* pack = TR ? gp.u2 : gp.v2;
  const int col = c0 + lane % 8 * 8;
  v8_t<DT> rows[4];
  const auto fetch = [&](int j) {
    const int i = j * kGradM + (lane & 31);
    int row = i < it.cnt ? rs.pairs[it.first + i] : -1;
    if ((unsigned)row >= (unsigned)rs.T) row = -1;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = __shfl(row, lane / 8 + 8 * q);
      rows[q] = load8<DT>(x, (size_t)max(r, 0) * ldx + col, r >= 0 && col < C);
    }
  };
  f32x4 acc[4][RT] = {};
  if (tiles) fetch(0);
  for (int j = 0; j < tiles; ++j) {
#pragma unroll
    for (int q = 0; q < 4; ++q) *(v8_t<DT>*)(stage + (lane / 8 + 8 * q) * kOutStride + lane % 8 * 8) = rows[q];
    if (j + 1 < tiles) fetch(j + 1);
    lds_order();
    v8_t<DT> xf[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const E* p = stage + (g * 8 + (li >> 2)) * kOutStride + (TR ? q * 16 + (li & 3) * 4 : (li & 3) * 16 + q * 4);
      xf[q] = read_across<DT>(p, p + 4 * kOutStride);
    }
    const size_t tile = it.tile + j;
    const int e = -gp.e[tile * 34 + kGradM + (TR ? 1 : 0)];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      v8_t<DT> vf[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p) vf[p] = __builtin_bit_cast(v8_t<DT>, pack[((tile * RT + r) * NP + p) * 64 + lane]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 s = DT == MOE_T_F16 ? f32x4{0, 0, 0, 0} : acc[q][r];
#pragma unroll
        for (int p = 0; p < NP; ++p) s = TR ? Mat<DT>::mma(vf[p], xf[q], s) : Mat<DT>::mma(xf[q], vf[p], s);
        if (DT == MOE_T_F16) {  // each tile has its own power of two
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[q][r][i] += __builtin_amdgcn_ldexpf(s[i], e);
        } else {
          acc[q][r] = s;
        }
      }
    }
    lds_order();
  }
  const size_t per = (size_t)d.R * (d.K + d.N);
  float* o = it.slot >= 0 ? gp.part + it.slot * per + (TR ? (size_t)d.R * d.K : 0) : out + (size_t)it.a * d.R * C;
  const float f = TR ? d.scale[it.a] : 1.0f;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (TR) {  // [N][R]: a lane holds 4 consecutive r of one column
        const int n = c0 + q * 16 + li, rr = r * 16 + g * 4;
        if (n < C && rr < d.R) *(f32x4*)(o + (size_t)n * d.R + rr) = acc[q][r] * f;
      } else {  // [R][K]: 4 consecutive columns of one r
        const int k = c0 + g * 16 + q * 4, rr = r * 16 + li;
        if (k < C && rr < d.R) *(f32x4*)(o + (size_t)rr * C + k) = acc[q][r];
      }
    }
}

// Workgroups [0, nA) take dA, [nA, nA + nB) dB, the rest dx.
template <int DT, int RT>
__global__ __launch_bounds__(kExpandThreads) void k_grad_out(AdapterArgs d, RowSet rs, GradPack gp, int items, int G,
                                                            const void* x, int64_t ldx, const void* dy, int64_t lddy,
                                                            const void* add, int64_t ldadd, void* dx, int64_t lddx,
                                                            float* d_a, float* d_b) {
  __shared__ SharedTile st;
  __shared__ __align__(16) typename Mat<DT>::elem lds[kExpandWaves][kGradM * kOutStride];
  typename Mat<DT>::elem* stage = lds[threadIdx.x >> 6];
  const int ka = (d.K + kOutCols - 1) / kOutCols, kb = (d.N + kOutCols - 1) / kOutCols;
  int b = blockIdx.x;
  if (b < items * ka) return grad_outer<DT, RT, false>(d, rs, gp, stage, b / ka, G, b % ka, x, ldx, d_a);
  b -= items * ka;
  if (b < items * kb) return grad_outer<DT, RT, true>(d, rs, gp, stage, b / kb, G, b % kb, dy, lddy, d_b);
  b -= items * kb;
  grad_dx<DT, RT>(d, rs, gp, &st, stage, b / ka, b % ka, add, ldadd, dx, lddx);
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
    const int incl = wave_prefix(ns, lane);
    if (a - a0 < 64) {
      slot += __shfl(incl - ns, a - a0);
      mine = __shfl(ns, a - a0);
    } else {
      slot += __shfl(incl, 63);
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
constexpr int kShrinkGroups = 256;  // workgroups wanted of a larger one

// Matrix fragments of a rank: 1, 2, 4 or 8 of 16.
int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

struct AdapterPlan {
  bool small;         // forward: grouped by the workgroups, 16-row tiles
  int M, tiles, all;  // forward: rows per tile, bound on tiles of adapters, and with the others
  int S;              // forward: K-segments
  int gtiles, G, items, slots;  // backward
  size_t part;                  // forward: [S][T][R]
  size_t v1, v2, u2, e, sums;   // backward
  size_t offsets, pairs, pos, sort, total;
};

AdapterPlan adapter_plan(const moe_adapters_t& d, int T) {
  AdapterPlan p{};
  p.small = T <= kSmallRows;
  p.M = p.small ? 16 : 32;
  p.tiles = (int)std::min<int64_t>(T, (int64_t)T / p.M + d.n + p.small);
  p.all = p.tiles + (p.small ? 0 : ceil_div(T, p.M));
  const int most = ceil_div(d.K, kSegment);
  p.S = p.small ? most : std::max(1, std::min(most, ceil_div(kShrinkGroups, std::max(1, ceil_div(T, p.M)))));
  p.gtiles = (int)std::min<int64_t>(T, (int64_t)T / kGradM + d.n);
  p.G = std::max(256, ceil_div(T, 32 * kGradM) * kGradM);
  p.items = T / p.G + d.n;
  p.slots = T > p.G ? 2 * (T / p.G) : 0;
  const int rt = rank_tiles(d.R), rb = (rt + 1) / 2, np = d.dtype == MOE_T_F16 ? 2 : 3;
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
  const size_t common = o;
  p.part = take((size_t)p.S * T * d.R * 4);
  const size_t forward = o;
  o = common;
  p.v1 = take((size_t)p.gtiles * rb * 4 * 1024);
  p.v2 = take((size_t)p.gtiles * rt * np * 1024);
  p.u2 = take((size_t)p.gtiles * rt * np * 1024);
  p.e = take((size_t)p.gtiles * 34 * 4);
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
  RowSet rs{ids, nullptr, nullptr, T, p.tiles};
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
  const int cols = ceil_div(d->N, 64 * kExpandWaves);
  const int groups = p.small ? 1 : std::min(2, cols);
  by_shape(*d, [&](auto dt, auto rt) {
    constexpr int DT = decltype(dt)::value, RT = decltype(rt)::value, RB = (RT + 1) / 2;
    const dim3 g1(p.all, p.S), g2(p.all, ceil_div(cols, groups));
    if (p.small) {
      k_shrink<DT, 1, RT><<<g1, kShrinkThreads, 0, s>>>(g, rs, x, ldx, part, direct);
      k_expand<DT, 1, RB><<<g2, kExpandThreads, 0, s>>>(g, rs, part, p.S, direct ? nullptr : u, add, ldadd, y, ldy, groups);
    } else {
      k_shrink<DT, 2, RT><<<g1, kShrinkThreads, 0, s>>>(g, rs, x, ldx, part, direct);
      k_expand<DT, 2, RB><<<g2, kExpandThreads, 0, s>>>(g, rs, part, p.S, direct ? nullptr : u, add, ldadd, y, ldy, groups);
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
  const RowSet rs{ids, offsets, pairs, T, p.gtiles};
  const GradPack gp{(u32x4*)(w + p.v1), (u32x4*)(w + p.v2), (u32x4*)(w + p.u2), (int32_t*)(w + p.e),
                    (float*)(w + p.sums), p.slots};
  const int ka = ceil_div(d->K, kOutCols), kb = ceil_div(d->N, kOutCols);
  const int dx_tiles = dx && T ? p.gtiles + ceil_div(T, kGradM) : 0;
  by_shape(*d, [&](auto dt, auto rt) {
    constexpr int DT = decltype(dt)::value, RT = decltype(rt)::value;
    if (T) k_grad_rows<DT, RT><<<p.gtiles, kShrinkThreads, 0, s>>>(g, rs, dy, lddy, u, gp);
    k_grad_out<DT, RT><<<p.items * (ka + kb) + dx_tiles * ka, kExpandThreads, 0, s>>>(
        g, rs, gp, p.items, p.G, x, ldx, dy, lddy, add, ldadd, dx, lddx, d_a, d_b);
  });
  if (p.slots) k_grad_sum<<<dim3(d->n, 64), 256, 0, s>>>(g, rs, gp.part, p.slots, p.G, d_a, d_b);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // extern "C"
