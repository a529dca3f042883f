// Low-rank adapters of many requests beside a shared projection
// (include/moe_adapter.h), on the matrix cores.
//
// Rows are taken in tiles of one adapter (16 rows for small batches, 64
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

// ---------------------------------------------------------------------------
// fp32 factors on 16-bit matrix instructions.  u and v are sums and are not
// rounded to 16 bits: a value is carried as a sum of 16-bit pieces, each the
// rounded rest of the ones before (two binary16 pieces hold 22 bits and no less
// than 2^-38 of the scale's largest, two bfloat16 16 bits, three 24).  binary16
// lacks fp32's range, so values are first scaled by a power of two per row (or per
// tile, where the contraction runs over rows) that brings the largest finite one
// to 2^13.
// ---------------------------------------------------------------------------
constexpr int kTopExp = 13;

// Power of two that scales a largest magnitude `top` as above (0 for 0).  Up to
// 2^140, which keeps every bit of subnormal values and has an inverse.
template <int DT>
__device__ __forceinline__ int scale_exp(float top) {
  if (DT == MOE_T_BF16 || top == 0.0f) return 0;
  return min(kTopExp + 1 - __builtin_amdgcn_frexp_expf(top), 140);
}

__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.0f;  // NaN too
}

// SIGN: the first piece is 0 only for 0, else at least the type's smallest step.
template <int DT, int NP, bool SIGN>
__device__ __forceinline__ void split_pieces(const float (&v)[8], int e, v8_t<DT> (&p)[NP]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float rest = DT == MOE_T_F16 ? __builtin_amdgcn_ldexpf(v[i], e) : v[i];
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      typename Mat<DT>::elem h = (typename Mat<DT>::elem)rest;
      if (SIGN && q == 0) {
        const uint16_t bits = __builtin_bit_cast(uint16_t, h);
        h = __builtin_bit_cast(typename Mat<DT>::elem, (uint16_t)(bits | (rest != 0.0f && !(bits & 0x7FFF) ? 1 : 0)));
      }
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

// Where the other factor is infinite the pieces' products cannot be added: a
// second piece of 0 or of the other sign gives NaN beside the first one's infinity.
// (In bfloat16 so can pieces whose products pass fp32's range.)  A result that is
// NaN is therefore formed again from the first pieces alone, which hold the
// values' signs, infinities and NaNs, and stays NaN only where the formula's is.
// Finite results never take that path and pay for looking for NaNs, 0 to 0.5 us of
// a forward call and 0 to 1 us of a backward one (1,801 rows of 6144, rank 64 27.0 ->
// 27.4; gradients of 2,048, rank 16 31.2 -> 31.5, rank 64 60.8 -> 61.8).
__device__ __forceinline__ bool has_nan(f32x4 v) {
  return __builtin_isunordered(v[0], v[1]) || __builtin_isunordered(v[2], v[3]);
}

// v, with what is NaN in it taken from `by`.
__device__ __forceinline__ f32x4 replace_nan(f32x4 v, f32x4 by) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = v[i] == v[i] ? v[i] : by[i];
  return v;
}

// The same for all of a lane's sums where the wavefront has a NaN: first(q) forms
// sums q again.  (One at a time, in a loop: that path must not cost the others
// registers.)
template <typename F>
__device__ __forceinline__ void redo_nan(f32x4 (&acc)[8], F first) {
  bool nan = false;
#pragma unroll
  for (int q = 0; q < 8; ++q) nan |= has_nan(acc[q]);
  const int n = __ballot(nan) ? 8 : 0;
#pragma unroll 1
  for (int q = 0; q < n; ++q) {
    const f32x4 v = first(q);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k == q) acc[k] = replace_nan(acc[k], v);
  }
}

// ---------------------------------------------------------------------------
// Tiles: up to M rows of one adapter.
// ---------------------------------------------------------------------------
constexpr int kSmallM = 16, kM = 64;  // rows per tile: of a small batch, otherwise

// A tile as a workgroup holds it in LDS, and as a pass's first launch leaves
// it in workspace for the next.  a: adapter, or n for rows without one; cnt:
// rows (0: no such tile); first: place of its rows in the sorted order; rank:
// 0 without an adapter; row: -1 past cnt.
struct SharedTile {
  int a, cnt, first, rank;
  int row[kM];
};
constexpr int kTileWords = sizeof(SharedTile) / 4;

// Which rows a call has and how they are grouped.  offsets == NULL: grouped by
// each workgroup itself from ids (find_tile up to 64 rows, else group_tile).
struct RowSet {
  const int32_t *ids, *offsets, *pairs;
  SharedTile* kept;  // [tiles]
  int T;
  int tiles;  // upper bound on tiles of adapters, a multiple of kXcds; with offsets, tiles of kM rows in order of
              // arrival follow, of which each stands for its rows without an adapter
};

// Workgroups go to the GPU's 8 dies in turn, and each die has its own L2.  The
// places of a launch are mapped so that a die takes consecutive tiles: it then
// reads few adapters' factors, and a tile's operands are read by the columns'
// workgroups through one L2.  (The launch's x size is a multiple of 8.)
constexpr int kXcds = 8;
__device__ __forceinline__ int tile_of_place(int place, int used) {  // -1: none
  const int per = (used + kXcds - 1) / kXcds, j = place / kXcds, t = place % kXcds * per + j;
  return j < per && t < used ? t : -1;
}

struct Tile {
  int a, cnt, first, row, rank;  // row: this lane's
};

__device__ __forceinline__ int at_lane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// A value that is the same in every lane, in a scalar register (stores that follow
// then wait for its load once, not each for all that is in flight).
__device__ __forceinline__ float uniform(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
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
  if (M == kSmallM && !rs.offsets) {
    int id = rs.ids[min(lane, rs.T - 1)];
    if ((unsigned)id >= (unsigned)n) id = n;
    const int rank = id < n ? rank_of(d, min(id, n - 1)) : 0;
    if (rs.T == 1) return {at_lane(id, 0), tile == 0, 0, lane == 0 ? 0 : -1, at_lane(rank, 0)};
    uint64_t same = __ballot(lane < rs.T);
    for (int b = 0; b < 11; ++b) {
      const bool one = (id >> b) & 1;
      const uint64_t v = __ballot(one);
      same &= one ? v : ~v;
    }
    const int nth = lanes_below(same);
    uint64_t lead = __ballot(lane < rs.T && nth % M == 0);
    for (int i = 0; i < tile; ++i) lead &= lead - 1;
    if (!lead) return {n, 0, 0, -1, 0};
    const int at = __builtin_ctzll(lead);
    const int a = at_lane(id, at), n0 = at_lane(nth, at);
    const uint64_t mine = __ballot(lane < rs.T && id == a && nth >= n0 && nth < n0 + M);
    const int cnt = __popcll(mine), bit = nth_bit(mine, M);
    return {a, cnt, 0, lane < cnt ? bit : -1, at_lane(rank, at)};
  }
  if (tile >= rs.tiles) {
    const int t0 = min((tile - rs.tiles) * M, rs.T), t = t0 + lane;
    const int id = rs.ids[min(t, rs.T - 1)];
    const uint64_t mine = __ballot(lane < M && t < rs.T && (unsigned)id >= (unsigned)n);
    const int cnt = __popcll(mine), bit = nth_bit(mine, M);
    return {n, cnt, 0, lane < cnt ? t0 + bit : -1, 0};
  }
  int used = 0;
  for (int a0 = 0; a0 < n && n > 64; a0 += 64) {
    int first, count;
    group_of(rs, a0 + lane, n, &first, &count);
    used += at_lane(wave_inclusive_scan((count + M - 1) / M), 63);
  }
  for (int a0 = 0, done = 0; a0 < n; a0 += 64) {
    int first, count;
    group_of(rs, a0 + lane, n, &first, &count);
    const int rank = rank_of(d, min(a0 + lane, n - 1));
    const int nt = (count + M - 1) / M, incl = wave_inclusive_scan(nt);
    if (a0 == 0) {
      tile = tile_of_place(tile, min(n > 64 ? used : at_lane(incl, 63), rs.tiles));
      if (tile < 0) break;
    }
    const uint64_t past = __ballot(incl > tile - done);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int j = tile - done - at_lane(incl - nt, at);
      const int i0 = at_lane(first, at) + j * M, cnt = min(M, at_lane(count, at) - j * M);
      int row = rs.pairs[min(i0 + lane, rs.T - 1)];
      if (lane >= cnt || (unsigned)row >= (unsigned)rs.T) row = -1;
      return {a0 + at, cnt, i0, row, at_lane(rank, at)};
    }
    done += at_lane(incl, 63);
  }
  return {n, 0, 0, -1, 0};
}

// find_tile by the first wavefront; stored to *keep where given.  Ends with a
// barrier.
template <int M>
__device__ __forceinline__ void share_tile(SharedTile* s, const AdapterArgs& d, const RowSet& rs, int tile,
                                           SharedTile* keep) {
  if (threadIdx.x < 64) {
    const Tile t = find_tile<M>(d, rs, tile);
    const auto put = [&](SharedTile* o) {
      o->row[threadIdx.x] = t.row;
      if (threadIdx.x == 0) {
        o->a = t.a;
        o->cnt = t.cnt;
        o->first = t.first;
        o->rank = t.rank;
      }
    };
    put(s);
    if (keep) put(keep);
  }
  __syncthreads();
}

// A tile of kM rows from at most kGroupRows ids of at most 64 adapters, by a whole
// workgroup of NT threads: it counts the adapters' rows, finds the tile's adapter,
// and takes that one's rows by their place among them.  Ends with a barrier.
// 1,801 rows of 8 adapters, 6144 wide, rank 64: 2 us longer than from a sorted
// order, which takes 4 and a launch; calls 27.4 and 29.5 us, 200 rows of 2048, rank 16
// 17.4 and 20.5, 4,096 rows of 64 adapters 84 and 87.  (Of 300 adapters 31.8 and 24.2.)
constexpr int kGroupRows = 4096;
struct GroupLds {
  int count[64];  // rows of each adapter
  int per[64];    // rows of the tile's adapter in each 64
};
template <int NT>
__device__ __forceinline__ void group_tile(SharedTile* s, const AdapterArgs& d, const RowSet& rs, int tile, GroupLds& L,
                                           SharedTile* kept) {
  constexpr int W = NT / 64, C = kGroupRows / NT;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = d.n, bits = 32 - __clz(n);
  int id[C];
#pragma unroll
  for (int c = 0; c < C; ++c) id[c] = rs.ids[min((c * W + wave) * 64 + lane, rs.T - 1)];
  if (tid < 64) L.count[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if ((c * W + wave) * 64 + lane >= rs.T || (unsigned)id[c] >= (unsigned)n) id[c] = -1;
    if ((c * W + wave) * 64 >= rs.T) continue;
    uint64_t same = __ballot(id[c] >= 0);
    for (int b = 0; b < bits; ++b) {
      const bool one = (id[c] >> b) & 1;
      const uint64_t v = __ballot(one);
      same &= one ? v : ~v;
    }
    if (id[c] >= 0 && lanes_below(same) == 0) atomicAdd(&L.count[id[c]], (int)__popcll(same));
  }
  __syncthreads();
  const int count = L.count[lane], nt = (count + kM - 1) / kM, incl = wave_inclusive_scan(nt), to = wave_inclusive_scan(count);
  tile = tile_of_place(tile, min(at_lane(incl, 63), rs.tiles));
  int a = n, cnt = 0, first = 0, j = 0;
  const uint64_t past = __ballot(incl > tile);
  if (tile >= 0 && past) {
    a = __builtin_ctzll(past);
    j = tile - at_lane(incl - nt, a);
    cnt = min(kM, at_lane(count, a) - j * kM);
    first = at_lane(to - count, a) + j * kM;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint64_t m = __ballot(id[c] == a);
    if (lane == 0) L.per[c * W + wave] = (int)__popcll(m);
  }
  __syncthreads();
  const int p = L.per[lane], before = wave_inclusive_scan(p) - p;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint64_t m = __ballot(id[c] == a);
    const int r = __shfl(before, c * W + wave) + lanes_below(m) - j * kM;
    if (id[c] == a && r >= 0 && r < cnt) s->row[r] = (c * W + wave) * 64 + lane;
  }
  if (tid < kM && tid >= cnt) s->row[tid] = -1;
  if (tid == 0) {
    s->a = a;
    s->cnt = cnt;
    s->first = first;
    s->rank = a < n ? rank_of(d, a) : 0;
  }
  __syncthreads();
  if (kept && tid < kTileWords) ((int*)kept)[tid] = ((const int*)s)[tid];
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

constexpr int kRowThreads = 512;
constexpr int kRowWaves = kRowThreads / kWave;

// What k_rows leaves: fragments by bands of 16 of a tile's 64 rows and blocks of
// 32 r.
struct RowsOut {
  float* sums;       // small batches: u [S][T][R] by row; else v [T][R] in the sorted order, or u by row (or NULL)
  u32x4* frag;       // [tiles][4][blocks][2 pieces][64]: contraction over r
  float* scale;      // [tiles][4][blocks][16]: what the products are multiplied by
  int blocks;
  const float* u;    // backward, where given: the forward pass's u, copied to
  float* u_sorted;   //   [T][R] in the sorted order
};

constexpr int cmin(int a, int b) { return a < b ? a : b; }

// (BYTES: no fewer for the wavefronts together, for what follows in k_small.)
template <int MT, int RT, bool ACROSS, int BYTES = 0>
struct RowsLds {
  static constexpr int M = MT * 16, W = RT * 16;
  static constexpr int KS = 64, XV = KS / 8, XS = KS + 8;  // columns per step; x's rows in LDS: vectors, stride
  static constexpr int FR = ACROSS ? KS : W, FV = ACROSS ? W / 8 : XV, FS = ACROSS ? W + 8 : XS;  // the factor's
  static constexpr int kStage = (M * XS + FR * FS) * 2;
  static_assert(kStage >= MT * RT * 1024, "a wavefront's sums fit its stage");
  SharedTile st;
  alignas(16) char lds[kRowWaves * kStage < BYTES ? BYTES : kRowWaves * kStage];
  alignas(16) float vs[M][W + 4];
};

// The long sums over a tile's rows: u[t][r] = <A_a[r], x[t]> (ACROSS false), or
// v[t][r] = s_a sum_c dy[t][c] B_a[c][r] (ACROSS), for MT bands of rows (z) and
// one block of r (y) per workgroup; the columns are split over its wavefronts,
// and in small batches over zs segments (z) first.  Splitting r instead of the
// columns reads x once per block but leaves whole sums, which are split into
// fragments here, once.
// Memory is read 128 contiguous bytes per row (8 lanes side by side: lanes that
// follow the fragments' layout, each in a row of its own, cost the address unit
// four times as many cycles); a wavefront's own LDS turns that into fragments,
// the next steps' loads in flight meanwhile.
// 2,048 rows of 6144 binary16, rank 16: 10.3 us, of which 1.2 find the tile, 3.5
// pass until the first steps have their data, 3.0 take the other two thirds, 1.0
// join and split the sums, the rest is the launch.  1,801 rows, rank 64: 16.4 us, 1.7
// of them grouping; its 120 workgroups are bound by what a CU loads (64 bytes a
// cycle), and more of them load more in all (the choice at RowsShape); with 1,024
// threads each 0.9 us longer.
// FUSED: the tile is in L already, and the sums stay in L.vs.
template <int DT, int MT, int RT, bool ACROSS, bool SMALL, bool FUSED = false, typename Lds>
__device__ __forceinline__ void rows_body(Lds& L, const AdapterArgs& d, const RowSet& rs, const void* x,
                                          int64_t ldx, const RowsOut& out, int tile, int y, int z, int zs) {
  typedef typename Mat<DT>::elem E;
  constexpr int M = Lds::M, W = Lds::W, NF = MT * RT, KS = Lds::KS, XV = Lds::XV, XS = Lds::XS, FR = Lds::FR, FV = Lds::FV,
                FS = Lds::FS, kStage = Lds::kStage;
  constexpr int XL = M * XV / 64, FL = FR * FV / 64;   // loads per lane
  SharedTile& st = L.st;
  char* lds = L.lds;
  auto& vs = L.vs;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  const int t0 = SMALL ? 0 : z * M, r0 = y * W;
  SharedTile* kept = r0 == 0 && z == 0 ? rs.kept + tile : nullptr;
  if (!ACROSS && !SMALL && !rs.offsets) {
    group_tile<kRowThreads>(&st, d, rs, tile, *(GroupLds*)lds, kept);
  } else if (!FUSED) {
    share_tile<SMALL ? kSmallM : kM>(&st, d, rs, tile, kept);
  }
  const int a = __builtin_amdgcn_readfirstlane(st.a), cnt = __builtin_amdgcn_readfirstlane(st.cnt) - t0;
  if (cnt <= 0 || a == d.n) return;
  const int rk = __builtin_amdgcn_readfirstlane(st.rank) - r0, R = d.R, C = ACROSS ? d.N : d.K;
  const int* strow = st.row + t0;
  const int first = st.first + t0;
  if (ACROSS && out.u)  // this block's columns of u
    for (int i = tid; i < min(cnt, M) * (W / 4); i += kRowThreads) {
      const int t = i / (W / 4), r = r0 + i % (W / 4) * 4;
      const f32x4 v = *(const f32x4*)(out.u + (size_t)max(strow[t], 0) * R + (r < R ? r : 0));
      if (r < R) *(f32x4*)(out.u_sorted + (size_t)(first + t) * R + r) = v;
    }
  if (rk <= 0) {
    if (!ACROSS && !SMALL && out.sums)
      for (int i = tid; i < min(cnt, M) * (W / 4); i += kRowThreads) {
        const int t = i / (W / 4), r = r0 + i % (W / 4) * 4;
        if (strow[t] >= 0 && r < R) *(f32x4*)(out.sums + (size_t)strow[t] * R + r) = f32x4{0, 0, 0, 0};
      }
    return;
  }
  const bool whole = rk % 8 == 0;
  const float f = ACROSS || !SMALL ? d.scale[a] : 1.0f;
  const int steps = (C + KS - 1) / KS, parts = (SMALL ? zs : 1) * kRowWaves;
  const int part = (SMALL ? z : 0) * kRowWaves + wave;
  const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
  E* xs = (E*)(lds + wave * kStage);
  E* fs = xs + M * XS;
  const int xc = lane % XV * 8;
  const E* xrow[XL];
  bool xok[XL];
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int r = strow[(lane + 64 * i) / XV];
    xok[i] = r >= 0;
    xrow[i] = (const E*)x + (size_t)max(r, 0) * ldx;
  }
  const E* fbase = (const E*)(ACROSS ? d.b : d.a) + (size_t)a * R * C + (size_t)r0 * (ACROSS ? 1 : C);
  constexpr int DEPTH = XL + FL <= 4 ? 4 : 2;
  u32x4 xn[DEPTH][XL], fn[DEPTH][FL];  // the next steps
  const auto fetch = [&](int s, u32x4 (&xn)[XL], u32x4 (&fn)[FL]) {
    const int c = s * KS + xc < C ? s * KS + xc : 0;
#pragma unroll
    for (int i = 0; i < FL; ++i) {
      const int row = (lane + 64 * i) / FV, fc = (lane + 64 * i) % FV * 8;
      const uint32_t at = ACROSS ? (uint32_t)min(s * KS + row, C - 1) * R + (fc < rk ? fc : 0)
                                 : (uint32_t)(row < rk ? row : 0) * C + c;
      fn[i] = load8<DT>(fbase, at);
    }
#pragma unroll
    for (int i = 0; i < XL; ++i) xn[i] = load8<DT>(xrow[i], c);
  };
  f32x4 acc[NF] = {};
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
    if (s + DEPTH < s1) fetch(s + DEPTH, xn, fn);
    lds_order();
#pragma unroll
    for (int h = 0; h < KS / 32; ++h) {
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
#pragma unroll
  for (int k = 0; k < DEPTH; ++k)
    if (s0 + k < s1) fetch(s0 + k, xn[k], fn[k]);
  for (int s = s0; s < s1; s += DEPTH) {
#pragma unroll
    for (int k = 0; k < DEPTH; ++k)
      if (s + k < s1) step(s + k, xn[k], fn[k]);
  }
  // the wavefronts' sums, added in order
#pragma unroll
  for (int q = 0; q < NF; ++q) *(f32x4*)(lds + wave * kStage + (q * 64 + lane) * 16) = acc[q];
  __syncthreads();
  if (tid < NF * 64) {
    f32x4 s = *(const f32x4*)(lds + tid * 16);
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) s += *(const f32x4*)(lds + w * kStage + tid * 16);
    if (ACROSS) s *= f;
    const int q = tid / 64, t = q / RT * 16 + li, c = q % RT * 16 + g * 4, r = r0 + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = c + i < rk ? s[i] : 0.0f;  // (zeros times an infinity otherwise)
    const int row = ACROSS ? (t < cnt ? first + t : -1) : strow[t];
    if (!FUSED && (SMALL || out.sums) && row >= 0 && r < R)
      *(f32x4*)(out.sums + ((size_t)(SMALL ? z : 0) * rs.T + row) * R + r) = s;
    if (!SMALL || FUSED) *(f32x4*)&vs[t][c] = s;
  }
  if (SMALL) return;
  __syncthreads();
  constexpr int BW = (RT + 1) / 2;  // blocks of 32 r here
  if (wave < MT * BW) {
    const int t = wave / BW * 16 + li, b = wave % BW;
    float v[8], top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = RT > 1 || g < 2 ? vs[t][b * 32 + g * 8 + i] : 0.0f;
      top = fmaxf(top, finite_abs(v[i]));
    }
    top = fmaxf(top, __builtin_bit_cast(float, partner<16>(__builtin_bit_cast(int, top))));
    top = fmaxf(top, __builtin_bit_cast(float, partner<32>(__builtin_bit_cast(int, top))));
    const int e = scale_exp<DT>(top);
    v8_t<DT> h[2];
    split_pieces<DT, 2, true>(v, e, h);
    const size_t at = ((size_t)tile * 4 + t0 / 16 + wave / BW) * out.blocks + y * BW + b;
    out.frag[(at * 2 + 0) * 64 + lane] = __builtin_bit_cast(u32x4, h[0]);
    out.frag[(at * 2 + 1) * 64 + lane] = __builtin_bit_cast(u32x4, h[1]);
    // below 2^-126 this factor loses bits of results that are far below the
    // 16-bit types' smallest step
    if (g == 0) out.scale[at * 16 + li] = __builtin_amdgcn_ldexpf(ACROSS ? 1.0f : f, -e);
  }
}

template <int DT, int MT, int RT, bool ACROSS, bool SMALL>
__global__ __launch_bounds__(kRowThreads) void k_rows(AdapterArgs d, RowSet rs, const void* x, int64_t ldx, RowsOut out) {
  __shared__ RowsLds<MT, RT, ACROSS> lds;
  rows_body<DT, MT, RT, ACROSS, SMALL>(lds, d, rs, x, ldx, out, blockIdx.x, blockIdx.y, blockIdx.z, gridDim.z);
}

constexpr int kOutThreads = 256;
constexpr int kOutWaves = kOutThreads / kWave;
// Wavefronts per SIMD that the second launches are held to.  Calls so and without:
// 1,801 rows of 6144, rank 64 27.4 and 29.7 us, 2,048 rows, rank 32 26.1 and 28.0,
// gradients of rank 16 31.5 and 34.0, but 4,096 rows of 64 adapters 84 and 79.  (4 at
// rank 64 is more than the registers: 31.9 us for the first.)
constexpr int out_waves(int RT) { return RT <= 4 ? 3 : 2; }

// ---------------------------------------------------------------------------
// Second launch of the forward pass.
// ---------------------------------------------------------------------------
// LDS of a small tile's u on its way to fragments.
template <int RB>
struct RowPack {
  float v[kSmallM][RB * 32 + 4];
  alignas(16) float scale[kSmallM];
  u32x4 frag[RB][2][64];
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

// Sums the S segments of a small tile's rows (also written to u, where given),
// and splits them into fragments.  Ends with a barrier.
template <int DT, int RB>
__device__ __forceinline__ void pack_rows(RowPack<RB>* p, const SharedTile& st, const float* part, int S, int T, int R,
                                          float f, float* u) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  const int rk = st.rank;
#pragma unroll
  for (int i0 = 0; i0 < kSmallM * RB * 8; i0 += kOutThreads) {
    const int i = i0 + tid, t = i / (RB * 8), r = i % (RB * 8) * 4;
    if (kSmallM * RB * 8 % kOutThreads && i >= kSmallM * RB * 8) break;
    const int row = st.row[t];
    f32x4 v = {0, 0, 0, 0};
    if (row >= 0 && r < rk) v = sum_segments(part + (size_t)row * R + r, (size_t)T * R, S);
    *(f32x4*)&p->v[t][r] = v;
    if (u && row >= 0 && r < R) *(f32x4*)(u + (size_t)row * R + r) = v;
  }
  __syncthreads();
  if (wave < RB) {
    const int b = wave;
    float v[8], top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p->v[li][b * 32 + g * 8 + i];
#pragma unroll
    for (int c = 0; c < RB * 8; c += 4) {  // a quarter of the row per lane group
      const f32x4 w = *(const f32x4*)&p->v[li][g * RB * 8 + c];
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, finite_abs(w[i]));
    }
    top = fmaxf(top, __builtin_bit_cast(float, partner<16>(__builtin_bit_cast(int, top))));
    top = fmaxf(top, __builtin_bit_cast(float, partner<32>(__builtin_bit_cast(int, top))));
    const int e = scale_exp<DT>(top);
    v8_t<DT> h[2];
    split_pieces<DT, 2, true>(v, e, h);
    p->frag[b][0][lane] = __builtin_bit_cast(u32x4, h[0]);
    p->frag[b][1][lane] = __builtin_bit_cast(u32x4, h[1]);
    if (b == 0 && g == 0) p->scale[li] = __builtin_amdgcn_ldexpf(f, -e);
  }
  __syncthreads();
}

// Column 8 i + q of 128 is lane i's column of product q, so that a lane ends
// with 8 consecutive columns and 16 lanes with 256 contiguous bytes of a row.
// B's rows pass through LDS, row 8 i + q at place 16 q + i (fragment reads then
// meet no bank conflict).
__device__ __forceinline__ int place_of(int n) { return n % 8 * 16 + n / 8; }

// y[t] = add[t] + s_a B_a u[t] for a small tile's rows, 128 columns per
// wavefront.  Bound by a chain of waits: the tile, the sums of u's segments, one
// run of B.  One token, 6144 wide, rank 16: 5.0 us (k_rows 4.0); 48 requests of 32
// adapters of rank up to 64, 6144 to 2048: 6.5 (7.2, for 11 MB of factors).
template <int DT, int RT>
__global__ __launch_bounds__(kOutThreads, out_waves(RT)) void k_expand_small(AdapterArgs d, RowSet rs, const float* part, int S,
                                                                            float* u, const void* add, int64_t ldadd, void* y,
                                                                            int64_t ldy) {
  typedef typename Mat<DT>::elem E;
  constexpr int RB = (RT + 1) / 2, VR = RT == 1 ? 2 : 4, BL = 128 * VR / 64, BS = VR * 8 + 8;
  __shared__ SharedTile st;
  __shared__ RowPack<RB> pk;
  __shared__ __align__(16) E lds[kOutWaves][128 * BS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  take_tile(&st, rs.kept + blockIdx.x);
  if (!__builtin_amdgcn_readfirstlane(st.cnt)) return;
  const int rk = __builtin_amdgcn_readfirstlane(st.rank), a = min(__builtin_amdgcn_readfirstlane(st.a), d.n - 1);
  const bool whole = rk % 8 == 0;
  E* bs = lds[wave];
  const E* bbase = (const E*)d.b + (size_t)a * d.N * d.R;
  const int n0 = (blockIdx.y * kOutWaves + wave) * 128, c = n0 + li * 8;
  if (RT == 1) {  // rank 16 fills half of the contraction; the other half reads zeros
#pragma unroll
    for (int i = 0; i < 2; ++i) *(u32x4*)(bs + (lane + 64 * i) * BS + 16) = u32x4{0, 0, 0, 0};
  }
  u32x4 bn[BL];
  const auto fetch = [&](int b) {
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int v = lane + 64 * i, r = b * 32 + v % VR * 8;
      bn[i] = load8<DT>(bbase, (uint32_t)min(n0 + v / VR, d.N - 1) * d.R + (r < rk ? r : 0));
    }
  };
  fetch(0);
  u32x4 av[4] = {};
  int row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    row[i] = st.row[g * 4 + i];
    if (add) av[i] = load8<DT>((const E*)add + (size_t)max(row[i], 0) * ldadd, c < d.N ? c : 0);
  }
  const float f0 = rk ? d.scale[a] : 0.0f;
  pack_rows<DT, RB>(&pk, st, part, S, rs.T, d.R, f0, blockIdx.y == 0 ? u : nullptr);
  const auto stage = [&](int b) {
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int v = lane + 64 * i, r = b * 32 + v % VR * 8;
      *(u32x4*)(bs + place_of(v / VR) * BS + v % VR * 8) = keep_upto(bn[i], rk - r, whole);
    }
    lds_order();
  };
  const auto factor = [&](int q) { return *(const v8_t<DT>*)(bs + (q * 16 + li) * BS + (RT == 1 ? min(g, 2) : g) * 8); };
  f32x4 acc[8] = {};
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    stage(b);
    if (b + 1 < RB) fetch(b + 1);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const v8_t<DT> bf = factor(q);
      acc[q] = Mat<DT>::mma(as_frag<DT>(pk.frag[b][0][lane]), bf, acc[q]);
      acc[q] = Mat<DT>::mma(as_frag<DT>(pk.frag[b][1][lane]), bf, acc[q]);
    }
    lds_order();
  }
  redo_nan(acc, [&](int q) {
    f32x4 v = {0, 0, 0, 0};
#pragma unroll 1
    for (int b = 0; b < RB; ++b) {
      if (RB > 1) {
        fetch(b);
        stage(b);
      }
      v = Mat<DT>::mma(as_frag<DT>(pk.frag[b][0][lane]), factor(q), v);
      lds_order();
    }
    return v;
  });
  const f32x4 f = *(const f32x4*)&pk.scale[g * 4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float o[8];
    unpack_vec<DT>(av[i], o);
#pragma unroll
    for (int q = 0; q < 8; ++q) o[q] = fmaf(acc[q][i], f[i], o[q]);
    if (row[i] >= 0 && c < d.N) *(u32x4*)((E*)y + (size_t)row[i] * ldy + c) = pack_vec<DT>(o);
  }
}

// Both products of a small tile in one launch, 128 columns of y per wavefront:
// every workgroup forms the tile's u for itself.  That costs the GPU about what
// the launch between did, and spares the host that launch (kSmallElems).  Bound by
// the same chain of waits: one token, 6144 wide, rank 16: 9.5 us.
template <int DT, int RT>
__global__ __launch_bounds__(kRowThreads) void k_small(AdapterArgs d, RowSet rs, const void* x, int64_t ldx, float* u,
                                                      const void* add, int64_t ldadd, void* y, int64_t ldy) {
  typedef typename Mat<DT>::elem E;
  constexpr int RB = (RT + 1) / 2, VR = RT == 1 ? 2 : 4, BL = 128 * VR / 64, BS = VR * 8 + 8;
  __shared__ RowsLds<1, RT, false, kRowWaves * 128 * BS * 2> L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  share_tile<kSmallM>(&L.st, d, rs, blockIdx.x, nullptr);
  if (!__builtin_amdgcn_readfirstlane(L.st.cnt)) return;
  const int rk = __builtin_amdgcn_readfirstlane(L.st.rank), a = min(__builtin_amdgcn_readfirstlane(L.st.a), d.n - 1);
  const bool whole = rk % 8 == 0;
  const E* bbase = (const E*)d.b + (size_t)a * d.N * d.R;
  const int n0 = (blockIdx.y * kRowWaves + wave) * 128, c = n0 + li * 8;
  u32x4 bn[RB][BL], av[4] = {};
  const auto fetch = [&](int b, u32x4 (&bn)[BL]) {
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int v = lane + 64 * i, r = b * 32 + v % VR * 8;
      bn[i] = load8<DT>(bbase, (uint32_t)min(n0 + v / VR, d.N - 1) * d.R + (r < rk ? r : 0));
    }
  };
#pragma unroll
  for (int b = 0; b < RB; ++b) fetch(b, bn[b]);
  int row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    row[i] = L.st.row[g * 4 + i];
    if (add) av[i] = load8<DT>((const E*)add + (size_t)max(row[i], 0) * ldadd, c < d.N ? c : 0);
  }
  if (rk > 0) rows_body<DT, 1, RT, false, true, true>(L, d, rs, x, ldx, RowsOut{}, 0, 0, 0, 1);
  __syncthreads();
  if (u && blockIdx.y == 0)
    for (int i = tid; i < kSmallM * (d.R / 4); i += kRowThreads) {
      const int t = i / (d.R / 4), r = i % (d.R / 4) * 4;
      f32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = r + q < rk ? L.vs[t][r + q] : 0.0f;
      if (L.st.row[t] >= 0) *(f32x4*)(u + (size_t)L.st.row[t] * d.R + r) = v;
    }
  // this wavefront's fragments of u
  float v[RB][8], top = 0.0f;
  const auto fetch_u = [&](int b, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = b * 32 + g * 8 + i;
      v[i] = (RT > 1 || g < 2) && r < rk ? L.vs[li][r] : 0.0f;
    }
  };
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    fetch_u(b, v[b]);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_abs(v[b][i]));
  }
  top = fmaxf(top, __builtin_bit_cast(float, partner<16>(__builtin_bit_cast(int, top))));
  top = fmaxf(top, __builtin_bit_cast(float, partner<32>(__builtin_bit_cast(int, top))));
  const int e = scale_exp<DT>(top);
  const float sc = __builtin_amdgcn_ldexpf(rk ? d.scale[a] : 0.0f, -e);
  E* bs = (E*)L.lds + wave * 128 * BS;
  if (RT == 1) {  // rank 16 fills half of the contraction; the other half reads zeros
#pragma unroll
    for (int i = 0; i < 2; ++i) *(u32x4*)(bs + (lane + 64 * i) * BS + 16) = u32x4{0, 0, 0, 0};
  }
  const auto stage = [&](int b, const u32x4 (&bn)[BL]) {
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int k = lane + 64 * i, r = b * 32 + k % VR * 8;
      *(u32x4*)(bs + place_of(k / VR) * BS + k % VR * 8) = keep_upto(bn[i], rk - r, whole);
    }
    lds_order();
  };
  const auto factor = [&](int q) { return *(const v8_t<DT>*)(bs + (q * 16 + li) * BS + (RT == 1 ? min(g, 2) : g) * 8); };
  f32x4 acc[8] = {};
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    v8_t<DT> h[2];
    split_pieces<DT, 2, false>(v[b], e, h);
    stage(b, bn[b]);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const v8_t<DT> bf = factor(q);
      acc[q] = Mat<DT>::mma(h[0], bf, acc[q]);
      acc[q] = Mat<DT>::mma(h[1], bf, acc[q]);
    }
    lds_order();
  }
  redo_nan(acc, [&](int q) {
    f32x4 s = {0, 0, 0, 0};
#pragma unroll 1
    for (int b = 0; b < RB; ++b) {
      float u[8];
      fetch_u(b, u);
      v8_t<DT> h[1];
      split_pieces<DT, 1, true>(u, e, h);
      if (RB > 1) {
        u32x4 bn[BL];
        fetch(b, bn);
        stage(b, bn);
      }
      s = Mat<DT>::mma(h[0], factor(q), s);
      lds_order();
    }
    return s;
  });
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = __shfl(sc, g * 4 + i);
    float o[8];
    unpack_vec<DT>(av[i], o);
#pragma unroll
    for (int q = 0; q < 8; ++q) o[q] = fmaf(acc[q][i], f, o[q]);
    if (row[i] >= 0 && c < d.N) *(u32x4*)((E*)y + (size_t)row[i] * ldy + c) = pack_vec<DT>(o);
  }
}

// Rows without an adapter (tile >= rs.tiles): out = add or zeros, u = 0.
template <int DT>
__device__ __forceinline__ void copy_none(SharedTile* st, const AdapterArgs& d, const RowSet& rs, int tile, const void* add,
                                          int64_t ldadd, void* out, int64_t ldo, int C, float* u) {
  typedef typename Mat<DT>::elem E;
  share_tile<kM>(st, d, rs, tile, nullptr);
  const int cnt = st->cnt, nv = C / 8;
  for (int i = threadIdx.x; i < cnt * nv; i += kOutThreads) {
    const int row = st->row[i / nv], c = i % nv * 8;
    u32x4 v = {0, 0, 0, 0};
    if (add) v = *(const u32x4*)((const E*)add + (size_t)row * ldadd + c);
    *(u32x4*)((E*)out + (size_t)row * ldo + c) = v;
  }
  if (u)
    for (int i = threadIdx.x; i < cnt * d.R; i += kOutThreads) u[(size_t)st->row[i / d.R] * d.R + i % d.R] = 0.0f;
}

constexpr int kCols = 128;  // columns that a workgroup of the second launch takes at a time

struct SpreadArgs {
  const u32x4* frag;
  const float* scale;
  const void* add;
  int64_t ldadd;
  void* out;
  int64_t ldo;
  float* u;      // forward: zeros for the rows without an adapter (or NULL)
  int passes;    // runs of 128 columns per workgroup
  int columns;   // workgroups of a tile; as many follow for the rows without an adapter, of which the first takes all
};
template <int DT, int RT, bool ACROSS>
struct SpreadLds {
  static constexpr int W = RT * 16, RB = (RT + 1) / 2;
  static constexpr int FS = ACROSS ? kCols + 16 : W + 8;   // row stride
  static constexpr int FR = ACROSS ? RB * 32 : kCols;      // rows
  SharedTile st;
  alignas(16) typename Mat<DT>::elem f[2][FR * FS];        // in turn
};

// The second launch of either pass, for a tile's rows and `passes` runs of 128
// columns: out[t] = add[t] + F v[t], with F = B_a times s_a (forward: rows of
// F in memory, v = u) or A_a^T (ACROSS: columns of F).  A band of 16 rows per
// wavefront, F's part shared in LDS, in two buffers: the next run's F and add
// load while this one is worked on.  Column 8 i + q of a run is lane i's
// column of product q (place_of); where the contraction runs across the rows
// of A, LDS holds their columns in that order, and 16 lanes read product q's
// across.
// Bound by memory, once the first run's data are there: 1,801 rows of 6144
// bfloat16, rank 64: 11.9 us for 44 MB of add and y (3.7 TB/s).
template <int DT, int RT, bool ACROSS>
__device__ __forceinline__ void spread_body(SpreadLds<DT, RT, ACROSS>& L, const AdapterArgs& d, const RowSet& rs,
                                            const SpreadArgs& sa, int tile, int chunk) {
  typedef typename Mat<DT>::elem E;
  typedef SpreadLds<DT, RT, ACROSS> Lds;
  constexpr int W = Lds::W, RB = Lds::RB, FS = Lds::FS, FL = W * kCols / 8 / kOutThreads;
  constexpr int FV = ACROSS ? kCols / 8 : W / 8;           // vectors of a row of F
  SharedTile& st = L.st;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  const int C = ACROSS ? d.K : d.N, R = d.R, passes = sa.passes;
  const u32x4* frag = sa.frag;
  const float* scale = sa.scale;
  const void* add = sa.add;
  void* out = sa.out;
  const int64_t ldadd = sa.ldadd, ldo = sa.ldo;
  if (chunk == sa.columns) {  // the tiles of rows without an adapter
    if (tile * kM < rs.T) copy_none<DT>(&st, d, rs, rs.tiles + tile, add, ldadd, out, ldo, C, sa.u);
    return;
  }
  take_tile(&st, rs.kept + tile);
  const int cnt = __builtin_amdgcn_readfirstlane(st.cnt);
  if (!cnt) return;
  const int rk = __builtin_amdgcn_readfirstlane(st.rank), a = __builtin_amdgcn_readfirstlane(st.a);
  const bool whole = rk % 8 == 0, mine = wave * 16 < cnt;
  const E* fbase = (const E*)(ACROSS ? d.a : d.b) + (size_t)a * R * C;
  u32x4 fn[FL], vf[RB][2], av[4] = {};
  const auto fetch = [&](int c0) {
#pragma unroll
    for (int i = 0; i < FL; ++i) {
      const int v = tid + kOutThreads * i, row = v / FV, c = v % FV * 8;
      if (ACROSS) fn[i] = load8<DT>(fbase, (uint32_t)(row < rk ? row : 0) * C + (c0 + c < C ? c0 + c : 0));
      else fn[i] = load8<DT>(fbase, (uint32_t)min(c0 + row, C - 1) * R + (c < rk ? c : 0));
    }
  };
  const int first = chunk * passes * kCols;
  fetch(first);
  const size_t band = ((size_t)tile * 4 + wave) * RB;
  f32x4 sc[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    // (blocks past the rank, and bands past the rows, hold anything: not used)
    vf[b][0] = frag[((band + b) * 2 + 0) * 64 + lane];
    vf[b][1] = frag[((band + b) * 2 + 1) * 64 + lane];
    sc[b] = *(const f32x4*)(scale + (band + b) * 16 + g * 4);
  }
  int row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = st.row[wave * 16 + g * 4 + i];
  const auto fetch_add = [&](int c0) {
    const int c = c0 + li * 8 < C ? c0 + li * 8 : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) av[i] = load8<DT>((const E*)add + (size_t)max(row[i], 0) * ldadd, c);
  };
  if (add && mine) fetch_add(first);
  if (ACROSS && RT == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) *(u32x4*)(L.f[i] + (tid / 16 + 16) * FS + tid % 16 * 8) = u32x4{0, 0, 0, 0};
  }
  constexpr bool kOneScale = DT == MOE_T_BF16 || RB == 1;  // else the blocks' powers of two differ
  for (int p = 0; p < passes; ++p) {
    const int c0 = first + p * kCols, c = c0 + li * 8;
    E* fs = L.f[p & 1];
#pragma unroll
    for (int i = 0; i < FL; ++i) {
      const int v = tid + kOutThreads * i, frow = v / FV, fc = v % FV * 8;
      if (ACROSS) {
        const v8_t<DT> w = as_frag<DT>(keep(fn[i], frow < rk && c0 + fc < C));
#pragma unroll
        for (int q = 0; q < 8; ++q) fs[frow * FS + q * 16 + fc / 8] = w[q];
      } else {
        *(u32x4*)(fs + place_of(frow) * FS + fc) = keep_upto(fn[i], rk - fc, whole);
      }
    }
    if (p + 1 < passes) fetch(c0 + kCols);
    __syncthreads();
    if (!mine || c0 >= C) continue;
    const auto factor = [&](int b, int q) {
      v8_t<DT> ff = {};
      if (ACROSS) {
        const E* at = fs + (b * 32 + g * 8 + (li >> 2)) * FS + q * 16 + (li & 3) * 4;
        ff = read_across<DT>(at, at + 4 * FS);
      } else if (RT > 1 || g < 2) {
        ff = *(const v8_t<DT>*)(fs + (q * 16 + li) * FS + b * 32 + g * 8);
      }
      return ff;
    };
    f32x4 tot[8] = {};
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      if (b * 32 >= rk) break;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const v8_t<DT> ff = factor(b, q);
        f32x4 s = kOneScale ? tot[q] : f32x4{0, 0, 0, 0};
        s = Mat<DT>::mma(as_frag<DT>(vf[b][0]), ff, s);
        s = Mat<DT>::mma(as_frag<DT>(vf[b][1]), ff, s);
        if (kOneScale) tot[q] = s;
        else
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[q][i] = fmaf(s[i], sc[b][i], tot[q][i]);
      }
    }
    redo_nan(tot, [&](int q) {
      f32x4 v = {0, 0, 0, 0};
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        if (b * 32 >= rk) break;
        const f32x4 s = Mat<DT>::mma(as_frag<DT>(vf[b][0]), factor(b, q), kOneScale ? v : f32x4{0, 0, 0, 0});
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = kOneScale ? s[i] : fmaf(s[i], sc[b][i], v[i]);
      }
      return v;
    });
    u32x4 res[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float o[8];
      unpack_vec<DT>(av[i], o);
      const float f = rk ? sc[0][i] : 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = kOneScale ? fmaf(tot[q][i], f, o[q]) : o[q] + tot[q][i];
      res[i] = pack_vec<DT>(o);
    }
    if (add && p + 1 < passes) fetch_add(c0 + kCols);
    // (past the L2s, whose dirty lines the launch's end would wait for)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row[i] >= 0 && c < C) __builtin_nontemporal_store(res[i], (u32x4*)((E*)out + (size_t)row[i] * ldo + c));
  }
}

template <int DT, int RT, bool ACROSS>
__global__ __launch_bounds__(kOutThreads, out_waves(RT)) void k_spread(AdapterArgs d, RowSet rs, SpreadArgs sa) {
  __shared__ SpreadLds<DT, RT, ACROSS> lds;
  spread_body<DT, RT, ACROSS>(lds, d, rs, sa, blockIdx.x, blockIdx.y);
}

// ---------------------------------------------------------------------------
// Backward pass, in two launches or three (kMergeTiles): k_grad_first forms v
// and, on the CUs that leaves free, dB, and k_grad_second dx and dA; or k_rows
// forms v, k_spread dx, and k_grad_weights dA and dB.  k_grad_sum adds the
// partial dA and dB of adapters whose rows several workgroups took.
// 2,048 rows of 4 adapters, 6144 wide: rank 16, binary16 15.3, 13.7 and 4.2 us for
// 4 passes over 25 MB and partial sums of 7; rank 64, bfloat16 16.4, 10.1 and 36.1,
// the last for making three pieces of each value of u and v in every workgroup,
// between barriers.
// ---------------------------------------------------------------------------
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
    const int incl = wave_inclusive_scan(ni), is = wave_inclusive_scan(ns);
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

constexpr int kGradM = 32;                // rows taken at a time
constexpr int kStride = 72;               // elements of an LDS row of 64 columns
constexpr int kOutCols = kOutWaves * 64;  // columns of a workgroup

// 32-row tiles of v or u held as fragments at a time (a multiple of 4).
template <int RT>
constexpr int kChunkTiles = RT <= 2 ? 8 : 4;

struct OuterArgs {
  const float *u, *v;  // [T][R]; v in the sorted order, u too where two launches follow k_rows
  int items, G, slots;
  const void *x, *dy;
  int64_t ldx, lddy;
  float *d_a, *d_b, *sums;  // sums: [slots][R K + R N], partial results
};

template <int DT, int RT, int H>
struct OuterLds {
  float top[kOutWaves * H];
  int ids[2][kChunkTiles<RT> * kGradM];  // rows of this chunk and of the next
  int redo;                              // whether a result is NaN
  union {
    struct {
      u32x4 frag[kChunkTiles<RT>][RT][kGradPieces<DT>][64];
      typename Mat<DT>::elem rows[kOutWaves * H][kGradM * kStride];
    };
    f32x4 half[H == 2 ? kOutWaves : 1][4 * cmin(RT, 4)][64];  // the second wavefronts' sums (of up to 4 r tiles)
  };
};

// A weight gradient's 64 columns per wavefront (H == 2: per two, which take
// tiles in turn) over an item's rows: the rows of x (dA = sum_t v x^T) or dy (TR:
// dB = s_a sum_t dy u^T) pass through LDS, 32 at a time, two such tiles in flight
// per wavefront, against v or u (IDS: in the order of arrival), which the
// workgroup holds as fragments for a chunk of tiles at a time.  In binary16 those
// share one power of two, the smallest so far; where a chunk brings a smaller
// one, the sums are rescaled.
// Rank 16, 6144 wide: the 256 rows of a chunk take 4.0 us on 192 workgroups, 6.3
// TB/s; 3.9 us pass before the first.  Four tiles in flight instead of two: no
// change.
template <int DT, int RT, int H, bool TR, bool IDS>
__device__ __forceinline__ void grad_outer(OuterLds<DT, RT, H>& L, const AdapterArgs& d, const RowSet& rs, const OuterArgs& ga,
                                           int item, int chunk) {
  typedef typename Mat<DT>::elem E;
  constexpr int CT = kChunkTiles<RT>, WV = kOutWaves * H, UW = (CT * RT + WV - 1) / WV;
  constexpr int CR = CT * kGradM;  // rows of a chunk
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  const int C = TR ? d.N : d.K, c0 = chunk * kOutCols + wave % kOutWaves * 64, half = wave / kOutWaves;
  const float* v = TR ? ga.u : ga.v;
  const E* x = (const E*)(TR ? ga.dy : ga.x);
  const int64_t ldx = TR ? ga.lddy : ga.ldx;
  const Item it = find_item(rs, d.n, item, ga.G);  // by every wavefront: no barrier
  if (it.a >= d.n || it.slot >= ga.slots) return;  // (past the slots: only for groups that overlap)
  const int rk = rank_of(d, it.a), tiles = rk ? (it.cnt + kGradM - 1) / kGradM : 0;
  E* stage = L.rows[wave];
  const int col = c0 + lane % 8 * 8, colc = col < C ? col : 0;
  const auto fetch_id = [&](int j0) {  // this thread's row of a chunk
    const int i = j0 * kGradM + tid;
    const int r = rs.pairs[min(it.first + min(i, it.cnt), rs.T - 1)];
    return i < it.cnt && (unsigned)r < (unsigned)rs.T ? r : -1;
  };
  const auto id_at = [&](int i) { return L.ids[i / CR & 1][i % CR]; };  // row of place i, this chunk or the next
  const auto id_of = [&](int j, int q) { return id_at(j * kGradM + lane / 8 + 8 * q); };
  u32x4 rows[2][4];  // the next two tiles
  const auto fetch = [&](int j, u32x4 (&rows)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) rows[q] = load8<DT>(x + (size_t)max(id_of(j, q), 0) * ldx, colc);
  };
  // this wavefront's part of a chunk of v: unit -> tile unit / RT, r tile unit % RT
  float w[UW][8];
  const auto fetch_v = [&](int j0) {
#pragma unroll
    for (int k = 0; k < UW; ++k) {
      const int unit = min(wave + k * WV, CT * RT - 1), r = min(unit % RT * 16 + li, d.R - 1);
      const int i = (j0 + unit / RT) * kGradM + g * 8;
      if (j0 + unit / RT >= tiles) break;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        w[k][q] = v[(size_t)(IDS ? max(id_at(i + q), 0) : it.first + min(i + q, it.cnt - 1)) * d.R + r];
    }
  };
  const auto pass = [&](auto first) {  // first: from the first pieces alone, for the results that are NaN; whether some are
    constexpr bool FIRST = decltype(first)::value;
    constexpr int NP = FIRST ? 1 : kGradPieces<DT>;
    f32x4 acc[4][RT] = {};
    int e = 0;
    bool any = false;
    int id = -1;
    if (tiles) {
      const int id0 = tid < CR ? fetch_id(0) : -1;
      if (!IDS) fetch_v(0);
      id = tid < CR ? fetch_id(CT) : -1;
      if (tid < CR) {
        L.ids[0][tid] = id0;
        L.ids[1][tid] = id;
      }
      __syncthreads();
      if (IDS) fetch_v(0);
      fetch(half, rows[0]);
      fetch(half + H, rows[1]);
      id = tid < CR ? fetch_id(2 * CT) : -1;
    }
    for (int j0 = 0; j0 < tiles; j0 += CT) {
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < UW; ++k) {
        const int unit = wave + k * WV, r = unit % RT * 16 + li, i = (j0 + unit / RT) * kGradM + g * 8;
        if (j0 + unit / RT >= tiles) break;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const bool row = IDS ? id_at(min(i + q, j0 * kGradM + CR - 1)) >= 0 : i + q < it.cnt;
          w[k][q] = unit < CT * RT && r < rk && row ? w[k][q] : 0.0f;
          top = fmaxf(top, finite_abs(w[k][q]));
        }
      }
      if (DT == MOE_T_F16) {
        top = __builtin_bit_cast(float, wave_max_u32(__builtin_bit_cast(uint32_t, top)));
        if (lane == 0) L.top[wave] = top;
      }
      __syncthreads();  // also: the last chunk's fragments and ids have been read
      if (j0 && tid < CR) {  // the next chunk's rows; and ask for those after
        L.ids[j0 / CT + 1 & 1][tid] = id;
        id = fetch_id(j0 + 2 * CT);
      }
      if (DT == MOE_T_F16) {
#pragma unroll
        for (int q = 0; q < WV; ++q) top = fmaxf(top, L.top[q]);
        if (top > 0.0f) {
          const int en = any ? min(e, scale_exp<DT>(top)) : scale_exp<DT>(top);
          if (any && en < e) {
            const float f = __builtin_amdgcn_ldexpf(1.0f, max(en - e, -126));  // (not 0: the sums may be infinite)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int r = 0; r < RT; ++r) acc[q][r] *= f;
          }
          e = en;
          any = true;
        }
      }
#pragma unroll
      for (int k = 0; k < UW; ++k) {
        const int unit = wave + k * WV;
        if (unit < CT * RT && j0 + unit / RT < tiles) {
          v8_t<DT> p[NP];
          split_pieces<DT, NP, FIRST>(w[k], e, p);
#pragma unroll
          for (int q = 0; q < NP; ++q) L.frag[unit / RT][unit % RT][q][lane] = __builtin_bit_cast(u32x4, p[q]);
        }
      }
      __syncthreads();
      if (j0 + CT < tiles) fetch_v(j0 + CT);
      const auto tile = [&](int j, u32x4 (&rows)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(u32x4*)(stage + (lane / 8 + 8 * q) * kStride + lane % 8 * 8) = keep(rows[q], id_of(j, q) >= 0 && col < C);
        if (j + 2 * H < tiles) fetch(j + 2 * H, rows);
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
      };
      const int j1 = min(j0 + CT, tiles);
      for (int j = j0 + half; j < j1; j += 2 * H) {
        tile(j, rows[0]);
        if (j + H < j1) tile(j + H, rows[1]);
      }
    }
    // the two wavefronts of each 64 columns, 4 r tiles at a time
#pragma unroll
    for (int r0 = 0; r0 < (H == 2 ? RT : 0); r0 += 4) {
      constexpr int RH = RT < 4 ? RT : 4;
      __syncthreads();
      if (half) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int r = 0; r < RH; ++r) L.half[wave % kOutWaves][q * RH + r][lane] = acc[q][r0 + r];
      }
      __syncthreads();
      if (!half) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int r = 0; r < RH; ++r) acc[q][r0 + r] += L.half[wave][q * RH + r][lane];
      }
    }
    bool nan = false;
    if (half || c0 >= C) return nan;
    const size_t per = (size_t)d.R * (d.K + d.N);
    float* out = TR ? ga.d_b : ga.d_a;
    float* o = it.slot >= 0 ? ga.sums + it.slot * per + (TR ? (size_t)d.R * d.K : 0) : out + (size_t)it.a * d.R * C;
    // (without rows: zero, whatever the scale)
    const float f = uniform(tiles ? __builtin_amdgcn_ldexpf(TR ? d.scale[it.a] : 1.0f, -e) : 0.0f);
    const auto put = [&](float* p, f32x4 v) {
      if (FIRST) {
        v = replace_nan(*(const f32x4*)p, v);
      } else {
        nan |= has_nan(v);
      }
      *(f32x4*)p = v;
    };
    // (past the rank: zeros, where the sums may hold zeros times an infinity)
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (TR) {  // [N][R]: a lane holds 4 consecutive r of one column
          const int n = c0 + q * 16 + li, rr = r * 16 + g * 4;
          f32x4 v = acc[q][r] * f;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = rr + i < rk ? v[i] : 0.0f;
          if (n < C && rr < d.R) put(o + (size_t)n * d.R + rr, v);
        } else {  // [R][K]: 4 consecutive columns of one r
          const int k = c0 + g * 16 + q * 4, rr = r * 16 + li;
          if (k < C && rr < d.R) put(o + (size_t)rr * C + k, rr < rk ? acc[q][r] * f : f32x4{0, 0, 0, 0});
        }
      }
    return nan;
  };
  if (tid == 0) L.redo = 0;
  const bool nan = pass(Const<false>{});
  if (!tiles) return;
  if (__ballot(nan) && lane == 0) L.redo = 1;
  __syncthreads();
  if (L.redo) pass(Const<true>{});
}

// Workgroups [0, rows_groups) form v (tile, block of r, bands: as k_rows), the
// rest dB.
template <int DT, int MT, int BT, int RT>
__global__ __launch_bounds__(kRowThreads) void k_grad_first(AdapterArgs d, RowSet rs, const void* dy, int64_t lddy, RowsOut out,
                                                           int blocks, int rows_groups, OuterArgs ga) {
  __shared__ union Lds {
    RowsLds<MT, BT, true> rows;
    OuterLds<DT, RT, 2> outer;
    __device__ Lds() {}
  } lds;
  const int b = blockIdx.x;
  if (b < rows_groups) {
    const int y = b / rs.tiles;
    return rows_body<DT, MT, BT, true, false>(lds.rows, d, rs, dy, lddy, out, b % rs.tiles, y % blocks, y / blocks, 1);
  }
  const int kb = (d.N + kOutCols - 1) / kOutCols;
  grad_outer<DT, RT, 2, true, true>(lds.outer, d, rs, ga, (b - rows_groups) / kb, (b - rows_groups) % kb);
}

// Workgroups [0, nA) take dA, the rest dx.
template <int DT, int RT>
__global__ __launch_bounds__(kOutThreads, out_waves(RT)) void k_grad_second(AdapterArgs d, RowSet rs, SpreadArgs sa, OuterArgs ga) {
  __shared__ union Lds {
    SpreadLds<DT, RT, true> spread;
    OuterLds<DT, RT, 1> outer;
    __device__ Lds() {}
  } lds;
  const int ka = (d.K + kOutCols - 1) / kOutCols, nA = ga.items * ka, b = blockIdx.x;
  if (b < nA) grad_outer<DT, RT, 1, false, false>(lds.outer, d, rs, ga, b / ka, b % ka);
  else spread_body<DT, RT, true>(lds.spread, d, rs, sa, (b - nA) % rs.tiles, (b - nA) / rs.tiles);
}

// Workgroups [0, nA) take dA, the rest dB.
template <int DT, int RT>
__global__ __launch_bounds__(2 * kOutThreads) void k_grad_weights(AdapterArgs d, RowSet rs, OuterArgs ga) {
  __shared__ OuterLds<DT, RT, 2> lds;
  const int ka = (d.K + kOutCols - 1) / kOutCols, kb = (d.N + kOutCols - 1) / kOutCols, nA = ga.items * ka;
  const int b = blockIdx.x;
  if (b < nA) grad_outer<DT, RT, 2, false, false>(lds, d, rs, ga, b / ka, b % ka);
  else grad_outer<DT, RT, 2, true, false>(lds, d, rs, ga, (b - nA) / kb, (b - nA) % kb);
}

// Sums the partial gradients of adapters that have several, in their order (4 to
// 6 us, mostly the launch).
__global__ __launch_bounds__(256) void k_grad_sum(AdapterArgs d, RowSet rs, const float* part, int slots, int G,
                                                  float* d_a, float* d_b) {
  const int a = blockIdx.x, lane = threadIdx.x & 63;
  int slot = 0, mine = 0;
  for (int a0 = 0; a0 <= a; a0 += 64) {
    int first, count;
    group_of(rs, a0 + lane, d.n, &first, &count);
    const int parts = (count + G - 1) / G, ns = parts > 1 ? parts : 0;
    const int incl = wave_inclusive_scan(ns);
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
    const f32x4 s = sum_segments(part + ((size_t)slot * (na + nb) + i) * 4, (na + nb) * 4, mine);
    if (i < na) ((f32x4*)d_a)[(size_t)a * na + i] = s;
    else ((f32x4*)d_b)[(size_t)a * nb + i - na] = s;
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
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

// Rows that each workgroup groups by itself, in tiles of 16: so (in two launches),
// and sorted first, 6144 wide: one row 9.0 and 15.0 us, 48 rows of 32 adapters 15.2
// and 21.0, 64 rows of 4 13.0 and 21.1.  (64: a lane each.)
constexpr int kSmallRows = 64;
// A small batch takes one launch (k_small) up to rank 64 where its workgroups load
// up to so many elements of x and A each, and fit the GPU at once.  Calls so and in
// two launches, of which 3.4 us are the second one's host time (GPU alone in
// brackets): rank 16, 6144 wide 12.9 and 16.0 us (9.5 and 8.9); rank 32, 2048 wide 12.9
// and 15.8 (7.3 and 8.6), 6144 wide 12.9 and 15.9 (11.4 and 9.6); rank 16, 10240 wide
// 12.9 and 15.9 (11.7 and 9.1); rank 64, 6144 wide 16.3 and 15.9 (16.6 and 10.1).
constexpr int kSmallTiles = 4;
constexpr int kSmallElems = 5 << 16;
constexpr int kSmallGroups = 256;
// Columns per K-segment of a small batch: two steps of every wavefront.  Those
// three calls with half as many 9.1, 16.7 and 13.0, with twice as many 9.2, 13.8, 13.8.
constexpr int kSegment = 1024;
constexpr int kWideRows = 4096;  // rows from which k_rows takes 64 r at a time (RowsShape)
constexpr int kWanted = 256;     // workgroups of k_grad_weights, one per CU
// Rank fragments up to which the gradients take two launches.  Two and three
// launches, 6144 wide, 4 adapters: 2,048 rows rank 16 31.4 and 36.5 us, rank 32 40.5
// and 44.3, rank 64 69.0 and 60.5 (the kernels' register and LDS needs add up);
// 8,000 rows, 2048 to 6144 wide, rank 16 65 and 93; 200 rows, 2048 wide 19.6 and
// 22.6.
constexpr int kMergeTiles = 2;
// Workgroups of k_spread below which none takes more than one run.  Calls of 1,801
// and 7,204 rows of 6144, rank 64: 27.4 and 83.3 us; 256: 29.7 and 93.4; 1,024: 27.8
// and 83.9; one run each: 27.7 and 85.3.
constexpr int kSpreadGroups = 512;

// Matrix fragments of a rank: 1, 2, 4 or 8 of 16.
int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

struct AdapterPlan {
  bool small;             // forward: 16-row tiles that the workgroups find from ids
  int tiles;              // bound on tiles of adapters (a multiple of kXcds, and no less than T / kM)
  int stiles, S;          // small: tiles, K-segments
  int rb;                 // blocks of 32 r
  int G, items, slots;    // weight gradients
  size_t kept, part, frag, scale, v, u, sums;
  size_t offsets, pairs, pos, sort, total;
};

AdapterPlan adapter_plan(const moe_adapters_t& d, int T) {
  AdapterPlan p{};
  p.small = T <= kSmallRows;
  p.tiles = ceil_div(std::min(T, T / kM + d.n), kXcds) * kXcds;
  p.stiles = std::min(T, T / kSmallM + d.n + 1);
  p.S = ceil_div(d.K, kSegment);
  p.rb = (rank_tiles(d.R) + 1) / 2;
  // Rows of an adapter per workgroup of its weight gradients: more leave the
  // last one working alone, fewer cost partial sums (R (K + N) floats each).
  // Rank 16, 4 adapters: 2,048 rows of 6144 31.4 us with 256, 39.0 with 512, 51.9 with
  // 1,024; 8,000 rows, 2048 to 6144 wide 64.7, 70.5, 86.3.  Above rank 32 a CU holds
  // one workgroup, so a launch has no more than there are CUs, or one per adapter
  // where that is more: rank 64, 2,048 rows of 6144 of 4 adapters whole 62 us, in parts
  // of 512 64; of one adapter whole 97, in parts of 512 55, of 352 66; 4,000 rows of
  // 2048 of 4 adapters whole 81, in parts of 512 47, of 352 44.  (Up to 256 rows are not split:
  // the sum would cost a launch.)
  const int tiles = rank_tiles(d.R), cols = ceil_div(d.K, kOutCols) + ceil_div(d.N, kOutCols), wanted = kWanted / cols;
  if (tiles <= kMergeTiles) p.G = std::max(256, ceil_div(T, 64 * kGradM) * kGradM);
  else if (wanted <= d.n) p.G = 2048;
  else p.G = std::min(2048, std::max(T <= 256 ? 256 : 128, ceil_div(T, (wanted - d.n) * kGradM) * kGradM));
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
  p.kept = take((size_t)std::max(p.tiles, p.stiles) * sizeof(SharedTile));
  p.part = take(p.small ? (size_t)p.S * T * d.R * 4 : 0);
  p.frag = take((size_t)p.tiles * 4 * p.rb * 2 * 1024);
  p.scale = take((size_t)p.tiles * 4 * p.rb * 16 * 4);
  p.v = take((size_t)T * d.R * 4);
  p.u = take(tiles > kMergeTiles ? (size_t)T * d.R * 4 : 0);
  p.sums = take((size_t)p.slots * d.R * ((size_t)d.K + d.N) * 4);
  p.total = o;
  return p;
}

// Calls f with the type and the number of rank fragments as constants.
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

// Bands and fragments of r per workgroup of k_rows: fewer workgroups re-read
// less, more fill the GPU.  At 6144 columns, rank 64 (mixed), bfloat16: 1,801
// rows 14.4 us with two bands and 32 r, 16.6 with one band and 64 r, 17.7 with
// one band and 32 r, 18.6 with two bands and 64 r; 7,204 rows 30.7 us with two
// bands and 64 r, 37.8 with 32 r, 32.6 with four bands and 32 r.  Rank 16, 1,801
// rows: 9.7 us with one band, 11.8 with two.
template <int RT>
struct RowsShape {
  static constexpr int BT = RT < 2 ? RT : 2, WT = RT < 4 ? RT : 4, MT = RT == 1 ? 1 : 2;
};

template <int DT, int RT, bool ACROSS>
void launch_rows(const AdapterPlan& p, const AdapterArgs& g, const RowSet& rs, const void* x, int64_t ldx,
                 const RowsOut& out, hipStream_t s) {
  constexpr int BT = RowsShape<RT>::BT, WT = RowsShape<RT>::WT, MT = RowsShape<RT>::MT;
  if (!ACROSS && p.small)
    k_rows<DT, 1, BT, ACROSS, true><<<dim3(p.stiles, ceil_div(g.R, BT * 16), p.S), kRowThreads, 0, s>>>(g, rs, x, ldx, out);
  else if (rs.T < kWideRows)
    k_rows<DT, MT, BT, ACROSS, false><<<dim3(p.tiles, ceil_div(g.R, BT * 16), 4 / MT), kRowThreads, 0, s>>>(g, rs, x, ldx, out);
  else
    k_rows<DT, 2, WT, ACROSS, false><<<dim3(p.tiles, ceil_div(g.R, WT * 16), 2), kRowThreads, 0, s>>>(g, rs, x, ldx, out);
}

template <int DT, int RT>
void launch_grad_first(const AdapterPlan& p, const AdapterArgs& g, const RowSet& rs, const void* dy, int64_t lddy,
                       const RowsOut& out, const OuterArgs& ga, hipStream_t s) {
  constexpr int BT = RowsShape<RT>::BT, WT = RowsShape<RT>::WT, MT = RowsShape<RT>::MT;
  const int kb = ceil_div(g.N, kOutCols);
  const auto launch = [&](auto kernel, int mt, int bt) {
    const int blocks = ceil_div(g.R, bt * 16), rows = rs.T ? p.tiles * blocks * (4 / mt) : 0;
    kernel<<<rows + p.items * kb, kRowThreads, 0, s>>>(g, rs, dy, lddy, out, blocks, rows, ga);
  };
  if (rs.T < kWideRows) launch(k_grad_first<DT, MT, BT, RT>, MT, BT);
  else launch(k_grad_first<DT, 2, WT, RT>, 2, WT);
}

// Runs of columns per workgroup of the second launch, and workgroups per tile.
void split_runs(const AdapterPlan& p, int width, SpreadArgs* sa) {
  const int runs = ceil_div(width, kCols);
  sa->passes = std::max(1, std::min(runs, (int)((int64_t)p.tiles * runs / kSpreadGroups)));
  sa->columns = ceil_div(runs, sa->passes);
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
  u32x4* frag = (u32x4*)(w + p.frag);
  float* scale = (float*)(w + p.scale);
  SharedTile* kept = (SharedTile*)(w + p.kept);
  if (p.small) {
    const RowSet rs{ids, nullptr, nullptr, kept, T, p.stiles};
    float* part = (float*)(w + p.part);
    by_shape(*d, [&](auto dt, auto rt) {
      constexpr int DT = decltype(dt)::value, RT = decltype(rt)::value;
      if constexpr (RT <= kSmallTiles) {
        const int groups = ceil_div(d->N, kRowWaves * kCols);
        if (p.stiles * groups <= kSmallGroups && (int64_t)(kSmallM + RT * 16) * d->K <= kSmallElems) {
          k_small<DT, RT><<<dim3(p.stiles, groups), kRowThreads, 0, s>>>(g, rs, x, ldx, u, add, ldadd, y, ldy);
          return;
        }
      }
      launch_rows<DT, RT, false>(p, g, rs, x, ldx, RowsOut{part, frag, scale, p.rb, nullptr, nullptr}, s);
      k_expand_small<DT, RT><<<dim3(p.stiles, ceil_div(d->N, kOutWaves * kCols)), kOutThreads, 0, s>>>(
          g, rs, part, p.S, u, add, ldadd, y, ldy);
    });
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
  }
  if (!offsets && (T > kGroupRows || d->n > 64)) {
    int32_t *o = (int32_t*)(w + p.offsets), *q = (int32_t*)(w + p.pairs);
    if (launch_sort(ids, T, 1, d->n, 1, T, o, q, (int32_t*)(w + p.pos), w + p.sort, s) != hipSuccess) return MOE_E_HIP;
    offsets = o;
    pairs = q;
  }
  const RowSet rs{ids, offsets, pairs, kept, T, p.tiles};
  SpreadArgs sa{frag, scale, add, ldadd, y, ldy, u, 0, 0};
  split_runs(p, d->N, &sa);
  by_shape(*d, [&](auto dt, auto rt) {
    constexpr int DT = decltype(dt)::value, RT = decltype(rt)::value;
    launch_rows<DT, RT, false>(p, g, rs, x, ldx, RowsOut{u, frag, scale, p.rb, nullptr, nullptr}, s);
    k_spread<DT, RT, false><<<dim3(p.tiles, sa.columns + 1), kOutThreads, 0, s>>>(g, rs, sa);
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
  u32x4* frag = (u32x4*)(w + p.frag);
  float *scale = (float*)(w + p.scale), *v = (float*)(w + p.v), *us = (float*)(w + p.u), *sums = (float*)(w + p.sums);
  const RowSet rs{ids, offsets, pairs, (SharedTile*)(w + p.kept), T, p.tiles};
  OuterArgs ga{u, v, p.items, p.G, p.slots, x, dy, ldx, lddy, d_a, d_b, sums};
  SpreadArgs sa{frag, scale, add, ldadd, dx, lddx, nullptr, 0, 0};
  split_runs(p, d->K, &sa);
  by_shape(*d, [&](auto dt, auto rt) {
    constexpr int DT = decltype(dt)::value, RT = decltype(rt)::value;
    const int ka = p.items * ceil_div(d->K, kOutCols), kb = p.items * ceil_div(d->N, kOutCols);
    if constexpr (RT <= kMergeTiles) {
      launch_grad_first<DT, RT>(p, g, rs, dy, lddy, RowsOut{v, frag, scale, p.rb, nullptr, nullptr}, ga, s);
      k_grad_second<DT, RT><<<ka + (dx && T ? p.tiles * (sa.columns + 1) : 0), kOutThreads, 0, s>>>(g, rs, sa, ga);
    } else {
      if (T) launch_rows<DT, RT, true>(p, g, rs, dy, lddy, RowsOut{v, frag, scale, p.rb, u, us}, s);
      if (T && dx) k_spread<DT, RT, true><<<dim3(p.tiles, sa.columns + 1), kOutThreads, 0, s>>>(g, rs, sa);
      ga.u = us;
      k_grad_weights<DT, RT><<<ka + kb, 2 * kOutThreads, 0, s>>>(g, rs, ga);
    }
  });
  if (p.slots)
    k_grad_sum<<<dim3(d->n, ceil_div((int64_t)d->R * (d->K + d->N), 2048)), 256, 0, s>>>(g, rs, sums, p.slots, p.G, d_a,
                                                                                         d_b);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // extern "C"
