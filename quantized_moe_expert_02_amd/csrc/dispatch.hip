// Tokens sorted by expert, their rows laid out and combined, and the
// gradients (include/moe_dispatch.h).
#include <algorithm>
#include <type_traits>

#include "rows.h"

namespace moe {

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kSortMaxBlocks = 128;
// Up to this many times 1,024 slots one workgroup sorts alone, each costing it
// about 1.3 us: with 8 instead, 4,800 slots of 256 experts 8.9 us (5 workgroups: 6.0), 8,000
// 12.8 (6.4).
constexpr int kSortOne = 4;
// Up to this many slots each workgroup counts all of them by itself, in one
// launch.  One launch and two (whose gap costs 3 us on the host and about 1 on the
// GPU): 4,800 slots 6.0 us and 7.8, 16,384 7.8 and 7.7, 32,768 10.6 and 8.7, 48,000
// 12.3 and 11.2, 65,536 14.7 and 10.0.
constexpr int kSortRead = 32768;

// Slots per workgroup (a multiple of kSortThreads) and number of workgroups.
struct SortSplit {
  int per_block, blocks;
};
SortSplit sort_split(int64_t n) {
  const int64_t chunks = (n + kSortThreads - 1) / kSortThreads;
  if (chunks <= kSortOne) return {kSortOne * kSortThreads, 1};
  const int64_t m = (chunks + kSortMaxBlocks - 1) / kSortMaxBlocks;
  return {(int)(m * kSortThreads), (int)((chunks + m - 1) / m)};
}

// Lanes of the wavefront that hold the same id (0 <= id < 2^bits; lanes with
// ok == false match nothing).
__device__ __forceinline__ uint64_t match_id(int id, bool ok, int bits) {
  uint64_t m = __ballot(ok);
  for (int b = 0; b < bits; ++b) {
    const bool one = (id >> b) & 1;
    const uint64_t v = __ballot(one);
    m &= one ? v : ~v;
  }
  return m;
}

// Per-workgroup expert counts, [blocks][E].
__global__ __launch_bounds__(kSortThreads) void k_sort_count(const int32_t* idx, int n, int E, int per_block,
                                                             int32_t* cnt) {
  __shared__ int h[kMaxExperts];
  const int tid = threadIdx.x;
  h[tid] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * per_block, hi = min(lo + per_block, (int64_t)n);
  for (int64_t i = lo + tid; i < hi; i += kSortThreads) {
    const int e = idx[i];
    if ((unsigned)e < (unsigned)E) atomicAdd(&h[e], 1);
  }
  __syncthreads();
  if (tid < E) cnt[(size_t)blockIdx.x * E + tid] = h[tid];
}

// Places every slot: a stable counting sort.  Thread e of each workgroup
// derives expert e's place from all workgroups' counts; then the slots are
// walked 1,024 at a time: a wavefront ranks its 64 slots by matching ids, and
// thread e turns the wavefronts' counts of expert e into places.  ONE: a single
// workgroup, which holds its slots in registers.  cnt == NULL: every workgroup
// counts all slots by itself.  Bound by its chain of steps, not by its 3 words per
// slot: 16,384 slots of 256 experts 7.8 us.
template <bool ONE>
__global__ __launch_bounds__(kSortThreads) void k_sort_place(const int32_t* idx, int n, int E, int bits, int align,
                                                             int rows, int per_block, const int32_t* cnt,
                                                             int32_t* offsets, int32_t* pairs, int32_t* pos) {
  __shared__ int wc[kSortWaves][kMaxExperts];
  __shared__ int wsum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, blk = blockIdx.x, blocks = gridDim.x;
  const int64_t lo = (int64_t)blk * per_block, hi = min(lo + per_block, (int64_t)n);

  int ids[kSortOne], ranks[kSortOne], same[kSortOne];  // ONE: same is the count of the id in the wavefront
  int total = 0, before = 0;
  if (ONE) {
    int* h = wc[0];
    h[tid] = 0;
#pragma unroll
    for (int c = 0; c < kSortOne; ++c) ids[c] = c * kSortThreads + tid < n ? idx[c * kSortThreads + tid] : -1;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kSortOne; ++c) {
      if (c * kSortThreads >= n) break;
      const bool ok = (unsigned)ids[c] < (unsigned)E;
      const uint64_t m = match_id(ids[c], ok, bits);
      ranks[c] = lanes_below(m);
      same[c] = __popcll(m);
      if (ok && ranks[c] == 0) atomicAdd(&h[ids[c]], same[c]);
    }
    __syncthreads();
    total = tid < E ? h[tid] : 0;
  } else if (!cnt) {
    int* h = wc[0];
    h[tid] = 0;
    __syncthreads();
    const auto count = [&](int from, int to) {
      for (int i0 = from + tid; i0 < to; i0 += 8 * kSortThreads) {
        int e[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) e[u] = idx[min(i0 + u * kSortThreads, n - 1)];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (i0 + u * kSortThreads < to && (unsigned)e[u] < (unsigned)E) atomicAdd(&h[e[u]], 1);
      }
    };
    count(0, (int)lo);
    __syncthreads();
    before = tid < E ? h[tid] : 0;
    __syncthreads();
    count((int)lo, n);
    __syncthreads();
    total = tid < E ? h[tid] : 0;
  } else if (tid < E) {
#pragma unroll 8
    for (int b = 0; b < blocks; ++b) {
      const int c = cnt[(size_t)b * E + tid];
      total += c;
      before += b < blk ? c : 0;
    }
  }
  const int padded = (total + align - 1) / align * align;
  int incl = padded;
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d);
    incl += lane >= d ? o : 0;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int start = incl - padded, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    start += w < wave ? wsum[w] : 0;
    all += wsum[w];
  }
  int place = start + before;  // thread e: of expert e's next slot
  if (tid < E && blk == tid % blocks)
    for (int r = start + total; r < start + padded; ++r) pairs[r] = -1;
  if (blk == 0) {
    if (tid < E) offsets[tid] = start;
    if (tid == 0) offsets[E] = all;
  }
  for (int64_t r = (int64_t)all + (int64_t)blk * kSortThreads + tid; r < rows; r += (int64_t)blocks * kSortThreads)
    pairs[r] = -1;

  const auto chunk = [&](int64_t i0, int id, int rank, int count) {
    const bool ok = (unsigned)id < (unsigned)E;
    for (int e = lane; e < E; e += 64) wc[wave][e] = 0;
    __atomic_signal_fence(__ATOMIC_SEQ_CST);  // one wavefront's LDS accesses stay in order
    if (ok && rank == 0) wc[wave][id] = count;
    __syncthreads();
    if (tid < E) {
      int c[kSortWaves];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) c[w] = wc[w][tid];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        wc[w][tid] = place;
        place += c[w];
      }
    }
    __syncthreads();
    const int64_t i = i0 + tid;
    if (i < hi) {
      const int r = ok ? wc[wave][id] + rank : -1;
      pos[i] = r;
      if (ok) pairs[r] = (int)i;
    }
    __syncthreads();
  };
  if (ONE) {
#pragma unroll
    for (int c = 0; c < kSortOne; ++c) {
      if (c * kSortThreads >= n) break;
      chunk(c * kSortThreads, ids[c], ranks[c], same[c]);
    }
  } else {
    for (int64_t i0 = lo; i0 < hi; i0 += kSortThreads) {
      const int id = i0 + tid < hi ? idx[i0 + tid] : -1;
      const uint64_t m = match_id(id, (unsigned)id < (unsigned)E, bits);
      chunk(i0, id, lanes_below(m), __popcll(m));
    }
  }
}

// Sort and rows of a small batch in one launch (align 1, up to kSmallSlots
// slots): every workgroup sorts all slots for itself, then lays out its part of
// one token's row; the first one also writes the order.  Bound by that chain of
// steps: one token of 6144 binary16, top-8 of 256 3.8 us, 128 tokens 9.0.
// So, and as sort and rows: 8 tokens 4.4 and 10.1 us, 50 5.9 and 10.7, 128 9.0 and
// 11.9, 200 (1,600 slots) 17.6 and 13.6.
constexpr int kSmallSlots = 1024;
constexpr int kSmallThreads = 256;

__global__ __launch_bounds__(kSmallThreads) void k_dispatch_small(const u32x4* x, int T, int nv, const int32_t* idx, int k,
                                                                int E, int bits, u32x4* xs, int32_t* offsets,
                                                                int32_t* pairs, int32_t* pos) {
  constexpr int W = kSmallThreads / kWave, C = kSmallSlots / kSmallThreads;
  __shared__ uint16_t wc[C * W][kMaxExperts];  // slots of each expert in each 64 slots, then those before
  __shared__ int start[kMaxExperts + 1], wsum[W], place[kSmallSlots];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = T * k, t = blockIdx.x;
  const int i = blockIdx.y * kSmallThreads + tid;
  u32x4 v = {0, 0, 0, 0};
  if (i < nv) v = x[(size_t)t * nv + i];
  int ids[C], ranks[C];
#pragma unroll
  for (int c = 0; c < C; ++c) ids[c] = c * kSmallThreads + tid < n ? idx[c * kSmallThreads + tid] : -1;
  const int chunks = (n + 63) / 64;
  for (int c = tid; c < chunks * E; c += kSmallThreads) wc[c / E][c % E] = 0;
  __syncthreads();
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (c * kSmallThreads >= n) break;
    const bool ok = (unsigned)ids[c] < (unsigned)E;
    const uint64_t m = match_id(ids[c], ok, bits);
    ranks[c] = lanes_below(m);
    if (ok && ranks[c] == 0) wc[c * W + wave][ids[c]] = (uint16_t)__popcll(m);
  }
  __syncthreads();
  const int per = (E + kSmallThreads - 1) / kSmallThreads;  // experts of this thread
  int total[kMaxExperts / kSmallThreads], mine = 0;
#pragma unroll
  for (int q = 0; q < kMaxExperts / kSmallThreads; ++q) {
    total[q] = 0;
    const int e = tid * per + q;
    if (q < per && e < E)
      for (int c = 0; c < chunks; ++c) {
        const int s = wc[c][e];
        wc[c][e] = (uint16_t)total[q];
        total[q] += s;
      }
    mine += total[q];
  }
  int incl = mine;
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d);
    incl += lane >= d ? o : 0;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int at = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    at += w < wave ? wsum[w] : 0;
    all += wsum[w];
  }
#pragma unroll
  for (int q = 0; q < kMaxExperts / kSmallThreads; ++q) {
    const int e = tid * per + q;
    if (q < per && e < E) start[e] = at;
    at += total[q];
  }
  if (tid == 0) start[E] = all;
  __syncthreads();
  const bool writes = blockIdx.x == 0 && blockIdx.y == 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int s = c * kSmallThreads + tid;
    if (s >= n) continue;
    const bool ok = (unsigned)ids[c] < (unsigned)E;
    const int r = ok ? start[ids[c]] + wc[c * W + wave][ids[c]] + ranks[c] : -1;
    place[s] = r;
    if (writes) {
      pos[s] = r;
      if (ok) pairs[r] = s;
      if (s >= all) pairs[s] = -1;
    }
  }
  if (writes)
    for (int e = tid; e <= E; e += kSmallThreads) offsets[e] = start[e];
  __syncthreads();
  if (i >= nv) return;
  for (int j = 0; j < k; ++j) {
    const int r = place[t * k + j];
    if (r >= 0) xs[(size_t)r * nv + i] = v;
  }
  for (int r = all + t; r < n; r += T) xs[(size_t)r * nv + i] = u32x4{0, 0, 0, 0};
}

// xs[pos(t,j)] = x[t], token by token, 16-byte vectors: x is read once.
// Workgroups past the tokens' zero the rows that hold no slot, a row per thread
// looked over.  Bound by the writes: 2,048 tokens of 6144 binary16, top-8: 40.4 us,
// 5.6 TB/s (a fill of 2 GiB reaches 6.9, a copy of 400 MB 5.4).
constexpr int kRowThreads = 256;  // most threads of a workgroup of the row kernels

// Rows past the last-level cache (256 MB) are read and written without a place
// in the caches.  Written so, they also leave no dirty lines in the dies' L2s,
// which the end of the launch would wait for.
template <bool STREAM>
__device__ __forceinline__ u32x4 load_row(const u32x4* p) {
  return STREAM ? __builtin_nontemporal_load(p) : *p;
}
template <bool STREAM>
__device__ __forceinline__ void store_row(u32x4* p, u32x4 v) {
  if (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// Zeros the rows whose pair is none of the n slots, or (pos given) a slot that
// lies elsewhere.
template <bool STREAM>
__device__ __forceinline__ void zero_pad_rows(const int32_t* pairs, const int32_t* pos, int rows, int n, int part, u32x4* out,
                                              int nv) {
  const int lane = threadIdx.x & 63, r0 = part * blockDim.x + (threadIdx.x & ~63u), r = r0 + lane;
  const int p = pairs[min(r, rows - 1)];
  const bool slot = (unsigned)p < (unsigned)n && (!pos || pos[p] == r);
  uint64_t pad = __ballot(r < rows && !slot);  // a wavefront looks over 64 rows
  for (; pad; pad &= pad - 1) {
    u32x4* o = out + (size_t)(r0 + __builtin_ctzll(pad)) * nv;
    for (int i = lane; i < nv; i += 64) store_row<STREAM>(o + i, u32x4{0, 0, 0, 0});
  }
}

template <bool STREAM>
__global__ __launch_bounds__(kRowThreads) void k_scatter_rows(const u32x4* x, int T, int nv, int k, int rows,
                                                              const int32_t* pos, const int32_t* pairs, u32x4* xs) {
  const int t = blockIdx.x;
  if (t >= T) return zero_pad_rows<STREAM>(pairs, nullptr, rows, T * k, t - T, xs, nv);
  const int32_t* p = pos + (size_t)t * k;
  for (int i = threadIdx.x; i < nv; i += blockDim.x) {
    const u32x4 v = x[(size_t)t * nv + i];
    for (int j = 0; j < k; ++j) {
      const int r = p[j];
      if (r >= 0) store_row<STREAM>(xs + (size_t)r * nv + i, v);
    }
  }
}

// y[t] = add[t] + sum_j w[t][j] o[pos(t,j)] (w == NULL: all ones), slots in
// order, 8 rows in flight.  Bound by reading o: 2,048 tokens of 6144 binary16,
// top-8, with add: 40.5 us, 6.2 TB/s; 8 tokens 3.6 us; 1,501 tokens of 2056 bfloat16,
// top-6, without weights: 9.0 us, 4.3 TB/s.
constexpr int kSlotsAtOnce = 8;

template <int DT, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void k_gather_sum(const u32x4* o, int rows, int nv, const float* w,
                                                            const int32_t* pos, int k, const u32x4* add, u32x4* y) {
  constexpr int VE = kVec<DT>;
  const int t = blockIdx.x, i = blockIdx.y * blockDim.x + threadIdx.x;
  if (i >= nv) return;
  float acc[VE] = {};
  if (add) unpack_vec<DT>(add[(size_t)t * nv + i], acc);
  constexpr int S = kSlotsAtOnce;
  for (int j0 = 0; j0 < k; j0 += S) {
    int r[S];
    float wj[S];
    u32x4 v[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int p = t * k + min(j0 + j, k - 1);
      r[j] = pos[p];
      if (j0 + j >= k || (unsigned)r[j] >= (unsigned)rows) r[j] = -1;
      wj[j] = w ? w[p] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < S; ++j)
      if (r[j] >= 0) v[j] = load_row<STREAM>(o + (size_t)r[j] * nv + i);  // (uniform)
#pragma unroll
    for (int j = 0; j < S; ++j) {
      if (r[j] < 0) continue;
      float f[VE];
      unpack_vec<DT>(v[j], f);
#pragma unroll
      for (int c = 0; c < VE; ++c) acc[c] = fmaf(wj[j], f[c], acc[c]);
    }
  }
  store_row<STREAM>(y + (size_t)t * nv + i, pack_vec<DT>(acc));
}

// d_o[pos(t,j)] = w dy[t]; dw[t][j] = <dy[t], o[pos(t,j)]>.  One workgroup per
// token, 8 slots at a time: their rows of o in flight together.  The workgroups
// past the tokens' zero padding rows.  Bound by reading o and writing d_o: 4,096
// tokens of 2048 bfloat16, top-8, groups padded to 64: 69.6 us, 5.1 TB/s.
template <int DT, bool STREAM_O, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void k_combine_grad(const u32x4* dy, const u32x4* o, int rows, int nv,
                                                              const float* w, const int32_t* pos,
                                                              const int32_t* pairs, int T, int k, u32x4* d_o,
                                                              float* dw) {
  constexpr int VE = kVec<DT>, S = kSlotsAtOnce, W = kRowThreads / kWave;
  __shared__ float part[W][S];
  const int t = blockIdx.x, tid = threadIdx.x;
  if (t >= T) return zero_pad_rows<STREAM>(pairs, pos, rows, T * k, t - T, d_o, nv);
  for (int j0 = 0; j0 < k; j0 += S) {
    int r[S];
    float wj[S], dot[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int p = t * k + min(j0 + j, k - 1);
      r[j] = pos[p];
      if (j0 + j >= k || (unsigned)r[j] >= (unsigned)rows) r[j] = -1;
      wj[j] = w[p];
      dot[j] = 0.0f;
    }
    for (int i = tid; i < nv; i += blockDim.x) {
      const u32x4 gv = dy[(size_t)t * nv + i];
      u32x4 v[S];
#pragma unroll
      for (int j = 0; j < S; ++j)
        if (r[j] >= 0) v[j] = load_row<STREAM_O>(o + (size_t)r[j] * nv + i);  // (uniform)
      float g[VE];
      unpack_vec<DT>(gv, g);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        if (r[j] < 0) continue;
        float f[VE], q[VE];
        unpack_vec<DT>(v[j], f);
#pragma unroll
        for (int c = 0; c < VE; ++c) {
          dot[j] = fmaf(g[c], f[c], dot[j]);
          q[c] = g[c] * wj[j];
        }
        store_row<STREAM>(d_o + (size_t)r[j] * nv + i, pack_vec<DT>(q));
      }
    }
#pragma unroll
    for (int j = 0; j < S; ++j) dot[j] = wave_sum_f32(dot[j]);
    if ((tid & 63) == 0) {
#pragma unroll
      for (int j = 0; j < S; ++j) part[tid >> 6][j] = dot[j];
    }
    __syncthreads();
    if (tid < S && j0 + tid < k) {
      float s = part[0][tid];
      for (int q = 1; q < (int)blockDim.x / kWave; ++q) s += part[q][tid];
      dw[(size_t)t * k + j0 + tid] = s;
    }
    if (j0 + S < k) __syncthreads();
  }
}

constexpr size_t kStream = (size_t)112 << 20;  // bytes of rows from which they are streamed

// Threads of a row kernel's workgroup: the row's vectors in as few equal parts as
// 256 threads allow (a 257-vector row: two parts of 192 threads).
int row_parts(int nv) { return (nv + kRowThreads - 1) / kRowThreads; }
int row_threads(int nv) {
  const int parts = row_parts(nv);
  return ((nv + parts - 1) / parts + kWave - 1) / kWave * kWave;
}

int id_bits(int E) {
  int b = 0;
  while ((1 << b) < E) ++b;
  return b;
}

// Rows given as [T][H] of `dtype`: a supported width and type.
int check_rows(int32_t dtype, int32_t T, int32_t H) {
  if (dtype != MOE_T_F16 && dtype != MOE_T_BF16 && dtype != MOE_T_F32) return MOE_E_INVAL;
  if (T < 0 || H <= 0) return MOE_E_INVAL;
  return H % 8 || H > kMaxWidth || T > kMaxRows ? MOE_E_UNSUPPORTED : MOE_OK;
}

int check_slots(int32_t T, int32_t k, int32_t rows) {
  if (T < 0 || k < 1 || rows < 0) return MOE_E_INVAL;
  return k > kMaxTopK ? MOE_E_UNSUPPORTED : MOE_OK;
}

}  // namespace

int check_sort_shape(int32_t T, int32_t k, int32_t E, int32_t align) {
  if (T < 0 || k < 1 || E < 1 || k > E || align < 1 || align > 1024) return MOE_E_INVAL;
  if (k > kMaxTopK || E > kMaxExperts || T > kMaxRows) return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

hipError_t launch_sort(const int32_t* idx, int T, int k, int E, int align, int rows, int32_t* offsets,
                       int32_t* pairs, int32_t* pos, void* ws, hipStream_t s) {
  const int n = T * k;
  const SortSplit sp = sort_split(n);
  int32_t* cnt = (int32_t*)ws;
  if (sp.blocks == 1) {
    k_sort_place<true><<<1, kSortThreads, 0, s>>>(idx, n, E, id_bits(E), align, rows, sp.per_block, cnt, offsets, pairs,
                                                 pos);
  } else {
    if (n > kSortRead) k_sort_count<<<sp.blocks, kSortThreads, 0, s>>>(idx, n, E, sp.per_block, cnt);
    else cnt = nullptr;
    k_sort_place<false><<<sp.blocks, kSortThreads, 0, s>>>(idx, n, E, id_bits(E), align, rows, sp.per_block, cnt, offsets,
                                                          pairs, pos);
  }
  return hipGetLastError();
}

}  // namespace moe

using namespace moe;

extern "C" {

int64_t moe_sort_rows(int32_t T, int32_t k, int32_t n_experts, int32_t align) {
  if (check_sort_shape(T, k, n_experts, align) != MOE_OK) return -1;
  int64_t r = (int64_t)T * k;
  if (align > 1) r = (r + std::min<int64_t>(n_experts, r) * (align - 1) + align - 1) / align * align;
  return r < ((int64_t)1 << 31) ? r : -1;
}

size_t moe_sort_workspace_bytes(int32_t T, int32_t k, int32_t n_experts) {
  if (check_sort_shape(T, k, n_experts, 1) != MOE_OK) return 0;
  const int blocks = sort_split((int64_t)T * k).blocks;
  return blocks > 1 && (int64_t)T * k > kSortRead ? round256((size_t)blocks * n_experts * 4) : 0;
}

int moe_sort(const int32_t* topk_idx, int32_t T, int32_t k, int32_t n_experts, int32_t align, int32_t* offsets,
             int32_t* pairs, int32_t* pos, void* ws, size_t ws_bytes, void* stream) {
  const int st = check_sort_shape(T, k, n_experts, align);
  if (st != MOE_OK) return st;
  const int64_t rows = moe_sort_rows(T, k, n_experts, align);
  if (rows < 0) return MOE_E_INVAL;
  if (bad(offsets, 4) || (T && (bad(topk_idx, 4) || bad(pairs, 4) || bad(pos, 4)))) return MOE_E_INVAL;
  const size_t need = moe_sort_workspace_bytes(T, k, n_experts);
  if (need && bad(ws, 16)) return MOE_E_INVAL;
  if (ws_bytes < need) return MOE_E_WORKSPACE;
  return launch_sort(topk_idx, T, k, n_experts, align, (int)rows, offsets, pairs, pos, ws, (hipStream_t)stream) ==
                 hipSuccess
             ? MOE_OK
             : MOE_E_HIP;
}

int moe_dispatch(const void* x, int32_t dtype, int32_t T, int32_t H, const int32_t* topk_idx, int32_t k,
                 int32_t n_experts, int32_t align, void* xs, int32_t* offsets, int32_t* pairs, int32_t* pos,
                 void* ws, size_t ws_bytes, void* stream) {
  int st = check_rows(dtype, T, H);
  if (st != MOE_OK) return st;
  st = check_sort_shape(T, k, n_experts, align);
  if (st != MOE_OK) return st;
  if (T && (bad(x, 16) || bad(xs, 16))) return MOE_E_INVAL;
  const int nv = (int)((size_t)H * elem_bytes(dtype) / 16), n = T * k;
  if (T && align == 1 && n <= kSmallSlots) {
    if (bad(offsets, 4) || bad(topk_idx, 4) || bad(pairs, 4) || bad(pos, 4)) return MOE_E_INVAL;
    k_dispatch_small<<<dim3(T, (nv + kSmallThreads - 1) / kSmallThreads), kSmallThreads, 0, (hipStream_t)stream>>>(
        (const u32x4*)x, T, nv, topk_idx, k, n_experts, id_bits(n_experts), (u32x4*)xs, offsets, pairs, pos);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
  }
  st = moe_sort(topk_idx, T, k, n_experts, align, offsets, pairs, pos, ws, ws_bytes, stream);
  if (st != MOE_OK || T == 0) return st;
  const int rows = (int)moe_sort_rows(T, k, n_experts, align);
  const int threads = row_threads(nv), grid = T + (rows + threads - 1) / threads;
  const auto launch = [&](auto kernel) {
    kernel<<<grid, threads, 0, (hipStream_t)stream>>>((const u32x4*)x, T, nv, k, rows, pos, pairs, (u32x4*)xs);
  };
  // 6144 wide, top-8, binary16, a call after another, plain and streamed: 50 MB of
  // rows 18.8 us and 18.5, 88 MB 22.1 and 23.6, 118 MB 31.1 and 29.4, 147 MB 42.6 and
  // 35.6, 201 MB 55.3 and 47.6.
  if ((size_t)n * nv * 16 >= kStream) launch(k_scatter_rows<true>);
  else launch(k_scatter_rows<false>);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

static int gather_sum(const void* o, int32_t dtype, int32_t rows, int32_t H, const float* w, const int32_t* pos,
                      int32_t T, int32_t k, const void* add, void* y, void* stream) {
  if (T == 0) return MOE_OK;
  if ((rows && bad(o, 16)) || bad(pos, 4) || bad(y, 16) || (add && !aligned_to(add, 16))) return MOE_E_INVAL;
  const int nv = (int)((size_t)H * elem_bytes(dtype) / 16);
  const dim3 grid(T, row_parts(nv));
  const int threads = row_threads(nv);
  const auto launch = [&](auto kernel) {
    kernel<<<grid, threads, 0, (hipStream_t)stream>>>((const u32x4*)o, rows, nv, w, pos, k, (const u32x4*)add,
                                                         (u32x4*)y);
  };
  // 6144 wide, top-8, binary16, plain and streamed: 101 MB of rows 23.1 and 22.5 us,
  // 201 MB 46.8 and 42.9, 403 MB 99.8 and 84.4; 25 MB 7.0 and 7.9.  (201 MB, y
  // written plainly and streamed: 42.8 and 40.4.)
  const bool stream_rows = (size_t)T * k * nv * 16 >= kStream;
  if (dtype == MOE_T_F16) stream_rows ? launch(k_gather_sum<MOE_T_F16, true>) : launch(k_gather_sum<MOE_T_F16, false>);
  else if (dtype == MOE_T_BF16) stream_rows ? launch(k_gather_sum<MOE_T_BF16, true>) : launch(k_gather_sum<MOE_T_BF16, false>);
  else stream_rows ? launch(k_gather_sum<MOE_T_F32, true>) : launch(k_gather_sum<MOE_T_F32, false>);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

int moe_dispatch_backward(const void* dxs, int32_t dtype, int32_t rows, int32_t H, const int32_t* pos, int32_t T,
                          int32_t k, const void* add, void* dx, void* stream) {
  int st = check_rows(dtype, T, H);
  if (st == MOE_OK) st = check_slots(T, k, rows);
  if (st != MOE_OK) return st;
  return gather_sum(dxs, dtype, rows, H, nullptr, pos, T, k, add, dx, stream);
}

int moe_combine(const void* o, int32_t dtype, int32_t rows, int32_t H, const float* topk_w, const int32_t* pos,
                int32_t T, int32_t k, const void* add, void* y, void* stream) {
  int st = check_rows(dtype, T, H);
  if (st == MOE_OK) st = check_slots(T, k, rows);
  if (st != MOE_OK) return st;
  if (T && bad(topk_w, 4)) return MOE_E_INVAL;
  return gather_sum(o, dtype, rows, H, topk_w, pos, T, k, add, y, stream);
}

int moe_combine_backward(const void* dy, const void* o, int32_t dtype, int32_t rows, int32_t H,
                         const float* topk_w, const int32_t* pos, const int32_t* pairs, int32_t T, int32_t k,
                         void* d_o, float* dw, void* stream) {
  int st = check_rows(dtype, T, H);
  if (st == MOE_OK) st = check_slots(T, k, rows);
  if (st != MOE_OK) return st;
  if (rows > kMaxSorted) return MOE_E_UNSUPPORTED;
  if (T == 0 && rows == 0) return MOE_OK;
  if (T && (bad(dy, 16) || bad(topk_w, 4) || bad(pos, 4) || bad(dw, 4))) return MOE_E_INVAL;
  if (rows && (bad(o, 16) || bad(d_o, 16) || bad(pairs, 4))) return MOE_E_INVAL;
  const int nv = (int)((size_t)H * elem_bytes(dtype) / 16);
  const int threads = row_threads(nv), grid = T + (rows + threads - 1) / threads;
  const auto launch = [&](auto kernel) {
    kernel<<<grid, threads, 0, (hipStream_t)stream>>>((const u32x4*)dy, (const u32x4*)o, rows, nv, topk_w, pos,
                                                         pairs, T, k, (u32x4*)d_o, dw);
  };
  // o is streamed where it and d_o together are that large, d_o where it is.  2048
  // wide, top-8, binary16, a call after another, o of 33 MB plain 12.8 us, o streamed
  // 14.9, both 15.1; 66 MB 26.5, 26.9, 27.2; 82 MB 36.1, 31.8, 34.4; 98 MB 44.6, 36.8,
  // 41.5; 131 MB 56.2, 49.5, 49.3; 164 MB, both 63.9 and o 69.0.
  const size_t bytes = (size_t)T * k * nv * 16;
  const auto by_size = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (bytes >= kStream) launch(k_combine_grad<DT, true, true>);
    else if (2 * bytes >= kStream) launch(k_combine_grad<DT, true, false>);
    else launch(k_combine_grad<DT, false, false>);
  };
  if (dtype == MOE_T_F16) by_size(std::integral_constant<int, MOE_T_F16>{});
  else if (dtype == MOE_T_BF16) by_size(std::integral_constant<int, MOE_T_BF16>{});
  else by_size(std::integral_constant<int, MOE_T_F32>{});
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // extern "C"
