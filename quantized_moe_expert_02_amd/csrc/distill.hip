// Distillation from a teacher's top logits (include/moe_distill.h).
//
// The loss needs one pass over a row: every thread keeps the largest logit it has
// met and the sum of exp((z - that) / tau), which is rescaled when a larger one
// comes; the threads' pairs are joined at the end.  The gradient is a second pass
// (read, write).  Both are bound by memory.
#include <algorithm>

#include "mat.h"
#include "moe_distill.h"

namespace moe {

namespace {

constexpr int kMaxEntries = 1024;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

struct DistillArgs {
  const void* z;
  int64_t ldz;
  int T, V, k;
  const int32_t* ids;
  const float* teacher;
  float c;  // log2(e) / tau
  float rtau;
  int chunk, chunks;  // columns of a workgroup, workgroups per row
  float* loss;
  float* stats;
  float2* part;  // [T][chunks]
  const float* dloss;
  void* dz;
  int64_t lddz;
};

// A running maximum m (NaN from the first NaN on) and the sum s of 2^((z - m) c).
struct Run {
  float m, s;
};

__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.0f : m; }

// NaN where either is (fmaxf passes NaNs over).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ Run join(Run a, Run b, float c) {
  const float m = larger(a.m, b.m), f = finite_or_0(m);
  return Run{m, a.s * __builtin_amdgcn_exp2f((a.m - f) * c) + b.s * __builtin_amdgcn_exp2f((b.m - f) * c)};
}

template <int STEP>
__device__ __forceinline__ Run partner_run(Run r) {
  return Run{__builtin_bit_cast(float, partner<STEP>(__builtin_bit_cast(int, r.m))),
             __builtin_bit_cast(float, partner<STEP>(__builtin_bit_cast(int, r.s)))};
}

__device__ __forceinline__ Run wave_join(Run r, float c) {
  r = join(r, partner_run<1>(r), c);
  r = join(r, partner_run<2>(r), c);
  r = join(r, partner_run<4>(r), c);
  r = join(r, partner_run<8>(r), c);
  r = join(r, partner_run<16>(r), c);
  return join(r, partner_run<32>(r), c);
}

template <int N>
__device__ __forceinline__ void add_run(Run& r, const float (&z)[N], float c) {
  float m = r.m;
#pragma unroll
  for (int i = 0; i < N; ++i) m = larger(m, z[i]);
  if (m != r.m) {
    r.s *= __builtin_amdgcn_exp2f((r.m - m) * c);
    r.m = m;
  }
  const float f = finite_or_0(r.m);
#pragma unroll
  for (int i = 0; i < N; ++i) r.s += __builtin_amdgcn_exp2f((z[i] - f) * c);
}

// The columns [c0, c1) of a row as unaligned ends and 16-byte vectors between, kBatch of
// them on their way per thread (results may be written over the row: without batches
// every load would wait for the store before it).  The first batch is requested where the
// object is made, ahead of what else a workgroup has to read.
constexpr int kBatch = 4;
template <int DT, bool STREAM, int TH>
struct RowScan {
  typedef typename RowType<DT>::elem elem;
  static constexpr int VEC = kVec<DT>;
  const u32x4* p;
  int c0, c1, head, vectors, tail;
  u32x4 x[kBatch];
  __device__ __forceinline__ RowScan(const elem* row, int c0_, int c1_) : c0(c0_), c1(c1_) {
    const int shift = (int)((uintptr_t)(row + c0) % 16 / sizeof(elem));
    head = min(c1, c0 + (shift ? VEC - shift : 0));
    vectors = (c1 - head) / VEC;
    tail = head + vectors * VEC;
    p = (const u32x4*)(row + head);
    if (vectors) load((int)threadIdx.x);
  }
  __device__ __forceinline__ void load(int v) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const u32x4* q = p + min(v + u * TH, vectors - 1);
      x[u] = STREAM ? __builtin_nontemporal_load(q) : *q;
    }
  }
  // one(i) for single columns, many(i, v) for the VEC columns from i
  template <typename One, typename Many>
  __device__ __forceinline__ void run(One one, Many many) {
    for (int v = threadIdx.x; v < vectors; v += kBatch * TH) {
      if (v >= kBatch * TH) load(v);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (v + u * TH < vectors) many(head + (v + u * TH) * VEC, x[u]);
    }
    ends(one);
  }
  template <typename One>
  __device__ __forceinline__ void ends(One one) const {
    if ((int)threadIdx.x < head - c0) one(c0 + threadIdx.x);
    if ((int)threadIdx.x < c1 - tail) one(tail + threadIdx.x);
  }
};

// The teacher's probabilities of row t, by one wavefront: top and norm with p = 2^((a
// - top) c) / norm.  False if the row keeps no entry.
struct Teacher {
  float top, norm;
  bool any;
};

__device__ __forceinline__ bool kept(int id, int V) { return (uint32_t)id < (uint32_t)V; }

__device__ __forceinline__ Teacher teacher_of(const DistillArgs& a, int t) {
  const int lane = threadIdx.x & 63;
  const int32_t* ids = a.ids + (int64_t)t * a.k;
  const float* in = a.teacher + (int64_t)t * a.k;
  Teacher r{-INFINITY, 0.0f, false};
  for (int j = lane; j < a.k; j += 64)
    if (kept(ids[j], a.V)) {
      r.any |= in[j] != -INFINITY;
      r.top = fmaxf(r.top, in[j]);
    }
  r.any = __ballot(r.any) != 0;
  if (!r.any) return r;
  r.top = wave_max_f32(r.top);
  for (int j = lane; j < a.k; j += 64)
    if (kept(ids[j], a.V)) r.norm += __builtin_amdgcn_exp2f((in[j] - r.top) * a.c);
  r.norm = wave_sum_f32(r.norm);
  return r;
}

// Loss and statistics of a row whose run is known, by one wavefront.
template <int DT>
__device__ __forceinline__ void finish_row(const DistillArgs& a, int t, const Teacher& te, Run run) {
  const int lane = threadIdx.x & 63;
  const typename RowType<DT>::elem* z = (const typename RowType<DT>::elem*)a.z + (int64_t)t * a.ldz;
  const float l = run.m == -INFINITY ? NAN : logf(run.s), norm = logf(te.norm);
  float loss = 0.0f;
  for (int j = lane; j < a.k; j += 64) {
    const int id = a.ids[(int64_t)t * a.k + j];
    if (!kept(id, a.V)) continue;
    const float d = a.teacher[(int64_t)t * a.k + j] - te.top, p = __builtin_amdgcn_exp2f(d * a.c) / te.norm;
    if (p == 0.0f) continue;
    loss += p * ((d * a.rtau - norm) - (((float)z[id] - run.m) * a.rtau - l));
  }
  loss = wave_sum_f32(loss);
  if (lane == 0) {
    a.loss[t] = loss;
    a.stats[2 * (int64_t)t] = run.m;
    a.stats[2 * (int64_t)t + 1] = l;
  }
}

__device__ __forceinline__ void drop_row(const DistillArgs& a, int t) {
  if (threadIdx.x == 0) a.loss[t] = a.stats[2 * (int64_t)t] = a.stats[2 * (int64_t)t + 1] = 0.0f;
}

// A workgroup of TH threads per row, or (PART) per chunk of one.  Bound by memory: 2,048 rows of
// 128,000 bfloat16, a tenth of them padding, 82 us (473 MB, 5.8 TB/s).
template <int DT, bool PART, bool STREAM, int TH>
__global__ __launch_bounds__(TH) void k_distill(DistillArgs a) {
  typedef typename RowType<DT>::elem elem;
  constexpr int VEC = kVec<DT>, W = TH / 64;
  __shared__ Run runs[W];
  const int t = PART ? blockIdx.x / a.chunks : blockIdx.x, ch = PART ? blockIdx.x % a.chunks : 0;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const elem* z = (const elem*)a.z + (int64_t)t * a.ldz;
  const int c0 = PART ? ch * a.chunk : 0, c1 = PART ? min(a.V, c0 + a.chunk) : a.V;
  RowScan<DT, STREAM, TH> scan(z, c0, c1);
  const Teacher te = teacher_of(a, t);
  if (!te.any) {
    if (!PART) drop_row(a, t);
    return;
  }
  Run r{-INFINITY, 0.0f};
  scan.run(
      [&](int i) {
        const float v[1] = {(float)z[i]};
        add_run(r, v, a.c);
      },
      [&](int, u32x4 x) {
        float v[VEC];
        unpack_vec<DT>(x, v);
        add_run(r, v, a.c);
      });
  r = wave_join(r, a.c);
  if (W > 1) {
    if (lane == 0) runs[wave] = r;
    __syncthreads();
    if (wave) return;
    r = runs[0];
#pragma unroll
    for (int i = 1; i < W; ++i) r = join(r, runs[i], a.c);
  }
  if (PART) {
    if (lane == 0) a.part[(int64_t)t * a.chunks + ch] = make_float2(r.m, r.s);
  } else {
    finish_row<DT>(a, t, te, r);
  }
}

// Joins the chunks of a row: a wavefront per row (4 rows of 32 chunks 2.8 us, its launch and waits).
template <int DT>
__global__ __launch_bounds__(64) void k_distill_join(DistillArgs a) {
  const int t = blockIdx.x, lane = threadIdx.x;
  const Teacher te = teacher_of(a, t);
  if (!te.any) return drop_row(a, t);
  Run r{-INFINITY, 0.0f};
  for (int i = lane; i < a.chunks; i += 64) {
    const float2 p = a.part[(int64_t)t * a.chunks + i];
    r = join(r, Run{p.x, p.y}, a.c);
  }
  finish_row<DT>(a, t, te, wave_join(r, a.c));
}

// The gradient of a chunk of a row.  The teacher's entries in the chunk are written
// after the others, each id once with the sum of its probabilities; their logits are
// read before anything is written, so that dz may be z.  Bound by memory: the 2,048 rows above
// 186 us (997 MB, 5.4 TB/s, what a copy reaches).
struct Entry {
  int id;   // -1: not in the chunk
  float p, z, sum;  // sum: of p over the entries of the same id; < 0 but for the first of them
};

template <int DT, bool STREAM, int TH>
__global__ __launch_bounds__(TH) void k_distill_grad(DistillArgs a) {
  typedef typename RowType<DT>::elem elem;
  constexpr int VEC = kVec<DT>;
  extern __shared__ Entry entry[];
  const int t = blockIdx.x / a.chunks, ch = blockIdx.x % a.chunks;
  const elem* z = (const elem*)a.z + (int64_t)t * a.ldz;
  elem* dz = (elem*)a.dz + (int64_t)t * a.lddz;
  const int c0 = ch * a.chunk, c1 = min(a.V, c0 + a.chunk);
  RowScan<DT, STREAM, TH> scan(z, c0, c1);
  const float m = a.stats[2 * (int64_t)t], l2 = a.stats[2 * (int64_t)t + 1] * kLog2e, w = a.dloss[t] * a.rtau;
  const Teacher te = teacher_of(a, t);
  const bool same = (uintptr_t)z % 16 == (uintptr_t)dz % 16;
  const auto put = [&](int i, const float (&v)[VEC]) {
    if (same) {
      const u32x4 o = pack_vec<DT>(v);
      if (STREAM) __builtin_nontemporal_store(o, (u32x4*)(dz + i));
      else *(u32x4*)(dz + i) = o;
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) dz[i + e] = (elem)v[e];
    }
  };
  if (!te.any) {
    const float zero[VEC] = {};
    for (int v = threadIdx.x; v < scan.vectors; v += TH) put(scan.head + v * VEC, zero);
    scan.ends([&](int i) { dz[i] = (elem)0.0f; });
    return;
  }
  const auto q = [&](float v) { return __builtin_amdgcn_exp2f(fmaf(v - m, a.c, -l2)); };
  // A product that is rounded to fp32 before it is to the rows' type, in every form of
  // the loop (the compiler may fuse the two), so that alignment does not show.
  const auto weighted = [&](float v) {
    float p = v * w;
    asm("" : "+v"(p));
    return p;
  };
  for (int j = threadIdx.x; j < a.k; j += TH) {
    const int id = a.ids[(int64_t)t * a.k + j];
    const bool here = id >= c0 && id < c1;
    Entry e{-1, 0.0f, 0.0f, -1.0f};
    if (here) {
      const float p = __builtin_amdgcn_exp2f((a.teacher[(int64_t)t * a.k + j] - te.top) * a.c) / te.norm;
      e = Entry{id, p, (float)z[id], -1.0f};
    }
    entry[j] = e;
  }
  __syncthreads();
  for (int j = threadIdx.x; j < a.k; j += TH) {
    const int id = entry[j].id;
    if (id < 0) continue;
    bool first = true;
    float sum = 0.0f;
#pragma unroll 4
    for (int i = 0; i < a.k; ++i) {
      const bool eq = entry[i].id == id;
      first &= !eq || i >= j;
      sum += eq ? entry[i].p : 0.0f;
    }
    if (first) entry[j].sum = sum;
  }
  scan.run([&](int i) { dz[i] = (elem)weighted(q((float)z[i])); },
           [&](int i, u32x4 x) {
             float v[VEC];
             unpack_vec<DT>(x, v);
#pragma unroll
             for (int e = 0; e < VEC; ++e) v[e] = weighted(q(v[e]));
             put(i, v);
           });
  __syncthreads();
  for (int j = threadIdx.x; j < a.k; j += TH) {
    const Entry e = entry[j];
    if (e.id >= 0 && !(e.sum < 0.0f)) dz[e.id] = (elem)weighted(q(e.z) - e.sum);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// Rows of up to 16 KB take a wavefront each (4,096 rows of 8,000 bfloat16 logits: 64
// threads 17.5 us, 512 25.6; gradient 41.5 and 48.2; of 16,000: 31.8 and 33.8, gradient 74
// and 65).
constexpr int64_t kShortRow = 16 << 10;
// Longer ones 512 threads, and where that makes too few workgroups, chunks of 16 to 64 KB,
// about 512 in all (loss of 64 rows of 128,000 bfloat16 logits: whole rows 14.1 us, 64 KB 9.9,
// 32 KB 10.4; 301 rows of 100,003 binary16: 22.1 and 20.9 (so whole from 256 rows); 4
// rows of 128,000 fp32: 13.9, 16 KB 6.3).  Up to 64 Ki columns the loss takes whole rows too, which
// is one launch instead of two and hardly longer on the GPU (whole and in chunks, us: 4 rows of
// 32,000 bfloat16 logits 5.3 and 6.5, 128 rows 5.8 and 7.9; of 64,000 7.4 and 6.6, 9.0 and
// 10.0; 4 rows of 64,000 fp32 8.5 and 6.2).  The gradient, which joins nothing, always takes
// chunks (2,048 rows of 128,000 bfloat16: whole rows 203, 64 KB 190).
constexpr int kWholeRows = 256, kWholeColumns = 64 << 10;

int chunk_of(int T, int V, int dtype, bool grad) {
  const int64_t b = (int64_t)elem_bytes(dtype), share = (int64_t)T * V * b / 512;
  const int64_t bytes = std::min<int64_t>(std::max<int64_t>(share, 16 << 10), 64 << 10);
  if (V * b <= kShortRow || (!grad && (T >= kWholeRows || V <= kWholeColumns))) return V;
  const int chunks = ceil_div(V * b, bytes);
  return std::min(V, ceil_div(ceil_div(V, chunks), 8) * 8);
}

// Logits too large for the last-level cache to keep are read and written past the caches
// (2,048 rows of 128,000 bfloat16: 94.4 us plainly, 85.7 streamed, gradient 208 and 190;
// 512 rows 29.3 and 25.9, gradient 57.7 and 51.6).
constexpr int64_t kStream = (int64_t)112 << 20;
bool streamed(int T, int V, int dtype) { return (int64_t)T * V * (int64_t)elem_bytes(dtype) >= kStream; }

int check_shape(int32_t T, int32_t V, int32_t dtype) {
  if (T < 0 || V < 1 || dtype < MOE_T_F16 || dtype > MOE_T_F32) return MOE_E_INVAL;
  return T > kMaxRows || V > (1 << 24) ? MOE_E_UNSUPPORTED : MOE_OK;
}

int check_distill(const void* z, int32_t dtype, int64_t ldz, int32_t T, int32_t V, const int32_t* ids,
                  const float* teacher, int32_t k, float tau) {
  const int st = check_shape(T, V, dtype);
  if (st != MOE_OK) return st;
  if (k < 1 || !(tau > 0.0f && tau < INFINITY) || ldz < V) return MOE_E_INVAL;
  if (tau < 0x1p-64f || tau > 0x1p64f) return MOE_E_UNSUPPORTED;
  if (k > kMaxEntries || ldz > (int64_t)1 << 36 || (int64_t)T * ldz > (int64_t)1 << 36) return MOE_E_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  return bad(z, (unsigned)elem_bytes(dtype)) || bad(ids, 4) || bad(teacher, 4) ? MOE_E_INVAL : MOE_OK;
}

template <typename F>
void by_type(int dtype, F f) {
  if (dtype == MOE_T_F16) f(Const<MOE_T_F16>{});
  else if (dtype == MOE_T_BF16) f(Const<MOE_T_BF16>{});
  else f(Const<MOE_T_F32>{});
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_distill_workspace_bytes(int32_t T, int32_t V, int32_t dtype) {
  if (check_shape(T, V, dtype) != MOE_OK || T == 0) return 0;
  const int chunks = ceil_div(V, chunk_of(T, V, dtype, false));
  return chunks > 1 ? (size_t)T * chunks * sizeof(float2) : 0;
}

int moe_distill_forward(const void* z, int32_t dtype, int64_t ldz, int32_t T, int32_t V, const int32_t* ids,
                        const float* teacher, int32_t k, float tau, float* loss, float* stats, void* ws,
                        size_t ws_bytes, void* stream) {
  const int st = check_distill(z, dtype, ldz, T, V, ids, teacher, k, tau);
  if (st != MOE_OK || T == 0) return st;
  if (bad(loss, 4) || bad(stats, 4)) return MOE_E_INVAL;
  const int chunk = chunk_of(T, V, dtype, false), chunks = ceil_div(V, chunk);
  if (chunks > 1 && bad(ws, 16)) return MOE_E_INVAL;
  if (ws_bytes < moe_distill_workspace_bytes(T, V, dtype)) return MOE_E_WORKSPACE;
  const hipStream_t s = (hipStream_t)stream;
  const DistillArgs a{z, ldz, T, V, k, ids, teacher, kLog2e / tau, 1.0f / tau, chunk, chunks, loss, stats,
                      (float2*)ws, nullptr, nullptr, 0};
  by_type(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (chunks == 1) {
      if (V * (int64_t)elem_bytes(dtype) <= kShortRow) k_distill<DT, false, false, 64><<<T, 64, 0, s>>>(a);
      else if (streamed(T, V, dtype)) k_distill<DT, false, true, 512><<<T, 512, 0, s>>>(a);
      else k_distill<DT, false, false, 512><<<T, 512, 0, s>>>(a);
    } else {
      k_distill<DT, true, false, 512><<<T * chunks, 512, 0, s>>>(a);
      k_distill_join<DT><<<T, 64, 0, s>>>(a);
    }
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

int moe_distill_backward(const void* z, int32_t dtype, int64_t ldz, int32_t T, int32_t V, const int32_t* ids,
                         const float* teacher, int32_t k, float tau, const float* stats, const float* dloss,
                         void* dz, int64_t lddz, void* stream) {
  const int st = check_distill(z, dtype, ldz, T, V, ids, teacher, k, tau);
  if (st != MOE_OK) return st;
  if (lddz < V || (dz == z && lddz != ldz)) return MOE_E_INVAL;
  if (lddz > (int64_t)1 << 36 || (int64_t)T * lddz > (int64_t)1 << 36) return MOE_E_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (bad(stats, 4) || bad(dloss, 4) || bad(dz, (unsigned)elem_bytes(dtype))) return MOE_E_INVAL;
  // (other workgroups may have written what one has yet to read)
  if (dz != z && rows_overlap(z, ldz, V, dz, lddz, V, T, (int64_t)elem_bytes(dtype))) return MOE_E_INVAL;
  const int chunk = chunk_of(T, V, dtype, true), chunks = ceil_div(V, chunk);
  const hipStream_t s = (hipStream_t)stream;
  const DistillArgs a{z, ldz, T, V, k, ids, teacher, kLog2e / tau, 1.0f / tau, chunk, chunks, nullptr,
                      (float*)stats, nullptr, dloss, dz, lddz};
  by_type(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const size_t lds = k * sizeof(Entry);
    if (V * (int64_t)elem_bytes(dtype) <= kShortRow) k_distill_grad<DT, false, 64><<<T * chunks, 64, lds, s>>>(a);
    else if (streamed(T, V, dtype)) k_distill_grad<DT, true, 512><<<T * chunks, 512, lds, s>>>(a);
    else k_distill_grad<DT, false, 512><<<T * chunks, 512, lds, s>>>(a);
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // extern "C"
