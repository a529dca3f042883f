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

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
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

// A running maximum m and the sum s of 2^((z - m) c).
struct Run {
  float m, s;
};

__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ Run join(Run a, Run b, float c) {
  const float m = fmaxf(a.m, b.m), f = finite_or_0(m);
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
  float m = z[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, z[i]);
  if (m > r.m) {
    r.s *= __builtin_amdgcn_exp2f((r.m - m) * c);
    r.m = m;
  }
  const float f = finite_or_0(r.m);
#pragma unroll
  for (int i = 0; i < N; ++i) r.s += __builtin_amdgcn_exp2f((z[i] - f) * c);
}

// The columns [c0, c1) of a row as unaligned ends and 16-byte vectors between:
// one(i) for single columns, many(i) for kVec columns from i.
template <int DT, typename One, typename Many>
__device__ __forceinline__ void over_row(const typename RowType<DT>::elem* row, int c0, int c1, One one, Many many) {
  constexpr int VEC = kVec<DT>;
  const int shift = (int)((uintptr_t)(row + c0) % 16 / sizeof(typename RowType<DT>::elem));
  const int head = min(c1, c0 + (shift ? VEC - shift : 0)), vectors = (c1 - head) / VEC, tail = head + vectors * VEC;
  if ((int)threadIdx.x < head - c0) one(c0 + threadIdx.x);
  for (int v = threadIdx.x; v < vectors; v += kThreads) many(head + v * VEC);
  if ((int)threadIdx.x < c1 - tail) one(tail + threadIdx.x);
}

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

// One workgroup per row, or (PART) per chunk of one.
template <int DT, bool PART>
__global__ __launch_bounds__(kThreads) void k_distill(DistillArgs a) {
  typedef typename RowType<DT>::elem elem;
  constexpr int VEC = kVec<DT>;
  __shared__ Run runs[kWaves];
  const int t = PART ? blockIdx.x / a.chunks : blockIdx.x, ch = PART ? blockIdx.x % a.chunks : 0;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const Teacher te = teacher_of(a, t);
  if (!te.any) {
    if (!PART) drop_row(a, t);
    return;
  }
  const elem* z = (const elem*)a.z + (int64_t)t * a.ldz;
  const int c0 = PART ? ch * a.chunk : 0, c1 = PART ? min(a.V, c0 + a.chunk) : a.V;
  Run r{-INFINITY, 0.0f};
  over_row<DT>(
      z, c0, c1,
      [&](int i) {
        const float v[1] = {(float)z[i]};
        add_run(r, v, a.c);
      },
      [&](int i) {
        float v[VEC];
        unpack_vec<DT>(*(const u32x4*)(z + i), v);
        add_run(r, v, a.c);
      });
  r = wave_join(r, a.c);
  if (lane == 0) runs[wave] = r;
  __syncthreads();
  if (wave) return;
  r = runs[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) r = join(r, runs[i], a.c);
  if (PART) {
    if (lane == 0) a.part[(int64_t)t * a.chunks + ch] = make_float2(r.m, r.s);
  } else {
    finish_row<DT>(a, t, te, r);
  }
}

// Joins the chunks of a row: a wavefront per row.
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
// read before anything is written, so that dz may be z.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_distill_grad(DistillArgs a) {
  typedef typename RowType<DT>::elem elem;
  constexpr int VEC = kVec<DT>;
  __shared__ int s_id[kMaxEntries];
  __shared__ float s_p[kMaxEntries];
  const int t = blockIdx.x / a.chunks, ch = blockIdx.x % a.chunks;
  const elem* z = (const elem*)a.z + (int64_t)t * a.ldz;
  elem* dz = (elem*)a.dz + (int64_t)t * a.lddz;
  const int c0 = ch * a.chunk, c1 = min(a.V, c0 + a.chunk);
  const Teacher te = teacher_of(a, t);
  const float m = a.stats[2 * (int64_t)t], l2 = a.stats[2 * (int64_t)t + 1] * kLog2e, w = a.dloss[t] * a.rtau;
  const auto q = [&](float v) { return __builtin_amdgcn_exp2f(fmaf(v - m, a.c, -l2)); };
  // A product that is rounded to fp32 before it is to the rows' type, in every form of
  // the loop (the compiler may fuse the two), so that alignment does not show.
  const auto weighted = [&](float v) {
    float p = v * w;
    asm("" : "+v"(p));
    return p;
  };
  constexpr int PER = kMaxEntries / kThreads;
  float own[PER], sum[PER];
  bool first[PER];
  if (te.any) {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int j = threadIdx.x + u * kThreads;
      if (j < a.k) {
        const int id = a.ids[(int64_t)t * a.k + j];
        const bool here = id >= c0 && id < c1;
        s_id[j] = here ? id : -1;
        s_p[j] = here ? __builtin_amdgcn_exp2f((a.teacher[(int64_t)t * a.k + j] - te.top) * a.c) / te.norm : 0.0f;
        own[u] = here ? (float)z[id] : 0.0f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int j = threadIdx.x + u * kThreads;
      first[u] = j < a.k && s_id[j] >= 0;
      sum[u] = 0.0f;
      if (first[u])
        for (int i = 0; i < a.k; ++i)
          if (s_id[i] == s_id[j]) {
            first[u] &= i >= j;
            sum[u] += s_p[i];
          }
    }
  }
  const bool same = (uintptr_t)z % 16 == (uintptr_t)dz % 16;
  over_row<DT>(
      z, c0, c1, [&](int i) { dz[i] = (elem)(te.any ? weighted(q((float)z[i])) : 0.0f); },
      [&](int i) {
        float v[VEC];
        if (te.any) {
          unpack_vec<DT>(*(const u32x4*)(z + i), v);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[e] = weighted(q(v[e]));
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[e] = 0.0f;
        }
        if (same) {
          *(u32x4*)(dz + i) = pack_vec<DT>(v);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) dz[i + e] = (elem)v[e];
        }
      });
  if (!te.any) return;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u)
    if (first[u]) dz[s_id[threadIdx.x + u * kThreads]] = (elem)weighted(q(own[u]) - sum[u]);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr int kTargetBlocks = 1024;
constexpr int kMinChunk = 8192;

// Columns per workgroup: whole rows where there are many.
int chunk_of(int T, int V) {
  const int chunks = std::min(ceil_div(kTargetBlocks, T), ceil_div(V, kMinChunk));
  return T >= kTargetBlocks / 2 ? V : (ceil_div(V, std::max(chunks, 1)) + 7) / 8 * 8;
}

int check_shape(int32_t T, int32_t V, int32_t dtype) {
  if (T < 0 || V < 1 || dtype < MOE_T_F16 || dtype > MOE_T_F32) return MOE_E_INVAL;
  return T > kMaxRows || V > (1 << 24) ? MOE_E_UNSUPPORTED : MOE_OK;
}

int check_distill(const void* z, int32_t dtype, int64_t ldz, int32_t T, int32_t V, const int32_t* ids,
                  const float* teacher, int32_t k, float tau) {
  const int st = check_shape(T, V, dtype);
  if (st != MOE_OK) return st;
  if (k < 1 || !(tau > 0.0f && tau < INFINITY) || ldz < V) return MOE_E_INVAL;
  if (k > kMaxEntries || ldz > (int64_t)1 << 40 || (int64_t)T * ldz > (int64_t)1 << 40) return MOE_E_UNSUPPORTED;
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
  const int chunks = ceil_div(V, chunk_of(T, V));
  return chunks > 1 ? (size_t)T * chunks * sizeof(float2) : 0;
}

int moe_distill_forward(const void* z, int32_t dtype, int64_t ldz, int32_t T, int32_t V, const int32_t* ids,
                        const float* teacher, int32_t k, float tau, float* loss, float* stats, void* ws,
                        size_t ws_bytes, void* stream) {
  const int st = check_distill(z, dtype, ldz, T, V, ids, teacher, k, tau);
  if (st != MOE_OK || T == 0) return st;
  if (bad(loss, 4) || bad(stats, 4)) return MOE_E_INVAL;
  const int chunk = chunk_of(T, V), chunks = ceil_div(V, chunk);
  if (chunks > 1 && bad(ws, 16)) return MOE_E_INVAL;
  if (ws_bytes < moe_distill_workspace_bytes(T, V, dtype)) return MOE_E_WORKSPACE;
  const hipStream_t s = (hipStream_t)stream;
  const DistillArgs a{z, ldz, T, V, k, ids, teacher, kLog2e / tau, 1.0f / tau, chunk, chunks, loss, stats,
                      (float2*)ws, nullptr, nullptr, 0};
  by_type(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (chunks == 1) {
      k_distill<DT, false><<<T, kThreads, 0, s>>>(a);
    } else {
      k_distill<DT, true><<<T * chunks, kThreads, 0, s>>>(a);
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
  if (lddz > (int64_t)1 << 40 || (int64_t)T * lddz > (int64_t)1 << 40) return MOE_E_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (bad(stats, 4) || bad(dloss, 4) || bad(dz, (unsigned)elem_bytes(dtype))) return MOE_E_INVAL;
  const int chunk = chunk_of(T, V), chunks = ceil_div(V, chunk);
  const hipStream_t s = (hipStream_t)stream;
  const DistillArgs a{z, ldz, T, V, k, ids, teacher, kLog2e / tau, 1.0f / tau, chunk, chunks, nullptr,
                      (float*)stats, nullptr, dloss, dz, lddz};
  by_type(dtype, [&](auto dt) { k_distill_grad<decltype(dt)::value><<<T * chunks, kThreads, 0, s>>>(a); });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // extern "C"
