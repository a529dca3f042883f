// Low-rank adapters of many requests beside a shared projection
// (include/moe_adapter.h).
#include <algorithm>

#include "rows.h"

namespace moe {

namespace {

struct AdapterArgs {
  const void *a, *b;
  const float* scale;
  const int32_t* ranks;
  int n, K, N, R;
};

__device__ __forceinline__ int rank_of(const AdapterArgs& d, int a) {
  return d.ranks ? min(max(d.ranks[a], 0), d.R) : d.R;
}

// u[t][r] = <A_a[r], x[t]>; a wavefront per (t, r).
template <int DT>
__global__ __launch_bounds__(64) void k_shrink(AdapterArgs d, const void* x, int64_t ldx, const int32_t* ids,
                                               float* u) {
  typedef typename RowType<DT>::elem E;
  const int t = blockIdx.x, r = blockIdx.y, a = ids[t];
  float s = 0.0f;
  if ((unsigned)a < (unsigned)d.n && r < rank_of(d, a)) {
    const E* A = (const E*)d.a + ((size_t)a * d.R + r) * d.K;
    const E* xt = (const E*)x + (size_t)t * ldx;
    for (int k = threadIdx.x; k < d.K; k += 64) s = fmaf((float)A[k], (float)xt[k], s);
  }
  s = wave_sum_f32(s);
  if (threadIdx.x == 0) u[(size_t)t * d.R + r] = s;
}

// v[t][r] = s_a sum_n dy[t][n] B_a[n][r]; a wavefront per (t, r).
template <int DT>
__global__ __launch_bounds__(64) void k_shrink_dy(AdapterArgs d, const void* dy, int64_t ld, const int32_t* ids,
                                                  float* v) {
  typedef typename RowType<DT>::elem E;
  const int t = blockIdx.x, r = blockIdx.y, a = ids[t];
  float s = 0.0f;
  if ((unsigned)a < (unsigned)d.n && r < rank_of(d, a)) {
    const E* B = (const E*)d.b + (size_t)a * d.N * d.R + r;
    const E* g = (const E*)dy + (size_t)t * ld;
    for (int n = threadIdx.x; n < d.N; n += 64) s = fmaf((float)B[(size_t)n * d.R], (float)g[n], s);
    s *= d.scale[a];
  }
  s = wave_sum_f32(s);
  if (threadIdx.x == 0) v[(size_t)t * d.R + r] = s;
}

// out[t][c] = add[t][c] + f * sum_r m(r, c) u[t][r]: the forward expansion
// (m = B_a[c][r], f = s_a) and the input's gradient (TR: m = A_a[r][c], f = 1).
template <int DT, bool TR>
__global__ __launch_bounds__(256) void k_expand(AdapterArgs d, const float* u, const int32_t* ids, const void* add,
                                                int64_t ldadd, void* out, int64_t ldo) {
  typedef typename RowType<DT>::elem E;
  const int t = blockIdx.x, c = blockIdx.y * 256 + threadIdx.x, a = ids[t];
  const int C = TR ? d.K : d.N;
  if (c >= C) return;
  float s = 0.0f;
  if ((unsigned)a < (unsigned)d.n) {
    const int rk = rank_of(d, a);
    for (int r = 0; r < rk; ++r) {
      const E m = TR ? ((const E*)d.a)[((size_t)a * d.R + r) * d.K + c] : ((const E*)d.b)[((size_t)a * d.N + c) * d.R + r];
      s = fmaf((float)m, u[(size_t)t * d.R + r], s);
    }
    if (!TR) s *= d.scale[a];
  }
  if (add) s += (float)((const E*)add)[(size_t)t * ldadd + c];
  ((E*)out)[(size_t)t * ldo + c] = (E)s;
}

// Weight gradients: dA_a[r][k] = sum_t v[t][r] x[t][k] (TR == false, out
// [R][C]) and dB_a[n][r] = s_a sum_t u[t][r] dy[t][n] (TR, out [C][R]).
template <int DT, bool TR>
__global__ __launch_bounds__(256) void k_outer(AdapterArgs d, const float* v, const void* x, int64_t ldx, int T,
                                               const int32_t* offsets, const int32_t* pairs, float* out) {
  typedef typename RowType<DT>::elem E;
  const int a = blockIdx.x, r = blockIdx.y, c = blockIdx.z * 256 + threadIdx.x;
  const int C = TR ? d.N : d.K;
  if (c >= C) return;
  float s = 0.0f;
  if (r < rank_of(d, a)) {
    const int i1 = min(T, offsets[a + 1]);
    for (int i = max(0, offsets[a]); i < i1; ++i) {
      const int t = pairs[i];
      if ((unsigned)t < (unsigned)T) s = fmaf(v[(size_t)t * d.R + r], (float)((const E*)x)[(size_t)t * ldx + c], s);
    }
    if (TR) s *= d.scale[a];
  }
  out[TR ? ((size_t)a * C + c) * d.R + r : ((size_t)a * d.R + r) * C + c] = s;
}

inline bool bad(const void* p, unsigned align) { return !p || !aligned_to(p, align); }
inline bool bad_ld(int64_t ld, int width) { return ld < width || ld % 8; }

int check_adapters(const moe_adapters_t* d, int32_t T) {
  if (!d || T < 0 || d->n < 1 || d->K <= 0 || d->N <= 0 || d->R <= 0) return MOE_E_INVAL;
  if (d->dtype != MOE_T_F16 && d->dtype != MOE_T_BF16) return MOE_E_INVAL;
  if (d->K % 8 || d->N % 8 || d->R % 8 || d->R > 128 || d->n > kMaxExperts || T > kMaxSlots) return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

int check_adapter_ptrs(const moe_adapters_t* d) {
  if (bad(d->a, 16) || bad(d->b, 16) || bad(d->scale, 4) || (d->ranks && !aligned_to(d->ranks, 4))) return MOE_E_INVAL;
  return MOE_OK;
}

// Workspace: u or v [T][R] fp32, then the rows' order when the call makes it
// (offsets, pairs, pos, the sort's scratch).
struct AdapterPlan {
  size_t u, offsets, pairs, pos, sort, total;
};
AdapterPlan adapter_plan(const moe_adapters_t& d, int T) {
  AdapterPlan p{};
  size_t o = 0;
  p.u = o; o += round256((size_t)T * d.R * 4);
  p.offsets = o; o += round256((size_t)(d.n + 1) * 4);
  p.pairs = o; o += round256((size_t)T * 4);
  p.pos = o; o += round256((size_t)T * 4);
  p.sort = o; o += moe_sort_workspace_bytes(T, 1, d.n);
  p.total = o;
  return p;
}

template <typename F16, typename BF16>
int by_type(int dtype, F16 f16, BF16 bf16) {
  if (dtype == MOE_T_F16) f16();
  else bf16();
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
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
  float* uu = u ? u : (float*)((char*)ws + p.u);
  const auto run = [&](auto shrink, auto expand) {
    shrink<<<dim3(T, g.R), 64, 0, s>>>(g, x, ldx, ids, uu);
    expand<<<dim3(T, (g.N + 255) / 256), 256, 0, s>>>(g, uu, ids, add, ldadd, y, ldy);
  };
  return by_type(
      d->dtype, [&] { run(k_shrink<MOE_T_F16>, k_expand<MOE_T_F16, false>); },
      [&] { run(k_shrink<MOE_T_BF16>, k_expand<MOE_T_BF16, false>); });
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
  float* v = (float*)(w + p.u);
  if (!offsets) {
    int32_t *o = (int32_t*)(w + p.offsets), *q = (int32_t*)(w + p.pairs);
    if (launch_sort(ids, T, 1, d->n, 1, T, o, q, (int32_t*)(w + p.pos), w + p.sort, s) != hipSuccess) return MOE_E_HIP;
    offsets = o;
    pairs = q;
  }
  const auto run = [&](auto shrink, auto expand, auto grad_a, auto grad_b) {
    if (T) shrink<<<dim3(T, g.R), 64, 0, s>>>(g, dy, lddy, ids, v);
    if (T && dx) expand<<<dim3(T, (g.K + 255) / 256), 256, 0, s>>>(g, v, ids, add, ldadd, dx, lddx);
    grad_a<<<dim3(g.n, g.R, (g.K + 255) / 256), 256, 0, s>>>(g, v, x, ldx, T, offsets, pairs, d_a);
    grad_b<<<dim3(g.n, g.R, (g.N + 255) / 256), 256, 0, s>>>(g, u, dy, lddy, T, offsets, pairs, d_b);
  };
  return by_type(
      d->dtype,
      [&] { run(k_shrink_dy<MOE_T_F16>, k_expand<MOE_T_F16, true>, k_outer<MOE_T_F16, false>, k_outer<MOE_T_F16, true>); },
      [&] {
        run(k_shrink_dy<MOE_T_BF16>, k_expand<MOE_T_BF16, true>, k_outer<MOE_T_BF16, false>, k_outer<MOE_T_BF16, true>);
      });
}

}  // extern "C"
