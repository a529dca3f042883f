// Gradient of the router's renormalised sigmoid weights (include/moe_dispatch.h).
#include <algorithm>

#include "rows.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// One workgroup per token: z_j of the kept slots (a wavefront per slot), the
// slots' dz, and dx = add + sum_j dz_j Wr[e_j].
//   w_j = s_j / S, so with m = sum_i dw_i w_i:  dz_j = w_j (1 - s_j) (dw_j - m).
template <int DT>
__global__ __launch_bounds__(kThreads) void k_route_grad_tokens(const u32x4* x, int nv, int E, int k,
                                                                const float* wr, const float* br,
                                                                const int32_t* idx, const float* dw,
                                                                const u32x4* add, u32x4* dx, float* dz_out) {
  __shared__ float z[kMaxTopK], dz[kMaxTopK];
  __shared__ int ex[kMaxTopK];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const u32x4* xt = x + (size_t)t * nv;
  for (int j = wave; j < k; j += kWaves) {
    const int e = idx[(size_t)t * k + j];
    const bool ok = (unsigned)e < (unsigned)E;
    float s = 0.0f;
    if (ok)
      for (int i = lane; i < nv; i += 64) {
        float f[8];
        unpack_vec<DT>(xt[i], f);
        const f32x4* r = (const f32x4*)(wr + ((size_t)e * nv + i) * 8);
        const f32x4 a = r[0], b = r[1];
#pragma unroll
        for (int c = 0; c < 4; ++c) s = fmaf(f[c], a[c], s);
#pragma unroll
        for (int c = 0; c < 4; ++c) s = fmaf(f[4 + c], b[c], s);
      }
    s = wave_sum_f32(s);
    if (lane == 0) {
      ex[j] = ok ? e : -1;
      z[j] = ok ? s + (br ? br[e] : 0.0f) : 0.0f;
    }
  }
  __syncthreads();
  if (wave == 0) {
    const bool ok = lane < k && ex[lane] >= 0;
    const float zj = ok ? z[lane] : 0.0f;
    const float s = ok ? 1.0f / (1.0f + expf(-zj)) : 0.0f;
    const float S = wave_sum_f32(s);
    const float w = ok ? s / S : 0.0f;
    const float g = ok ? dw[(size_t)t * k + lane] : 0.0f;
    const float m = wave_sum_f32(g * w);
    const float d = ok ? w * (1.0f / (1.0f + expf(zj))) * (g - m) : 0.0f;
    if (lane < k) {
      dz[lane] = d;
      dz_out[(size_t)t * k + lane] = d;
    }
  }
  __syncthreads();
  for (int i = tid; i < nv; i += kThreads) {
    float acc[8] = {};
    if (add) unpack_vec<DT>(add[(size_t)t * nv + i], acc);
    for (int j = 0; j < k; ++j) {
      if (ex[j] < 0) continue;
      const f32x4* r = (const f32x4*)(wr + ((size_t)ex[j] * nv + i) * 8);
      const f32x4 a = r[0], b = r[1];
      const float d = dz[j];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[c] = fmaf(d, a[c], acc[c]);
        acc[4 + c] = fmaf(d, b[c], acc[4 + c]);
      }
    }
    dx[(size_t)t * nv + i] = pack_vec<DT>(acc);
  }
}

// dWr[e] = sum over the expert's rows of dz x[t]; a thread per 8 columns.
template <int DT>
__global__ __launch_bounds__(64) void k_route_grad_weights(const u32x4* x, int nv, int k, const float* dz,
                                                           const int32_t* offsets, const int32_t* pairs, int rows,
                                                           int n, float* dwr, float* db) {
  const int e = blockIdx.x, i = blockIdx.y * 64 + threadIdx.x;
  const int r0 = max(0, offsets[e]), r1 = min(rows, offsets[e + 1]);
  float acc[8] = {}, sum = 0.0f;
  for (int r = r0; r < r1; ++r) {
    const int p = pairs[r];
    if ((unsigned)p >= (unsigned)n) continue;
    const float d = dz[p];
    sum += d;
    if (i < nv) {
      float f[8];
      unpack_vec<DT>(x[(size_t)(p / k) * nv + i], f);
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] = fmaf(d, f[c], acc[c]);
    }
  }
  if (i < nv) {
    f32x4* o = (f32x4*)(dwr + ((size_t)e * nv + i) * 8);
    o[0] = f32x4{acc[0], acc[1], acc[2], acc[3]};
    o[1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
  }
  if (i == 0) db[e] = sum;
}

inline bool bad(const void* p, unsigned align) { return !p || !aligned_to(p, align); }

int check_shape(int32_t T, int32_t k, int32_t E, int32_t H, int32_t rows) {
  const int st = check_sort_shape(T, k, E, 1);
  if (st != MOE_OK) return st;
  if (H <= 0 || rows < 0) return MOE_E_INVAL;
  return H % 8 || H > kMaxWidth ? MOE_E_UNSUPPORTED : MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_route_backward_workspace_bytes(int32_t T, int32_t k, int32_t n_experts, int32_t H, int32_t rows) {
  if (check_shape(T, k, n_experts, H, rows) != MOE_OK) return 0;
  return round256(std::max<size_t>(1, (size_t)T * k * 4));
}

int moe_route_backward(const void* x, int32_t dtype, int32_t T, int32_t H, int32_t n_experts, int32_t k,
                       const float* router_w, const float* router_b, const int32_t* topk_idx, const float* dw,
                       const int32_t* offsets, const int32_t* pairs, int32_t rows, const void* add, void* dx,
                       float* d_router_w, float* d_router_b, void* ws, size_t ws_bytes, void* stream) {
  if (dtype != MOE_T_F16 && dtype != MOE_T_BF16) return MOE_E_INVAL;
  const int st = check_shape(T, k, n_experts, H, rows);
  if (st != MOE_OK) return st;
  if (bad(router_w, 16) || (router_b && !aligned_to(router_b, 4)) || bad(d_router_w, 16) || bad(d_router_b, 4) ||
      bad(offsets, 4) || bad(ws, 16) || (rows && bad(pairs, 4)))
    return MOE_E_INVAL;
  if (T && (bad(x, 16) || bad(dx, 16) || (add && !aligned_to(add, 16)) || bad(topk_idx, 4) || bad(dw, 4)))
    return MOE_E_INVAL;
  if (ws_bytes < moe_route_backward_workspace_bytes(T, k, n_experts, H, rows)) return MOE_E_WORKSPACE;
  const int nv = H / 8, E = n_experts;
  float* dz = (float*)ws;
  const hipStream_t s = (hipStream_t)stream;
  const auto launch = [&](auto tokens, auto weights) {
    if (T) {
      tokens<<<T, kThreads, 0, s>>>((const u32x4*)x, nv, E, k, router_w, router_b, topk_idx, dw, (const u32x4*)add,
                                    (u32x4*)dx, dz);
      if (hipGetLastError() != hipSuccess) return MOE_E_HIP;
    }
    weights<<<dim3(E, (nv + 63) / 64), 64, 0, s>>>((const u32x4*)x, nv, k, dz, offsets, pairs, rows, T * k, d_router_w,
                                                  d_router_b);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
  };
  if (dtype == MOE_T_F16) return launch(k_route_grad_tokens<MOE_T_F16>, k_route_grad_weights<MOE_T_F16>);
  return launch(k_route_grad_tokens<MOE_T_BF16>, k_route_grad_weights<MOE_T_BF16>);
}

}  // extern "C"
