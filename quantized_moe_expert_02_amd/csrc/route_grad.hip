// Gradient of the router's renormalised sigmoid weights (include/moe_dispatch.h).
//
//   z_j = b[e_j] + <x, Wr[e_j]>, s_j = sigmoid(z_j), w_j = s_j / sum s, and with
//   m = sum_i dw_i w_i:  dz_j = w_j (1 - s_j) (dw_j - m)
//   dx = sum_j dz_j Wr[e_j];  dWr[e] = sum of dz x over e's slots
//
// The products touch k of E experts per token: T k H multiply-adds in each of
// the three steps, but as rows gathered from Wr they are T k H fp32 words (403
// MB for 2,048 tokens, top-8, 6144 wide) out of the 6 MB of Wr.  The two steps
// that gather Wr therefore run by column slice: a workgroup holds all experts'
// 64 (32 above 512 experts) columns in LDS and takes a range of tokens, so
// that Wr and x each cross the memory a few times only.
#include <algorithm>
#include <type_traits>

#include "rows.h"

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;

struct RouteArgs {
  const u32x4* x;
  const float* wr;
  const int32_t* idx;
  int T, H, E, k;
  uint32_t per_k;  // ceil(2^32 / k): p / k by multiplication (exact for p < 2^27, k <= 32), 0 for k = 1
};

__device__ __forceinline__ int token_of(const RouteArgs& a, int p) {
  return a.per_k ? (int)__umulhi((uint32_t)p, a.per_k) : p;
}

// All experts' columns [c0, c0 + CW) of Wr into LDS rows of CW + 4 floats;
// columns past H are zero.
template <int CW>
__device__ __forceinline__ void load_slice(const RouteArgs& a, int c0, float* w) {
  constexpr int V = CW / 4;
  for (int i = threadIdx.x; i < a.E * V; i += kThreads) {
    const int e = i / V, c = i % V * 4;
    f32x4 v = {0, 0, 0, 0};
    if (c0 + c < a.H) v = *(const f32x4*)(a.wr + (size_t)e * a.H + c0 + c);
    *(f32x4*)(w + e * (CW + 4) + c) = v;
  }
}

// Lanes that share a row of a slice, 8 columns each, and rows per wavefront.
template <int CW>
constexpr int kLanes = CW / 8;

// Partial logits [slices][T k]: a group of CW / 8 lanes per slot, 64 slots per
// turn of a wavefront.
template <int DT, int EC, int CW>
__global__ __launch_bounds__(kThreads) void k_route_dots(RouteArgs a, int range, float* zpart) {
  __shared__ __align__(16) float w[EC * (CW + 4)];  // E <= EC
  constexpr int L = kLanes<CW>, P = 64 / L;  // lanes per slot, slots per step
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane / L, cl = lane % L;
  const int c0 = blockIdx.x * CW, nv = a.H / 8, cv = min(c0 / 8 + cl, nv - 1);
  load_slice<CW>(a, c0, w);
  __syncthreads();
  const int n = a.T * a.k, p1 = min((int)(blockIdx.y + 1) * range * a.k, n);
  float* out = zpart + (size_t)blockIdx.x * n;
  for (int base = blockIdx.y * range * a.k + wave * 64; base < p1; base += kWaves * 64) {
    int e = a.idx[min(base + lane, n - 1)];
    if ((unsigned)e >= (unsigned)a.E) e = 0;  // dropped: the sum is not used
    u32x4 xv[L];
#pragma unroll
    for (int s = 0; s < L; ++s) xv[s] = a.x[(size_t)token_of(a, min(base + s * P + sub, n - 1)) * nv + cv];
    float mine = 0.0f;
#pragma unroll
    for (int s = 0; s < L; ++s) {
      const float* r = w + __shfl(e, s * P + sub) * (CW + 4) + cl * 8;
      const f32x4 lo = *(const f32x4*)r, hi = *(const f32x4*)(r + 4);
      if (c0 + CW > a.H && c0 / 8 + cl >= nv) xv[s] = u32x4{0, 0, 0, 0};  // past the last column
      float f[8];
      unpack_vec<DT>(xv[s], f);
      float z = 0.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) z = fmaf(f[c], lo[c], z);
#pragma unroll
      for (int c = 0; c < 4; ++c) z = fmaf(f[4 + c], hi[c], z);
      z += __builtin_bit_cast(float, partner<1>(__builtin_bit_cast(int, z)));
      z += __builtin_bit_cast(float, partner<2>(__builtin_bit_cast(int, z)));
      if (L == 8) z += __builtin_bit_cast(float, partner<4>(__builtin_bit_cast(int, z)));
      if (cl == s) mine = z;  // slot base + s P + sub
    }
    const int p = base + cl * P + sub;
    if (p < p1) out[p] = mine;
  }
}

// dz of every slot from the partial logits: 64 / k tokens per workgroup, four
// threads per slot over the slices.
constexpr int kSlotThreads = 256;
__global__ __launch_bounds__(kSlotThreads) void k_route_slots(RouteArgs a, int slices, const float* zpart, const float* br,
                                                             const float* dw, float* dz) {
  __shared__ float part[4][64], sg[64], gw[64];
  const int l = threadIdx.x & 63, q = threadIdx.x >> 6, n = a.T * a.k, per = 64 / a.k;
  const int p0 = blockIdx.x * per * a.k, np = min(per * a.k, n - p0), p = min(p0 + l, n - 1);
  float z = 0.0f;
  for (int s = slices * q / 4; s < slices * (q + 1) / 4; s += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = zpart[(size_t)min(s + i, slices - 1) * n + p];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s + i < slices * (q + 1) / 4) z += v[i];
  }
  part[q][l] = z;
  __syncthreads();
  if (q) return;
  const int e = a.idx[p];
  const bool ok = l < np && (unsigned)e < (unsigned)a.E;
  z = (part[0][l] + part[1][l]) + (part[2][l] + part[3][l]);
  if (ok && br) z += br[e];
  const float s = ok ? 1.0f / (1.0f + expf(-z)) : 0.0f, g = ok ? dw[p] : 0.0f;
  sg[l] = s;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);  // one wavefront from here on: LDS keeps its order
  const int first = l / a.k * a.k;
  float S = 0.0f;
  for (int j = 0; j < a.k; ++j) S += sg[min(first + j, 63)];
  const float w = ok ? s / S : 0.0f;
  gw[l] = g * w;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  float m = 0.0f;
  for (int j = 0; j < a.k; ++j) m += gw[min(first + j, 63)];
  if (l < np) dz[p] = ok ? w * (1.0f / (1.0f + expf(z))) * (g - m) : 0.0f;
}

// dx[t] = add[t] + sum_j dz_j Wr[e_j], 64 columns of 8 tokens (32 of 16) per
// turn of a wavefront.
template <int DT, int EC, int CW>
__global__ __launch_bounds__(kThreads) void k_route_dx(RouteArgs a, int range, const float* dz, const u32x4* add, u32x4* dx) {
  __shared__ __align__(16) float w[EC * (CW + 4)];  // E <= EC
  constexpr int L = kLanes<CW>, P = 64 / L;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane / L, cl = lane % L;
  const int c0 = blockIdx.x * CW, nv = a.H / 8, cv = c0 / 8 + cl;
  load_slice<CW>(a, c0, w);
  __syncthreads();
  const int n = a.T * a.k, t1 = min((int)(blockIdx.y + 1) * range, a.T);
  for (int base = blockIdx.y * range + wave * P; base < t1; base += kWaves * P) {
    const int t = base + sub, tt = min(t, a.T - 1), cc = min(cv, nv - 1);
    float acc[8] = {};
    if (add) unpack_vec<DT>(add[(size_t)tt * nv + cc], acc);
    for (int j0 = 0; j0 < a.k; j0 += L) {
      const int p = min(tt * a.k + j0 + cl, n - 1);
      int e = a.idx[p];
      float d = dz[p];
      if (j0 + cl >= a.k || (unsigned)e >= (unsigned)a.E) e = -1;
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const int ej = __shfl(e, sub * L + j);
        const float dj = __shfl(d, sub * L + j);
        const float* r = w + max(ej, 0) * (CW + 4) + cl * 8;
        const f32x4 lo = *(const f32x4*)r, hi = *(const f32x4*)(r + 4);
        if (ej >= 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            acc[c] = fmaf(dj, lo[c], acc[c]);
            acc[4 + c] = fmaf(dj, hi[c], acc[4 + c]);
          }
        }
      }
    }
    if (t < t1 && cv < nv) dx[(size_t)t * nv + cv] = pack_vec<DT>(acc);
  }
}

// The same three steps for few slots, whose rows of Wr are gathered directly:
// one workgroup per token.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_route_grad_tokens(RouteArgs a, const float* br, const float* dw, const u32x4* add,
                                                                u32x4* dx, float* dz_out) {
  __shared__ float z[kMaxTopK], dz[kMaxTopK];
  __shared__ int ex[kMaxTopK];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, k = a.k, nv = a.H / 8;
  const u32x4* xt = a.x + (size_t)t * nv;
  for (int j = wave; j < k; j += kWaves) {
    const int e = a.idx[(size_t)t * k + j];
    const bool ok = (unsigned)e < (unsigned)a.E;
    float s = 0.0f;
    if (ok)
      for (int i = lane; i < nv; i += 64) {
        float f[8];
        unpack_vec<DT>(xt[i], f);
        const f32x4* r = (const f32x4*)(a.wr + ((size_t)e * nv + i) * 8);
        const f32x4 lo = r[0], hi = r[1];
#pragma unroll
        for (int c = 0; c < 4; ++c) s = fmaf(f[c], lo[c], s);
#pragma unroll
        for (int c = 0; c < 4; ++c) s = fmaf(f[4 + c], hi[c], s);
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
      const f32x4* r = (const f32x4*)(a.wr + ((size_t)ex[j] * nv + i) * 8);
      const f32x4 lo = r[0], hi = r[1];
      const float d = dz[j];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[c] = fmaf(d, lo[c], acc[c]);
        acc[4 + c] = fmaf(d, hi[c], acc[4 + c]);
      }
    }
    dx[(size_t)t * nv + i] = pack_vec<DT>(acc);
  }
}

// dWr[e] = sum over the expert's rows of dz x[t], and db[e]: a workgroup per
// expert and 512 columns, a thread per 8 columns, the rows split over its
// wavefronts, 8 in flight for each.
constexpr int kSumThreads = 512;
template <int DT>
__global__ __launch_bounds__(kSumThreads) void k_route_weights(const u32x4* x, int nv, int E, int k, uint32_t per_k,
                                                              const float* dz, const int32_t* offsets, const int32_t* pairs,
                                                              int rows, int n, float* dwr, float* db) {
  constexpr int W = kSumThreads / kWave, U = 8;
  __shared__ f32x4 red[W][2][64];
  __shared__ float bred[W];
  const int e = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = blockIdx.x * 64 + lane;
  const int r0 = min(max(0, offsets[e]), rows), r1 = max(r0, min(rows, offsets[e + 1]));
  const int ic = min(i, nv - 1), cnt = r1 - r0;
  const int a0 = r0 + (int)((int64_t)cnt * wave / W), a1 = r0 + (int)((int64_t)cnt * (wave + 1) / W);
  float acc[8] = {}, sum = 0.0f;
  for (int b0 = a0; b0 < a1; b0 += 64) {  // 64 slots: a lane each
    const int rr = b0 + lane;
    int p = rr < a1 ? pairs[rr] : -1;
    const bool ok = (unsigned)p < (unsigned)n;
    const float d = ok ? dz[p] : 0.0f;
    sum += d;
    int t = ok ? p : 0;
    if (per_k) t = (int)__umulhi((uint32_t)t, per_k);
    const int m = min(64, a1 - b0);
    const uint64_t used = __ballot(ok);
    for (int s = 0; s < m; s += U) {
      u32x4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = x[(size_t)__builtin_amdgcn_readlane(t, min(s + u, 63)) * nv + ic];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!(used >> min(s + u, 63) & 1)) continue;  // padding: x is not used
        const float du = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, d), min(s + u, 63)));
        float f[8];
        unpack_vec<DT>(v[u], f);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = fmaf(du, f[c], acc[c]);
      }
    }
  }
  red[wave][0][lane] = f32x4{acc[0], acc[1], acc[2], acc[3]};
  red[wave][1][lane] = f32x4{acc[4], acc[5], acc[6], acc[7]};
  sum = wave_sum_f32(sum);
  if (lane == 0) bred[wave] = sum;
  __syncthreads();
  if (threadIdx.x < 128) {
    const int h = threadIdx.x & 1, l = threadIdx.x >> 1, c = blockIdx.x * 64 + l;
    f32x4 s = red[0][h][l];
#pragma unroll
    for (int w = 1; w < W; ++w) s += red[w][h][l];
    if (c < nv) *(f32x4*)(dwr + ((size_t)e * nv + c) * 8 + h * 4) = s;
  }
  if (threadIdx.x == 0 && blockIdx.x == 0) {
    float s = 0.0f;
    for (int w = 0; w < W; ++w) s += bred[w];
    db[e] = s;
  }
}

inline bool bad(const void* p, unsigned align) { return !p || !aligned_to(p, align); }
inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

int check_shape(int32_t T, int32_t k, int32_t E, int32_t H, int32_t rows) {
  const int st = check_sort_shape(T, k, E, 1);
  if (st != MOE_OK) return st;
  if (H <= 0 || rows < 0) return MOE_E_INVAL;
  return H % 8 || H > kMaxWidth ? MOE_E_UNSUPPORTED : MOE_OK;
}

constexpr int kWideSlice = 512;    // experts up to which a slice has 64 columns
constexpr int kSliceGroups = 512;  // workgroups of the slice kernels

struct RoutePlan {
  bool gather;  // few slots: rows of Wr gathered
  int slices, ranges, range;
  size_t dz, z, total;
};
RoutePlan route_plan(int T, int k, int E, int H) {
  RoutePlan p{};
  p.gather = (int64_t)T * k <= E;
  p.slices = ceil_div(H, E <= kWideSlice ? 64 : 32);
  p.ranges = std::max(1, std::min(kSliceGroups / p.slices, ceil_div(T, 32)));
  p.range = ceil_div(std::max(T, 1), p.ranges);
  p.dz = 0;
  p.z = round256(std::max<size_t>(4, (size_t)T * k * 4));
  p.total = p.z + (p.gather ? 0 : round256((size_t)p.slices * T * k * 4));
  return p;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_route_backward_workspace_bytes(int32_t T, int32_t k, int32_t n_experts, int32_t H, int32_t rows) {
  if (check_shape(T, k, n_experts, H, rows) != MOE_OK) return 0;
  return route_plan(T, k, n_experts, H).total;
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
  const RoutePlan p = route_plan(T, k, n_experts, H);
  if (ws_bytes < p.total) return MOE_E_WORKSPACE;
  const uint32_t per_k = k == 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + k - 1) / k);
  const RouteArgs a{(const u32x4*)x, router_w, topk_idx, T, H, n_experts, k, per_k};
  const int nv = H / 8, n = T * k;
  float *dz = (float*)((char*)ws + p.dz), *z = (float*)((char*)ws + p.z);
  const hipStream_t s = (hipStream_t)stream;
  const u32x4* addv = (const u32x4*)add;
  u32x4* dxv = (u32x4*)dx;
  const dim3 grid(p.slices, p.ranges), sums(ceil_div(nv, 64), n_experts);
  const auto run = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const auto slices = [&](auto dots, auto to_dx) {
      dots<<<grid, kThreads, 0, s>>>(a, p.range, z);
      k_route_slots<<<ceil_div(T, 64 / k), kSlotThreads, 0, s>>>(a, p.slices, z, router_b, dw, dz);
      to_dx<<<grid, kThreads, 0, s>>>(a, p.range, dz, addv, dxv);
    };
    if (T && p.gather) k_route_grad_tokens<DT><<<T, kThreads, 0, s>>>(a, router_b, dw, addv, dxv, dz);
    else if (T && n_experts <= 64) slices(k_route_dots<DT, 64, 64>, k_route_dx<DT, 64, 64>);
    else if (T && n_experts <= 256) slices(k_route_dots<DT, 256, 64>, k_route_dx<DT, 256, 64>);
    else if (T && n_experts <= kWideSlice) slices(k_route_dots<DT, kWideSlice, 64>, k_route_dx<DT, kWideSlice, 64>);
    else if (T) slices(k_route_dots<DT, kMaxExperts, 32>, k_route_dx<DT, kMaxExperts, 32>);
    k_route_weights<DT><<<sums, kSumThreads, 0, s>>>((const u32x4*)x, nv, n_experts, k, per_k, dz, offsets, pairs, rows, n,
                                                    d_router_w, d_router_b);
  };
  if (dtype == MOE_T_F16) run(std::integral_constant<int, MOE_T_F16>{});
  else run(std::integral_constant<int, MOE_T_BF16>{});
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // extern "C"
