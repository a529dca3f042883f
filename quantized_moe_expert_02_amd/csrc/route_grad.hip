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
// that Wr and x each cross the memory a few times only.  What bounds them is the
// vector unit: 8 multiply-adds of a lane come with about 14 other instructions.
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
};

// All experts' columns [c0, c0 + CW) of Wr into LDS rows; columns past H are
// zero, and so is one row more, which dropped slots read.
template <int CW>
__device__ __forceinline__ void load_slice(const RouteArgs& a, int c0, float* w) {
  constexpr int V = CW / 4, U = 9;  // loads in flight (all of them for 256 experts)
  const int n = (a.E + 1) * V;
  for (int i0 = threadIdx.x; i0 < n; i0 += U * kThreads) {
    f32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads, e = min(i / V, a.E - 1), c = c0 + i % V * 4;
      v[u] = *(const f32x4*)(a.wr + (size_t)e * a.H + (c < a.H ? c : 0));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= a.E * V || c0 + i % V * 4 >= a.H) v[u] = f32x4{0, 0, 0, 0};
      if (i < n) *(f32x4*)(w + i * 4) = v[u];
    }
  }
}

// A row of a slice is shared by CW / 8 lanes, 8 columns each.  A lane reads its
// 8 as two 16-byte halves, and lanes of odd rows take the second half first:
// two neighbouring rows then cover different LDS banks, whichever experts they
// are.
template <int CW>
constexpr int kLanes = CW / 8;

// The slots of the token that a lane group works on, L at a time, one per lane:
// the experts' places in LDS.
template <int CW>
__device__ __forceinline__ int slot_place(const RouteArgs& a, int t, int j) {
  int e = a.idx[min(min(t, a.T - 1) * a.k + j, a.T * a.k - 1)];
  if (j >= a.k || (unsigned)e >= (unsigned)a.E) e = a.E;
  return e * CW;
}

// Partial logits [slices][T k], 64 / L tokens per turn of a wavefront.  2,048
// tokens, top-8 of 256, 6144 wide: 16.0 us, of which about 5 fill the slices.
template <int DT, int EC, int CW>
__global__ __launch_bounds__(kThreads) void k_route_dots(RouteArgs a, int range, float* zpart) {
  __shared__ __align__(16) float w[(EC + 1) * CW];  // E <= EC
  constexpr int L = kLanes<CW>, P = 64 / L;  // lanes per token, tokens per turn
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane / L, cl = lane % L, odd = sub & 1;
  const int c0 = blockIdx.x * CW, nv = a.H / 8, cv = c0 / 8 + cl;
  const int n = a.T * a.k, t1 = min((int)(blockIdx.y + 1) * range, a.T), first = blockIdx.y * range + wave * P;
  u32x4 xn = {0, 0, 0, 0};
  int pn = 0;
  const auto fetch_x = [&](int base) { xn = a.x[(size_t)min(base + sub, a.T - 1) * nv + min(cv, nv - 1)]; };
  if (first < t1) {
    fetch_x(first);
    pn = slot_place<CW>(a, first + sub, cl);
  }
  load_slice<CW>(a, c0, w);
  __syncthreads();
  const float *wa = w + cl * 8 + odd * 4, *wb = w + cl * 8 + 4 - odd * 4;
  float* out = zpart + (size_t)blockIdx.x * n;
  for (int base = first; base < t1; base += kWaves * P) {
    const int t = base + sub;
    float f[8];
    {
      u32x4 x = cv < nv ? xn : u32x4{0, 0, 0, 0};
      if (odd) x = u32x4{x[2], x[3], x[0], x[1]};
      unpack_vec<DT>(x, f);
    }
    if (base + kWaves * P < t1) fetch_x(base + kWaves * P);
    for (int j0 = 0; j0 < a.k; j0 += L) {
      const int place = pn;
      if (j0 + L < a.k) pn = slot_place<CW>(a, t, j0 + L + cl);
      else if (base + kWaves * P < t1) pn = slot_place<CW>(a, t + kWaves * P, cl);
      float mine = 0.0f;
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const int at = __shfl(place, sub * L + j);
        const f32x4 r0 = *(const f32x4*)(wa + at), r1 = *(const f32x4*)(wb + at);
        float z = f[0] * r0[0];
#pragma unroll
        for (int c = 1; c < 4; ++c) z = fmaf(f[c], r0[c], z);
#pragma unroll
        for (int c = 0; c < 4; ++c) z = fmaf(f[4 + c], r1[c], z);
        z += __builtin_bit_cast(float, partner<1>(__builtin_bit_cast(int, z)));
        z += __builtin_bit_cast(float, partner<2>(__builtin_bit_cast(int, z)));
        if (L == 8) z += __builtin_bit_cast(float, partner<4>(__builtin_bit_cast(int, z)));
        if (cl == j) mine = z;
      }
      if (t < t1 && j0 + cl < a.k) out[(size_t)t * a.k + j0 + cl] = mine;
    }
  }
}

// Work items of the weights' gradient: up to kItemRows sorted rows of one
// expert (an expert without rows has one, which writes zeros).
constexpr int kItemRows = 128;
struct Item {
  int e, r0, r1;  // e < 0: none
  int slot;       // partial sum it writes, or -1: the result itself
  int parts;      // the expert's items, in its first one (else 0)
};

// Fills items[0, most) from the groups; one workgroup of 256 threads.  The
// experts' first items and slots first, then a thread looks up each item's expert.
struct ItemLds {
  int item[kMaxExperts], slot[kMaxExperts], r0[kMaxExperts], r1[kMaxExperts], sums[2][4];
};
__device__ __forceinline__ void make_items(ItemLds& L, const int32_t* offsets, int E, int rows, int most, Item* items) {
  constexpr int per = kItemRows;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int at = 0, slots = 0;
  for (int e0 = 0; e0 < E; e0 += 256) {
    const int e = e0 + tid;
    int r0 = 0, r1 = 0;
    if (e < E) {
      r0 = min(max(0, offsets[e]), rows);
      r1 = max(r0, min(rows, offsets[e + 1]));
    }
    const int parts = (int)(((int64_t)r1 - r0 + per - 1) / per), ni = e < E ? max(1, parts) : 0, ns = parts > 1 ? parts : 0;
    int ii = ni, is = ns;
    for (int d = 1; d < 64; d <<= 1) {
      const int oi = __shfl_up(ii, d), os = __shfl_up(is, d);
      ii += lane >= d ? oi : 0;
      is += lane >= d ? os : 0;
    }
    if (lane == 63) {
      L.sums[0][wave] = ii;
      L.sums[1][wave] = is;
    }
    __syncthreads();
    int i0 = at + ii - ni, s0 = slots + is - ns;
    for (int w = 0; w < 4; ++w) {
      i0 += w < wave ? L.sums[0][w] : 0;
      s0 += w < wave ? L.sums[1][w] : 0;
      at += L.sums[0][w];
      slots += L.sums[1][w];
    }
    if (e < E) {
      L.item[e] = i0;
      L.slot[e] = s0;
      L.r0[e] = r0;
      L.r1[e] = r1;
    }
    __syncthreads();
  }
  for (int i = tid; i < most; i += 256) {
    Item it = {-1, 0, 0, -1, 0};
    if (i < at) {
      int lo = 0, hi = E;  // L.item[lo] <= i < L.item[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (L.item[mid] <= i) lo = mid;
        else hi = mid;
      }
      const int r0 = L.r0[lo], r1 = L.r1[lo];
      const int j = i - L.item[lo], parts = (int)(((int64_t)r1 - r0 + per - 1) / per), from = r0 + j * per;
      it = {lo, from, min(r1, from + per), parts > 1 ? L.slot[lo] + j : -1, j ? 0 : parts};
    }
    items[i] = it;
  }
}

// sigmoid(z) e^-top for a token's kept slots, top being their largest logit or 0
// if that is less: the factor cancels in w = s / sum s, and without it every s of
// a token is 0 in fp32 where all its logits lie below about -88 (0 / 0).
__device__ __forceinline__ float scaled_sigmoid(float z, float top) { return 1.0f / (expf(top) + expf(top - z)); }

// dz of every slot from the partial logits: 64 / k tokens per workgroup, four
// threads per slot over the slices.  The last workgroup makes the items of the
// launch after next.
constexpr int kSlotThreads = 256;
__global__ __launch_bounds__(kSlotThreads) void k_route_slots(RouteArgs a, int slices, const float* zpart, const float* br,
                                                             const float* dw, float* dz, const int32_t* offsets, int rows,
                                                             int most, Item* items) {
  __shared__ union {
    ItemLds items;
    struct {
      float part[4][64], sg[64], gw[64];
    };
  } L;
  auto& part = L.part;
  float *sg = L.sg, *gw = L.gw;
  if (blockIdx.x == gridDim.x - 1) return make_items(L.items, offsets, a.E, rows, most, items);
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
  gw[l] = ok ? z : -INFINITY;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);  // one wavefront from here on: LDS keeps its order
  const int first = l / a.k * a.k;
  float top = -INFINITY;
  for (int j = 0; j < a.k; ++j) top = fmaxf(top, gw[min(first + j, 63)]);
  const float s = ok ? scaled_sigmoid(z, fminf(top, 0.0f)) : 0.0f, g = ok ? dw[p] : 0.0f;
  sg[l] = s;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  float S = 0.0f;
  for (int j = 0; j < a.k; ++j) S += sg[min(first + j, 63)];
  const float w = ok ? s / S : 0.0f;
  gw[l] = g * w;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  float m = 0.0f;
  for (int j = 0; j < a.k; ++j) m += gw[min(first + j, 63)];
  if (l < np) dz[p] = ok ? w * (1.0f / (1.0f + expf(z))) * (g - m) : 0.0f;
}

// dx[t] = add[t] + sum_j dz_j Wr[e_j], as k_route_dots (15.2 us there).
template <int DT, int EC, int CW>
__global__ __launch_bounds__(kThreads) void k_route_dx(RouteArgs a, int range, const float* dz, const u32x4* add, u32x4* dx) {
  __shared__ __align__(16) float w[(EC + 1) * CW];
  constexpr int L = kLanes<CW>, P = 64 / L;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane / L, cl = lane % L, odd = sub & 1;
  const int c0 = blockIdx.x * CW, nv = a.H / 8, cv = c0 / 8 + cl;
  const int n = a.T * a.k, t1 = min((int)(blockIdx.y + 1) * range, a.T), first = blockIdx.y * range + wave * P;
  u32x4 an = {0, 0, 0, 0};
  int pn = 0;
  float dn = 0.0f;
  const auto fetch_add = [&](int base) { an = add[(size_t)min(base + sub, a.T - 1) * nv + min(cv, nv - 1)]; };
  const auto fetch = [&](int t, int j) {
    pn = slot_place<CW>(a, t, j);
    dn = dz[min(min(t, a.T - 1) * a.k + j, n - 1)];
    if (j >= a.k) dn = 0.0f;
  };
  if (first < t1) {
    if (add) fetch_add(first);
    fetch(first + sub, cl);
  }
  load_slice<CW>(a, c0, w);
  __syncthreads();
  const float *wa = w + cl * 8 + odd * 4, *wb = w + cl * 8 + 4 - odd * 4;
  for (int base = first; base < t1; base += kWaves * P) {
    const int t = base + sub;
    float acc[8];
    unpack_vec<DT>(an, acc);
    if (add && base + kWaves * P < t1) fetch_add(base + kWaves * P);
    f32x4 s0 = {0, 0, 0, 0}, s1 = s0;
    for (int j0 = 0; j0 < a.k; j0 += L) {
      const int place = pn;
      const float d = dn;
      if (j0 + L < a.k) fetch(t, j0 + L + cl);
      else if (base + kWaves * P < t1) fetch(t + kWaves * P, cl);
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const int at = __shfl(place, sub * L + j);
        const float dj = __shfl(d, sub * L + j);
        const f32x4 r0 = *(const f32x4*)(wa + at), r1 = *(const f32x4*)(wb + at);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s0[c] = fmaf(dj, r0[c], s0[c]);
          s1[c] = fmaf(dj, r1[c], s1[c]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      acc[c] += odd ? s1[c] : s0[c];
      acc[4 + c] += odd ? s0[c] : s1[c];
    }
    // (past the L2s, whose dirty lines the launch's end would wait for: 58.7 -> 56.5 us)
    if (t < t1 && cv < nv) __builtin_nontemporal_store(pack_vec<DT>(acc), dx + (size_t)t * nv + cv);
  }
}

// The same three steps for few tokens, whose rows of Wr are gathered directly:
// one workgroup per token, a wavefront per slot and then a thread per 8 columns.
// Bound by three waits for memory in turn: 100 tokens, top-8 of 256, 6144 wide 10.5
// us; 45 tokens, 2048 wide 5.5.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_route_grad_tokens(RouteArgs a, const float* br, const float* dw, const u32x4* add,
                                                                u32x4* dx, float* dz_out) {
  constexpr int U = 4;  // vectors, or slots, in flight
  __shared__ float z[kMaxTopK], dz[kMaxTopK];
  __shared__ int ex[kMaxTopK];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, k = a.k, nv = a.H / 8;
  const u32x4* xt = a.x + (size_t)t * nv;
  const f32x4* w4 = (const f32x4*)a.wr;
  for (int j = wave; j < k; j += kWaves) {
    const int e = a.idx[(size_t)t * k + j];
    const bool ok = (unsigned)e < (unsigned)a.E;
    const f32x4* r = w4 + (size_t)(ok ? e : 0) * nv * 2;
    float s = 0.0f;
    for (int i0 = lane; i0 < nv; i0 += 64 * U) {
      u32x4 x[U];
      f32x4 lo[U], hi[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = min(i0 + 64 * u, nv - 1);
        x[u] = xt[i];
        lo[u] = r[i * 2];
        hi[u] = r[i * 2 + 1];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + 64 * u >= nv) continue;
        float f[8];
        unpack_vec<DT>(x[u], f);
#pragma unroll
        for (int c = 0; c < 4; ++c) s = fmaf(f[c], lo[u][c], s);
#pragma unroll
        for (int c = 0; c < 4; ++c) s = fmaf(f[4 + c], hi[u][c], s);
      }
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
    const float top = wave_max_f32(ok ? zj : -INFINITY);
    const float s = ok ? scaled_sigmoid(zj, fminf(top, 0.0f)) : 0.0f;
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
    for (int j0 = 0; j0 < k; j0 += U) {
      f32x4 lo[U], hi[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const f32x4* r = w4 + ((size_t)max(ex[min(j0 + u, k - 1)], 0) * nv + i) * 2;
        lo[u] = r[0];
        hi[u] = r[1];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j0 + u >= k || ex[j0 + u] < 0) continue;
        const float d = dz[j0 + u];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[c] = fmaf(d, lo[u][c], acc[c]);
          acc[4 + c] = fmaf(d, hi[u][c], acc[4 + c]);
        }
      }
    }
    dx[(size_t)t * nv + i] = pack_vec<DT>(acc);
  }
}

// dWr[e] = sum over an item's rows of dz x[t], and db[e]: a workgroup per item
// and Q * 256 columns.  Half a wavefront takes a row (a lane 8 columns of each
// 256), the rows are split over the W wavefronts, 8 KB or more in flight for
// each.  With 8 runs of columns a die takes one of them, so that its L2 keeps
// that part of x over all experts.  items == NULL: an expert each.
template <int DT, int W, int Q>
__global__ __launch_bounds__(W * kWave) void k_route_weights(const u32x4* x, int nv, int E, uint32_t per_k, const float* dz,
                                                            const int32_t* offsets, const int32_t* pairs, int rows, int n,
                                                            const Item* items, int chunks, float* dwr, float* db,
                                                            float* sums, float* bsums, int slots) {
  constexpr int U = Q == 1 ? 8 : Q == 2 ? 6 : 4;  // rows in flight per half
  __shared__ f32x4 red[W][Q][2][32];
  __shared__ float bred[W];
  const int j = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  Item it;
  if (items) {
    it = items[j];
  } else {
    it.e = j;
    it.r0 = min(max(0, offsets[it.e]), rows);
    it.r1 = max(it.r0, min(rows, offsets[it.e + 1]));
    it.slot = -1;
    it.parts = 0;
  }
  if (it.e < 0 || it.slot >= slots) return;  // (past the slots: only for groups that overlap)
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5, l = lane & 31;
  int cc[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) cc[q] = min((chunk * Q + q) * 32 + l, nv - 1);
  const int cnt = it.r1 - it.r0;
  const int a0 = it.r0 + cnt * wave / W, a1 = it.r0 + cnt * (wave + 1) / W;
  float acc[Q][8] = {};
  float sum = 0.0f;
  for (int b0 = a0; b0 < a1; b0 += 64) {  // 64 slots: a lane each
    const int rr = b0 + lane;
    const int p = rr < a1 ? pairs[rr] : -1;
    const bool ok = (unsigned)p < (unsigned)n;
    const float d = ok ? dz[p] : 0.0f;
    sum += d;
    int t = ok ? p : 0;
    if (per_k) t = (int)__umulhi((uint32_t)t, per_k);
    if (!ok) t = -1;
    const int m = min(64, a1 - b0);
    for (int s = 0; s < m; s += 2 * U) {
      u32x4 v[U][Q];
      int tt[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        tt[u] = __shfl(t, min(s + 2 * u + half, 63));
        const u32x4* row = x + (size_t)max(tt[u], 0) * nv;
#pragma unroll
        for (int q = 0; q < Q; ++q) v[u][q] = row[cc[q]];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float du = __shfl(d, min(s + 2 * u + half, 63));
        if (s + 2 * u + half < m && tt[u] >= 0) {  // else padding: x is not used
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            float f[8];
            unpack_vec<DT>(v[u][q], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[q][i] = fmaf(du, f[i], acc[q][i]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      acc[q][i] += __builtin_bit_cast(float, partner<32>(__builtin_bit_cast(int, acc[q][i])));
    if (!half) {
      red[wave][q][0][l] = f32x4{acc[q][0], acc[q][1], acc[q][2], acc[q][3]};
      red[wave][q][1][l] = f32x4{acc[q][4], acc[q][5], acc[q][6], acc[q][7]};
    }
  }
  sum = wave_sum_f32(sum);
  if (lane == 0) bred[wave] = sum;
  __syncthreads();
  float* o = it.slot >= 0 ? sums + (size_t)it.slot * nv * 8 : dwr + (size_t)it.e * nv * 8;
  for (int i = threadIdx.x; i < Q * 64; i += W * kWave) {  // 4 columns each, in their order
    const int q = i / 64, c = i % 64 / 2, h = i & 1, col = (chunk * Q + q) * 32 + c;
    f32x4 s = red[0][q][h][c];
#pragma unroll
    for (int w = 1; w < W; ++w) s += red[w][q][h][c];
    if (col < nv) *(f32x4*)(o + (size_t)col * 8 + h * 4) = s;
  }
  if (threadIdx.x == 0 && chunk == 0) {
    float s = 0.0f;
    for (int w = 0; w < W; ++w) s += bred[w];
    (it.slot >= 0 ? bsums[it.slot] : db[it.e]) = s;
  }
}

// Adds the partial sums of experts that have several (in consecutive slots).
__global__ __launch_bounds__(256) void k_route_sum(const Item* items, int H, const float* sums, const float* bsums, int slots,
                                                  float* dwr, float* db) {
  const Item it = items[blockIdx.x];
  if (it.e < 0 || it.parts < 2) return;
  const int m = min(it.parts, slots - it.slot), i = blockIdx.y * 256 + threadIdx.x;
  if (m <= 0) return;
  if (i < H / 4) {
    const f32x4* p = (const f32x4*)(sums + (size_t)it.slot * H) + i;
    constexpr int U = 8;  // in flight
    f32x4 s = {0, 0, 0, 0};
    for (int j = 0; j < m; j += U) {
      f32x4 v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) v[k] = p[(size_t)min(j + k, m - 1) * (H / 4)];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (j + k < m) s += v[k];
    }
    *(f32x4*)(dwr + (size_t)it.e * H + i * 4) = s;
  }
  if (i < 64) {
    float s = 0.0f;
    for (int j = i; j < m; j += 64) s += bsums[it.slot + j];
    s = wave_sum_f32(s);
    if (i == 0) db[it.e] = s;
  }
}

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

int check_shape(int32_t T, int32_t k, int32_t E, int32_t H, int32_t rows) {
  const int st = check_sort_shape(T, k, E, 1);
  if (st != MOE_OK) return st;
  if (H <= 0 || rows < 0) return MOE_E_INVAL;
  return H % 8 || H > kMaxWidth || rows > kMaxSorted ? MOE_E_UNSUPPORTED : MOE_OK;
}

constexpr int kWideSlice = 512;    // experts up to which a slice has 64 columns
// Tokens up to which rows of Wr are gathered, in two launches instead of five.
// Calls gathered and by slices, 6144 wide, even router: 512 tokens, 2 of 8 experts
// 19.5 and 28.3 us, 8 of 64 21.1 and 27.0, 8 of 256 24.9 and 27.4 (800 tokens 37.8 and
// 38.7); 100 tokens 17 and 27; 2048 wide, 512 tokens 17 and 27 with any.  A skewed
// router (zipf 1.1) leaves an expert's rows to one workgroup: 300 tokens, 8 of 64
// experts 26.6 and 28.0, 8 of 256 27.6 and 29.2, 512 tokens 25.5 and 28.4, 35.6 and 30.4,
// 36.5 and 33.1 (800 tokens 56.5 and 41.2), 2048 wide 17.4, 20.7, 21.4 and 27.5.
constexpr int kGatherTokens = 512;
constexpr int kSliceGroups = 512;  // workgroups of the slice kernels

struct RoutePlan {
  bool gather;  // few tokens: rows of Wr gathered
  int slices, ranges, range;
  int items, slots;  // of the weights' gradient (bounds; none where rows are gathered)
  size_t dz, z, item, sums, bsums, total;
};
RoutePlan route_plan(int T, int k, int E, int H, int rows) {
  RoutePlan p{};
  p.gather = T <= kGatherTokens;
  p.slices = ceil_div(H, E <= kWideSlice ? 64 : 32);
  p.ranges = std::max(1, std::min(kSliceGroups / p.slices, ceil_div(T, 32)));
  p.range = ceil_div(std::max(T, 1), p.ranges);
  size_t o = 0;
  const auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += round256(bytes);
    return at;
  };
  p.dz = take(std::max<size_t>(4, (size_t)T * k * 4));
  if (!p.gather) {
    p.items = E + rows / kItemRows;
    p.slots = 2 * (rows / kItemRows);
    p.z = take((size_t)p.slices * T * k * 4);
    p.item = take((size_t)p.items * sizeof(Item));
    p.sums = take((size_t)p.slots * H * 4);
    p.bsums = take((size_t)p.slots * 4);
  }
  p.total = o;
  return p;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_route_backward_workspace_bytes(int32_t T, int32_t k, int32_t n_experts, int32_t H, int32_t rows) {
  if (check_shape(T, k, n_experts, H, rows) != MOE_OK) return 0;
  return route_plan(T, k, n_experts, H, rows).total;
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
  const RoutePlan p = route_plan(T, k, n_experts, H, rows);
  if (ws_bytes < p.total) return MOE_E_WORKSPACE;
  // p / k by multiplication with ceil(2^32 / k): exact for p < 2^27, k <= 32; 0 for k = 1
  const uint32_t per_k = k == 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + k - 1) / k);
  const RouteArgs a{(const u32x4*)x, router_w, topk_idx, T, H, n_experts, k};
  const int n = T * k;
  float *dz = (float*)((char*)ws + p.dz), *z = (float*)((char*)ws + p.z);
  const hipStream_t s = (hipStream_t)stream;
  const u32x4* addv = (const u32x4*)add;
  u32x4* dxv = (u32x4*)dx;
  const dim3 grid(p.slices, p.ranges);
  Item* items = p.gather ? nullptr : (Item*)((char*)ws + p.item);
  float *sums = (float*)((char*)ws + p.sums), *bsums = (float*)((char*)ws + p.bsums);
  const auto run = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const auto slices = [&](auto dots, auto to_dx) {
      dots<<<grid, kThreads, 0, s>>>(a, p.range, z);
      k_route_slots<<<ceil_div(T, 64 / k) + 1, kSlotThreads, 0, s>>>(a, p.slices, z, router_b, dw, dz, offsets, rows, p.items,
                                                                     items);
      to_dx<<<grid, kThreads, 0, s>>>(a, p.range, dz, addv, dxv);
    };
    if (T && p.gather) k_route_grad_tokens<DT><<<T, kThreads, 0, s>>>(a, router_b, dw, addv, dxv, dz);
    else if (T && n_experts <= 64) slices(k_route_dots<DT, 64, 64>, k_route_dx<DT, 64, 64>);
    else if (T && n_experts <= 256) slices(k_route_dots<DT, 256, 64>, k_route_dx<DT, 256, 64>);
    else if (T && n_experts <= kWideSlice) slices(k_route_dots<DT, kWideSlice, 64>, k_route_dx<DT, kWideSlice, 64>);
    else if (T) slices(k_route_dots<DT, kMaxExperts, 32>, k_route_dx<DT, kMaxExperts, 32>);
    const auto weights = [&](auto kernel, int W, int Q) {
      const int chunks = ceil_div(H, 256 * Q);
      kernel<<<(items ? p.items : n_experts) * chunks, W * kWave, 0, s>>>((const u32x4*)x, H / 8, n_experts, per_k, dz, offsets,
                                                                        pairs, rows, n, items, chunks, d_router_w, d_router_b,
                                                                        sums, bsums, items ? p.slots : 0);
    };
    // An eighth of the width per workgroup where that is 256 to 768 columns; two
    // wavefronts and 128 rows at most: 2,048 tokens, top-8 of 256, 6144 wide, a
    // skewed router: 20 us (64 rows: 19, but twice the partial sums; 256: 26; one
    // wavefront 24, eight and 512 rows 32).
    const int runs = ceil_div(H, 8 * 256);
    if (runs == 1) weights(k_route_weights<DT, 2, 1>, 2, 1);
    else if (runs == 2) weights(k_route_weights<DT, 2, 2>, 2, 2);
    else weights(k_route_weights<DT, 2, 3>, 2, 3);
    if (items && p.slots)
      k_route_sum<<<dim3(p.items, ceil_div(H, 1024)), 256, 0, s>>>(items, H, sums, bsums, p.slots, d_router_w,
                                                                  d_router_b);
  };
  if (dtype == MOE_T_F16) run(std::integral_constant<int, MOE_T_F16>{});
  else run(std::integral_constant<int, MOE_T_BF16>{});
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // extern "C"
