// Entry points of include/moe_w4.h, packing, and the sum of split products; the
// products themselves are in w4_few.hip, w4_rows.hip and w4_grad.hip.
#include "w4.h"

namespace moe {

namespace {

// The splits' partial sums added in their order.  Bound by its launch (45 rows of 2080: 3.9 us).
template <int DT>
__global__ __launch_bounds__(256) void k_w4_sum(W4Args a, int width) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = width / 4, row = i / per;
  if (row >= a.T) return;
  const int c = (int)(i % per) * 4;
  f32x4 v{};
  for (int s = 0; s < a.split; ++s) v += *(const f32x4*)(a.part + ((int64_t)s * a.T + row) * width + c);
  W4Args o = a;
  o.part = nullptr;
  put4<DT>(o, width, 0, row, c, v);
}

// ---------------------------------------------------------------------------
// Packing.
// ---------------------------------------------------------------------------
struct PackArgs {
  uint8_t* packed;
  size_t stride, soff, zoff;
  int N, K, NB, KB, group, SG, dtype;
  uint8_t* q;
  uint16_t* scales;
  int8_t* zeros;
};

// Nibbles 0 .. 7 to 0 2 4 6 1 3 5 7 (even columns to the low half), and back.
__device__ __forceinline__ uint32_t to_halves(uint32_t v) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) o |= (v >> (4 * i) & 15) << (4 * (i / 2 + (i & 1) * 4));
  return o;
}
__device__ __forceinline__ uint32_t from_halves(uint32_t v) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) o |= (v >> (4 * (i / 2 + (i & 1) * 4)) & 15) << (4 * i);
  return o;
}

// One workgroup per block and matrix; a pass over memory, once per model.
template <bool PACK>
__global__ __launch_bounds__(64) void k_w4_pack(PackArgs a) {
  const int lane = threadIdx.x, li = lane & 15, g = lane >> 4;
  const size_t block = blockIdx.x;
  const int nb = (int)(block / a.KB), kb = (int)(block % a.KB), e = blockIdx.y, row = nb * kBlockRows + li;
  uint8_t* w = a.packed + (size_t)e * a.stride;
  const bool in = row < a.N;
  const size_t r = (size_t)e * a.N + row;
  u32x4* mine = (u32x4*)(w + block * kBlockBytes) + lane;
  u32x4 d{0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
  if (!PACK) d = *mine;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = kb * kBlockCols + 32 * j + 8 * g;
    if (!in || c >= a.K) continue;
    // (K is a multiple of 32: a dword of canonical codes is aligned)
    uint32_t* at = (uint32_t*)(a.q + (r * a.K + c) / 2);
    if (PACK) d[j] = to_halves(*at ^ 0x88888888u);
    else *at = from_halves(d[j]) ^ 0x88888888u;
  }
  if (PACK) *mine = d;
  const int width = kBlockCols / a.SG, groups = a.K / a.group;
  for (int i = lane; i < 16 * a.SG; i += 64) {
    const int rr = nb * kBlockRows + i / a.SG, c = kb * kBlockCols + i % a.SG * width;
    const bool have = rr < a.N && c < a.K;
    uint16_t* s = (uint16_t*)(w + a.soff) + block * 16 * a.SG + i;
    int8_t* z = (int8_t*)(w + a.zoff) + block * 16 * a.SG + i;
    const size_t from = ((size_t)e * a.N + rr) * groups + c / a.group;
    if (PACK) {
      *s = have ? a.scales[from] : 0;
      if (a.zeros) *z = have ? a.zeros[from] : 0;
    } else if (have && c % a.group == 0) {
      a.scales[from] = *s;
      if (a.zeros) a.zeros[from] = *z;
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr int64_t kMaxLd = 1 << 22;
constexpr int kFewRows = 16;

W4Layout w4_layout(const moe_w4_dims_t& d) {
  W4Layout l;
  l.NB = ceil_div(d.N, kBlockRows);
  l.KB = ceil_div(d.K, kBlockCols);
  l.SG = d.group == 32 ? 4 : d.group == 64 ? 2 : 1;
  const size_t blocks = (size_t)l.NB * l.KB;
  l.soff = blocks * kBlockBytes;
  l.zoff = l.soff + round256(blocks * 16 * l.SG * 2);
  l.stride = l.zoff + (d.zeros ? round256(blocks * 16 * l.SG) : 0);
  return l;
}

int check_w4(const moe_w4_dims_t* d) {
  if (!d || d->n < 1 || d->N <= 0 || d->K <= 0 || d->group <= 0 || (d->zeros != 0 && d->zeros != 1)) return MOE_E_INVAL;
  if (d->dtype != MOE_T_F16 && d->dtype != MOE_T_BF16) return MOE_E_INVAL;
  if (d->K % d->group) return MOE_E_INVAL;
  if (d->K % 32 || d->K > kMaxWidth || d->N % 8 || d->N > (1 << 20) || d->n > kMaxExperts ||
      (int64_t)d->n * d->N > (1 << 24))
    return MOE_E_UNSUPPORTED;
  if (d->group != 32 && d->group != 64 && d->group % 128 && d->group != d->K) return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

int check_w4_rows(const moe_w4_dims_t* d, int32_t T) {
  const int st = check_w4(d);
  if (st != MOE_OK) return st;
  if (T < 0) return MOE_E_INVAL;
  return T > kMaxRows || (int64_t)T * std::max(d->N, d->K) > kMaxElems ? MOE_E_UNSUPPORTED : MOE_OK;
}

// Up to 16 rows of one matrix, or half as many rows as experts (us, few and many rows' kernel:
// 256 experts, 2048 x 1024, by Zipf's law, 64 rows 17.9 and 21.1, 128 23.3 and 23.4, 512 53 and
// 48, 4,096 128 and 82; 128 experts, 6144 x 2048, evenly, 64 rows 87 and 97, 128 164 and 169).
// More of one matrix, up to 512, where that kernel passes over the columns once and, 16 rows
// at a time, decodes at most 40 Ki blocks (us, few and many rows' kernel with its sum: 2048 x
// 2048, 64 rows 7.4 and 14.3, 256 14.0 and 18.9, 512 21.0 and 21.6; 6144 x 6144, 32 rows 15.1
// and 16.4, 48 23.4 and 20.3; 6144 x 2048 with groups of 32 and zero points, 96 rows 18.7 and
// 20.3, 256 33.3 and 27.8; 32,000 x 2048, 24 rows 21.9 and 18.8; in several passes, 512 rows of
// 40 x 16384 26.8 and 20.0, 300 of 8 x 65536 73 and 33; bfloat16, whose codes take more
// instructions, 2048 x 2048, 64 rows 7.7 and 14.3, 256 15.2 and 18.7, 512 22.3 and 21.8).
constexpr int kFewRowsMost = 512, kOnePass = 48;
constexpr int64_t kFewBlocks = 40 << 10;

bool few_rows(const moe_w4_dims_t& d, int T) {
  if (T <= std::max(kFewRows, d.n / 2)) return true;
  const int KB = ceil_div(d.K, kBlockCols);
  return d.n == 1 && T <= kFewRowsMost && KB <= kOnePass &&
         (int64_t)ceil_div(T, 16) * ceil_div(d.N, kBlockRows) * KB <= kFewBlocks;
}

// Measured in us.  One matrix: tiles of 128 rows where they give nearly two workgroups
// per CU, else 64 (6144 x 6144, 2,048 rows: forward 128 x 192 147, 64 x 256 186; 8,192 rows,
// gradient 128 rows 550, 64 642; 2,048 rows of 2048 x 6144: forward 64 x 256 68, 128 x 192
// 96, gradient 64 rows 62, 128 66), and 32 for up to 32 rows.  Experts: forward 96 x
// 256 (256 experts, 2048 x 1024, 15,565 rows by Zipf's law: 135, 64 x 256 138, 128 x 192 206;
// 64 experts, 6144 x 2048, 16,384 rows: 463, 532, 513); gradient 64 rows, or 128 where they
// have nearly that many on average (the same: 87 and 107; 530 and 472).
// The sums are split while all workgroups are resident at once (6144 x 6144, 64 rows: 4
// parts 19.7, 8 13.8, 12 17.1, with 24 tiles).
constexpr int kTwoPerCU = 460, kOnePerCU = 256, kStepsPerPart = 3;

// Tiles of BM rows that a call is expected to have: of the experts that can have rows, half
// are taken to have a tile that is not full.
int64_t likely_tiles(const moe_w4_dims_t& d, int T, int BM) {
  return d.n > 1 ? T / BM + (std::min(d.n, T) + 1) / 2 : ceil_div(T, BM);
}

TilePlan plan_tiles(const moe_w4_dims_t& d, int T, bool grad) {
  TilePlan p;
  const int avg = ceil_div(T, d.n);
  const auto blocks = [&](int MT, int R) {
    return likely_tiles(d, T, 16 * MT) * (grad ? ceil_div(d.K, kGradCols) : ceil_div(d.N, 64 * R));
  };
  p.R = 4;
  if (d.n > 1) {
    p.MT = !grad ? 6 : avg <= 96 ? 4 : 8;
  } else if (T <= 32) {
    p.MT = 2;
  } else if (blocks(8, 3) >= kTwoPerCU) {
    p.MT = 8;
    p.R = 3;
  } else {
    p.MT = 4;
  }
  p.groups = grad ? ceil_div(d.K, kGradCols) : ceil_div(d.N, 64 * p.R);
  const int steps = grad ? ceil_div(d.N, kStepRows) : ceil_div(d.K, kBlockCols);
  p.split = (int)std::max<int64_t>(1, std::min<int64_t>(kOnePerCU / blocks(p.MT, p.R), steps / kStepsPerPart));
  return p;
}

// The gradient by the kernel for few rows, in tiles of 16 or 32 rows: where that makes at
// most a workgroup per CU, and the steps are few enough for eight wavefronts
// (us, 16 or 32 rows a tile, and split over workgroups: 6144 x 6144, 16 rows 14.9, 16.9 and
// 14.8, 64 rows 26.5, 19.4 and 23.5, 128 rows 38.0, 36.5 and 29.3; 2048 x 2048, 64 rows 7.5,
// 9.1 and 14.7, 256 rows 11.6, 9.4 and 19.9; 128,000 x 2048, 8 rows 282, 316 and 59; 8 experts
// of 1024 x 1024, 64 rows 5.7, 6.3 and 10.3; 16 of 2048 x 512, 128 rows 7.0, 8.0 and 12.7).
// 0: the other kernel.
constexpr int kFewSteps = 96;

int few_grad_rows(const moe_w4_dims_t& d, int T) {
  if (ceil_div(d.N, kStepRows) > kFewSteps) return 0;
  const int groups = ceil_div(d.K, 64);
  for (int M = 1; M <= 2; ++M)
    if (likely_tiles(d, T, 16 * M) * groups <= kCUs) return M;
  return 0;
}

size_t part_bytes(const moe_w4_dims_t& d, int T, const TilePlan& p, bool grad) {
  return p.split > 1 ? (size_t)p.split * T * (grad ? d.K : d.N) * 4 : 0;
}

int check_call(const moe_w4_dims_t* d, const void* packed, const void* x, int64_t ldx, int into, int32_t T,
               const int32_t* offsets, const void* add, int64_t ldadd, const void* y, int64_t ldy, int out) {
  if (bad(packed, 256)) return MOE_E_INVAL;
  if (offsets ? !aligned_to(offsets, 4) : d->n != 1) return MOE_E_INVAL;
  if (T == 0) return MOE_OK;
  if (bad(x, 16) || bad_ld(ldx, into) || bad(y, 16) || bad_ld(ldy, out)) return MOE_E_INVAL;
  if (add && (!aligned_to(add, 16) || bad_ld(ldadd, out))) return MOE_E_INVAL;
  return ldx > kMaxLd || ldy > kMaxLd || (add && ldadd > kMaxLd) ? MOE_E_UNSUPPORTED : MOE_OK;
}

// Rows are read while others are written: y shares no memory with x, and with add only where it is add.
bool outputs_overlap(const W4Args& a, int into, int out) {
  const bool same = a.add == a.y && (a.ldadd == a.ldy || a.T == 1);
  return rows_overlap(a.x, a.ldx, into, a.y, a.ldy, out, a.T, 2) ||
         (a.add && !same && rows_overlap(a.add, a.ldadd, out, a.y, a.ldy, out, a.T, 2));
}

void launch_sum(const W4Args& a, int dtype, int width, hipStream_t s) {
  const int blocks = ceil_div((int64_t)a.T * (width / 4), 256);
  if (dtype == MOE_T_F16) k_w4_sum<MOE_T_F16><<<blocks, 256, 0, s>>>(a, width);
  else k_w4_sum<MOE_T_BF16><<<blocks, 256, 0, s>>>(a, width);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_w4_packed_bytes(const moe_w4_dims_t* d) {
  return check_w4(d) == MOE_OK ? (size_t)d->n * w4_layout(*d).stride : 0;
}

static int pack_call(const moe_w4_dims_t* d, const void* q, const void* scales, const void* zeros, const void* packed,
                     bool pack, void* stream) {
  const int st = check_w4(d);
  if (st != MOE_OK) return st;
  if (bad(q, 16) || bad(scales, 2) || bad(packed, 256) || (d->zeros != 0) != (zeros != nullptr)) return MOE_E_INVAL;
  const W4Layout l = w4_layout(*d);
  const PackArgs a{(uint8_t*)packed, l.stride, l.soff, l.zoff, d->N, d->K, l.NB, l.KB, d->group, l.SG, d->dtype,
                   (uint8_t*)q, (uint16_t*)scales, (int8_t*)zeros};
  const dim3 grid((unsigned)(l.NB * l.KB), (unsigned)d->n);
  if (pack) k_w4_pack<true><<<grid, 64, 0, (hipStream_t)stream>>>(a);
  else k_w4_pack<false><<<grid, 64, 0, (hipStream_t)stream>>>(a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

int moe_w4_pack(const moe_w4_dims_t* d, const void* q, const void* scales, const void* zeros, void* packed,
                void* stream) {
  return pack_call(d, q, scales, zeros, packed, true, stream);
}

int moe_w4_unpack(const moe_w4_dims_t* d, const void* packed, void* q, void* scales, void* zeros, void* stream) {
  return pack_call(d, q, scales, zeros, packed, false, stream);
}

int32_t moe_w4_few_rows(const moe_w4_dims_t* d, int32_t T) {
  return check_w4_rows(d, T) == MOE_OK && few_rows(*d, T) ? 1 : 0;
}

size_t moe_w4_workspace_bytes(const moe_w4_dims_t* d, int32_t T, int32_t backward) {
  if (check_w4_rows(d, T) != MOE_OK || T == 0 || (backward ? few_grad_rows(*d, T) != 0 : few_rows(*d, T))) return 0;
  return part_bytes(*d, T, plan_tiles(*d, T, backward != 0), backward != 0);
}

int moe_w4_forward(const moe_w4_dims_t* d, const void* packed, const void* x, int64_t ldx, int32_t T,
                   const int32_t* offsets, const void* add, int64_t ldadd, void* y, int64_t ldy, void* ws,
                   size_t ws_bytes, void* stream) {
  int st = check_w4_rows(d, T);
  if (st == MOE_OK) st = check_call(d, packed, x, ldx, d->K, T, offsets, add, ldadd, y, ldy, d->N);
  if (st != MOE_OK || T == 0) return st;
  const W4Layout l = w4_layout(*d);
  const hipStream_t s = (hipStream_t)stream;
  W4Args a{(const uint8_t*)packed, l.stride, l.soff, l.zoff, d->n, d->N, d->K, l.NB, l.KB, x, ldx, T, offsets, add,
           ldadd, y, ldy, nullptr, 1};
  if (few_rows(*d, T)) {
    if (outputs_overlap(a, d->K, d->N)) return MOE_E_INVAL;
    launch_w4_few(a, *d, l, s);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
  }
  const TilePlan p = plan_tiles(*d, T, false);
  const size_t need = part_bytes(*d, T, p, false);
  if (need) {
    if (bad(ws, 16)) return MOE_E_INVAL;
    if (ws_bytes < need) return MOE_E_WORKSPACE;
    a.part = (float*)ws;
    a.split = p.split;
  }
  if (outputs_overlap(a, d->K, d->N)) return MOE_E_INVAL;
  launch_w4_rows(a, *d, l, p, s);
  if (need) launch_sum(a, d->dtype, d->N, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

int moe_w4_backward(const moe_w4_dims_t* d, const void* packed, const void* dy, int64_t lddy, int32_t T,
                    const int32_t* offsets, const void* add, int64_t ldadd, void* dx, int64_t lddx, void* ws,
                    size_t ws_bytes, void* stream) {
  int st = check_w4_rows(d, T);
  if (st == MOE_OK) st = check_call(d, packed, dy, lddy, d->N, T, offsets, add, ldadd, dx, lddx, d->K);
  if (st != MOE_OK || T == 0) return st;
  const W4Layout l = w4_layout(*d);
  const hipStream_t s = (hipStream_t)stream;
  W4Args a{(const uint8_t*)packed, l.stride, l.soff, l.zoff, d->n, d->N, d->K, l.NB, l.KB, dy, lddy, T, offsets, add,
           ldadd, dx, lddx, nullptr, 1};
  if (const int M = few_grad_rows(*d, T)) {
    if (outputs_overlap(a, d->N, d->K)) return MOE_E_INVAL;
    launch_w4_grad_few(a, *d, l, M, s);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
  }
  const TilePlan p = plan_tiles(*d, T, true);
  const size_t need = part_bytes(*d, T, p, true);
  if (need) {
    if (bad(ws, 16)) return MOE_E_INVAL;
    if (ws_bytes < need) return MOE_E_WORKSPACE;
    a.part = (float*)ws;
  }
  a.split = p.split;
  if (outputs_overlap(a, d->N, d->K)) return MOE_E_INVAL;
  launch_w4_grad(a, *d, l, p, s);
  if (need) launch_sum(a, d->dtype, d->K, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // extern "C"
