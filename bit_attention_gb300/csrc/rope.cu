// rope.cu -- per-head norms of queries and keys with the position rotation in
// the same pass, and its backward: kernels and the C ABI of
// include/sage_rope.h.
//
// Both are bound by HBM: the forward reads and writes each element once (4
// bytes an element), the backward reads x and g and writes dx (6 bytes).  A
// row of D channels is held by D / 8 lanes, 16 bytes each; the norm's sum goes
// through shuffles among them, and so does the half layout's partner chunk
// (rot is a multiple of 16, so a chunk's partners are one whole chunk).
// A warp takes kH times 2 (D = 128) or 4 neighbouring heads of one token, 512
// consecutive bytes an instruction: the token's cos and sin, four times a
// chunk's bytes, are loaded once into registers and serve all of them, and the
// kH loads are in flight together.  (A warp that goes on with its token's heads,
// the next ones' loads in flight, was slower: 96 registers instead of 64 leave
// 20 warps an SM.)
// 16384 tokens of 32 + 8 heads of 128: forward 59 us, 5.8 TB/s; 8192 tokens of 16 +
// 16 heads: backward 41 us, 4.9 TB/s (128 registers leave it 16 warps an SM, which
// issue in 54% of cycles).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/sage_rope.h"
#include "host.h"
#include "ptx.cuh"

namespace sagefp4 {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kBwdThreads = 256, kBwdBlocks = 2;  // resident an SM
constexpr unsigned kAll = 0xffffffffu;

struct RopeSide {     // q or k
  const uint16_t* x;  // forward: input; backward: the forward's input (norm = 1)
  const uint16_t* g;  // backward: gradient of y
  uint16_t* y;        // forward: y; backward: dx
  Strides sx, sg, sy;
  const void* w;
  float* partial;     // backward: [blocks][D]
  int H, segs;        // heads, segments of heads (kH rows a lane group each)
};

struct RopeParams {
  RopeSide side[2];
  const int32_t* pos;
  const float* cs;
  int32_t* status;
  long long pos_b;
  int tokens, N, max_pos, rot, norm, wf32;
  int blocks0;  // backward: the blocks below take q, the others k
  float eps;
};

// Eight channels as four FP32 pairs: the arithmetic below is on pairs, half the
// instructions (the forward would otherwise be bound by them and not by HBM).
struct Eight {
  uint64_t v[4];
};
__device__ __forceinline__ uint64_t unpack_bf(uint32_t w) {
  return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ Eight unpack8(const uint4& u) {
  return Eight{{unpack_bf(u.x), unpack_bf(u.y), unpack_bf(u.z), unpack_bf(u.w)}};
}
__device__ __forceinline__ uint32_t pack_bf(uint64_t v) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi2(v)), "f"(lo2(v)));
  return r;
}
__device__ __forceinline__ uint4 pack8(const Eight& f) {
  return uint4{pack_bf(f.v[0]), pack_bf(f.v[1]), pack_bf(f.v[2]), pack_bf(f.v[3])};
}
__device__ __forceinline__ Eight load8(const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  return Eight{{pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w)}};
}
__device__ __forceinline__ Eight load_weight(const void* w, int f32, int d) {
  return f32 ? load8(static_cast<const float*>(w) + d)
             : unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + d));
}
__device__ __forceinline__ Eight mul8(const Eight& a, const Eight& b) {
  return Eight{{mul2(a.v[0], b.v[0]), mul2(a.v[1], b.v[1]), mul2(a.v[2], b.v[2]), mul2(a.v[3], b.v[3])}};
}
__device__ __forceinline__ Eight mul8(const Eight& a, float f) {
  const uint64_t g = pack2(f, f);
  return mul8(a, Eight{{g, g, g, g}});
}
__device__ __forceinline__ Eight fma8(const Eight& a, const Eight& b, const Eight& c) {
  return Eight{{fma2(a.v[0], b.v[0], c.v[0]), fma2(a.v[1], b.v[1], c.v[1]), fma2(a.v[2], b.v[2], c.v[2]),
                fma2(a.v[3], b.v[3], c.v[3])}};
}
__device__ __forceinline__ float dot8(const Eight& a, const Eight& b) {
  const uint64_t s = fma2(a.v[0], b.v[0], mul2(a.v[1], b.v[1])), t = fma2(a.v[2], b.v[2], mul2(a.v[3], b.v[3]));
  const uint64_t u = add2(s, t);
  return lo2(u) + hi2(u);
}

// Sum over the kC lanes of a row's group.
template <int kC>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = kC / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The lane's share of its token's rotation: y = x c + o s, where o are the
// partners of its eight channels, in lane `partner` (half layout) or their
// neighbours (interleaved), and s has the sign that belongs to the channel.
// Lanes past the rotated channels keep c = 1, s = 0.  (By the opposite angle:
// x c - o s.)
struct Angles {
  Eight c, s;
  int partner;
};

template <bool kInter>
__device__ __forceinline__ void load_angles(Angles& a, const float* row, int lane, int rot) {
  a.partner = lane;
#pragma unroll
  for (int e = 0; e < 4; e++) a.c.v[e] = pack2(1.0f, 1.0f), a.s.v[e] = 0;
  if (8 * lane >= rot) return;
  if constexpr (kInter) {
    const float4 c = *reinterpret_cast<const float4*>(row + 4 * lane);
    const float4 s = *reinterpret_cast<const float4*>(row + rot / 2 + 4 * lane);
    a.c = Eight{{pack2(c.x, c.x), pack2(c.y, c.y), pack2(c.z, c.z), pack2(c.w, c.w)}};
    a.s = Eight{{pack2(-s.x, s.x), pack2(-s.y, s.y), pack2(-s.z, s.z), pack2(-s.w, s.w)}};
  } else {
    const int half = rot / 16, at = 8 * (lane < half ? lane : lane - half);
    a.partner = lane < half ? lane + half : lane - half;
    a.c = load8(row + at);
    a.s = load8(row + rot / 2 + at);
    if (lane < half) a.s = mul8(a.s, -1.0f);
  }
}

// The partners of a lane's channels.
template <bool kInter, int kC>
__device__ __forceinline__ uint4 partners(const uint4& u, const Angles& a) {
  if constexpr (kInter)
    return uint4{__byte_perm(u.x, 0, 0x1032), __byte_perm(u.y, 0, 0x1032), __byte_perm(u.z, 0, 0x1032),
                 __byte_perm(u.w, 0, 0x1032)};
  else
    return uint4{__shfl_sync(kAll, u.x, a.partner, kC), __shfl_sync(kAll, u.y, a.partner, kC),
                 __shfl_sync(kAll, u.z, a.partner, kC), __shfl_sync(kAll, u.w, a.partner, kC)};
}

// The table row of position `at`, or NULL (recorded) for one outside the table.
__device__ __forceinline__ const float* table_row(const RopeParams& p, int at) {
  if (at >= 0 && at < p.max_pos) return p.cs + static_cast<long long>(at) * p.rot;
  atomicCAS(p.status, 0, SAGE_FP4_EINDEX);
  return nullptr;
}

// kH rows of a lane group, heads h0 + i * kG; zeros past the last head.
template <int kG, int kH>
__device__ __forceinline__ void load_rows(uint4 (&raw)[kH], const uint16_t* x, long long stride, int h0, int H) {
#pragma unroll
  for (int i = 0; i < kH; i++)
    raw[i] = h0 + i * kG < H ? *reinterpret_cast<const uint4*>(x + (h0 + i * kG) * stride) : uint4{0, 0, 0, 0};
}

// Grid (blocks of one token a warp, q's and k's head segments).
template <int D, bool kInter, int kH>
__global__ void __launch_bounds__(kRopeThreads) rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kC = D / 8, kG = 32 / kC;
  const int lane = threadIdx.x % kC, grp = (threadIdx.x & 31) / kC;
  const int token = blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32, seg = blockIdx.y;
  if (static_cast<unsigned>(token) >= static_cast<unsigned>(p.tokens)) return;  // the whole warp; unsigned: past 2^31 too
  const int b = p.N == p.tokens ? 0 : token / p.N, n = token - b * p.N;
  const int at = p.pos[b * p.pos_b + n];
  const bool isk = seg >= p.side[0].segs;
  const RopeSide& S = p.side[isk];
  const int h0 = (seg - (isk ? p.side[0].segs : 0)) * (kH * kG) + grp;
  uint4 raw[kH];
  load_rows<kG, kH>(raw, S.x + b * S.sx.b + n * S.sx.n + 8 * lane, S.sx.h, h0, S.H);
  const float* row = table_row(p, at);
  Angles a;
  load_angles<kInter>(a, row, lane, row ? p.rot : 0);
  if (p.norm) {
    // the weights go into the angles: y = r (x (c w) + o (s w of the partner))
    const Eight w = load_weight(S.w, p.wf32, 8 * lane);
    Eight wo = kInter ? w : load_weight(S.w, p.wf32, 8 * a.partner);
    if constexpr (kInter) {
#pragma unroll
      for (int e = 0; e < 4; e++) wo.v[e] = pack2(hi2(w.v[e]), lo2(w.v[e]));
    }
    a.c = mul8(a.c, w);
    a.s = mul8(a.s, wo);
  }
  uint16_t* y = S.y + b * S.sy.b + n * S.sy.n + 8 * lane;
#pragma unroll
  for (int i = 0; i < kH; i++) {
    const Eight f = unpack8(raw[i]), o = unpack8(partners<kInter, kC>(raw[i], a));
    Eight z = fma8(o, a.s, mul8(f, a.c));
    if (p.norm) z = mul8(z, rsqrtf(group_sum<kC>(dot8(f, f)) * (1.0f / D) + p.eps));
    if (h0 + i * kG < S.H) *reinterpret_cast<uint4*>(y + (h0 + i * kG) * S.sy.h) = row ? pack8(z) : uint4{0, 0, 0, 0};
  }
}

// Grid of blocks0 blocks for q, then the blocks for k; a warp strides over
// (token, head segment) units of its side and keeps its share of dw in
// registers; the block's sum goes to its row of `partial`.
template <int D, bool kInter, bool kNorm, int kH>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocks) rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kC = D / 8, kG = 32 / kC, kGroups = kBwdThreads / kC, kWarps = kBwdThreads / 32;
  const bool isk = static_cast<int>(blockIdx.x) >= p.blocks0;
  const RopeSide& S = p.side[isk];
  const int block = blockIdx.x - (isk ? p.blocks0 : 0);
  const int blocks = isk ? gridDim.x - p.blocks0 : p.blocks0;
  const int lane = threadIdx.x % kC, grp = (threadIdx.x & 31) / kC;
  const int stride = blocks * kWarps, dtoken = stride / S.segs, dseg = stride - dtoken * S.segs;
  Eight w, dw{};
  if (kNorm) w = load_weight(S.w, p.wf32, 8 * lane);
  int token = (block * kWarps + static_cast<int>(threadIdx.x) / 32) / S.segs;
  int seg = block * kWarps + static_cast<int>(threadIdx.x) / 32 - token * S.segs;
  for (; token < p.tokens && token >= 0; token += dtoken + (seg + dseg >= S.segs), seg += dseg - (seg + dseg >= S.segs ? S.segs : 0)) {
    const int h0 = seg * (kH * kG) + grp;
    const int b = p.N == p.tokens ? 0 : token / p.N, n = token - b * p.N;
    const int at = p.pos[b * p.pos_b + n];
    uint4 rx[kH], rg[kH];
    load_rows<kG, kH>(rg, S.g + b * S.sg.b + n * S.sg.n + 8 * lane, S.sg.h, h0, S.H);
    if (kNorm) load_rows<kG, kH>(rx, S.x + b * S.sx.b + n * S.sx.n + 8 * lane, S.sx.h, h0, S.H);
    const float* row = table_row(p, at);
    Angles a;
    load_angles<kInter>(a, row, lane, row ? p.rot : 0);
    a.s = mul8(a.s, -1.0f);  // back
    if (!row) {  // left out: nothing for dw
#pragma unroll
      for (int i = 0; i < kH; i++) rg[i] = uint4{0, 0, 0, 0};
    }
    uint16_t* dx = S.y + b * S.sy.b + n * S.sy.n + 8 * lane;
#pragma unroll
    for (int i = 0; i < kH; i++) {
      // the gradient of n
      Eight f = fma8(unpack8(partners<kInter, kC>(rg[i], a)), a.s, mul8(unpack8(rg[i]), a.c));
      if (kNorm) {
        const Eight v = unpack8(rx[i]), fv = mul8(f, v);
        // rows that are not there or are left out: r of zeros would be infinite for eps = 0, and dw NaN
        const float ms = group_sum<kC>(dot8(v, v)) * (1.0f / D) + p.eps;
        const float r = row && h0 + i * kG < S.H ? rsqrtf(ms) : 0.0f;
        const float c = group_sum<kC>(dot8(fv, w)) * (1.0f / D) * r * r;  // mean(g' w xh) r
        const uint64_t r2 = pack2(r, r), m2 = pack2(-c * r, -c * r);
        dw = fma8(fv, Eight{{r2, r2, r2, r2}}, dw);
        f = fma8(v, Eight{{m2, m2, m2, m2}}, mul8(mul8(f, w), r));  // r (g' w - x c)
      }
      if (h0 + i * kG < S.H) *reinterpret_cast<uint4*>(dx + (h0 + i * kG) * S.sy.h) = row ? pack8(f) : uint4{0, 0, 0, 0};
    }
  }
  if (kNorm) {
    __shared__ float sum[kGroups][D + 4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      sum[threadIdx.x / kC][8 * lane + 2 * e] = lo2(dw.v[e]);
      sum[threadIdx.x / kC][8 * lane + 2 * e + 1] = hi2(dw.v[e]);
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < kGroups; j++) t += sum[j][threadIdx.x];
      S.partial[static_cast<size_t>(block) * D + threadIdx.x] = t;
    }
  }
}

// The blocks' partial sums of dw, in their order: grid (D / 16, q and k),
// thread (column, share of the blocks).
template <int D>
__global__ void __launch_bounds__(256) rope_dw_kernel(const float* pq, int nq, float* dwq, const float* pk, int nk,
                                                      float* dwk) {
  const float* part = blockIdx.y ? pk : pq;
  const int n = blockIdx.y ? nk : nq, col = blockIdx.x * 16 + threadIdx.x % 16, share = threadIdx.x / 16;
  float t = 0.0f;
#pragma unroll 8
  for (int i = share; i < n; i += 16) t += part[static_cast<size_t>(i) * D + col];
  __shared__ float sum[16][17];
  sum[share][threadIdx.x % 16] = t;
  __syncthreads();
  if (share == 0) {
    t = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; j++) t += sum[j][threadIdx.x];
    (blockIdx.y ? dwk : dwq)[col] = t;
  }
}

constexpr int kFwdHeads = 4, kBwdHeads = 4;  // rows of a lane group at a time
constexpr int kMaxBwdBlocks = 1024;          // rows of `partial` for each of q and k

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

bool desc_ok(const sage_rope_desc* d) {
  if (!d || d->B < 0 || d->N < 0 || d->Hq < 0 || d->Hk < 0) return false;
  if (d->D != 64 && d->D != 128) return false;
  if (d->rot < 16 || d->rot > d->D || d->rot % 16) return false;
  if ((d->interleaved | d->norm | d->weight_f32) & ~1) return false;
  if (d->max_pos < 0 || !(d->eps >= 0.0f) || !isfinite(d->eps)) return false;
  if (static_cast<long long>(d->B) * d->N > INT32_MAX) return false;
  if (d->Hq > 65535 || d->Hk > 65535) return false;
  if (d->pos_b_stride < 0 || (d->B > 1 && d->pos_b_stride > (int64_t(1) << 60) / d->B)) return false;
  return true;
}

bool pointers_ok(const sage_rope_desc* d) {
  if (!is_aligned(d->positions, 4) || !is_aligned(d->cos_sin, 16) || !is_aligned(d->status, 4)) return false;
  return !d->norm || (is_aligned(d->q_weight, 16) && is_aligned(d->k_weight, 16));
}

bool strides_or_dense(const sage_fp4_strides* in, const sage_rope_desc* d, int H, Strides* out) {
  const int64_t D = d->D;
  const sage_fp4_strides dense = {int64_t(d->N) * H * D, D, int64_t(H) * D};
  return take_strides(in ? *in : dense, d->B, H, d->N, D, out);
}

void fill(RopeParams& p, const sage_rope_desc* d, int heads) {
  p.pos = d->positions;
  p.cs = d->cos_sin;
  p.status = d->status;
  p.pos_b = d->pos_b_stride;
  p.tokens = d->B * d->N;
  p.N = d->N;
  p.max_pos = d->max_pos;
  p.rot = d->rot;
  p.norm = d->norm;
  p.wf32 = d->weight_f32;
  p.eps = d->eps;
  p.side[0].H = d->Hq;
  p.side[1].H = d->Hk;
  p.side[0].w = d->q_weight;
  p.side[1].w = d->k_weight;
  for (RopeSide& s : p.side) s.segs = ceil_div(s.H, heads * (256 / d->D));
}

template <int D, int kH>
void fwd_launch(const RopeParams& p, int inter, cudaStream_t st) {
  const dim3 grid(ceil_div(p.tokens, kRopeThreads / 32), p.side[0].segs + p.side[1].segs);
  if (inter)
    rope_fwd_kernel<D, true, kH><<<grid, kRopeThreads, 0, st>>>(p);
  else
    rope_fwd_kernel<D, false, kH><<<grid, kRopeThreads, 0, st>>>(p);
}

template <int D>
void bwd_launch(const RopeParams& p, int inter, int blocks, cudaStream_t st) {
  if (inter) {
    if (p.norm)
      rope_bwd_kernel<D, true, true, kBwdHeads><<<blocks, kBwdThreads, 0, st>>>(p);
    else
      rope_bwd_kernel<D, true, false, kBwdHeads><<<blocks, kBwdThreads, 0, st>>>(p);
  } else {
    if (p.norm)
      rope_bwd_kernel<D, false, true, kBwdHeads><<<blocks, kBwdThreads, 0, st>>>(p);
    else
      rope_bwd_kernel<D, false, false, kBwdHeads><<<blocks, kBwdThreads, 0, st>>>(p);
  }
}

size_t rope_ws_bytes(const sage_rope_desc* d) {
  return d->norm ? 2 * size_t(kMaxBwdBlocks) * d->D * sizeof(float) : 256;
}

}  // namespace
}  // namespace sagefp4

using namespace sagefp4;

extern "C" {

int sage_rope_fwd(const sage_rope_desc* desc, const void* q, const sage_fp4_strides* q_strides, const void* k,
                  const sage_fp4_strides* k_strides, void* q_out, const sage_fp4_strides* q_out_strides, void* k_out,
                  const sage_fp4_strides* k_out_strides, void* stream) {
  if (!desc_ok(desc)) return SAGE_FP4_EINVAL;
  const long long rows = static_cast<long long>(desc->B) * desc->N * (static_cast<long long>(desc->Hq) + desc->Hk);
  if (rows == 0) return SAGE_FP4_OK;
  if (!pointers_ok(desc)) return SAGE_FP4_EINVAL;
  RopeParams p = {};
  if (!strides_or_dense(q_strides, desc, desc->Hq, &p.side[0].sx) ||
      !strides_or_dense(k_strides, desc, desc->Hk, &p.side[1].sx) ||
      !strides_or_dense(q_out_strides, desc, desc->Hq, &p.side[0].sy) ||
      !strides_or_dense(k_out_strides, desc, desc->Hk, &p.side[1].sy))
    return SAGE_FP4_EINVAL;
  if (desc->Hq && (!is_aligned(q, 16) || !is_aligned(q_out, 16))) return SAGE_FP4_EINVAL;
  if (desc->Hk && (!is_aligned(k, 16) || !is_aligned(k_out, 16))) return SAGE_FP4_EINVAL;
  int sms = 0;
  if (const int rc = check_device_103(&sms)) return rc;
  // One head a lane group where the rows are too few to fill the card one head
  // deep: the pass is then a chain of latencies, and shorter (32 + 8 heads of 128,
  // one and four heads deep: 8 tokens 7.3 and 9.3 us, 256 both 9.3, 1024 15.5 and
  // 13.4, 2048 23.7 and 15.5).
  const bool few = rows * (desc->D / 8) < static_cast<long long>(sms) * 2048;
  fill(p, desc, few ? 1 : kFwdHeads);
  p.side[0].x = static_cast<const uint16_t*>(q);
  p.side[1].x = static_cast<const uint16_t*>(k);
  p.side[0].y = static_cast<uint16_t*>(q_out);
  p.side[1].y = static_cast<uint16_t*>(k_out);
  if (p.side[0].segs + p.side[1].segs > 65535) return SAGE_FP4_EINVAL;  // rows of the launch's grid
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (desc->D == 64)
    few ? fwd_launch<64, 1>(p, desc->interleaved, st) : fwd_launch<64, kFwdHeads>(p, desc->interleaved, st);
  else
    few ? fwd_launch<128, 1>(p, desc->interleaved, st) : fwd_launch<128, kFwdHeads>(p, desc->interleaved, st);
  return launched(cudaGetLastError());
}

size_t sage_rope_workspace_bytes(const sage_rope_desc* desc) { return desc_ok(desc) ? rope_ws_bytes(desc) : 0; }

int sage_rope_bwd(const sage_rope_desc* desc, const void* gq, const sage_fp4_strides* gq_strides, const void* gk,
                  const sage_fp4_strides* gk_strides, const void* q, const sage_fp4_strides* q_strides, const void* k,
                  const sage_fp4_strides* k_strides, void* dq, const sage_fp4_strides* dq_strides, void* dk,
                  const sage_fp4_strides* dk_strides, float* dq_weight, float* dk_weight, void* workspace,
                  size_t workspace_bytes, void* stream) {
  if (!desc_ok(desc)) return SAGE_FP4_EINVAL;
  if (desc->norm && (!is_aligned(dq_weight, 4) || !is_aligned(dk_weight, 4))) return SAGE_FP4_EINVAL;
  const long long tokens = static_cast<long long>(desc->B) * desc->N;
  const long long rows = tokens * (static_cast<long long>(desc->Hq) + desc->Hk);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int sms = 0;
  RopeParams p = {};
  if (rows) {
    if (!pointers_ok(desc) || !is_aligned(workspace, 256) || workspace_bytes < rope_ws_bytes(desc))
      return SAGE_FP4_EINVAL;
    const sage_fp4_strides* st6[6] = {gq_strides, gk_strides, q_strides, k_strides, dq_strides, dk_strides};
    Strides* to6[6] = {&p.side[0].sg, &p.side[1].sg, &p.side[0].sx, &p.side[1].sx, &p.side[0].sy, &p.side[1].sy};
    for (int i = 0; i < 6; i++)
      if (!strides_or_dense(st6[i], desc, i % 2 ? desc->Hk : desc->Hq, to6[i])) return SAGE_FP4_EINVAL;
    if (desc->Hq && (!is_aligned(gq, 16) || !is_aligned(dq, 16) || (desc->norm && !is_aligned(q, 16))))
      return SAGE_FP4_EINVAL;
    if (desc->Hk && (!is_aligned(gk, 16) || !is_aligned(dk, 16) || (desc->norm && !is_aligned(k, 16))))
      return SAGE_FP4_EINVAL;
  }
  if (const int rc = check_device_103(&sms)) return rc;
  if (!rows) {
    if (!desc->norm) return SAGE_FP4_OK;
    if (cudaMemsetAsync(dq_weight, 0, desc->D * sizeof(float), st) != cudaSuccess ||
        cudaMemsetAsync(dk_weight, 0, desc->D * sizeof(float), st) != cudaSuccess)
      return SAGE_FP4_ECUDA;
    return SAGE_FP4_OK;
  }
  fill(p, desc, kBwdHeads);
  p.side[0].g = static_cast<const uint16_t*>(gq);
  p.side[1].g = static_cast<const uint16_t*>(gk);
  p.side[0].x = static_cast<const uint16_t*>(q);
  p.side[1].x = static_cast<const uint16_t*>(k);
  p.side[0].y = static_cast<uint16_t*>(dq);
  p.side[1].y = static_cast<uint16_t*>(dk);
  p.side[0].partial = static_cast<float*>(workspace);
  p.side[1].partial = p.side[0].partial + size_t(kMaxBwdBlocks) * desc->D;
  // Blocks in proportion to the sides' units, as many as are resident in all,
  // one at least each.
  const int warps = kBwdThreads / 32;
  const long long nq0 = (tokens * p.side[0].segs + warps - 1) / warps, nk0 = (tokens * p.side[1].segs + warps - 1) / warps;
  const long long cap = kBwdBlocks * sms < kMaxBwdBlocks ? kBwdBlocks * sms : kMaxBwdBlocks;
  long long nq = nq0, nk = nk0;
  if (nq + nk > cap) {
    nq = cap * nq0 / (nq0 + nk0);
    nk = cap - nq;
    if (nq0 && !nq) nq = 1;
    if (nk0 && !nk) nk = 1;
  }
  p.blocks0 = static_cast<int>(nq);
  const int blocks = static_cast<int>(nq + nk);
  if (desc->D == 64)
    bwd_launch<64>(p, desc->interleaved, blocks, st);
  else
    bwd_launch<128>(p, desc->interleaved, blocks, st);
  if (desc->norm) {
    const dim3 grid(desc->D / 16, 2);
    if (desc->D == 64)
      rope_dw_kernel<64><<<grid, 256, 0, st>>>(p.side[0].partial, static_cast<int>(nq), dq_weight, p.side[1].partial,
                                               static_cast<int>(nk), dk_weight);
    else
      rope_dw_kernel<128><<<grid, 256, 0, st>>>(p.side[0].partial, static_cast<int>(nq), dq_weight, p.side[1].partial,
                                                static_cast<int>(nk), dk_weight);
  }
  return launched(cudaGetLastError());
}

int sage_rope_get_status(int32_t* status, void* stream) { return read_status(status, stream); }

}  // extern "C"
