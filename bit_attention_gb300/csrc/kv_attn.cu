// kv_attn.cu -- attention of new tokens over the paged cache: the C ABI
// (include/sage_kv.h), the plan of a call's work and the join of partial
// results (kv_attn.cuh describes both).
#include "kv_attn.cuh"
#include "layout.cuh"

namespace sagefp4 {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint64_t kWaitNs = 1500ull * 1000ull * 1000ull;  // bounded waits: 1.5 s
constexpr int kPlanThreads = 512;

// Sum of v over the threads before this one, and over all of them (*total).
__device__ __forceinline__ long long block_scan(long long v, long long* warps, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(kAll, s, o);
    if (lane >= o) s += x;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = s;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 32; i++) {
    const long long x = warps[i];
    if (i < warp) before += x;
    all += x;
  }
  *total = all;
  return before + s - v;
}

// The entries of a call, in the order of the sequences: one block.  A few
// hundred sequences or entries are one round each.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ KvView c,
                                                            const __grid_constant__ AttnArgs a,
                                                            const __grid_constant__ AttnWork w, int rows) {
  griddep_launch_dependents();
  __shared__ long long warps[kPlanThreads / 32];
  __shared__ int4 seq[kPlanThreads];  // q0, nq, len, first entry of this round's sequences
  long long units = 0, base = 0;
  for (int b0 = 0; b0 < c.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int4 s{0, 0, 0, 0};
    if (b < c.B) {
      const int2 r = seq_rows(c, b, a.T);
      s = int4{r.x, r.y - r.x, seq_len(c, b), 0};
    }
    long long entries, at = block_scan((static_cast<long long>(s.y) * a.G + rows - 1) / rows, warps, &entries);
    s.w = static_cast<int>(at);
    seq[threadIdx.x] = s;
    __syncthreads();
    for (int j0 = 0; j0 < entries; j0 += kPlanThreads) {
      const int j = j0 + threadIdx.x;
      PlanEntry e{};
      if (j < entries) {
        int lo = 0, hi = kPlanThreads;  // the last sequence whose first entry is <= j
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (seq[mid].w <= j)
            lo = mid;
          else
            hi = mid;
        }
        // of several with that first entry, all but the last are empty
        const int4 q = seq[lo];
        e = make_entry(a, rows, q.x, q.y, q.z, b0 + lo, (j - q.w) * rows);
      }
      long long sum;
      const long long cum = units + block_scan(j < entries ? e.tiles + w.lead_units : 0, warps, &sum);
      if (j < entries && base + j < w.capacity) {
        w.entry[base + j] = e;
        w.cum[base + j] = cum;
      }
      // bounds that overlap could ask for more entries than rows exist
      if (base + j0 + kPlanThreads <= w.capacity || base + entries <= w.capacity) {
        units += sum;
      } else {
        flag_index(c.status);
        units = 0;
        base = w.capacity;
        b0 = c.B;
        break;
      }
    }
    base += entries;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    w.head->units = units;
    w.head->entries = units ? static_cast<int>(base) : 0;
  }
}

__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// The same for a call of at most 32 entries (and so sequences), by one warp
// without a barrier: calls of a few rows wait for little else.  One token of one
// sequence over 4097: 2.8 us, with plan_kernel 3.8.
constexpr int kFew = 32;
__global__ void __launch_bounds__(32) plan_few_kernel(const __grid_constant__ KvView c, const __grid_constant__ AttnArgs a,
                                                      const __grid_constant__ AttnWork w, int rows) {
  griddep_launch_dependents();
  const int lane = threadIdx.x;
  int q0 = 0, nq = 0, len = 0;
  if (lane < c.B) {
    const int2 r = seq_rows(c, lane, a.T);
    q0 = r.x, nq = r.y - r.x, len = seq_len(c, lane);
  }
  // a sequence has at most capacity entries, so that the sums stay small
  const int mine = static_cast<int>((static_cast<long long>(nq) * a.G + rows - 1) / rows);
  const int end = warp_scan(mine), entries = __shfl_sync(kAll, end, 31);
  int b = 0;  // the sequence of entry `lane`: the number of those that end at or before it
  for (int i = 0; i < c.B; i++) b += __shfl_sync(kAll, end, i) <= lane;
  const int first = __shfl_sync(kAll, end - mine, b & 31);
  q0 = __shfl_sync(kAll, q0, b & 31);
  nq = __shfl_sync(kAll, nq, b & 31);
  len = __shfl_sync(kAll, len, b & 31);
  // bounds that overlap could ask for more entries than rows exist
  const bool fits = entries <= w.capacity;
  PlanEntry e{};
  if (fits && lane < entries) e = make_entry(a, rows, q0, nq, len, b, (lane - first) * rows);
  const int cost = fits && lane < entries ? e.tiles + w.lead_units : 0, sum = warp_scan(cost);
  if (fits && lane < entries) {
    w.entry[lane] = e;
    w.cum[lane] = sum - cost;
  }
  if (lane == 31) {
    if (!fits) flag_index(c.status);
    w.head->units = sum;
    w.head->entries = fits ? entries : 0;
  }
}

// An entry's partial results (step kernel): of the workers [w0, w1]; none to
// join where it lies in one share.
struct Parts {
  long long w0, w1;
  __device__ __forceinline__ Parts(const AttnWork& w, int heads, int h, int j) {
    const long long units = w.head->units, share = share_of(units * heads, w.workers, w.min_share);
    const long long start = units * h + w.cum[j];
    // a border within the lead units or at the first tile has moved to the start
    w0 = (start + w.lead_units) / share;
    w1 = (start + w.lead_units + w.entry[j].tiles - 1) / share;
  }
  // the first one's piece began the entry, the others' did not
  __device__ __forceinline__ size_t slot(long long i) const { return 2 * static_cast<size_t>(i) + (i == w0); }
};

__device__ __forceinline__ void write_row(const AttnArgs& a, const PlanEntry& e, int h, int r, int d4, const float4& v,
                                          float m, float l) {
  const int rr = e.row0 + r, i = rr / a.G, hq = h * a.G + rr - i * a.G;
  const long long tok = e.q0 + i;
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  *reinterpret_cast<uint2*>(a.o + tok * a.orow.t + hq * a.orow.h + 4 * d4) = uint2{bf2(v.x * inv, v.y * inv), bf2(v.z * inv, v.w * inv)};
  if (a.lse && d4 == 0) a.lse[tok * a.Hq + hq] = l > 0.0f ? (m + lg2_approx(l)) * kLn2 : -INFINITY;
}

__device__ __forceinline__ void add_scaled(float4& acc, const float4& v, float f) {
  acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y), acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
}

// Chunk kernel's partials: grid (worker whose share may begin an entry that
// others go on with, 32 rows).  A lane has one row, a warp D / 32 neighbouring
// 4-channel columns.  An entry has few parts here, and the time is that of the loads that
// wait on one another: the worker's own note of the entry saves a search through
// the plan (8192-token prompt, 37 MB of parts: 10.6 us; with the search 17).
template <int D>
__global__ void __launch_bounds__(256) combine_chunk_kernel(const __grid_constant__ KvView c,
                                                            const __grid_constant__ AttnArgs a,
                                                            const __grid_constant__ AttnWork w) {
  griddep_wait();
  const int w0 = blockIdx.x;
  const int2 at = w.open[w0];  // entry, head
  const long long units = w.head->units;
  if (units == 0 || at.x < 0) return;
  const PlanEntry e = w.entry[at.x];
  // the last of its tiles lies `past` units behind the border of w0's share
  const long long share = share_of(units * c.H, w.workers, w.min_share);
  const long long past = units * at.y + w.cum[at.x] + w.lead_units + e.tiles - 1 - share * (w0 + 1);
  const int w1 = w0 + 1 + (past < share ? 0 : static_cast<int>(past / share));
  const int r = blockIdx.y * 32 + (threadIdx.x & 31), d0 = threadIdx.x >> 5;
  if (r >= min(e.nq * a.G - e.row0, kChunkRows)) return;
  // the first one's piece began the entry, the others' did not
  auto slot = [&](int i) { return 2 * static_cast<size_t>(i) + (i == w0); };
  constexpr int kN = D / 4 / 8;
  float m = -INFINITY, l = 0.0f;
  float4 acc[kN] = {};
#pragma unroll 2
  for (int i = w0; i <= w1; i++) {
    const float2 ml = w.part_ml[slot(i) * kChunkRows + r];
    const float4* o = reinterpret_cast<const float4*>(w.part_o) + slot(i) * (D / 4) * kChunkRows + r;
    float4 v[kN];
#pragma unroll
    for (int k = 0; k < kN; k++) v[k] = o[static_cast<size_t>(d0 * kN + k) * kChunkRows];
    // in two steps each: over E4M3 what a part is relative to counts V's scale, and its
    // sum makes up for that, so that a factor may be below FP32 where the product is not
    const float mn = fmaxf(m, ml.x), sub = mn == -INFINITY ? 0.0f : mn;
    const float h0 = ex2_approx(0.5f * (m - sub)), h1 = ex2_approx(0.5f * (ml.x - sub)), f0 = h0 * h0, f1 = h1 * h1;
    l = l * h0 * h0 + ml.y * h1 * h1;
#pragma unroll
    for (int k = 0; k < kN; k++) {
      acc[k] = float4{acc[k].x * f0, acc[k].y * f0, acc[k].z * f0, acc[k].w * f0};
      add_scaled(acc[k], v[k], f1);
    }
    m = mn;
  }
  const int rr = e.row0 + r, q = rr / a.G, hq = at.y * a.G + rr - q * a.G;
  const long long tok = e.q0 + q;
  uint16_t* out = a.o + tok * a.orow.t + hq * a.orow.h + 4 * kN * d0;
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int k = 0; k < kN; k += 2)
    *reinterpret_cast<uint4*>(out + 4 * k) = uint4{bf2(acc[k].x * inv, acc[k].y * inv), bf2(acc[k].z * inv, acc[k].w * inv),
                                                  bf2(acc[k + 1].x * inv, acc[k + 1].y * inv),
                                                  bf2(acc[k + 1].z * inv, acc[k + 1].w * inv)};
  if (a.lse && d0 == 0) a.lse[tok * a.Hq + hq] = l > 0.0f ? (m + lg2_approx(l)) * kLn2 : -INFINITY;
}

// Step kernel's partials: grid (entry, head, 256 / kSplit consecutive
// 4-channel columns of the rows); a lane has one column, and kSplit warps share
// out the parts.
template <int D, int kSplit>
__global__ void __launch_bounds__(256) combine_step_kernel(const __grid_constant__ KvView c,
                                                           const __grid_constant__ AttnArgs a,
                                                           const __grid_constant__ AttnWork w, int rows) {
  griddep_wait();
  const int j = blockIdx.x, h = blockIdx.y;
  if (j >= w.head->entries) return;
  const Parts parts(w, c.H, h, j);
  if (parts.w0 == parts.w1) return;
  const PlanEntry e = w.entry[j];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = warp % kSplit;
  const int at = (blockIdx.z * (8 / kSplit) + warp / kSplit) * 32 + lane, r = at / (D / 4), d4 = at % (D / 4);
  const bool live = r < min(e.nq * a.G - e.row0, rows);
  float m = -INFINITY, l = 0.0f;
  float4 acc{};
  if (live) {
#pragma unroll 4
    for (long long i = parts.w0 + share; i <= parts.w1; i += kSplit) {
      const float2 ml = w.part_ml[parts.slot(i) * rows + r];
      const float4 o = reinterpret_cast<const float4*>(w.part_o)[parts.slot(i) * rows * (D / 4) + at];
      const float mn = fmaxf(m, ml.x), sub = mn == -INFINITY ? 0.0f : mn;
      const float f0 = ex2_approx(m - sub), f1 = ex2_approx(ml.x - sub);
      l = l * f0 + ml.y * f1;
      acc = float4{acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0};
      add_scaled(acc, o, f1);
      m = mn;
    }
  }
  if constexpr (kSplit > 1) {
    __shared__ float4 so[8][32];
    __shared__ float2 sml[8][32];
    so[warp][lane] = acc;
    sml[warp][lane] = float2{m, l};
    __syncthreads();
    if (share != 0) return;
#pragma unroll
    for (int i = 1; i < kSplit; i++) m = fmaxf(m, sml[warp + i][lane].x);
    l = 0.0f;
    acc = float4{};
#pragma unroll
    for (int i = 0; i < kSplit; i++) {
      const float2 ml = sml[warp + i][lane];
      const float f = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - m);
      l = fmaf(ml.y, f, l);
      add_scaled(acc, so[warp + i][lane], f);
    }
  }
  if (live) write_row(a, e, h, r, d4, acc, m, l);
}

// How a call of these sizes runs and the workspace's parts.
//
// A sequence's query rows for one key/value head are G times its new tokens.
// Where they are few on average, the step kernel reads the cache at HBM's rate
// and its tiles of 8 or 16 rows waste little; above that the chunk kernel's tiles
// of 128 rows cost one pass instead of several.  Two passes are still cheaper over
// a quantized cache, whose conversion holds the chunk kernel up.  32 sequences of
// 4096 tokens, 8 key/value heads of 128, step and chunk kernel:
//   rows    bf16         E4M3         NVFP4
//   16      118, 122 us  81, 134
//   32      196, 124     116, 134     105, 128
//   64      351, 124     198, 134
// Tiles of 8 rows leave registers for 12 warps an SM instead of 8: one token of 64
// sequences of 8192, NVFP4 142 us, with 16 rows 167; bf16 337 and 346.
struct Way {
  bool step;
  int rows;     // of an entry
  int workers, lead_units, min_share, capacity;
  size_t entry, cum, open, ml, o, total;
};
Way way_of(const sage_kv_cache* c, int B, int T, int Hq, int sms) {
  const int H = c->H, D = c->D;
  Way w;
  const long long G = Hq / H, avg = B > 0 ? T * G / B : 0;
  if (sms > kMaxSms) sms = kMaxSms;
  w.step = avg <= (c->format == SAGE_KV_BF16 ? 16 : 32);
  w.rows = !w.step ? kChunkRows : avg <= 8 ? 8 : 16;
  w.workers = !w.step ? sms : sms * (avg <= 8 ? 12 : 8);  // warps that fit by registers
  // Filling and draining the chunk kernel's pipeline and writing an entry out
  // take about as long as two tiles.
  w.lead_units = w.step ? 0 : 2;
  w.min_share = w.lead_units + (w.step ? 1 : 2);
  w.capacity = static_cast<int>(T * G / w.rows) + B;
  w.entry = 256;
  w.cum = w.entry + align256(size_t(w.capacity) * sizeof(PlanEntry));
  w.open = w.cum + align256(size_t(w.capacity) * sizeof(long long));
  w.ml = w.open + align256(w.step ? 0 : size_t(w.workers) * sizeof(int2));
  w.o = w.ml + align256(size_t(2) * w.workers * w.rows * sizeof(float2));
  w.total = w.o + size_t(2) * w.workers * w.rows * D * sizeof(float);
  return w;
}

template <int D>
cudaError_t launch_combine(const KvView& c, const AttnArgs& a, const AttnWork& work, const Way& w, int sms, cudaStream_t st) {
  if (!w.step && w.workers == 1) return cudaSuccess;
  if (!w.step) return launch_after(combine_chunk_kernel<D>, dim3(w.workers - 1, kChunkRows / 32), 256, 0, st, c, a, work);
  // A sequence and head lies in about workers / (capacity * heads) shares.  Where
  // that is a handful one thread joins them; a long sequence that is alone lies in
  // hundreds, which eight warps share out (one token in E4M3 with one and with
  // eight: over 131072, 155 and 81 us; 16 sequences of 4096, 50 and 46; 64 of 4096,
  // 120 and 126).
  const int columns = w.rows * (D / 4);
  if (static_cast<long long>(w.capacity) * c.H >= 2 * sms)
    return launch_after(combine_step_kernel<D, 1>, dim3(w.capacity, c.H, (columns + 255) / 256), 256, 0, st, c, a, work, w.rows);
  return launch_after(combine_step_kernel<D, 8>, dim3(w.capacity, c.H, columns / 32), 256, 0, st, c, a, work, w.rows);
}

bool sizes_ok(const sage_kv_cache* c, int B, int T, int Hq) {
  return cache_ok(c) && B >= 0 && T >= 0 && Hq >= 1 && Hq <= 65535 && Hq % c->H == 0 &&
         static_cast<long long>(T) * Hq <= INT32_MAX - kChunkRows;  // row numbers, a tile's end too, are ints
}

int attn(const sage_kv_cache* cache, const sage_kv_batch* batch, const void* q, sage_kv_rows q_rows, void* o,
         sage_kv_rows o_rows, float* lse, int T, int Hq, int causal, int window, float scale, void* workspace,
         size_t workspace_bytes, void* stream, uint64_t wait_ns, int withhold) {
  if (!batch_ok(batch, true) || !sizes_ok(cache, batch->B, T, Hq)) return SAGE_FP4_EINVAL;
  if ((causal & ~1) || window < 0 || !(scale > 0.0f && scale <= 1.0e30f)) return SAGE_FP4_EINVAL;
  if (T == 0 || batch->B == 0) return SAGE_FP4_OK;
  Strides s;
  if (!cache_pointers_ok(cache) || !is_aligned(q, 16) || !is_aligned(o, 16) || (lse && !is_aligned(lse, 4)) ||
      !take_strides(sage_fp4_strides{0, q_rows.h, q_rows.t}, 1, Hq, T, cache->D, &s) ||
      !take_strides(sage_fp4_strides{0, o_rows.h, o_rows.t}, 1, Hq, T, cache->D, &s))
    return SAGE_FP4_EINVAL;
  if (!is_aligned(workspace, 256) || workspace_bytes < way_of(cache, batch->B, T, Hq, kMaxSms).total)
    return SAGE_FP4_EINVAL;
  int sms = 0;
  if (const int rc = check_device_103(&sms)) return rc;
  const KvView c = view_of(cache, batch);
  const AttnArgs a{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(o), lse, q_rows, o_rows, T, Hq, Hq / c.H, causal,
                   window, scale * kLog2e};
  const Way way = way_of(cache, c.B, T, Hq, sms);
  if (withhold && way.step) return SAGE_FP4_EINVAL;  // that kernel waits for nothing
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const AttnWork w{reinterpret_cast<PlanHead*>(ws), reinterpret_cast<PlanEntry*>(ws + way.entry),
                   reinterpret_cast<long long*>(ws + way.cum), reinterpret_cast<float*>(ws + way.o),
                   reinterpret_cast<float2*>(ws + way.ml), reinterpret_cast<int2*>(ws + way.open), way.capacity, way.workers, way.lead_units, way.min_share, wait_ns, withhold};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (way.capacity <= kFew)
    plan_few_kernel<<<1, 32, 0, st>>>(c, a, w, way.rows);
  else
    plan_kernel<<<1, kPlanThreads, 0, st>>>(c, a, w, way.rows);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = way.step ? launch_attn_step(c, a, w, way.rows, cache->D, cache->format, st)
                 : launch_attn_chunk(c, a, w, cache->D, cache->format, st);
  if (e == cudaSuccess)
    e = cache->D == 64 ? launch_combine<64>(c, a, w, way, sms, st) : launch_combine<128>(c, a, w, way, sms, st);
  return launched(e);
}

}  // namespace
}  // namespace sagefp4

using namespace sagefp4;

extern "C" {

size_t sage_kv_attn_workspace_bytes(const sage_kv_cache* cache, int B, int T, int Hq) {
  return sizes_ok(cache, B, T, Hq) ? way_of(cache, B, T, Hq, kMaxSms).total : 0;
}

int sage_kv_attn(const sage_kv_cache* cache, const sage_kv_batch* batch, const void* q, sage_kv_rows q_rows, void* o,
                 sage_kv_rows o_rows, float* lse, int T, int Hq, int causal, int window, float scale, void* workspace,
                 size_t workspace_bytes, void* stream) {
  return attn(cache, batch, q, q_rows, o, o_rows, lse, T, Hq, causal, window, scale, workspace, workspace_bytes, stream, kWaitNs,
              0);
}

int sage_kv_attn_stall_test(const sage_kv_cache* cache, const sage_kv_batch* batch, const void* q, sage_kv_rows q_rows,
                            void* o, sage_kv_rows o_rows, int T, int Hq, uint64_t wait_limit_ns, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (wait_limit_ns < 1000000 || wait_limit_ns > kWaitNs) return SAGE_FP4_EINVAL;
  return attn(cache, batch, q, q_rows, o, o_rows, nullptr, T, Hq, 1, 0, 0.125f, workspace, workspace_bytes, stream,
              wait_limit_ns, 1);
}

}  // extern "C"
