// kv_cache.cu -- writing rows into the paged key/value cache and reading them
// back: kernels and C ABI (include/sage_kv.h).
//
// Both are bound by HBM.  A row of D channels is held by D / 8 lanes, 16 bytes
// of bf16 each.  Writing: the row's largest magnitude (E4M3) goes through
// shuffles among its lanes, a 16-channel group's (NVFP4) through one; a lane
// has several rows in flight, of k and of v, and asks for them before the chain
// of small loads (sequence bounds, length, page) that says where they go.
// 65536 tokens of 8 heads of 128: bf16 86 us (6.2 TB/s), E4M3 69 (5.9), NVFP4 71
// (4.9, where converting bounds it: issue in 80% of cycles); back again 86, 75 and 71
// (issue in 64% and 70%).
#include "kv.cuh"

namespace sagefp4 {
namespace {

constexpr int kThreads = 256;      // of append
// of read, with the rows of a lane group: 65536 tokens of 8 heads of 128 in E4M3,
// 75 us; 8 rows 96, 2 rows 77
constexpr int kReadThreads = 128, kReadRows = 4;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Largest magnitudes of eight bf16 values, of the even and the odd ones: their
// bits without the sign are in the magnitudes' order.
__device__ __forceinline__ uint32_t max8(const uint4& u) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(u.x & kAbs, u.y & kAbs), __vmaxu2(u.z & kAbs, u.w & kAbs));
}
__device__ __forceinline__ float larger_half(uint32_t m) { return __uint_as_float(max(m << 16, m & 0xffff0000u)); }

// The E8M0 byte of a row: the smallest power of two that brings amax (a bf16
// value) to 448 = 1.75 * 2^8 or less.  At least 17 and at most 246, so that
// every code times its scale is a normal, finite bf16 value (2^-9 * 2^-110 the
// smallest, 448 * 2^119 the largest; with 247 a magnitude above 1.875 * 2^127
// would round to a code of 256 and read back as infinity).
__device__ __forceinline__ uint32_t e4m3_scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
  return static_cast<uint32_t>(min(max(e, 17), 246));
}

// The sequence of packed row t (warp-wide), -1 for none: the number of
// sequences that end at or before t.
__device__ __forceinline__ int find_sequence(const KvView& c, int t, int T) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  bool bad = false;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const int b = b0 + lane;
    int q0 = 0, q1 = 0x7fffffff;
    if (b < c.B) {
      q0 = c.cu_q[b];
      q1 = c.cu_q[b + 1];
      bad |= q0 < 0 || q1 < q0 || q1 > T;
    }
    n += __popc(__ballot_sync(kAll, q1 <= t));
  }
  if (bad) flag_index(c.status);
  return n < c.B ? n : -1;
}

// One warp: kRows heads a lane group of packed token t, of k and of v.
template <int kFmt, int D, int kRows>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ KvView c, const uint16_t* k,
                                                          sage_kv_rows kr, const uint16_t* v, sage_kv_rows vr, int T,
                                                          int pieces) {
  constexpr int kC = D / 8, kGroups = 32 / kC;
  const long long warp = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  if (warp >= static_cast<long long>(T) * pieces) return;
  const int t = pieces == 1 ? static_cast<int>(warp) : static_cast<int>(warp / pieces);
  const int lane = threadIdx.x % kC, grp = (threadIdx.x & 31) / kC;
  const int h0 = static_cast<int>(warp - static_cast<long long>(t) * pieces) * (kGroups * kRows) + grp;
  uint4 raw[2][kRows];
#pragma unroll
  for (int s = 0; s < 2; s++) {
    const uint16_t* src = (s ? v + t * vr.t + h0 * vr.h : k + t * kr.t + h0 * kr.h) + 8 * lane;
    const long long step = kGroups * (s ? vr.h : kr.h);
#pragma unroll
    for (int i = 0; i < kRows; i++)
      raw[s][i] = h0 + i * kGroups < c.H ? *reinterpret_cast<const uint4*>(src + i * step) : uint4{0, 0, 0, 0};
  }
  const int b = find_sequence(c, t, T);
  if (b < 0) return;
  const int2 rows = seq_rows(c, b, T);
  const int pos = seq_len(c, b) - (rows.y - t);
  if (t < rows.x || t >= rows.y || pos < 0) return;
  const long long row0 = row_of(c, b, 0, pos);
  if (row0 < 0) return;
  const long long row1 = row0 + (static_cast<long long>(h0) << c.page_shift);
  const int dr = kGroups << c.page_shift;  // rows from one of the group's heads to its next
#pragma unroll
  for (int s = 0; s < 2; s++) {
    uint8_t* codes = (s ? c.vc : c.kc) + row1 * row_bytes<kFmt>(D);
    uint8_t* scales = (s ? c.vs : c.ks) + row1 * row_scales<kFmt>(D);
#pragma unroll
    for (int i = 0; i < kRows; i++) {
      const bool on = h0 + i * kGroups < c.H;
      if constexpr (kFmt == kBf16) {
        if (on) *reinterpret_cast<uint4*>(codes + static_cast<long long>(i) * dr * (2 * D) + 16 * lane) = raw[s][i];
      } else if constexpr (kFmt == kE4m3) {
        uint32_t top = max8(raw[s][i]);
#pragma unroll
        for (int o = kC / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(kAll, top, o));
        const uint32_t byte = e4m3_scale_byte(larger_half(top));
        const float up = __uint_as_float((254u - byte) << 23);  // 2^(127 - byte)
        float f[8];
        unpack8(raw[s][i], f);
        uint2 w;
        w.x = cvt_e4m3x2(f[0] * up, f[1] * up) | cvt_e4m3x2(f[2] * up, f[3] * up) << 16;
        w.y = cvt_e4m3x2(f[4] * up, f[5] * up) | cvt_e4m3x2(f[6] * up, f[7] * up) << 16;
        if (on) {
          *reinterpret_cast<uint2*>(codes + static_cast<long long>(i) * dr * D + 8 * lane) = w;
          if (lane == 0) scales[static_cast<long long>(i) * dr] = static_cast<uint8_t>(byte);
        }
      } else {
        float f[8];
        unpack8(raw[s][i], f);
        uint32_t top = max8(raw[s][i]);
        top = __vmaxu2(top, __shfl_xor_sync(kAll, top, 1));
        const uint32_t s8 = cvt_e4m3(__fdiv_rn(larger_half(top), 6.0f));
        const float sc = e4m3_to_f32(s8), inv = sc > 0.0f ? __frcp_rn(sc) : 0.0f;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] = f[e] * inv;
        if (on) {
          *reinterpret_cast<uint32_t*>(codes + static_cast<long long>(i) * dr * (D / 2) + 4 * lane) = sc > 0.0f ? cvt_e2m1x8(y) : 0u;
          if ((lane & 1) == 0) scales[static_cast<long long>(i) * dr * (D / 16) + lane / 2] = static_cast<uint8_t>(s8);
        }
      }
    }
  }
}

// Block (tile of tokens of one sequence, head, k or v).
template <int kFmt, int D>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ KvView c, uint16_t* ko, Strides sk,
                                                        uint16_t* vo, Strides sv, int N, int tiles) {
  constexpr int kC = D / 8, kGroups = kReadThreads / kC, kRows = kReadRows;
  const int b = blockIdx.x / tiles, tile = blockIdx.x - b * tiles, h = blockIdx.y;
  const bool isk = blockIdx.z == 0;
  const int lane = threadIdx.x % kC, grp = threadIdx.x / kC, j0 = tile * (kGroups * kRows) + grp;
  const int len = seq_len(c, b);
  const Strides& s = isk ? sk : sv;
  uint16_t* out = (isk ? ko : vo) + b * s.b + h * s.h + 8 * lane;
  long long row[kRows];
#pragma unroll
  for (int i = 0; i < kRows; i++) {
    // 16 tokens from a multiple of 16 on are neighbours
    const int j = j0 + i * kGroups, in = (i * kGroups) % 16;
    if (in == 0)
      row[i] = j - grp < len && j - grp < N ? row_of(c, b, h, j - grp) : -1;
    else
      row[i] = row[i - 1];
  }
#pragma unroll
  for (int i = kRows - 1; i >= 0; i--) {
    const int j = j0 + i * kGroups;
    row[i] = row[i] >= 0 && j < len && j < N ? row[i] + (i * kGroups) % 16 + grp : -1;
  }
  uint4 w[kRows];
#pragma unroll
  for (int i = 0; i < kRows; i++)
    w[i] = row[i] >= 0 ? load_chunk<kFmt, D>(isk ? c.kc : c.vc, isk ? c.ks : c.vs, row[i], lane) : uint4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kRows; i++) {
    const int j = j0 + i * kGroups;
    if (j < N) *reinterpret_cast<uint4*>(out + j * s.n) = w[i];
  }
}

template <int kFmt, int D, int kRows>
void append_launch(const KvView& c, const void* k, sage_kv_rows kr, const void* v, sage_kv_rows vr, int T,
                   cudaStream_t st) {
  const int per = 32 / (D / 8) * kRows, pieces = (c.H + per - 1) / per;
  const long long warps = static_cast<long long>(T) * pieces;
  const unsigned blocks = static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32));
  append_kernel<kFmt, D, kRows><<<blocks, kThreads, 0, st>>>(c, static_cast<const uint16_t*>(k), kr,
                                                             static_cast<const uint16_t*>(v), vr, T, pieces);
}

// A lane group takes as many heads as it needs to have all of them in one warp, up
// to four: idle rows cost as much as others, and a warp's search for its place
// serves all its rows.  65536 tokens in NVFP4 with one, two, four heads a lane
// group: 8 heads of 128, 93, 77, 71 us; 4 heads, 51, 43, 66; 1 head, 33, 43, 69.
template <int kFmt, int D>
void append_rows(const KvView& c, const void* k, sage_kv_rows kr, const void* v, sage_kv_rows vr, int T, cudaStream_t st) {
  constexpr int kGroups = 32 / (D / 8);
  if (c.H <= kGroups)
    append_launch<kFmt, D, 1>(c, k, kr, v, vr, T, st);
  else if (c.H <= 2 * kGroups)
    append_launch<kFmt, D, 2>(c, k, kr, v, vr, T, st);
  else
    append_launch<kFmt, D, 4>(c, k, kr, v, vr, T, st);
}

template <int kFmt, int D>
void read_launch(const KvView& c, void* ko, Strides sk, void* vo, Strides sv, int N, cudaStream_t st) {
  const int per = kReadThreads / (D / 8) * kReadRows, tiles = (N + per - 1) / per;
  read_kernel<kFmt, D><<<dim3(static_cast<unsigned>(c.B) * tiles, c.H, 2), kReadThreads, 0, st>>>(
      c, static_cast<uint16_t*>(ko), sk, static_cast<uint16_t*>(vo), sv, N, tiles);
}

bool rows_ok(const void* p, const sage_kv_rows& r, int T, int H) {
  Strides s;
  return is_aligned(p, 16) && take_strides(sage_fp4_strides{0, r.h, r.t}, 1, H, T, 128, &s);
}

}  // namespace
}  // namespace sagefp4

using namespace sagefp4;

extern "C" {

int sage_kv_append(const sage_kv_cache* cache, const sage_kv_batch* batch, const void* k, sage_kv_rows k_rows,
                   const void* v, sage_kv_rows v_rows, int T, void* stream) {
  if (!cache_ok(cache) || !batch_ok(batch, true) || T < 0) return SAGE_FP4_EINVAL;
  if (T == 0 || batch->B == 0) return SAGE_FP4_OK;
  if (!cache_pointers_ok(cache) || !rows_ok(k, k_rows, T, cache->H) || !rows_ok(v, v_rows, T, cache->H))
    return SAGE_FP4_EINVAL;
  if (static_cast<long long>(T) * cache->H > (1LL << 32)) return SAGE_FP4_EINVAL;  // blocks of the launch
  int sms = 0;
  if (const int rc = check_device_103(&sms)) return rc;
  const KvView c = view_of(cache, batch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define SAGE_KV_CASE(F)                                                  \
  case F:                                                                \
    if (cache->D == 64)                                                  \
      append_rows<F, 64>(c, k, k_rows, v, v_rows, T, st);                \
    else                                                                 \
      append_rows<F, 128>(c, k, k_rows, v, v_rows, T, st);               \
    break;
  switch (cache->format) {
    SAGE_KV_CASE(kBf16)
    SAGE_KV_CASE(kE4m3)
    SAGE_KV_CASE(kNvfp4)
  }
#undef SAGE_KV_CASE
  return launched(cudaGetLastError());
}

int sage_kv_read(const sage_kv_cache* cache, const sage_kv_batch* batch, void* k_out,
                 const sage_fp4_strides* k_strides, void* v_out, const sage_fp4_strides* v_strides, int N,
                 void* stream) {
  if (!cache_ok(cache) || !batch_ok(batch, false) || N < 0 || N > INT32_MAX - 1024) return SAGE_FP4_EINVAL;
  if (N == 0 || batch->B == 0) return SAGE_FP4_OK;
  const int64_t H = cache->H, D = cache->D;
  const sage_fp4_strides dense = {H * N * D, N * D, D};
  Strides sk, sv;
  if (!cache_pointers_ok(cache) || !is_aligned(k_out, 16) || !is_aligned(v_out, 16) ||
      !take_strides(k_strides ? *k_strides : dense, batch->B, H, N, D, &sk) ||
      !take_strides(v_strides ? *v_strides : dense, batch->B, H, N, D, &sv))
    return SAGE_FP4_EINVAL;
  if ((static_cast<long long>(N) + 31) / 32 * batch->B > INT32_MAX) return SAGE_FP4_EINVAL;  // blocks of the launch
  int sms = 0;
  if (const int rc = check_device_103(&sms)) return rc;
  const KvView c = view_of(cache, batch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define SAGE_KV_CASE(F)                                          \
  case F:                                                        \
    if (cache->D == 64)                                          \
      read_launch<F, 64>(c, k_out, sk, v_out, sv, N, st);        \
    else                                                         \
      read_launch<F, 128>(c, k_out, sk, v_out, sv, N, st);       \
    break;
  switch (cache->format) {
    SAGE_KV_CASE(kBf16)
    SAGE_KV_CASE(kE4m3)
    SAGE_KV_CASE(kNvfp4)
  }
#undef SAGE_KV_CASE
  return launched(cudaGetLastError());
}

int sage_kv_get_status(const sage_kv_cache* cache, void* stream) {
  return cache ? read_status(cache->status, stream) : SAGE_FP4_EINVAL;
}

}  // extern "C"
