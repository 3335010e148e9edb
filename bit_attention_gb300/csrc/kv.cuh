// kv.cuh -- what the paged cache's kernels share: the device view of a cache
// and a batch, its index checks, the row formats.  Internal to the library.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sage_kv.h"
#include "host.h"
#include "ptx.cuh"

namespace sagefp4 {

constexpr int kBf16 = SAGE_KV_BF16, kE4m3 = SAGE_KV_E4M3, kNvfp4 = SAGE_KV_NVFP4;

struct KvView {
  uint8_t *kc, *vc, *ks, *vs;
  const int32_t *cu_q, *kv_len, *table;
  long long table_stride;
  int32_t* status;
  int num_pages, page_shift, H, B, max_pages;
};

template <int kFmt>
__host__ __device__ constexpr int row_bytes(int D) {
  return kFmt == kBf16 ? 2 * D : kFmt == kE4m3 ? D : D / 2;
}
template <int kFmt>
__host__ __device__ constexpr int row_scales(int D) {
  return kFmt == kBf16 ? 0 : kFmt == kE4m3 ? 1 : D / 16;
}

__device__ __forceinline__ void flag_index(int32_t* status) { atomicCAS(status, 0, SAGE_FP4_EINDEX); }

// The longest sequence: ends of tiles and of steps past it are ints too.
constexpr int kMaxLen = INT32_MAX - 4095;

// Tokens of sequence b in the cache, 0 (recorded) for a length that its table
// cannot hold.
__device__ __forceinline__ int seq_len(const KvView& c, int b) {
  const int n = c.kv_len[b];
  if (n >= 0 && n <= kMaxLen && n <= (static_cast<long long>(c.max_pages) << c.page_shift)) return n;
  flag_index(c.status);
  return 0;
}

// The packed rows of sequence b's new tokens, [first, end); none (recorded)
// where they leave [0, T] or run backwards.
__device__ __forceinline__ int2 seq_rows(const KvView& c, int b, int T) {
  const int q0 = c.cu_q[b], q1 = c.cu_q[b + 1];
  if (q0 >= 0 && q1 >= q0 && q1 <= T) return int2{q0, q1};
  flag_index(c.status);
  return int2{0, 0};
}

// Row index (page * H + h) * page_size + slot of token j of sequence b, head h
// (0 <= j < seq_len); -1 (recorded) for a page that the cache does not have.
__device__ __forceinline__ long long row_of(const KvView& c, int b, int h, int j) {
  const int page = c.table[b * c.table_stride + (j >> c.page_shift)];
  if (page < 0 || page >= c.num_pages) {
    flag_index(c.status);
    return -1;
  }
  return ((static_cast<long long>(page) * c.H + h) << c.page_shift) + (j & ((1 << c.page_shift) - 1));
}

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight E2M1 codes (element 0 in bits 0-3) -> four FP16 pairs, exact.
__device__ __forceinline__ void e2m1x8_to_h2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Four E4M3 codes -> two FP16 pairs, exact.
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t w, uint32_t (&h)[2]) {
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
}
__device__ __forceinline__ float2 h2_to_f2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// FP16 pair times a scale -> bf16 pair.  Exact for codes times their scale:
// four significant bits for E4M3 times a power of two, two times four for
// E2M1 times E4M3, within bf16's exponents.
__device__ __forceinline__ uint32_t h2_scaled_bf2(uint32_t h, float s) {
  const float2 f = h2_to_f2(h);
  return bf2(f.x * s, f.y * s);
}

// Eight consecutive channels (d = 8 * chunk) of a stored row as bf16.
template <int kFmt, int D>
__device__ __forceinline__ uint4 load_chunk(const uint8_t* codes, const uint8_t* scales, long long row, int chunk) {
  if constexpr (kFmt == kBf16) {
    return *reinterpret_cast<const uint4*>(codes + row * (2 * D) + 16 * chunk);
  } else if constexpr (kFmt == kE4m3) {
    const uint2 c = *reinterpret_cast<const uint2*>(codes + row * D + 8 * chunk);
    const float s = __uint_as_float(static_cast<uint32_t>(scales[row]) << 23);
    uint32_t a[2], b[2];
    e4m3x4_to_h2(c.x, a);
    e4m3x4_to_h2(c.y, b);
    return uint4{h2_scaled_bf2(a[0], s), h2_scaled_bf2(a[1], s), h2_scaled_bf2(b[0], s), h2_scaled_bf2(b[1], s)};
  } else {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + row * (D / 2) + 4 * chunk);
    const float s = e4m3_to_f32(scales[row * (D / 16) + chunk / 2]);
    uint32_t h[4];
    e2m1x8_to_h2(c, h);
    return uint4{h2_scaled_bf2(h[0], s), h2_scaled_bf2(h[1], s), h2_scaled_bf2(h[2], s), h2_scaled_bf2(h[3], s)};
  }
}

// ------------------------------------------------------------------ host
inline bool cache_ok(const sage_kv_cache* c) {
  if (!c || (c->D != 64 && c->D != 128) || c->H < 1 || c->H > 65535 || c->num_pages < 0) return false;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return false;
  return c->format == SAGE_KV_BF16 || c->format == SAGE_KV_E4M3 || c->format == SAGE_KV_NVFP4;
}
inline bool cache_pointers_ok(const sage_kv_cache* c) {
  if (!is_aligned(c->k_codes, 16) || !is_aligned(c->v_codes, 16) || !is_aligned(c->status, 4)) return false;
  return c->format == SAGE_KV_BF16 || (is_aligned(c->k_scales, 16) && is_aligned(c->v_scales, 16));
}
// Sequences, table rows; the table's offsets stay within 2^62.
inline bool batch_ok(const sage_kv_batch* b, bool new_tokens) {
  if (!b || b->B < 0 || b->max_pages < 0) return false;
  if (b->B == 0) return true;
  if ((new_tokens && !is_aligned(b->cu_q, 4)) || !is_aligned(b->kv_len, 4)) return false;
  if (b->max_pages == 0) return true;
  return is_aligned(b->block_table, 4) && b->table_stride >= b->max_pages && b->table_stride <= (int64_t(1) << 31);
}
inline KvView view_of(const sage_kv_cache* c, const sage_kv_batch* b) {
  KvView v;
  v.kc = static_cast<uint8_t*>(c->k_codes);
  v.vc = static_cast<uint8_t*>(c->v_codes);
  v.ks = c->k_scales;
  v.vs = c->v_scales;
  v.status = c->status;
  v.cu_q = b->cu_q;
  v.kv_len = b->kv_len;
  v.table = b->block_table;
  v.table_stride = b->table_stride;
  v.num_pages = c->num_pages;
  v.page_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
  v.H = c->H;
  v.B = b->B;
  v.max_pages = b->max_pages;
  return v;
}

}  // namespace sagefp4
