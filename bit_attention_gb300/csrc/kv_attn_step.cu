// kv_attn_step.cu -- attention of a few new tokens over the paged cache: the
// form for single tokens.  Bound by HBM: every stored key and value is read
// once for all query heads of its group.
//
// The unit of work is a warp, which walks its own share of the KV tiles and
// shares nothing with other warps: its buffers in shared memory are its own, and
// it waits for its own copies alone.  It takes up to
// 8 * kNt query rows (new tokens x heads of the group) against kKeys keys a
// step, with warp-level MMAs in the transposed form that wastes nothing on
// eight rows: S^T = K Q^T (M = keys, N = rows), O^T += V^T P^T (M = channels,
// K = keys).
//
// Stored rows come by asynchronous copies into the warp's own two buffers of 4
// KB of K and 4 KB of V (a step of 16, 32 or 64 keys).  Every copy instruction
// reads 512 consecutive bytes, which HBM serves at 7.4 TB/s (64-byte pieces of
// eight rows: 5.5); K's buffer is refilled as soon as S^T is formed and V's as
// soon as O^T is, so that a step or more is in flight: 8 KB a warp, 96 KB an SM.
// 64 sequences of 512 to 16384 tokens, 32 query and 8 key/value heads of 128:
// 1.14 GB of E4M3 in 185 us, 6.2 TB/s.
// The operands' free orders fit them to whole 16-byte chunks: in S^T the order
// of the channels along K is free as long as Q has the same, so lane q of a
// row's four takes whole chunks of it; in O^T the order of the channels along M
// is free, so lane group g takes whole chunks of four keys' rows, whose values
// it interleaves by pairs.  Rows and chunks are permuted in the buffer so that
// these reads touch all bank groups.  P^T comes out of the accumulators' layout
// by movmatrix.
//
// Quantized rows are taken as FP16: E4M3 codes without their scales, which
// multiply the scores of a key (K) or its probability (V, through a second
// running maximum that includes the scale, so that the largest weight is 1);
// E2M1 codes times their E4M3 scales, exact in FP16 (six significant bits,
// 2^-10 .. 2688).  Q becomes FP16 after its row is scaled by the power of two
// that brings its largest magnitude to 2^14 .. 2^15: bf16's eight bits fit
// while a channel is above 2^-28 of the row's largest.  P is rounded to FP16
// (the largest weight raised to 2^11 .. 2^15: half a step is 2^-11 relative down
// to 2^-25 of it, and 2^-36 of it below) or, for a bf16 cache, to bf16; sums and
// statistics are FP32.
#include "kv_attn.cuh"
#include "umma.cuh"

namespace sagefp4 {
namespace {

constexpr int kThreads = 128;
constexpr int kBuffers = 2;  // of a warp; the code below counts on two
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;

template <int kFmt>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kFmt == kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t h2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two E4M3 bytes (in the low 16 bits) -> FP16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b)));
  return r;
}

// size: 16, or 0 for zeros
__device__ __forceinline__ void copy_async16(uint32_t dst, const uint8_t* src, uint32_t size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}

template <int kBytes>
__device__ __forceinline__ void load_shared(uint32_t (&w)[kBytes / 4], uint32_t src) {
  if constexpr (kBytes == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(src) : "memory");
  else if constexpr (kBytes == 8)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(src) : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(src) : "memory");
}
__device__ __forceinline__ uint32_t load_shared_u8(uint32_t src) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(src) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_shared_u16(uint32_t src) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(src) : "memory");
  return v;
}

// A step's rows: how lanes share them out, and the buffer that holds them.
template <int kFmt, int D>
struct Step {
  static constexpr int kRow = row_bytes<kFmt>(D);
  static constexpr int kKeys = 4096 / kRow;  // 16, 32, 64 (128 for D = 64 in 4 bits)
  static constexpr int kG = kKeys / 16;      // groups of 16 keys; a page holds whole groups
  // K: chunks of a lane in a row, chunk j at kChunk * (q + 4j), kVals channels each
  static constexpr int kChunk = kRow / 4 < 16 ? kRow / 4 : 16;
  static constexpr int kChunks = kRow / 4 / kChunk;
  static constexpr int kVals = kChunk * D / kRow;
  // V: chunks of a lane in a row, chunk j at kVChunk * (g + 8j), kVVals channels each
  static constexpr int kVChunk = kRow / 8 < 16 ? kRow / 8 : 16;
  static constexpr int kVChunks = kRow / 8 / kVChunk;
  static constexpr int kVVals = kVChunk * D / kRow;
  static constexpr int kScales = row_scales<kFmt>(D);  // bytes of a row
  // the buffer: each group's K and V rows, then the groups' scales, K and V
  static constexpr int kPer = kRow / 16;  // 16-byte chunks of a row
  static constexpr int kCopies = kRow / 32;  // copy instructions (512 bytes) of a group's 16 rows
  static constexpr int kKBytes = 16 * kRow, kGroup = 2 * kKBytes;
  static constexpr int kScaleOff = kG * kGroup, kScaleGroup = 32 * kScales;
  static constexpr int kBuffer = kScaleOff + (kG * kScaleGroup + 127) / 128 * 128;

  // Where chunk ch of row r of a group lies.  K is read by eight lanes as two
  // neighbouring rows x four chunks; V as rows 0, 2, 4, 6 (or 1, 3, ...) x two
  // neighbouring chunks (halves, quarters of one where rows are short), so its
  // even rows come first.
  static __device__ __forceinline__ int place_k(int r, int ch) {
    return r * kRow + 16 * (kRow >= 128 ? ch ^ (4 * (r & 1)) : ch);
  }
  static __device__ __forceinline__ int place_v(int r, int ch) {
    const int pos = ((r >> 1) & 3) | ((r & 1) << 2) | (r & 8);
    return pos * kRow + 16 * (kRow >= 128 ? ch ^ (2 * (pos & 3)) : kRow == 64 ? ch ^ (pos & 2) : ch);
  }

  // The table's entries of the step's groups; asked for a step before they are
  // looked at.  Groups outside [begin, end) have none (-1).
  static __device__ __forceinline__ void look_up(const KvView& c, int b, int key0, int begin, int end, int (&page)[kG]) {
#pragma unroll
    for (int i = 0; i < kG; i++) {
      const int key = key0 + 16 * i;
      page[i] = key >= begin && key < end ? c.table[b * c.table_stride + (key >> c.page_shift)] : -1;
    }
  }

  // Bit i: the cache does not have the page of group i (recorded, where the
  // group is in [begin, end)).
  static __device__ __forceinline__ uint32_t missing(const KvView& c, int key0, int begin, int end, const int (&page)[kG]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kG; i++)
      if (static_cast<unsigned>(page[i]) >= static_cast<unsigned>(c.num_pages)) {
        m |= 1u << i;
        if (key0 + 16 * i >= begin && key0 + 16 * i < end) flag_index(c.status);
      }
    return m;
  }

  // First row of every group in the cache (of page 0 where there is none).
  static __device__ __forceinline__ void locate(const KvView& c, int h, int key0, uint32_t gone, const int (&page)[kG],
                                                long long (&row)[kG]) {
#pragma unroll
    for (int i = 0; i < kG; i++)
      row[i] = ((static_cast<long long>((gone >> i) & 1u ? 0 : page[i]) * c.H + h) << c.page_shift) +
               ((key0 + 16 * i) & ((1 << c.page_shift) - 1));
  }

  // Ask for K, and for the scales that go into the scores or into P.  kAllThere:
  // no group is missing, and (V) every key lies before the piece's end.
  template <bool kAllThere>
  static __device__ __forceinline__ void issue_k(uint32_t buf, const KvView& c, uint32_t gone, const long long (&row)[kG]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kG; i++) {
      const bool there = kAllThere || !((gone >> i) & 1u);
      const uint8_t* k = c.kc + row[i] * kRow + 16 * lane;
#pragma unroll
      for (int j = 0; j < kCopies; j++) {
        const int at = 32 * j + lane;
        copy_async16(buf + i * kGroup + place_k(at / kPer, at % kPer), k + 512 * j, there ? 16 : 0);
      }
      // 16 rows' scales are one run of 16 kScales bytes
      if constexpr (kFmt == kE4m3) {
        if (lane < 2)
          copy_async16(buf + kScaleOff + i * kScaleGroup + 16 * lane, (lane ? c.vs : c.ks) + row[i], there ? 16 : 0);
      } else if constexpr (kFmt == kNvfp4) {
        if (lane < kScales)
          copy_async16(buf + kScaleOff + i * kScaleGroup + 16 * lane, c.ks + row[i] * kScales + 16 * lane, there ? 16 : 0);
      }
    }
  }

  // Ask for V; keys at `end` and beyond become zeros (what a free slot holds
  // may be NaN).
  template <bool kAllThere>
  static __device__ __forceinline__ void issue_v(uint32_t buf, const KvView& c, int key0, int end, uint32_t gone,
                                                 const long long (&row)[kG]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kG; i++) {
      const bool there = kAllThere || !((gone >> i) & 1u);
      const uint8_t* v = c.vc + row[i] * kRow + 16 * lane;
#pragma unroll
      for (int j = 0; j < kCopies; j++) {
        const int at = 32 * j + lane;
        copy_async16(buf + i * kGroup + kKBytes + place_v(at / kPer, at % kPer), v + 512 * j,
                     kAllThere || (there && key0 + 16 * i + at / kPer < end) ? 16 : 0);
      }
      if constexpr (kFmt == kNvfp4) {
        if (lane < kScales)
          copy_async16(buf + kScaleOff + i * kScaleGroup + 16 * (kScales + lane), c.vs + row[i] * kScales + 16 * lane,
                         there ? 16 : 0);
      }
    }
  }

  uint32_t k[2][kRow / 16];                  // keys g, g + 8 of the current group
  uint32_t v[4][kRow / 32];                  // keys 2q, 2q + 1, 2q + 8, 2q + 9
  uint32_t ks[2], vs[kFmt == kNvfp4 ? 4 : 2];  // E4M3: bytes of keys g, g + 8; NVFP4: of the lane's channels

  __device__ __forceinline__ void take_k(uint32_t buf, int i) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; e++) {
#pragma unroll
      for (int j = 0; j < kChunks; j++) {
        uint32_t w[kChunk / 4];
        load_shared<kChunk>(w, buf + i * kGroup + (kChunk == 16 ? place_k(g + 8 * e, q + 4 * j) : place_k(g + 8 * e, 0) + 8 * q));
#pragma unroll
        for (int x = 0; x < kChunk / 4; x++) k[e][j * (kChunk / 4) + x] = w[x];
      }
      const uint32_t sc = buf + kScaleOff + i * kScaleGroup + (g + 8 * e) * kScales;
      if constexpr (kFmt == kE4m3) ks[e] = load_shared_u8(sc);
      if constexpr (kFmt == kNvfp4) ks[e] = D == 128 ? load_shared_u16(sc + 2 * q) : load_shared_u8(sc + q);
    }
  }
  // live: keys of the group before the piece's end (the scale in a free slot may be NaN)
  __device__ __forceinline__ void take_v(uint32_t buf, int i, int live) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int e = 0; e < 4; e++) {
#pragma unroll
      for (int j = 0; j < kVChunks; j++) {
        uint32_t w[kVChunk / 4];
        const int r = 8 * (e >> 1) + 2 * q + (e & 1), at = kVChunk * (g + 8 * j);
        load_shared<kVChunk>(w, buf + i * kGroup + kKBytes + place_v(r, at / 16) + at % 16);
#pragma unroll
        for (int x = 0; x < kVChunk / 4; x++) v[e][j * (kVChunk / 4) + x] = w[x];
      }
      if constexpr (kFmt == kNvfp4) {
        const int at = 8 * (e >> 1) + 2 * q + (e & 1);
        vs[e] = load_shared_u8(buf + kScaleOff + i * kScaleGroup + (16 + at) * kScales + (D == 128 ? g : g >> 1));
        if (at >= live) vs[e] = 0;
      }
    }
  }
  // E4M3: V's scale bytes of keys g, g + 8 (they go into P)
  static __device__ __forceinline__ uint32_t v_scale(uint32_t buf, int i, int e) {
    return load_shared_u8(buf + kScaleOff + i * kScaleGroup + 16 + ((threadIdx.x & 31) >> 2) + 8 * e);
  }

  // A operand of K step s: {key g, g + 8} x {pair 0, pair 1}.
  // Called for s = 0, 1, ... in turn: hold keeps what one conversion gave.
  template <int s>
  __device__ __forceinline__ void k_operand(uint32_t (&a)[4], uint32_t (&hold)[2][4]) const {
#pragma unroll
    for (int e = 0; e < 2; e++) {
      if constexpr (kFmt == kBf16) {
        a[e] = k[e][2 * s], a[2 + e] = k[e][2 * s + 1];
      } else if constexpr (kFmt == kE4m3) {
        uint32_t h[2];
        e4m3x4_to_h2(k[e][s], h);
        a[e] = h[0], a[2 + e] = h[1];
      } else {
        if constexpr (s % 2 == 0) {
          e2m1x8_to_h2(k[e][s / 2], hold[e]);
          const uint32_t byte = D == 128 ? (ks[e] >> (8 * (s / 4))) & 255u : ks[e];
          const uint32_t sc = e4m3x2_to_h2(byte | byte << 8);
#pragma unroll
          for (int x = 0; x < 4; x++) hold[e][x] = mul_h2(hold[e][x], sc);
        }
        a[e] = hold[e][2 * (s % 2)], a[2 + e] = hold[e][2 * (s % 2) + 1];
      }
    }
  }

  // A operands of the M tiles: tile t has channels 2t (rows g) and 2t + 1 (rows
  // g + 8) of the lane group's share; x: word of the share (2, 4 or 8 channels),
  // from which tiles kFrom * x .. come.
  static constexpr int kFrom = kFmt == kBf16 ? 1 : kFmt == kE4m3 ? 2 : 4;
  __device__ __forceinline__ void v_operands(int x, const uint32_t (&sc)[2], uint32_t (&a)[kFrom][4]) const {
#pragma unroll
    for (int e = 0; e < 2; e++) {  // keys 2q, 2q + 1, then 2q + 8, 2q + 9
      const uint32_t u0 = v[2 * e][x], u1 = v[2 * e + 1][x];
      if constexpr (kFmt == kBf16) {
        a[0][2 * e] = __byte_perm(u0, u1, 0x5410);
        a[0][2 * e + 1] = __byte_perm(u0, u1, 0x7632);
      } else if constexpr (kFmt == kE4m3) {
#pragma unroll
        for (int y = 0; y < 2; y++) {
          uint32_t h[2];
          e4m3x4_to_h2(__byte_perm(u0, u1, y ? 0x7362 : 0x5140), h);
          a[y][2 * e] = h[0], a[y][2 * e + 1] = h[1];
        }
      } else {
        uint32_t lo[4], hi[4];
        e2m1x8_to_h2((u0 & 0x0f0f0f0fu) | ((u1 << 4) & 0xf0f0f0f0u), lo);
        e2m1x8_to_h2(((u0 >> 4) & 0x0f0f0f0fu) | (u1 & 0xf0f0f0f0u), hi);
#pragma unroll
        for (int y = 0; y < 4; y++) a[y][2 * e] = mul_h2(lo[y], sc[e]), a[y][2 * e + 1] = mul_h2(hi[y], sc[e]);
      }
    }
  }
};

template <int kFmt, int D, int kNt, int s = 0>
__device__ __forceinline__ void scores(const Step<kFmt, D>& S, const uint32_t (&q)[kNt][D / 16][2], float (&acc)[kNt][4],
                                       uint32_t (&hold)[2][4]) {
  if constexpr (s < D / 16) {
    uint32_t a[4];
    S.template k_operand<s>(a, hold);
#pragma unroll
    for (int n = 0; n < kNt; n++) mma16<kFmt>(acc[n], a, q[n][s][0], q[n][s][1]);
    scores<kFmt, D, kNt, s + 1>(S, q, acc, hold);
  }
}

__device__ __forceinline__ float over_keys_max(float v) {  // over the lanes of a row
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float over_keys_sum(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

template <int kFmt, int D, int kNt>
__global__ void __launch_bounds__(kThreads, kNt == 1 ? 3 : 2)
    step_kernel(const __grid_constant__ KvView c, const __grid_constant__ AttnArgs a, const __grid_constant__ AttnWork work) {
  using P = Step<kFmt, D>;
  constexpr int kTiles = D / 16;  // M tiles of O^T
  constexpr int kRows = 8 * kNt, kKeys = P::kKeys, kG = P::kG;
  constexpr bool kVScale = kFmt == kE4m3;  // V's scales go into P
  // A weight at its row's maximum is 2^kRaise, and none exceeds 2^(kRaise + kGrow)
  constexpr float kGrow = 4.0f, kRaise = kFmt == kBf16 ? 0.0f : 11.0f;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  // neighbouring shares lie on different SMs
  const int worker = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  extern __shared__ uint8_t smem[];
  const uint32_t ring = smem_addr(smem) + (threadIdx.x >> 5) * kBuffers * P::kBuffer;
  griddep_launch_dependents();
  griddep_wait();  // the plan
  Walk walk(work, c.H, worker);
  while (walk.next(work)) {
    const PlanEntry e = walk.entry(work);
    const int rows = min(e.nq * a.G - e.row0, kRows);
    const int begin = first_key(a, e.len, e.nq, e.row0), first = walk.t * kTile;
    const int end = min(e.len, (walk.t + walk.tiles) * kTile);  // keys of the piece
    // Copies are committed as K, V, K, V, ...: of step s into buffer s % 2
    int page[kG];                  // table entries of the step to be asked for next
    uint32_t gone[kBuffers] = {};  // groups without a page, of the steps in the buffers
    if (walk.tiles) {
      P::look_up(c, e.b, first, begin, end, page);
#pragma unroll
      for (int n = 0; n < kBuffers; n++) {
        const int key0 = first + n * kKeys;
        long long row[kG];
        if (key0 < end) {
          gone[n] = P::missing(c, key0, begin, end, page);
          P::locate(c, walk.h, key0, gone[n], page, row);
          P::template issue_k<false>(ring + n * P::kBuffer, c, gone[n], row);
        }
        cp_async_commit();
        if (key0 < end) P::template issue_v<false>(ring + n * P::kBuffer, c, key0, end, gone[n], row);
        cp_async_commit();
        P::look_up(c, e.b, key0 + kKeys, begin, end, page);
      }
    }
    // ---- Q: row 8n + g in the channel order of the lane's K chunks
    uint32_t qf[kNt][D / 16][2];
    float rf[kNt][2];  // what turns an accumulator into a score in log2 units, rows 8n + 2q, + 1
#pragma unroll
    for (int n = 0; n < kNt; n++) {
      const int r = 8 * n + g, rr = e.row0 + r, i = rr / a.G, gq = rr - i * a.G;
      const uint16_t* src = a.q + (e.q0 + i) * a.qr.t + (walk.h * a.G + gq) * a.qr.h;
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < D / 16; s++) {
        const int d = P::kVals * (q + 4 * (s / (P::kVals / 4))) + 4 * (s % (P::kVals / 4));
        const uint2 w = r < rows ? *reinterpret_cast<const uint2*>(src + d) : uint2{0, 0};
        qf[n][s][0] = w.x, qf[n][s][1] = w.y;
        if constexpr (kFmt != kBf16)
          top = max(max(top, (w.x << 16) & 0x7fffffffu), max(w.x & 0x7fff0000u, max((w.y << 16) & 0x7fffffffu, w.y & 0x7fff0000u)));
      }
      float f = a.scale_log2;
      if constexpr (kFmt != kBf16) {
        top = max(top, __shfl_xor_sync(kAll, top, 1));
        top = max(top, __shfl_xor_sync(kAll, top, 2));
        const int up = min(14 + 127 - static_cast<int>(top >> 23), 126);  // exponent of the scaling
        const float m = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        f *= __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
        for (int s = 0; s < D / 16; s++)
#pragma unroll
          for (int x = 0; x < 2; x++)
            qf[n][s][x] = h2_of(__uint_as_float(qf[n][s][x] << 16) * m, __uint_as_float(qf[n][s][x] & 0xffff0000u) * m);
      }
      rf[n][0] = __shfl_sync(kAll, f, 8 * q);      // lane of row 2q
      rf[n][1] = __shfl_sync(kAll, f, 8 * q + 4);  // of row 2q + 1
    }
    int2 see[kNt][2];
#pragma unroll
    for (int n = 0; n < kNt; n++)
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const int r = 8 * n + 2 * q + x;
        see[n][x] = r < rows ? key_range(a, e.len, e.nq, (e.row0 + r) / a.G) : int2{0, 0};
      }
    // the keys [clear0, clear1) are seen by every row (rows of one entry see
    // ranges that move on with the token)
    const int clear0 = key_range(a, e.len, e.nq, (e.row0 + rows - 1) / a.G).x, clear1 = key_range(a, e.len, e.nq, e.row0 / a.G).y;
    float o[kTiles][kNt][4];
#pragma unroll
    for (int t = 0; t < kTiles; t++)
#pragma unroll
      for (int n = 0; n < kNt; n++)
#pragma unroll
        for (int x = 0; x < 4; x++) o[t][n][x] = 0.0f;
    // The largest score so far (log2 units), which weights are relative to, and this
    // lane's part of their sum; E4M3: the largest of score - m + log2 of V's scale,
    // which P is relative to besides.  A score of any size is subtracted first:
    // what remains is small, and nothing is lost by adding to that.
    float m[kNt][2], l[kNt][2], mw[kNt][2];
#pragma unroll
    for (int n = 0; n < kNt; n++)
#pragma unroll
      for (int x = 0; x < 2; x++) m[n][x] = mw[n][x] = -INFINITY, l[n][x] = 0.0f;

    uint32_t buf = ring;
    for (int key0 = first; key0 < end; key0 += kKeys) {
      cp_async_wait<2 * kBuffers - 1>();
      __syncwarp();  // lanes read what others copied
      // ---- S^T
      float s[kG][kNt][4];
      float vx[kVScale ? kG : 1][2];  // exponents of V's scales
      P S;
#pragma unroll
      for (int i = 0; i < kG; i++) {
        S.take_k(buf, i);
#pragma unroll
        for (int n = 0; n < kNt; n++)
#pragma unroll
          for (int x = 0; x < 4; x++) s[i][n][x] = 0.0f;
        uint32_t hold[2][4];
        scores<kFmt, D, kNt>(S, qf, s[i], hold);
        float kf[2] = {1.0f, 1.0f};
        if constexpr (kFmt == kE4m3) {
#pragma unroll
          for (int x = 0; x < 2; x++) {
            kf[x] = __uint_as_float(S.ks[x] << 23);
            vx[i][x] = __uint_as_float(0x4b000000u | P::v_scale(buf, i, x)) - (8388608.0f + 127.0f);  // byte - 127
          }
        }
#pragma unroll
        for (int n = 0; n < kNt; n++)
#pragma unroll
          for (int x = 0; x < 4; x++) s[i][n][x] *= kf[x >> 1] * rf[n][x & 1];
      }
      // keys that the row does not see, and groups whose page does not exist
      if (key0 < clear0 || key0 + kKeys > clear1 || gone[0]) {
#pragma unroll
        for (int i = 0; i < kG; i++)
#pragma unroll
          for (int x = 0; x < 2; x++) {
            const int key = (gone[0] >> i) & 1u ? -1 : key0 + 16 * i + 8 * x + g;
#pragma unroll
            for (int n = 0; n < kNt; n++)
#pragma unroll
              for (int y = 0; y < 2; y++)
                if (key < see[n][y].x || key >= see[n][y].y) s[i][n][2 * x + y] = -INFINITY;
          }
      }
      // ---- K's buffer takes the step after the next
      const int next = key0 + kBuffers * kKeys;
      uint32_t gone_next = 0;
      long long row[kG];
      bool all = false;
      __syncwarp();
      if (next < end) {
        gone_next = P::missing(c, next, begin, end, page);
        P::locate(c, walk.h, next, gone_next, page, row);
        all = gone_next == 0 && next + kKeys <= end;
        if (all)
          P::template issue_k<true>(buf, c, 0, row);
        else
          P::template issue_k<false>(buf, c, gone_next, row);
        P::look_up(c, e.b, next + kKeys, begin, end, page);
      }
      cp_async_commit();
      // ---- softmax.  The maxima that P and the row sum are relative to move
      // (for all rows, and with them O and the sums) only when a value has
      // outgrown its own by kGrow: FP16's range has room for that, and most
      // steps then need one vote instead of reductions over the lanes.
      uint32_t p[kG][kNt][2];
      auto or_zero = [](float x) { return x == -INFINITY ? 0.0f : x; };
      // the largest s - sub + log2 of V's scale of a row among this lane's keys
      auto with_scale = [&](int n, int y, float sub) {
        float t = -INFINITY;
#pragma unroll
        for (int i = 0; i < kG; i++)
          t = max3f(t, (s[i][n][y] - sub) + vx[kVScale ? i : 0][0], (s[i][n][2 + y] - sub) + vx[kVScale ? i : 0][1]);
        return t;
      };
      float top[kNt][2];
      bool grown = false;
#pragma unroll
      for (int n = 0; n < kNt; n++)
#pragma unroll
        for (int y = 0; y < 2; y++) {
          float t = -INFINITY;
#pragma unroll
          for (int i = 0; i < kG; i++) t = max3f(t, s[i][n][y], s[i][n][2 + y]);
          top[n][y] = t;
          if constexpr (kVScale)
            grown |= with_scale(n, y, or_zero(m[n][y])) > mw[n][y] + kGrow || t > m[n][y] + 16.0f;
          else
            grown |= t > m[n][y] + kGrow;
        }
      if (__any_sync(kAll, grown)) {
#pragma unroll
        for (int n = 0; n < kNt; n++)
#pragma unroll
          for (int y = 0; y < 2; y++) {
            const float t = fmaxf(m[n][y], over_keys_max(top[n][y]));
            const float d = t == -INFINITY ? 0.0f : m[n][y] - t, al = ex2_approx(d);  // 0 on the row's first keys
            m[n][y] = t;
            l[n][y] *= al;
            float aw = al;
            if constexpr (kVScale) {
              // O's reference, relative to the new maximum, before and after
              const float old = mw[n][y] == -INFINITY ? -INFINITY : mw[n][y] + d;
              const float tw = fmaxf(old, over_keys_max(with_scale(n, y, or_zero(t))));
              aw = tw == -INFINITY ? 1.0f : ex2_approx(old - tw);
              mw[n][y] = tw;
            }
#pragma unroll
            for (int t2 = 0; t2 < kTiles; t2++) o[t2][n][y] *= aw, o[t2][n][2 + y] *= aw;
          }
      }
#pragma unroll
      for (int n = 0; n < kNt; n++)
#pragma unroll
        for (int y = 0; y < 2; y++) {
          const float sub = or_zero(m[n][y]);
          const float subw = kVScale ? or_zero(mw[n][y]) - kRaise : 0.0f;
#pragma unroll
          for (int i = 0; i < kG; i++) {
            float d0 = s[i][n][y] - sub, d1 = s[i][n][2 + y] - sub;
            if constexpr (!kVScale && kRaise != 0.0f) d0 += kRaise, d1 += kRaise;
            const float p0 = ex2_approx(d0), p1 = ex2_approx(d1);
            l[n][y] += p0 + p1;
            if constexpr (kVScale) {
              s[i][n][y] = ex2_approx(d0 + (vx[i][0] - subw));
              s[i][n][2 + y] = ex2_approx(d1 + (vx[i][1] - subw));
            } else {
              s[i][n][y] = p0, s[i][n][2 + y] = p1;
            }
          }
        }
#pragma unroll
      for (int i = 0; i < kG; i++)
#pragma unroll
        for (int n = 0; n < kNt; n++)
#pragma unroll
          for (int x = 0; x < 2; x++)
            p[i][n][x] = transpose8x8(kFmt == kBf16 ? bf2(s[i][n][2 * x], s[i][n][2 * x + 1])
                                                    : h2_of(s[i][n][2 * x], s[i][n][2 * x + 1]));
      // ---- O^T
      cp_async_wait<2 * kBuffers - 1>();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kG; i++) {
        S.take_v(buf, i, end - key0 - 16 * i);
        uint32_t sc[2] = {0, 0};
        if constexpr (kFmt == kNvfp4) {
          sc[0] = e4m3x2_to_h2(S.vs[0] | S.vs[1] << 8);
          sc[1] = e4m3x2_to_h2(S.vs[2] | S.vs[3] << 8);
        }
#pragma unroll
        for (int x = 0; x < P::kRow / 32; x++) {
          uint32_t va[P::kFrom][4];
          S.v_operands(x, sc, va);
#pragma unroll
          for (int y = 0; y < P::kFrom; y++)
#pragma unroll
            for (int n = 0; n < kNt; n++) mma16<kFmt>(o[P::kFrom * x + y][n], va[y], p[i][n][0], p[i][n][1]);
        }
      }
      // ---- and V's
      __syncwarp();
      if (all)
        P::template issue_v<true>(buf, c, next, end, 0, row);
      else if (next < end)
        P::template issue_v<false>(buf, c, next, end, gone_next, row);
      cp_async_commit();
      gone[0] = gone[1];
      gone[1] = gone_next;
      buf = buf == ring ? ring + P::kBuffer : ring;
    }

    // ---- the piece's results: rows 8n + 2q + y; M tile u has channels
    // channel(u), + 1 of the lane group
    auto channel = [&](int u) { return P::kVVals * (g + 8 * (2 * u / P::kVVals)) + 2 * u % P::kVVals; };
    const bool whole = walk.first && walk.last;
    const size_t slot = 2 * static_cast<size_t>(worker) + (walk.first ? 1 : 0);
#pragma unroll
    for (int n = 0; n < kNt; n++)
#pragma unroll
      for (int y = 0; y < 2; y++) {
        // the sum and o relative to the row's maximum (the first raised, but for E4M3)
        const float up = kVScale ? 1.0f : __uint_as_float((127u - static_cast<uint32_t>(kRaise)) << 23);
        const float sum = over_keys_sum(l[n][y]) * up;
        const int r = 8 * n + 2 * q + y;
        if (r >= rows) continue;
        float f = sum > 0.0f ? up : 0.0f;
        if constexpr (kVScale)
          if (sum > 0.0f) f = ex2_approx(mw[n][y] - kRaise);
        if (whole) {
          if (sum > 0.0f) f *= 1.0f / sum;
          const int rr = e.row0 + r, i = rr / a.G, gq = rr - i * a.G;
          const long long tok = e.q0 + i;
          const int hq = walk.h * a.G + gq;
          uint16_t* dst = a.o + tok * a.orow.t + hq * a.orow.h;
#pragma unroll
          for (int t = 0; t < kTiles; t += 4)
            *reinterpret_cast<uint4*>(dst + channel(t)) =
                uint4{bf2(o[t][n][y] * f, o[t][n][2 + y] * f), bf2(o[t + 1][n][y] * f, o[t + 1][n][2 + y] * f),
                      bf2(o[t + 2][n][y] * f, o[t + 2][n][2 + y] * f), bf2(o[t + 3][n][y] * f, o[t + 3][n][2 + y] * f)};
          if (a.lse && g == 0) a.lse[tok * a.Hq + hq] = sum > 0.0f ? (m[n][y] + lg2_approx(sum)) * kLn2 : -INFINITY;
        } else {
          float* dst = work.part_o + (slot * kRows + r) * D;
#pragma unroll
          for (int t = 0; t < kTiles; t += 2)
            *reinterpret_cast<float4*>(dst + channel(t)) =
                float4{o[t][n][y] * f, o[t][n][2 + y] * f, o[t + 1][n][y] * f, o[t + 1][n][2 + y] * f};
          if (g == 0) work.part_ml[slot * kRows + r] = float2{m[n][y], sum};
        }
      }
  }
}

template <int kFmt, int D, int kNt>
cudaError_t launch_rows(const KvView& c, const AttnArgs& a, const AttnWork& w, cudaStream_t st) {
  constexpr int kShared = kThreads / 32 * kBuffers * Step<kFmt, D>::kBuffer;
  static_assert((kNt == 1 ? 3 : 2) * (kShared + 1024) <= 228 * 1024, "shared memory of an SM");
  const cudaError_t e = set_shared_once<&step_kernel<kFmt, D, kNt>>(kShared);
  if (e != cudaSuccess) return e;
  return launch_after(step_kernel<kFmt, D, kNt>, dim3(w.workers / (kThreads / 32)), kThreads, kShared, st, c, a, w);
}

template <int kFmt, int D>
cudaError_t launch(const KvView& c, const AttnArgs& a, const AttnWork& w, int rows, cudaStream_t st) {
  return rows == 8 ? launch_rows<kFmt, D, 1>(c, a, w, st) : launch_rows<kFmt, D, 2>(c, a, w, st);
}

}  // namespace

cudaError_t launch_attn_step(const KvView& c, const AttnArgs& a, const AttnWork& w, int rows, int D, int format,
                             cudaStream_t st) {
  if (format == kBf16) return D == 64 ? launch<kBf16, 64>(c, a, w, rows, st) : launch<kBf16, 128>(c, a, w, rows, st);
  if (format == kE4m3) return D == 64 ? launch<kE4m3, 64>(c, a, w, rows, st) : launch<kE4m3, 128>(c, a, w, rows, st);
  return D == 64 ? launch<kNvfp4, 64>(c, a, w, rows, st) : launch<kNvfp4, 128>(c, a, w, rows, st);
}

}  // namespace sagefp4
