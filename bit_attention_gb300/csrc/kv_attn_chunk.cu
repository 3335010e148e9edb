// kv_attn_chunk.cu -- attention of many new tokens over the paged cache on the
// 5th-generation tensor cores.
//
// S = Q K^T and O += P V run as tcgen05.mma kind::f16, FP32 in tensor memory.  A
// CTA takes two row tiles of 128 query rows against one stream of KV tiles of
// 128 keys:
//   warpgroups 0, 1  softmax of row tile 0, 1: a thread owns a row; it reads
//                    its 128 scores from tensor memory, writes P over them as
//                    the A operand of P V, rescales O where a row maximum has
//                    grown by more than 2^8 (else P simply grows past its
//                    reference, up to 2^8), loads Q and writes the results
//   warpgroup 2      gathers K and V rows by page into the operand layout:
//                    copies of 16 bytes for bf16; codes through registers,
//                    converted, for the quantized formats
//   warpgroup 3      one warp issues the MMAs
// The two tiles alternate: while one's softmax works, the tensor cores compute
// the other's P V and next S; P V starts on the first 64 keys' P.
//
// Bound by that alternation: a pair of tiles takes 2050 cycles of MMA at the
// tensor cores' rate (2780 measured: S reads both operands from shared memory,
// at its bandwidth), and the chain of one tile's S, softmax and P V 3200.  A
// prompt of 8192 tokens, 32 query and 8 key/value heads of 128, bf16: 373 us,
// 1.47 PFLOP/s, tensor pipe busy 66%; 1121 new tokens over 37000 in E4M3, whose
// conversion keeps the gather at 3300 .. 3600 cycles a pair: 199 us, 1.12 PFLOP/s.
//
// Operand types.  For a bf16 cache both products are bf16.  For the quantized
// ones they are FP16, into which stored values convert in two instructions a
// pair instead of six (measured on 128 keys of E4M3: 840 cycles a tile instead
// of 2050): E2M1 codes times E4M3 scales are exact there, and E4M3 codes are
// multiplied by their scale relative to the largest scale of 32 keys (a warp's
// share of a tile), whose exponent enters the scores (K) or P's exponent (V); Scales
// below says where that is exact and what else is done.  Q's rows are scaled by the power
// of two that brings their largest magnitude to 2^14 .. 2^15: bf16's eight bits
// fit while a channel is above 2^-28 of it.  P is rounded to bf16 (2^-8
// relative) or FP16 (weights of 2^7 at the reference: 2^-11 relative down to
// 2^-21, 2^-32 below); the row sums take the FP32 values.
#include "kv_attn.cuh"
#include "umma.cuh"

namespace sagefp4 {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = kChunkRows;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.0f;  // log2 of how far P may grow past its reference before O is rescaled
// Registers of a thread of the softmax, gather and control warpgroups; twice
// the first and the others make 512, four times the launch's 128.  Converting
// wants more than copying: over E4M3, 400 tokens against 16000 in 3 sequences,
// 104 for it 210 us, 112 (176 for the softmax) 228, 88 290; over bf16, a prompt
// of 8192 tokens, 96 396 us, 104 (40 for control) 418.
template <int kFmt>
struct Regs {
  static constexpr uint32_t kSoft = 184, kGather = kFmt == kBf16 ? 96 : 104, kCtl = kFmt == kBf16 ? 48 : 40;
  static_assert(2 * kSoft + kGather + kCtl == 512, "register split");
};

template <int D>
struct Smem {
  static constexpr int kHalf = 128 * 128;             // 128 rows of 64 bf16 values
  static constexpr int kOperand = D / 64 * kHalf;     // one Q, K or V tile
  static constexpr int kSlots = D == 64 ? 8 : 4;      // ring of K and V tiles, alternating
  static constexpr int kQ = 0;                        // two row tiles
  static constexpr int kRing = 2 * kOperand;
  static constexpr int kStage = kRing + kSlots * kOperand;  // [8 softmax warps][32 rows][64 channels] of results
  static constexpr int kBar = kStage + 8 * 4096;
  static constexpr int kMask = kBar + 32 * 8;         // [8 tiles][4] words: keys that exist
  static constexpr int kScale = kMask + 8 * 16;       // [8 tiles][4] log2 of V's scale of 32 keys (E4M3)
  static constexpr int kKScale = kScale + 8 * 16;     // [8 tiles][4] K's scale of 32 keys (E4M3), 0: wide
  static constexpr int kBytes = kKScale + 8 * 16;     // [kInfo tiles][2][128] scale bytes of K and V (E4M3, wide rows)
  static constexpr int kInfo = D == 64 ? 8 : 4;       // (a tile's are read before the one three tiles on is written)
  static constexpr int kMisc = kBytes + kInfo * 256;        // tensor-memory address, abort flag, V scales
                                                           // seen, pieces to redo [8 softmax warps]
  static constexpr int kAlloc = kMisc + 48 + 1024;    // with room to align to 1024
};
static_assert(Smem<128>::kAlloc <= 227 * 1024 && Smem<64>::kAlloc <= 227 * 1024, "shared memory");

enum {
  B_FULL = 0,    // + slot: the tile is in shared memory
  B_EMPTY = 8,   // + slot: the MMAs that read it have completed
  B_QFULL = 16,  // + row tile: the piece's Q is in shared memory
  B_QEMPTY = B_QFULL + 2,  // every S of the piece has completed
  B_S,           // + row tile: S is in tensor memory (and the P V before it in O)
  B_P = B_S + 2, // + 2 * row tile + half: P of 64 keys is in tensor memory
  B_O = B_P + 4, // + row tile: the piece's last P V has completed
  B_OFREE = B_O + 2,  // + row tile: the piece's O has been read
  B_DRAIN = B_OFREE + 2,
  B_COUNT
};
static_assert(B_COUNT <= 32, "barriers");

// tensor-memory columns: S (P over its first 64), O
constexpr uint32_t kTmS = 0, kTmO = 256;

// Rows of an entry, up to kRows.
__device__ __forceinline__ int entry_rows(const PlanEntry& e, int G) { return min(e.nq * G - e.row0, kRows); }

__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// An E4M3 byte -> that FP16 value twice.
__device__ __forceinline__ uint32_t e4m3_to_h2(uint32_t byte) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(byte * 0x101u)));
  return r;
}

// Eight E4M3 codes -> four FP16 pairs, exact.
__device__ __forceinline__ void e4m3x8_to_h2(uint32_t lo, uint32_t hi, uint32_t (&h)[4]) {
  uint32_t a[2], b[2];
  e4m3x4_to_h2(lo, a);
  e4m3x4_to_h2(hi, b);
  h[0] = a[0], h[1] = a[1], h[2] = b[0], h[3] = b[1];
}

// Two bf16 values times f -> FP16.
__device__ __forceinline__ uint32_t bf2_to_h2(uint32_t w, float f) {
  return h2_of(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
}

// The bits 0 .. n - 1 of a word (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? kAll : (1u << n) - 1u;
}

// ------------------------------------------------------------------ gather
// A warp's 32 rows of a tile: the codes of a lane's share of them in registers,
// in pieces of 16 channels, D / 16 lanes to a row.  Rows 16 g .. of the warp's 32
// are neighbours in the cache (a page has 16 tokens or more), so two addresses
// make all of them (an address of each row by shuffles: attention of 400 tokens
// over 16000 in E4M3, 3 sequences, 249 us; this 212).
template <int kFmt, int D>
struct Gather {
  static constexpr int kBytes = row_bytes<kFmt>(D);
  static constexpr int kWords = kFmt == kE4m3 ? 4 : 2;  // of a piece
  static constexpr int kLanes = D / 16, kSteps = kLanes, kStep = 32 / kLanes;
  uint32_t code[kSteps][kWords];
  uint32_t scale[kFmt == kNvfp4 ? kSteps : 1];  // E4M3: of the lane's own row; NVFP4: of its pieces

  // E4M3: the scale of the lane's own row, -1: none (asked for before the codes, which
  // are wanted later)
  __device__ __forceinline__ void load_scale(const uint8_t* scales, long long row) { scale[0] = row >= 0 ? scales[row] : 0u; }

  // row: this lane's row of the cache (key 32 * warp + lane of the tile), or -1;
  // here: the lanes that have one, of each 16 the first ones
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, long long row, uint32_t here) {
    const int lane = threadIdx.x & 31, q = lane / kLanes, c = lane % kLanes;
    const uint8_t *from[2], *sc[2];
#pragma unroll
    for (int g = 0; g < 2; g++) {
      const long long r = __shfl_sync(kAll, row, 16 * g) + q;
      from[g] = codes + r * kBytes + 4 * kWords * c;
      if constexpr (kFmt == kNvfp4) sc[g] = scales + r * (D / 16) + c;
    }
    // (not kept in L1, which shared memory leaves little of)
    auto get = [&](int i, bool on) {
      const int g = i * kStep / 16, o = i * kStep % 16;
      if constexpr (kWords == 4) {
        const uint4 v = on ? __ldcg(reinterpret_cast<const uint4*>(from[g] + o * kBytes)) : uint4{0, 0, 0, 0};
        code[i][0] = v.x, code[i][1] = v.y, code[i][2] = v.z, code[i][3] = v.w;
      } else {
        const uint2 v = on ? __ldcg(reinterpret_cast<const uint2*>(from[g] + o * kBytes)) : uint2{0, 0};
        code[i][0] = v.x, code[i][1] = v.y;
        scale[i] = on ? __ldcg(sc[g] + o * (D / 16)) : 0u;
      }
    };
    if (here == kAll) {
#pragma unroll
      for (int i = 0; i < kSteps; i++) get(i, true);
    } else {
#pragma unroll
      for (int i = 0; i < kSteps; i++) get(i, (here >> (i * kStep + q)) & 1);
    }
  }

  // The rows as FP16 (E4M3: times `mine`, an FP16 pair, of the lane's own row) to the
  // tile's rows from base (a multiple of 32) on.  Chunk ch (8 channels) of row r stands at
  // chunk ch ^ (r & 7) of the row's 128 bytes.  For D = 128, where a row's second
  // four lanes write the other half of the tile, those take their pieces' second
  // chunks first, so that eight lanes' 16 bytes fall into eight bank groups.
  __device__ __forceinline__ void store(uint32_t tile, int base, uint32_t mine) const {
    const int lane = threadIdx.x & 31, q = lane / kLanes, c = lane % kLanes;
    const bool x = c >= 4;
    const uint32_t rows = tile + (c >> 2) * (128 * 128) + (base + q) * 128;
    const int ch = 2 * (c & 3) + x;
#pragma unroll
    for (int i = 0; i < kSteps; i++) {
      const uint32_t f = kFmt == kE4m3 ? __shfl_sync(kAll, mine, i * kStep + q) : e4m3_to_h2(scale[kFmt == kNvfp4 ? i : 0]);
      const uint32_t at = rows + i * kStep * 128 + ((ch ^ ((q + i * kStep) & 7)) << 4);
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const bool second = (k != 0) != x;
        uint32_t h[4];
        if constexpr (kFmt == kE4m3)
          e4m3x8_to_h2(second ? code[i][2] : code[i][0], second ? code[i][3] : code[i][1], h);
        else
          e2m1x8_to_h2(second ? code[i][1] : code[i][0], h);
        st_shared16(at ^ (k << 4), uint4{mul_h2(h[0], f), mul_h2(h[1], f), mul_h2(h[2], f), mul_h2(h[3], f)});
      }
    }
  }
};

// E4M3: the scales of a warp's 32 rows of a tile.  Codes are multiplied by 2^7 (so
// that they use FP16's range) and by their scale relative to the largest of the 32,
// which enters the scores (K) or P's exponents (V), as long as little is lost by it:
// K scales within 2^21 (exact in FP16: 18 + 21 bits from 2^15.8 down), V scales within
// 2^8 or of rows of zeros.  (V's values are exact then; P is relative to the largest
// weight times that scale and its smallest step 2^-32 of it, so that among 32 values of
// like sizes a weight is off by 2^-32 of the largest, and by 2^-24 at the limit.)  The
// others are `wide`: codes are taken without their scales, which the softmax then
// applies to each key; a tile of these takes six times as long.
// A scale byte of 17 (a row of zeros, or below 2^-101 in magnitude) is taken for zeros;
// V's scales count as 2^-80 at least, so that the row sum, relative to weights that
// count V's scale, stays within FP32, and lower rows lose bits (half a step 2^-112).
struct Scales {
  static constexpr uint32_t kZero = 17, kLeastV = 47, kSpreadK = 21, kSpreadV = 8;
  // a share whose V scales are further apart may leave weights of the least out of
  // the row sum: its rows are done again
  static constexpr int kMostV = 92;
  static constexpr uint32_t kBias = 127 + 7;
  uint32_t top_k, top_v, mine_k, mine_v;  // largest; this lane's factors
  uint32_t seen;                          // V's scales in eights, a bit each
  bool wide;

  static __device__ __forceinline__ uint32_t largest(uint32_t v) {
    uint32_t r;
    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(r) : "r"(v));
    return r;
  }
  static __device__ __forceinline__ uint32_t smallest(uint32_t v) {
    uint32_t r;
    asm volatile("redux.sync.min.u32 %0, %1, 0xffffffff;" : "=r"(r) : "r"(v));
    return r;
  }
  // 2^(7 - d) as an FP16 pair
  static __device__ __forceinline__ uint32_t factor(uint32_t d) {
    const float f = __uint_as_float((kBias - d) << 23);
    return h2_of(f, f);
  }
  // k, v: the lane's scale bytes, 0 where it has no row
  __device__ __forceinline__ Scales(uint32_t k, uint32_t v) {
    const bool kz = k <= kZero, vz = v <= kZero;
    const uint32_t least = v < kLeastV ? kLeastV : v;
    top_k = largest(kz ? kZero + 1 : k);
    top_v = largest(least);
    wide = top_k > smallest(kz ? 255u : k) + kSpreadK || top_v > smallest(vz ? 255u : least) + kSpreadV;
    mine_k = kz ? 0u : factor(wide ? 0 : top_k - k);
    mine_v = vz ? 0u : factor(wide ? least - v : top_v - v);
    seen = 1u << (top_v / 8);
    // (a wide share's weights are summed by themselves: only the sum's own range counts)
    if (wide) seen |= 1u << (min(smallest(v ? least : 255u) + (126 - kMostV), 255u) / 8);
  }
  // of a CTA's shares
  static __device__ __forceinline__ bool apart(uint32_t all) { return all && (31 - __clz(all)) - (__ffs(all) - 1) > kMostV / 8 - 1; }
};

// 32 bf16 rows to an operand tile by asynchronous 16-byte copies; a missing
// row (-1) becomes zeros.
template <int D>
__device__ __forceinline__ void copy_rows(uint32_t tile, int base, const uint8_t* src, long long row_off) {
  constexpr int kPer = D / 8, kStep = 32 / kPer;
  const int lane = threadIdx.x & 31, ch = lane % kPer;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const long long off = __shfl_sync(kAll, row_off, i * kStep + lane / kPer);
    const int r = base + i * kStep + lane / kPer;
    cp_async16(tile + (ch >> 3) * (128 * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4), src + (off >= 0 ? off : 0) + 16 * ch,
               off >= 0);
  }
}

// ------------------------------------------------------------------ softmax
// kWipe: an infinite O becomes 0 by a factor of 0.  (FP16 weights need it not: what an
// infinite one leaves in every channel of O shows later.)
template <int D, bool kWipe = false>
__device__ __forceinline__ void rescale_o(uint32_t tO, float alpha) {
#pragma unroll 1
  for (int j = 0; j < D; j += 8) {
    uint32_t o[8];
    tmem_ld8(tO + j, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; e++) o[e] = !kWipe || alpha > 0.0f ? __float_as_uint(__uint_as_float(o[e]) * alpha) : 0u;
    tmem_st8(tO + j, o);
  }
  tmem_wait_st();
}

struct Row {
  float ref, l;  // what a thread's row is relative to, its sum
};

// A tile with wide rows (E4M3), each score by itself: a call that reads them from
// tensor memory twice, eight at a time, so that the fast path keeps its registers.
template <int D>
__device__ __noinline__ Row wide_tile(uint32_t tS, uint32_t tO, uint32_t bar_p, uint32_t info, uint32_t bytes, int see0, int see1, float factor, Row x) {
  constexpr float kRaise = 7.0f;
  using L = Smem<D>;
  const uint32_t mask = info + L::kMask, kscale = info + L::kKScale, vlog = info + L::kScale;
  // keys c .. c + 7: log2 scores (-inf: not seen), and the exponents of V's scales
  auto look = [&](int c, float (&u)[8], float (&v)[8]) {
    uint32_t r[8];
    tmem_ld8(tS + c, r);
    const int g = c >> 5;
    const uint32_t on = (ld_shared4(mask + 4 * g) & bits_below(see1 - 32 * g) & ~bits_below(see0 - 32 * g)) >> (c & 31);
    const float kf = __uint_as_float(ld_shared4(kscale + 4 * g)), vx = __uint_as_float(ld_shared4(vlog + 4 * g));
    const uint32_t kb[2] = {ld_shared4(bytes + c), ld_shared4(bytes + c + 4)};
    const uint32_t vb[2] = {ld_shared4(bytes + 128 + c), ld_shared4(bytes + 128 + c + 4)};
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const uint32_t k = (kb[e / 4] >> (8 * (e % 4))) & 255u, w = (vb[e / 4] >> (8 * (e % 4))) & 255u;
      const float f = kf > 0.0f ? kf : k > Scales::kZero ? __uint_as_float((k + 127 - Scales::kBias) << 23) : 0.0f;
      v[e] = kf > 0.0f ? vx : static_cast<float>(static_cast<int>(max(w, Scales::kLeastV) - Scales::kBias));
      u[e] = (on >> e) & 1 ? __uint_as_float(r[e]) * (factor * f) : -INFINITY;
    }
  };
  float u[8], v[8], top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < kTile; c += 8) {
    look(c, u, v);
#pragma unroll
    for (int e = 0; e < 8; e++) top = fmaxf(top, u[e] + v[e]);
  }
  if (__any_sync(kAll, top > x.ref + kGrow)) {
    const float to = fmaxf(x.ref, top), alpha = to == -INFINITY ? 1.0f : ex2_approx(x.ref - to);
    x.ref = to;
    const bool some = __any_sync(kAll, x.l > 0.0f);
    x.l *= alpha;
    if (some) rescale_o<D>(tO, alpha);
  }
  const float sub = (x.ref == -INFINITY ? 0.0f : x.ref) - kRaise;
#pragma unroll 1
  for (int c = 0; c < kTile; c += 8) {
    look(c, u, v);
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const float d0 = u[2 * e] - sub, d1 = u[2 * e + 1] - sub;
      x.l += ex2_approx(d0) + ex2_approx(d1);
      p[e] = h2_of(ex2_approx(d0 + v[2 * e]), ex2_approx(d1 + v[2 * e + 1]));
    }
    tmem_st4(tS + c / 2, p);  // over scores that have been read
    if (c % 64 == 56) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(bar_p + 8 * (c / 64));
    }
  }
  return x;
}

// ------------------------------------------------------------------ rows of huge scores
// The tile loop takes a row's reference from a score times its factor with one
// rounding, the sum of that and P's raise with another.  Beyond 2^19 (log2
// units) these no longer leave P's exponents where FP16 and FP32 hold them.  Pieces
// of a warp's rows in which a reference ends there, or whose sum or O an infinite
// weight has gone through (every channel of O then), are done again here, a row at a
// time: every score is rounded first and the largest subtracted before anything
// else.  So it is for any row of finite scores; how long it takes matters little,
// while a second path in the tile loop cost 2 to 9% of that.
constexpr float kHuge = 0x1p19f;

// Of the piece that the walk is at, the warp's rows from `at` of the entry on;
// results go where the tile loop's went.
template <int kFmt, int D>
__device__ __forceinline__ void redo_rows(const KvView& c, const AttnArgs& a, const AttnWork& work, const Walk& walk, int at) {
  constexpr int kC = D / 8, kG = 32 / kC;
  const int lane = threadIdx.x & 31, ch = lane % kC, grp = lane / kC;
  const int slot = walk.first && walk.last ? -1 : 2 * static_cast<int>(blockIdx.x) + (walk.first ? 1 : 0);
  const PlanEntry en = walk.entry(work);
  const int b = en.b, h = walk.h;
  auto each = [](const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; i++) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  };
  for (int r = 0; r < 32 && at + r < entry_rows(en, a.G); r++) {
    const int rr = en.row0 + at + r, i = rr / a.G, hq = h * a.G + rr - i * a.G;
    const long long tok = en.q0 + i;
    const uint16_t* qr = a.q + tok * a.qr.t + hq * a.qr.h;
    const int2 see = key_range(a, en.len, en.nq, i);
    const int first = max(walk.t * kTile, see.x), end = min((walk.t + walk.tiles) * kTile, see.y);
    float top = -INFINITY, l = 0.0f, o[8] = {};
    for (int j0 = first; j0 < end; j0 += 32) {
      // a lane's key, then a lane group's channels of every kG-th key's value
      const long long row = j0 + lane < end ? row_of(c, b, h, j0 + lane) : -1;
      float s = row >= 0 ? 0.0f : -INFINITY;
#pragma unroll 1
      for (int x = 0; x < kC; x++) {
        float k[8], f[8];
        each(*reinterpret_cast<const uint4*>(qr + 8 * x), f);
        each(row >= 0 ? load_chunk<kFmt, D>(c.kc, c.ks, row, x) : uint4{0, 0, 0, 0}, k);
#pragma unroll
        for (int e = 0; e < 8; e++) s = fmaf(f[e], k[e], s);
      }
      s = row >= 0 ? __fmul_rn(s, a.scale_log2) : -INFINITY;
      float to = s;
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) to = fmaxf(to, __shfl_xor_sync(kAll, to, i));
      to = fmaxf(top, to);
      if (to == -INFINITY) continue;
      const float alpha = ex2_approx(top - to), p = ex2_approx(s - to);
      top = to;
      l = fmaf(l, alpha, p);  // a lane's own keys
#pragma unroll
      for (int e = 0; e < 8; e++) o[e] *= alpha;
#pragma unroll 1
      for (int i = grp; i < 32; i += kG) {
        const long long vr = __shfl_sync(kAll, row, i);
        const float pi = __shfl_sync(kAll, p, i);
        float v[8];
        each(vr >= 0 ? load_chunk<kFmt, D>(c.vc, c.vs, vr, ch) : uint4{0, 0, 0, 0}, v);
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = fmaf(pi, v[e], o[e]);
      }
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) {
      l += __shfl_xor_sync(kAll, l, i);
#pragma unroll
      for (int e = 0; e < 8; e++) o[e] += i >= kC ? __shfl_xor_sync(kAll, o[e], i) : 0.0f;
    }
    if (slot < 0) {
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      uint16_t* dst = a.o + tok * a.orow.t + hq * a.orow.h + 8 * ch;
      if (grp == 0)
        *reinterpret_cast<uint4*>(dst) = uint4{bf2(o[0] * inv, o[1] * inv), bf2(o[2] * inv, o[3] * inv),
                                               bf2(o[4] * inv, o[5] * inv), bf2(o[6] * inv, o[7] * inv)};
      if (a.lse && lane == 0) a.lse[tok * a.Hq + hq] = l > 0.0f ? (top + lg2_approx(l)) * kLn2 : -INFINITY;
    } else {
      float4* part = reinterpret_cast<float4*>(work.part_o) + static_cast<size_t>(slot) * (D / 4) * kRows + at + r;
      if (grp == 0) {
        part[static_cast<size_t>(2 * ch) * kRows] = float4{o[0], o[1], o[2], o[3]};
        part[static_cast<size_t>(2 * ch + 1) * kRows] = float4{o[4], o[5], o[6], o[7]};
      }
      if (lane == 0) work.part_ml[static_cast<size_t>(slot) * kRows + at + r] = float2{top, l};
    }
  }
}

// Of all the CTA's pieces, those whose bit is set (the last bit: of the 32nd and all
// after it), once the tile loops are through and nobody waits for this warp.
template <int kFmt, int D>
__device__ __noinline__ void redo_pieces(const KvView& c, const AttnArgs& a, const AttnWork& work, uint32_t pieces, int at) {
  Walk walk(work, c.H, blockIdx.x);
  for (int n = 0; walk.next(work);) {
    if (walk.tiles == 0 || (at & 128) >= entry_rows(walk.entry(work), a.G)) continue;
    if ((pieces >> min(n++, 31)) & 1) redo_rows<kFmt, D>(c, a, work, walk, at);
  }
}

// ------------------------------------------------------------------ kernel
template <int kFmt, int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ KvView c, const __grid_constant__ AttnArgs a, const __grid_constant__ AttnWork work) {
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
  auto bar = [&](int i) { return sbase + L::kBar + 8 * i; };
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  uint32_t* spread = reinterpret_cast<uint32_t*>(smem + L::kMisc + 8);
  uint32_t* lost = reinterpret_cast<uint32_t*>(smem + L::kMisc + 16);
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + L::kMask);
  float* vlog = reinterpret_cast<float*>(smem + L::kScale);
  float* kscale = reinterpret_cast<float*>(smem + L::kKScale);
  constexpr bool kHalf = kFmt != kBf16;     // FP16 operands
  constexpr bool kScales = kFmt == kE4m3;   // K's and V's scales enter the scores and P
  constexpr float kRaise = kHalf ? 7.0f : 0.0f;
  const WaitCtl ctl{c.status, abort, work.wait_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kSlots; s++) {
      mbar_init(bar(B_FULL + s), 4);   // the gather's warps
      mbar_init(bar(B_EMPTY + s), 1);  // commit
    }
    mbar_init(bar(B_QEMPTY), 1);
    for (int m = 0; m < 2; m++) {
      mbar_init(bar(B_QFULL + m), 4);
      mbar_init(bar(B_S + m), 1);
      mbar_init(bar(B_P + 2 * m), 4);
      mbar_init(bar(B_P + 2 * m + 1), 4);
      mbar_init(bar(B_O + m), 1);
      mbar_init(bar(B_OFREE + m), 4);
    }
    mbar_init(bar(B_DRAIN), 1);
    *abort = 0;
    *spread = 0;
    for (int i = 0; i < 8; i++) lost[i] = 0;
    mbar_fence_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_addr(tslot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  griddep_launch_dependents();
  griddep_wait();  // the plan
  Walk walk(work, c.H, blockIdx.x);

  if (wg < 2) {
    // ---- softmax of row tile m
    regs_inc<Regs<kFmt>::kSoft>();
    const int m = wg, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes + kTmS + 128 * m, tO = tmem + lanes + kTmO + 128 * m;
    const int r = 128 * m + row;  // of the entry
    int g = 0, pieces = 0, tile0 = 0, q_pieces = 0;  // tiles and pieces of this row tile so far, and of the CTA
    bool ok = true;
    if (threadIdx.x == 0) work.open[blockIdx.x] = int2{-1, 0};
    // A piece as this thread sees it.
    struct Mine {
      long long out, lse;  // where its row goes (elements; -1: no such row)
      int2 see;            // keys that it sees
      int t, tiles, slot;  // KV tiles; where partial results go (-1: the piece is the whole entry)
      float factor;        // from accumulator to score (log2 units), but for K's scales
      bool on;             // the entry has this row tile
    };
    // The next piece, with its Q brought into operand form (while the piece
    // before it still waits for its last product).  Rows that see no key are
    // written on the way.
    auto open = [&](Mine& x) {
      while (walk.next(work)) {
        const PlanEntry e = walk.entry(work);
        const int rows = entry_rows(e, a.G), rr = e.row0 + r, i = rr / a.G, hq = walk.h * a.G + rr - i * a.G;
        const bool live = r < rows;
        const long long tok = e.q0 + i;
        x.out = live ? tok * a.orow.t + hq * a.orow.h : -1;
        x.lse = tok * a.Hq + hq;
        x.see = live ? key_range(a, e.len, e.nq, i) : int2{0, 0};
        x.t = walk.t, x.tiles = walk.tiles;
        x.slot = walk.first && walk.last ? -1 : 2 * static_cast<int>(blockIdx.x) + (walk.first ? 1 : 0);
        if (threadIdx.x == 0 && walk.first && !walk.last) work.open[blockIdx.x] = int2{walk.j - 1, walk.h};
        x.on = 128 * m < rows;
        x.factor = a.scale_log2;
        if (walk.tiles == 0) {
          if (live) {
#pragma unroll
            for (int j = 0; j < D; j += 8) *reinterpret_cast<uint4*>(a.o + x.out + j) = uint4{0, 0, 0, 0};
            if (a.lse) a.lse[x.lse] = -INFINITY;
          }
          continue;
        }
        if (q_pieces > 0 && !(ok = wait_warp(bar(B_QEMPTY), (q_pieces - 1) & 1, ctl))) return false;
        if (x.on) {
          // the warp's 32 rows, whole rows by D / 8 lanes
          const long long off = live ? 2 * (tok * a.qr.t + hq * a.qr.h) : -1;
          copy_rows<D>(sbase + L::kQ + m * L::kOperand, 32 * (warp & 3), reinterpret_cast<const uint8_t*>(a.q), off);
          cp_async_commit();
          cp_async_wait<0>();
          if constexpr (kHalf) {
            __syncwarp();
            const uint32_t dst = sbase + L::kQ + m * L::kOperand + 128 * row;
            auto at = [&](int j) { return dst + (j >> 3) * (128 * 128) + (((j & 7) ^ (row & 7)) << 4); };
            uint32_t top = 0;  // the row's largest magnitude, as bf16 bits in either half
            uint4 v[D / 8];
#pragma unroll
            for (int j = 0; j < D / 8; j++) {
              v[j] = ld_shared16(at(j));
              top = __vmaxu2(__vmaxu2(__vmaxu2(top, v[j].x & 0x7fff7fffu), __vmaxu2(v[j].y & 0x7fff7fffu, v[j].z & 0x7fff7fffu)),
                             v[j].w & 0x7fff7fffu);
            }
            top = max(top & 0xffffu, top >> 16);
            const int up = min(14 + 127 - static_cast<int>(top >> 7), 126);
            const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            x.factor *= __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
            for (int j = 0; j < D / 8; j++)
              st_shared16(at(j), uint4{bf2_to_h2(v[j].x, f), bf2_to_h2(v[j].y, f), bf2_to_h2(v[j].z, f), bf2_to_h2(v[j].w, f)});
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_QFULL + m));
        q_pieces++;
        return true;
      }
      return false;
    };
    // The rows of Q of the entry after the current piece's, towards L2.
    auto prefetch_q = [&]() {
      if (walk.left == 0) return;
      const bool wrap = walk.j == work.head->entries;
      const PlanEntry e = work.entry[wrap ? 0 : walk.j];
      const int rr = e.row0 + r, i = rr / a.G, hq = (walk.h + wrap) * a.G + rr - i * a.G;
      if (r < entry_rows(e, a.G)) {
        const uint16_t* q = a.q + (e.q0 + i) * a.qr.t + hq * a.qr.h;
#pragma unroll
        for (int j = 0; j < D; j += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + j));
      }
    };
    Mine cur;
    bool have = open(cur);
    while (have) {
      prefetch_q();
      // what P and O are relative to (log2 units; with V's scale, where that
      // enters), and the row sum, relative to the same
      float ref = -INFINITY, l = 0.0f;
      for (int k = 0; cur.on && k < cur.tiles; k++, g++) {
        if (!(ok = wait_warp(bar(B_S + m), g & 1, ctl))) break;
        tc_fence_after();
        if constexpr (kScales) {
          const float4 f = *reinterpret_cast<const float4*>(kscale + 4 * ((tile0 + k) & 7));
          if (fminf(fminf(f.x, f.y), fminf(f.z, f.w)) == 0.0f) {
            const int t = tile0 + k, at = 4 * (t & 7), k0 = (cur.t + k) * kTile;
            const Row x = wide_tile<D>(tS, tO, bar(B_P + 2 * m), sbase + 4 * at,
                                       sbase + L::kBytes + 256 * (t % L::kInfo), cur.see.x - k0, cur.see.y - k0, cur.factor,
                                       Row{ref, l});
            ref = x.ref, l = x.l;
            continue;
          }
        }
        uint32_t s[4][32];
        float t[4];  // maxima of 32 scores each
#pragma unroll
        for (int j = 0; j < 4; j++) tmem_ld32_max(tS + 32 * j, s[j], t[j]);
        const uint4 mw = *reinterpret_cast<const uint4*>(mask + 4 * ((tile0 + k) & 7));
        // of the keys 32 j ..: from accumulator to score, and the exponent of V's scale
        float cx[4] = {cur.factor, cur.factor, cur.factor, cur.factor}, vx[4] = {};
        if constexpr (kScales) {
          const float4 f = *reinterpret_cast<const float4*>(kscale + 4 * ((tile0 + k) & 7));
          const float4 v = *reinterpret_cast<const float4*>(vlog + 4 * ((tile0 + k) & 7));
          cx[0] *= f.x, cx[1] *= f.y, cx[2] *= f.z, cx[3] *= f.w;
          vx[0] = v.x, vx[1] = v.y, vx[2] = v.z, vx[3] = v.w;
        }
        tmem_wait_ld();
        const int k0 = (cur.t + k) * kTile;
        const int2 see = cur.see;
        const bool whole = (mw.x & mw.y & mw.z & mw.w) == kAll && see.x <= k0 && see.y >= k0 + kTile;
        if (!__all_sync(kAll, whole)) {
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const uint32_t on = (j == 0 ? mw.x : j == 1 ? mw.y : j == 2 ? mw.z : mw.w) & bits_below(see.y - k0 - 32 * j) &
                                ~bits_below(see.x - k0 - 32 * j);
#pragma unroll
            for (int e = 0; e < 32; e++)
              if (!(on & (1u << e))) s[j][e] = __float_as_uint(-INFINITY);
            // a factor that has underflowed (a row of zeros) would make NaN of these;
            // any small one gives the same scores to the others
            cx[j] = fmaxf(cx[j], 1.1754944e-38f);
            t[j] = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 2) t[j] = max3f(t[j], __uint_as_float(s[j][e]), __uint_as_float(s[j][e + 1]));
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; j++)
          top = fmaxf(top, fmaf(t[j], cx[j], vx[j]));
        // also from -inf, on the row's first visible keys
        if (__any_sync(kAll, top > ref + kGrow)) {
          const float to = fmaxf(ref, top);
          const float alpha = to == -INFINITY ? 1.0f : ex2_approx(ref - to);
          ref = to;
          const bool some = __any_sync(kAll, l > 0.0f);  // else O holds nothing, or nothing yet
          l *= alpha;
          if (some) rescale_o<D, !kHalf>(tO, alpha);
        }
        const float sub = (ref == -INFINITY ? 0.0f : ref) - kRaise;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float cj = cx[j], vj = vx[j];
          const uint64_t c2 = pack2(cj, cj), n2 = pack2(vj - sub, vj - sub);
          uint64_t acc0 = 0, acc1 = 0;
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; e++) {
            const uint64_t y = fma2(pack2(__uint_as_float(s[j][2 * e]), __uint_as_float(s[j][2 * e + 1])), c2, n2);
            const float p0 = ex2_approx(lo2(y)), p1 = ex2_approx(hi2(y));
            if (e & 1)
              acc1 = add2(acc1, pack2(p0, p1));
            else
              acc0 = add2(acc0, pack2(p0, p1));
            p[e] = kHalf ? h2_of(p0, p1) : bf2(p0, p1);
          }
          const uint64_t acc = add2(acc0, acc1);
          const float sum = lo2(acc) + hi2(acc);
          l = kScales ? fmaf(sum, ex2_approx(-vj), l) : l + sum;
          tmem_st16(tS + 16 * j, p);
          if (j & 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P + 2 * m + (j >> 1)));
          }
        }
      }
      if (!ok) break;
      tile0 += cur.tiles;
      Mine next;
      have = open(next);
      if (!ok) break;
      if (cur.on) {
        // ---- the piece's results
        if (!(ok = wait_warp(bar(B_O + m), pieces & 1, ctl))) break;
        tc_fence_after();
        const float base = ref - kRaise;  // l is the sum of 2^(score - base)
        if (cur.slot < 0) {
          // through shared memory, 64 channels at a time, so that eight lanes write
          // 128 consecutive bytes of a row
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
          const uint32_t stage = sbase + L::kStage + 4096 * warp;
          long long to[8];
#pragma unroll
          for (int n = 0; n < 8; n++) to[n] = __shfl_sync(kAll, cur.out, 4 * n + (lane >> 3));
          const int ch = lane & 7;
#pragma unroll
          for (int j = 0; j < D; j += 64) {
            __syncwarp();
#pragma unroll
            for (int x0 = 0; x0 < 8; x0 += 4) {
              uint32_t o[32];
              tmem_ld32(tO + j + 8 * x0, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 4; x++) {
                uint32_t w[4];
#pragma unroll
                for (int n = 0; n < 4; n++) {
                  const uint32_t* v = &o[8 * x + 2 * n];
                  w[n] = l > 0.0f ? bf2(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv) : 0u;
                }
                st_shared16(stage + 128 * lane + (((x0 + x) ^ (lane & 7)) << 4), uint4{w[0], w[1], w[2], w[3]});
              }
            }
            __syncwarp();
#pragma unroll
            for (int n = 0; n < 8; n++) {
              const int r4 = 4 * n + (lane >> 3);
              const uint4 v = ld_shared16(stage + 128 * r4 + ((ch ^ (r4 & 7)) << 4));
              if (to[n] >= 0) *reinterpret_cast<uint4*>(a.o + to[n] + j + 8 * ch) = v;
            }
          }
          if (cur.out >= 0 && a.lse) a.lse[cur.lse] = l > 0.0f ? (base + lg2_approx(l)) * kLn2 : -INFINITY;
        } else {
          float4* part = reinterpret_cast<float4*>(work.part_o) + static_cast<size_t>(cur.slot) * (D / 4) * kRows + r;
#pragma unroll
          for (int j = 0; j < D; j += 32) {
            uint32_t o[32];
            __syncwarp();
            tmem_ld32(tO + j, o);
            tmem_wait_ld();
            if (cur.out >= 0) {
#pragma unroll
              for (int n = 0; n < 8; n++)
                part[static_cast<size_t>(j / 4 + n) * kRows] =
                    float4{__uint_as_float(o[4 * n]), __uint_as_float(o[4 * n + 1]), __uint_as_float(o[4 * n + 2]),
                           __uint_as_float(o[4 * n + 3])};
            }
          }
          if (cur.out >= 0) work.part_ml[static_cast<size_t>(cur.slot) * kRows + r] = float2{l > 0.0f ? base : -INFINITY, l};
        }
        uint32_t o[8];
        __syncwarp();
        tmem_ld8(tO, o);
        tmem_wait_ld();
        pieces++;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_OFREE + m));
        const bool gone = fabsf(ref) > kHuge || !(l < INFINITY) || !(fabsf(__uint_as_float(o[0])) < INFINITY);
        if (__any_sync(kAll, cur.out >= 0 && ref != -INFINITY && gone) && lane == 0) lost[warp] |= 1u << min(pieces - 1, 31);
      }
      cur = next;
    }
    __syncwarp();
    const uint32_t redo = kScales && __any_sync(kAll, Scales::apart(*spread)) ? kAll : lost[warp];
    if (ok && redo) redo_pieces<kFmt, D>(c, a, work, redo, 128 * m + 32 * (warp & 3));
    tc_fence_before();
  } else if (wg == 2) {
    // ---- gather: warp w of four takes keys 32 w .. of every tile
    regs_dec<Regs<kFmt>::kGather>();
    const int w = warp & 3;
    int n = 0, tiles = 0;  // slots filled so far, tiles of the CTA
    bool ok = true;
    auto filled = [&](int s) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_FULL + s % L::kSlots));
    };
    auto slot = [&](int s) { return sbase + L::kRing + (s % L::kSlots) * L::kOperand; };
    // The stream of tiles, looked up one tile before it is needed: the lane's key
    // in the table (-1: none there), and what makes its row of it.
    int page = -1, at = -1, head = 0;
    int key = 0, left = 0, begin = 0, len = 0;  // the lane's key in the next tile, tiles left in the piece, its entry's keys
    const int32_t* table = nullptr;  // its row of the table
    bool more = true;
    auto look_up = [&]() {
      while (left == 0) {
        if (!(more = walk.next(work))) return;
        left = walk.tiles;
        const PlanEntry e = walk.entry(work);
        begin = first_key(a, e.len, e.nq, e.row0);
        len = e.len;
        table = c.table + e.b * c.table_stride;
        key = walk.t * kTile + 32 * w + lane;
      }
      const bool there = key >= begin && key < len;
      page = there ? table[key >> c.page_shift] : -1;
      at = there ? key & ((1 << c.page_shift) - 1) : -1;
      head = walk.h;
      key += kTile;
      left--;
    };
    auto row_found = [&]() -> long long {
      if (at < 0) return -1;
      if (page >= 0 && page < c.num_pages) return ((static_cast<long long>(page) * c.H + head) << c.page_shift) + at;
      flag_index(c.status);
      return -1;
    };
    look_up();
    if constexpr (kFmt == kBf16) {
      int shown = 0;  // slots handed to the MMAs; copies of the others are in flight
      while (ok && more) {
        const long long row = row_found();
        const uint32_t here = __ballot_sync(kAll, row >= 0);
        const long long off = row >= 0 ? row * (2 * D) : -1;
        look_up();
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
          if (n >= L::kSlots) {
            const uint32_t e = bar(B_EMPTY + n % L::kSlots), par = (n / L::kSlots - 1) & 1;
            // the ring is full: hand over what has been asked for, then wait
            if (!__all_sync(kAll, mbar_test_wait(e, par))) {
              cp_async_wait<0>();
              while (shown < n) filled(shown++);
            }
            if (!(ok = wait_warp(e, par, ctl))) break;
          }
          // the mask words of tile (tiles - 8) have been read: this slot's
          // release followed P V of tile (tiles - 5) or later
          if (kv == 0 && lane == 0) mask[4 * (tiles & 7) + w] = here;
          copy_rows<D>(slot(n), 32 * w, kv ? c.vc : c.kc, off);
          cp_async_commit();
          n++;
          if (n - shown > 2) {
            cp_async_wait<2>();
            filled(shown++);
          }
        }
        tiles++;
      }
      cp_async_wait<0>();
      while (ok && shown < n) filled(shown++);
    } else {
      // codes of the next K and V tile wait in registers while the ones before
      // them are converted
      Gather<kFmt, D> gk, gv;
      auto free_slot = [&](int s) {
        return s < L::kSlots || wait_warp(bar(B_EMPTY + s % L::kSlots), (s / L::kSlots - 1) & 1, ctl);
      };
      bool have = more;
      long long row = row_found();
      uint32_t here = __ballot_sync(kAll, row >= 0);
      if (have) {
        if constexpr (kScales) gk.load_scale(c.ks, row), gv.load_scale(c.vs, row);
        gk.load(c.kc, c.ks, row, here);
        gv.load(c.vc, c.vs, row, here);
        look_up();
      }
      while (have) {
        if (!(ok = free_slot(n))) break;
        uint32_t mine_k = 0, mine_v = 0;
        if constexpr (kScales) {
          const uint32_t sk = gk.scale[0], sv = gv.scale[0];
          const Scales x(sk, sv);
          mine_k = x.mine_k, mine_v = x.mine_v;
          if (x.wide) {
            uint8_t* to = smem + L::kBytes + 256 * (tiles % L::kInfo) + 32 * w + lane;
            to[0] = static_cast<uint8_t>(sk), to[128] = static_cast<uint8_t>(sv);
          }
          if (lane == 0) {
            kscale[4 * (tiles & 7) + w] = x.wide ? 0.0f : __uint_as_float((x.top_k + 127 - Scales::kBias) << 23);
            vlog[4 * (tiles & 7) + w] = static_cast<float>(static_cast<int>(x.top_v - Scales::kBias));
            atomicOr(spread, x.seen);
          }
        }
        if (lane == 0) mask[4 * (tiles & 7) + w] = here;
        gk.store(slot(n), 32 * w, mine_k);
        filled(n++);
        have = more;
        if (have) {
          row = row_found();
          here = __ballot_sync(kAll, row >= 0);
          if constexpr (kScales) gk.load_scale(c.ks, row), gv.load_scale(c.vs, row);
          gk.load(c.kc, c.ks, row, here);
          look_up();
        }
        if (!(ok = free_slot(n))) break;
        gv.store(slot(n), 32 * w, mine_v);
        filled(n++);
        if (have) gv.load(c.vc, c.vs, row, here);
        tiles++;
      }
    }
  } else {
    regs_dec<Regs<kFmt>::kCtl>();
    if (warp == 12) {
      // ---- MMA issue.  Order: S0(0) S1(0), then for every tile k PV0(k)
      // S0(k + 1) PV1(k) S1(k + 1)
      const uint32_t id_s = kHalf ? idesc_fp16(128, 128) : idesc_bf16(128, 128);
      const uint32_t id_o = (kHalf ? idesc_fp16(128, D) : idesc_bf16(128, D)) | kIdescBmn;
      int n = 0;             // ring position of the current tile's K; its V follows
      int g[2] = {0, 0};     // tiles of each row tile so far
      int pieces[2] = {0, 0}, q_pieces = 0;
      bool ok = true;
      const bool held = work.withhold && blockIdx.x == 0;
      auto slot = [&](int s) { return sbase + L::kRing + (s % L::kSlots) * L::kOperand; };
      auto wait_full = [&](int s) { return wait_warp(bar(B_FULL + s % L::kSlots), (s / L::kSlots) & 1, ctl); };
      auto issue_s = [&](int m, int s) {
        umma_qk<D>(tmem + kTmS + 128 * m, desc_kmajor(sbase + L::kQ + m * L::kOperand), desc_kmajor(slot(s)), id_s);
        if (!held) tc_commit(bar(B_S + m));
      };
      while (ok && walk.next(work)) {
        if (walk.tiles == 0) continue;
        const int nm = entry_rows(walk.entry(work), a.G) > 128 ? 2 : 1;
        ok = wait_full(n);
        for (int m = 0; ok && m < 2; m++) {
          if (!(ok = wait_warp(bar(B_QFULL + m), q_pieces & 1, ctl))) break;
          tc_fence_after();
          if (m < nm && elect_one()) issue_s(m, n);
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) {
          tc_commit(bar(B_EMPTY + n % L::kSlots));
          if (walk.tiles == 1) tc_commit(bar(B_QEMPTY));
        }
        __syncwarp();
        for (int k = 0; ok && k < walk.tiles; k++, n += 2) {
          const bool more = k + 1 < walk.tiles;
          if (!(ok = wait_full(n + 1))) break;
          for (int m = 0; ok && m < nm; m++) {
            const uint32_t tO = tmem + kTmO + 128 * m, tP = tmem + kTmS + 128 * m, dv = desc_mnmajor(slot(n + 1), 128 * 128);
            if (k == 0 && pieces[m] > 0 && !(ok = wait_warp(bar(B_OFREE + m), (pieces[m] - 1) & 1, ctl))) break;
            if (!(ok = wait_warp(bar(B_P + 2 * m), g[m] & 1, ctl))) break;
            tc_fence_after();
            if (elect_one()) umma_pv<0, 4>(tO, tP, dv, id_o, k > 0);
            __syncwarp();
            if (!(ok = wait_warp(bar(B_P + 2 * m + 1), g[m] & 1, ctl))) break;
            tc_fence_after();
            if (elect_one()) {
              umma_pv<4, 8>(tO, tP, dv, id_o, true);
              if (m == nm - 1) tc_commit(bar(B_EMPTY + (n + 1) % L::kSlots));
              if (!more) tc_commit(bar(B_O + m));
            }
            __syncwarp();
            g[m]++;
            if (!more) continue;
            if (m == 0 && !(ok = wait_full(n + 2))) break;
            tc_fence_after();
            if (elect_one()) {
              issue_s(m, n + 2);
              if (m == nm - 1) {
                tc_commit(bar(B_EMPTY + (n + 2) % L::kSlots));
                if (k + 2 == walk.tiles) tc_commit(bar(B_QEMPTY));
              }
            }
            __syncwarp();
          }
        }
        for (int m = 0; m < nm; m++) pieces[m]++;
        q_pieces++;
      }
      // every MMA issued completes before tensor memory is freed
      if (elect_one()) tc_commit(bar(B_DRAIN));
      __syncwarp();
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar(B_DRAIN), 0) && globaltimer_ns() - t0 < work.wait_ns) {
      }
    }
  }
  // the roles leave from their own code paths
  __syncwarp();
  named_barrier(1, kThreads);
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int kFmt, int D>
cudaError_t launch(const KvView& c, const AttnArgs& a, const AttnWork& w, cudaStream_t st) {
  const cudaError_t e = set_shared_once<&chunk_kernel<kFmt, D>>(Smem<D>::kAlloc);
  if (e != cudaSuccess) return e;
  return launch_after(chunk_kernel<kFmt, D>, dim3(w.workers), kThreads, Smem<D>::kAlloc, st, c, a, w);
}

}  // namespace

cudaError_t launch_attn_chunk(const KvView& c, const AttnArgs& a, const AttnWork& w, int D, int format, cudaStream_t st) {
  if (format == kBf16) return D == 64 ? launch<kBf16, 64>(c, a, w, st) : launch<kBf16, 128>(c, a, w, st);
  if (format == kE4m3) return D == 64 ? launch<kE4m3, 64>(c, a, w, st) : launch<kE4m3, 128>(c, a, w, st);
  return D == 64 ? launch<kNvfp4, 64>(c, a, w, st) : launch<kNvfp4, 128>(c, a, w, st);
}

}  // namespace sagefp4
