// umma.cuh -- inline-PTX wrappers of the 16-bit tensor-core forms that the
// paged cache's attention uses: tcgen05.mma kind::f16 with bf16 operands, its
// operand layouts, bounded waits, cp.async.
#pragma once

#include "ptx.cuh"

namespace sagefp4 {

// Instruction descriptor of kind::f16: bf16 A and B (formats 1 in bits 7-9 and
// 10-12), FP32 accumulator (bits 4-5 = 1), N >> 3 in bits 17-22, M >> 4 in
// bits 24-28; both operands K-major, B MN-major with bit 16.
__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t M, uint32_t N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
constexpr uint32_t kIdescBmn = 1u << 16;
// The same with FP16 A and B (formats 0).
__host__ __device__ constexpr uint32_t idesc_fp16(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// Operand tiles are rows of 128 bytes (64 values) whose 16-byte chunks are
// XOR-permuted by row & 7, on a 1024-byte boundary, eight rows 1024 bytes
// apart.  K-major: rows are M or N, the 64 values a run of K; MN-major: rows
// are K, the 64 values a run of N, and the next run of N starts block_stride
// bytes later.  Of the 64-bit descriptor (ptx.cuh's smem_desc) only the low
// word varies: the start address, and the leading offset above it.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (kSwizzle128B << 29);
__device__ __forceinline__ uint32_t desc_kmajor(uint32_t tile) { return (tile >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mnmajor(uint32_t tile, uint32_t block_stride) {
  return (tile >> 4) | ((block_stride >> 4) << 16);
}

// D[tmem] (+)= A x B, K = 16: A and B in shared memory, or A in tensor memory
// (128 rows in lanes, a row's 16 values in 8 consecutive 32-bit columns).
// Operands are the low descriptor words plus kA, kB (units of 16 bytes).
template <uint32_t kA, uint32_t kB>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\t"
      "add.u32 x, %1, %5;\n\tadd.u32 y, %2, %6;\n\t"
      "mov.b64 da, {x, %7};\n\tmov.b64 db, {y, %7};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kB), "n"(kDescHigh)
      : "memory");
}
template <uint32_t kA, uint32_t kB>  // kA: tensor-memory columns
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 db;\n\t"
      "add.u32 x, %1, %5;\n\tadd.u32 y, %2, %6;\n\t"
      "mov.b64 db, {y, %7};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kB), "n"(kDescHigh)
      : "memory");
}

// All K steps of S = Q K^T (D channels; both K-major, 64-channel halves 16 KB
// apart) and of O (+)= P V (128 keys; V MN-major, a step of 16 keys is 2 KB).
template <int D, int kStep = 0>
__device__ __forceinline__ void umma_qk(uint32_t d, uint32_t q, uint32_t k, uint32_t idesc) {
  if constexpr (kStep < D / 16) {
    constexpr uint32_t kOff = 1024 * (kStep / 4) + 2 * (kStep % 4);
    umma_ss<kOff, kOff>(d, q, k, idesc, kStep > 0);
    umma_qk<D, kStep + 1>(d, q, k, idesc);
  }
}
// Steps kStep .. kEnd - 1 of the latter's eight.
template <int kStep, int kEnd>
__device__ __forceinline__ void umma_pv(uint32_t d, uint32_t p, uint32_t v, uint32_t idesc, bool accumulate) {
  if constexpr (kStep < kEnd) {
    umma_ts<8 * kStep, 128 * kStep>(d, p, v, idesc, kStep > 0 || accumulate);
    umma_pv<kStep + 1, kEnd>(d, p, v, idesc, accumulate);
  }
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Each thread of the warp reads 32 consecutive columns of its lane as FP32 and,
// in the same instruction, their maximum (sm_103a).  Valid after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld32_max(uint32_t taddr, uint32_t (&r)[32], float& mx) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(mx)
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t dst, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint32_t ld_shared4(uint32_t src) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(src) : "memory");
  return v;
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void named_barrier(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// Bounded waits: every role of a CTA shares an abort flag; a wait that runs out
// sets it and records SAGE_FP4_ETIMEOUT, and every other wait then gives up.
struct WaitCtl {
  int32_t* status;
  volatile int* abort;
  uint64_t limit;
};

// By a whole warp, which leaves together.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const WaitCtl& c) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    int stop = 0;
    if ((threadIdx.x & 31) == 0) {
      if (*c.abort) {
        stop = 1;
      } else if (globaltimer_ns() - t0 > c.limit) {
        *c.abort = 1;
        atomicCAS(c.status, 0, -3);  // SAGE_FP4_ETIMEOUT
        stop = 1;
      }
    }
    if (__shfl_sync(0xffffffffu, stop, 0)) return false;
  }
}

}  // namespace sagefp4
