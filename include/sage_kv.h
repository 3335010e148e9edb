/* sage_kv.h -- C ABI of the paged key/value cache and of attention over it on
 * sm_103a (libsagefp4.so).
 *
 * The cache holds the keys and values of many sequences in pages of
 * `page_size` tokens.  A batch says which pages are whose and how long each
 * sequence is, all in device memory, so that one captured graph serves
 * changing lengths:
 *   cu_q   int32 [B + 1]: the rows cu_q[b] .. cu_q[b + 1] - 1 of a call's
 *          packed tensors [T][heads][D] are the new tokens of sequence b;
 *          rows behind cu_q[B] belong to nobody and are left as they were;
 *   kv_len int32 [B]: the tokens of sequence b in the cache, the new ones
 *          (its last cu_q[b + 1] - cu_q[b]) among them;
 *   block_table int32 [B][max_pages], rows table_stride apart: the page of
 *          tokens p * page_size .. of sequence b is block_table[b][p].
 * New token i of a sequence has position kv_len - (its number of new tokens)
 * + i; a negative position is a token that the cache does not hold.
 *
 * Formats of the stored rows (one token, one head, D channels):
 *   SAGE_KV_BF16   the bf16 values;
 *   SAGE_KV_E4M3   8-bit E4M3 codes with one power-of-two scale a row (E8M0:
 *                  2^(byte - 127)), the smallest that brings the row's largest
 *                  magnitude to 448 or less, the byte from 17 (a row of zeros)
 *                  to 246; code = E4M3_rn(x / scale), saturating at 448 (only
 *                  above 1.75 * 2^127), and code * scale is a finite bf16 value;
 *   SAGE_KV_NVFP4  4-bit E2M1 codes, two a byte, the even channel in the low
 *                  nibble, with one E4M3 scale per 16 channels, by the group
 *                  rule of sage_fp4.h (code * scale is a bf16 value).
 * So what a row reads back as is exact in bf16, and attention over a quantized
 * cache is attention over exactly these bf16 values, whatever the sizes of the rows
 * around one and whether they are seen (but E4M3 rows below 2^-101 in magnitude may
 * count as zeros; where 32 neighbouring values differ by more than 2^8 calls of many
 * rows take longer).  Over quantized caches queries enter in FP16, relative to their
 * row's largest magnitude: exact down to 2^-28 of it.
 *
 * Layout of the buffers (contiguous, 16-byte aligned, k and v alike):
 *   codes  [num_pages][H][page_size][D], [D / 2] bytes for NVFP4;
 *   scales E4M3: uint8 [num_pages][H][page_size]; NVFP4: uint8
 *          [num_pages][H][page_size][D / 16]; BF16: none (NULL).
 *
 * D is 64 or 128; page_size a power of two from 16 to 1024; H >= 1.  Inputs must
 * be finite.  Slots past a sequence's length may hold anything, NaN included.
 * The pages that new tokens land in must be their sequence's alone; two tokens
 * that are given one slot leave it with unspecified contents.
 *
 * Indexes found out of range on the device set *status to SAGE_FP4_EINDEX and
 * are left out: a page outside [0, num_pages) (its tokens are not written, read
 * as zeros, and are not attended to); a kv_len outside [0, max_pages *
 * page_size] or above 2^31 - 4096 (the sequence counts as empty); new tokens outside [0, T] or
 * fewer than none (the sequence has none).  Where cu_q runs backwards anywhere,
 * any of the batch's new tokens may be left out, and their rows of an output
 * hold anything.
 * Attention does not look at a page that its window hides from all of a
 * sequence's new tokens: such a page may be gone from the table and the cache.
 *
 * An output's elements share memory neither with each other nor with an input's.
 *
 * Errors as in sage_fp4.h; calls are asynchronous on `stream` and allocate
 * nothing. */
#ifndef SAGE_KV_H
#define SAGE_KV_H

#include <stddef.h>
#include <stdint.h>

#include "sage_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SAGE_KV_BF16 0
#define SAGE_KV_E4M3 1
#define SAGE_KV_NVFP4 2

typedef struct sage_kv_cache {
  void *k_codes, *v_codes;      /* 16-byte aligned */
  uint8_t *k_scales, *v_scales; /* 16-byte aligned; NULL for SAGE_KV_BF16 */
  int32_t *status;              /* one int32 of device memory, zero-initialised by the caller */
  int32_t num_pages, page_size, H, D, format;
} sage_kv_cache;

typedef struct sage_kv_batch {
  const int32_t *cu_q;        /* not read by sage_kv_read */
  const int32_t *kv_len;
  const int32_t *block_table;
  int64_t table_stride;       /* >= max_pages */
  int32_t B, max_pages;
} sage_kv_batch;

/* Element strides of a packed bf16 [T][heads][D] tensor: between tokens and
 * between heads (>= 0, multiples of 8), D contiguous, 16-byte aligned. */
typedef struct sage_kv_rows {
  int64_t t, h;
} sage_kv_rows;

/* Quantize the new tokens' keys and values k, v (bf16, T rows of cache->H
 * heads) into their slots.  One launch. */
int sage_kv_append(const sage_kv_cache *cache, const sage_kv_batch *batch, const void *k, sage_kv_rows k_rows,
                   const void *v, sage_kv_rows v_rows, int T, void *stream);

/* The first N tokens of every sequence back as bf16 [B][H][N][D] through the
 * strides (NULL: contiguous); tokens at kv_len and beyond are zeros.  One
 * launch. */
int sage_kv_read(const sage_kv_cache *cache, const sage_kv_batch *batch, void *k_out,
                 const sage_fp4_strides *k_strides, void *v_out, const sage_fp4_strides *v_strides, int N,
                 void *stream);

/* Bytes of device workspace sage_kv_attn needs (0 for bad sizes). */
size_t sage_kv_attn_workspace_bytes(const sage_kv_cache *cache, int B, int T, int Hq);

/* Attention of the new tokens' queries q (bf16, T rows of Hq heads; query head
 * h reads key/value head h / (Hq / H), Hq a multiple of H) over their
 * sequences' cached tokens: o = softmax(scale * q K^T) V in bf16 and, where lse
 * is given, the natural-log log-sum-exp of the scaled scores, float [T][Hq].
 * causal = 1: a query at position p sees the tokens j <= p; 0: all kv_len.
 * window > 0: only j > p - window; 0: no window.  A row that sees nothing gets
 * o = 0 and lse = -inf.  scale: positive, at most 1e30.  Sums and softmax
 * statistics are FP32; a score may be of any size that FP32 holds (rows beyond
 * 2^18 are far slower where a call has many rows).  workspace: 256-byte aligned, no initialisation; calls
 * sharing one must be ordered. */
int sage_kv_attn(const sage_kv_cache *cache, const sage_kv_batch *batch, const void *q, sage_kv_rows q_rows, void *o,
                 sage_kv_rows o_rows, float *lse, int T, int Hq, int causal, int window, float scale, void *workspace,
                 size_t workspace_bytes, void *stream);

/* Failure-detection test: sage_kv_attn (causal, scale 1/8) with one signal
 * withheld: the first CTA never announces its first scores, so that its bounded
 * waits run out after wait_limit_ns (1 ms to 1.5 s; sage_kv_attn uses 1.5 s).
 * Copies and tensor-core operations in flight are waited for, tensor memory is
 * freed, nothing faults, *status becomes SAGE_FP4_ETIMEOUT, and the other CTAs
 * complete; o is left partly written.  EINVAL for a limit out of range and for
 * calls of so few rows that they run in the kernel without waits. */
int sage_kv_attn_stall_test(const sage_kv_cache *cache, const sage_kv_batch *batch, const void *q, sage_kv_rows q_rows,
                            void *o, sage_kv_rows o_rows, int T, int Hq, uint64_t wait_limit_ns, void *workspace,
                            size_t workspace_bytes, void *stream);

/* Synchronise `stream`, read the status word, reset it to 0 and return it, or
 * SAGE_FP4_ECUDA if the copy failed. */
int sage_kv_get_status(const sage_kv_cache *cache, void *stream);

#ifdef __cplusplus
}
#endif
#endif
