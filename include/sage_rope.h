/* sage_rope.h -- C ABI of the query/key preparation in front of attention on
 * sm_103a (libsagefp4.so): an optional root-mean-square norm of every head and
 * the rotary position rotation, in one pass, with its backward.
 *
 * For a row x of D channels (one token, one head of q or k):
 *   n  = x * r * w          r = 1 / sqrt(mean(x^2) + eps)  (norm = 1)
 *   n  = x                                                 (norm = 0)
 *   y  = n, its first `rot` channels rotated by the angles of the token's
 *        position: the pair (u, v) of angle a becomes
 *        (u cos a - v sin a, v cos a + u sin a).  Pair i is (i, i + rot/2)
 *        in the half layout, (2i, 2i + 1) in the interleaved one.
 * and, given the gradient g of y (rotated back: g' = the rotation by -a of g):
 *   dx = r * (g' w - xh * mean(g' w xh)),  xh = x r;  dw = sum over rows of g' xh
 *   dx = g'                                                (norm = 0)
 * All arithmetic is FP32 on bf16 inputs, rounded once to bf16; dw stays FP32.
 * (So mean(x^2) has to be an FP32 number, and not 0 where eps = 0: a row of zeros,
 * or of magnitudes below 2^-70, then has no norm and gives NaN or infinity.)
 *
 * The library takes cos and sin from the caller's table, cos_sin[max_pos][rot]
 * (FP32, cos of pair i at i, sin at rot/2 + i), so that a table made in 64 bits
 * keeps far positions exact and carries any scaling for long contexts.
 *
 * Tensors: bf16, element (b, n, h, d) at b*b_stride + n*n_stride + h*h_stride + d
 * (sage_fp4_strides of sage_fp4.h; strides >= 0, multiples of 8), 16-byte
 * aligned, on the current device; NULL strides mean contiguous [B][N][H][D].
 * An output may be the input itself with the same strides, and no other
 * overlap, also not among an output's elements.  D is 64 or 128; rot a multiple of 16, 16 <= rot <= D.  B, N, Hq,
 * Hk >= 0 (an empty problem succeeds; sage_rope_bwd then still writes zeros to
 * dw).  B * N <= 2^31 - 1.
 *
 * Positions: int32 [B][N] with stride pos_b_stride between batches (0: one row
 * for every batch).  A position outside [0, max_pos) is found on the device:
 * that token's outputs (and its share of dw) are zero and *status becomes
 * SAGE_FP4_EINDEX.
 *
 * Errors as in sage_fp4.h; calls are asynchronous on `stream` and allocate
 * nothing. */
#ifndef SAGE_ROPE_H
#define SAGE_ROPE_H

#include <stddef.h>
#include <stdint.h>

#include "sage_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct sage_rope_desc {
  int32_t B, N, Hq, Hk, D;
  int32_t rot;          /* rotated channels */
  int32_t interleaved;  /* 0: half layout, 1: adjacent pairs */
  int32_t norm;         /* 1: norm with q_weight / k_weight */
  int32_t weight_f32;   /* weights are FP32 (1) or bf16 (0) */
  int32_t max_pos;
  float eps;            /* >= 0, finite */
  int64_t pos_b_stride;
  const int32_t *positions; /* 4-byte aligned */
  const float *cos_sin;     /* [max_pos][rot], 16-byte aligned */
  const void *q_weight, *k_weight; /* [D], 16-byte aligned; read where norm = 1 */
  int32_t *status;      /* one int32 of device memory, zero-initialised by the caller */
} sage_rope_desc;

/* y of q and k: one launch. */
int sage_rope_fwd(const sage_rope_desc *desc, const void *q, const sage_fp4_strides *q_strides, const void *k,
                  const sage_fp4_strides *k_strides, void *q_out, const sage_fp4_strides *q_out_strides, void *k_out,
                  const sage_fp4_strides *k_out_strides, void *stream);

/* Bytes of device workspace sage_rope_bwd needs (0 for bad sizes; 256 where
 * norm = 0). */
size_t sage_rope_workspace_bytes(const sage_rope_desc *desc);

/* dq, dk (bf16) and, where norm = 1, dq_weight and dk_weight (FP32 [D]) from
 * the outputs' gradients gq, gk and the forward's inputs q, k (not read where
 * norm = 0).  Two launches (norm = 0: one).  The sums behind dw run in a fixed
 * order: repeated calls give the same bits on one device.  workspace:
 * 256-byte aligned; calls sharing one must be ordered. */
int sage_rope_bwd(const sage_rope_desc *desc, const void *gq, const sage_fp4_strides *gq_strides, const void *gk,
                  const sage_fp4_strides *gk_strides, const void *q, const sage_fp4_strides *q_strides, const void *k,
                  const sage_fp4_strides *k_strides, void *dq, const sage_fp4_strides *dq_strides, void *dk,
                  const sage_fp4_strides *dk_strides, float *dq_weight, float *dk_weight, void *workspace,
                  size_t workspace_bytes, void *stream);

/* Synchronise `stream`, read the status word, reset it to 0 and return it
 * (SAGE_FP4_OK, SAGE_FP4_EINDEX), or SAGE_FP4_ECUDA if the copy failed. */
int sage_rope_get_status(int32_t *status, void *stream);

#ifdef __cplusplus
}
#endif
#endif
