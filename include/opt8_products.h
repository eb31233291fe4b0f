/*
 * opt8_products.h -- C ABI of the operators between a language model's
 * weights and their gradients, for AMD Instinct MI355X (gfx950): 8-bit
 * floating point with a scale for each block of 128 values (quantiser and
 * matrix product) and the gated feed-forward block (forward and backward).
 * Library: libopt8.so, beside the optimizer steps of opt8.h, whose status
 * codes, error channel (opt8_last_error) and conventions these share: device
 * pointers on the current HIP device, owned by the caller and valid until the
 * work queued on hip_stream has finished; arguments checked before anything is
 * queued (on a validation error nothing is queued or modified); calls are
 * asynchronous to the host.  No call allocates, copies from the host, keeps
 * anything for a later one or needs opt8_init_codebooks; every call may be
 * captured into a graph.  Concurrent calls on different streams must not share
 * an output or a workspace.
 *
 * Matrices are row-major with `ld` elements from one row to the next.
 * Operands that feed the matrix cores (every input, and the 8-bit outputs)
 * start on a 16-byte boundary, have ld*size a multiple of 16, and own the last
 * 16 bytes of their last row whole (rows are read in pieces of 16 bytes; what
 * lies behind a row's end is ignored, and never written).  Other outputs need their
 * element's own alignment only and are faster on 16 bytes.  No count of rows
 * or columns exceeds 2^22 (d and f: 2^20), no matrix 2^37 elements, no ld 2^38,
 * and no ld*size of a matrix that feeds the matrix cores 2^23 bytes.  An output may
 * not overlap another buffer of the call; halves of one wider matrix (the same
 * ld, columns side by side) are apart, other spans that meet are refused.
 *
 * Status codes of these calls: OPT8_E_NULL (a required pointer), OPT8_E_SIZE
 * (counts, ld, workspace), OPT8_E_MODE (an unknown type, block or act, or a
 * type where it does not belong), OPT8_E_ALIGN, OPT8_E_ALIAS, and OPT8_E_HIP
 * (a launch failed; with more than one launch those before it are queued).
 */
#ifndef OPT8_PRODUCTS_H_
#define OPT8_PRODUCTS_H_

#include "opt8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define OPT8_FP8_BLOCK 128   /* values along the contraction that share a scale */

typedef enum {
  OPT8_TYPE_BF16 = 0,
  OPT8_TYPE_FP16 = 1,
  OPT8_TYPE_FP32 = 2,
  OPT8_TYPE_E4M3 = 3,        /* OCP E4M3 (finite and NaN), largest value 448     */
  OPT8_TYPE_E5M2 = 4         /* OCP E5M2, largest value 57344                    */
} opt8_type;

typedef enum {
  OPT8_FP8_BLOCK_ROW = 0,    /* a scale for each row and 128 columns             */
  OPT8_FP8_BLOCK_TILE = 1    /* a scale for each 128 rows and 128 columns        */
} opt8_fp8_block;

typedef enum {
  OPT8_ACT_SILU = 0,         /* g * sigmoid(g)                                   */
  OPT8_ACT_GELU = 1,         /* g * Phi(g), Phi the normal distribution          */
  OPT8_ACT_GELU_TANH = 2     /* its tanh form: 0.044715, sqrt(2/pi)              */
} opt8_act;

/* 8-bit codes and scales of x [rows, cols] (bf16, fp16 or fp32), of x
 * transposed, or of both from one read of x.  With fmax the format's largest
 * value, a block's scale is
 *   s = max(max|x| / fmax, 2^-126)          (fp32, rounded once)
 * and a value's code the one nearest to x * (1/s) (fp32, ties to even).  The
 * last blocks of a row or column are shorter.  NaN keeps a NaN code and does
 * not count for the maximum; a block that holds an infinity has an infinite
 * scale, zero codes for its finite values and NaN codes for its infinities.
 * Scales lie block-major: scale[b][i] is that of columns 128b..128b+127 of row
 * i (ROW; [ceil(cols/128), rows]) or of rows 128i..128i+127 (TILE;
 * [ceil(cols/128), ceil(rows/128)]), dense.  scale_t likewise for x transposed
 * (of which qt has cols rows of ldt).  Either pair may be NULL, not both. */
typedef struct opt8_fp8_quant {
  const void* x;
  void* q;             /* codes [rows, cols], or NULL                                 */
  float* scale;
  void* qt;            /* codes of x transposed [cols, rows], or NULL                 */
  float* scale_t;
  int64_t rows, cols;  /* >= 0; an empty x queues nothing                             */
  int64_t ldx;         /* x: element alignment is enough                              */
  int64_t ldq, ldt;    /* multiples of 16                                             */
  int32_t x_type;      /* OPT8_TYPE_BF16, FP16 or FP32                                */
  int32_t q_type;      /* OPT8_TYPE_E4M3 or E5M2                                      */
  int32_t block;       /* opt8_fp8_block                                              */
} opt8_fp8_quant;
int opt8_fp8_quantize(const opt8_fp8_quant* quant, void* hip_stream);

/* C[m][n] = sum over blocks b of 128 k of
 *     (scale_a[b][m] * scale_b[b][n]) * sum over k in b of A[m][k]*B[n][k]
 * for A [m, k] with ROW scales and B [n, k] with ROW or TILE scales (n/128 for
 * n), as opt8_fp8_quantize lays them out; C, bf16 or fp16, rounded once from
 * fp32.  Sums over blocks are fp32; within a block the 8-bit matrix
 * instruction adds 8 products at a time on a grid 2^-13 of the largest one's
 * power of two.  That cuts 1e-5 of a typical result on normal values, 3e-5 with
 * a few loud channels, and at most 3.3e-4 in the mean: below a 16-bit result's
 * half step, but why there is no 32-bit one.  The product of the two scales is formed
 * first, in fp32, and has to be a normal number: below 2^-126 the block's term loses
 * bits or all of it, and from 2^128 on it is infinite, or NaN where its sum is 0.
 * The three products of a linear layer y = x w^T are: y from x and w (TILE); the
 * input's gradient from dy and w transposed (TILE); the weight's gradient from
 * dy transposed and x transposed (ROW).  k == 0 stores zeros. */
typedef struct opt8_fp8_product {
  const void* a;
  const float* scale_a;
  const void* b;
  const float* scale_b;
  void* c;
  int64_t m, n, k;     /* >= 0; m == 0 or n == 0 queues nothing                       */
  int64_t lda, ldb;    /* >= k, multiples of 16                                       */
  int64_t ldc;         /* >= n                                                        */
  int32_t a_type;      /* OPT8_TYPE_E4M3 or E5M2                                      */
  int32_t b_type;      /* OPT8_TYPE_E4M3                                              */
  int32_t c_type;      /* OPT8_TYPE_BF16 or FP16                                      */
  int32_t block_b;     /* opt8_fp8_block                                              */
} opt8_fp8_product;
int opt8_fp8_matmul(const opt8_fp8_product* product, void* hip_stream);

/* Gated feed-forward block: g = x w_gate^T, u = x w_up^T, h = act(g) * u for
 * x [rows, d] and w_gate, w_up [f, d], in one kernel: fp32 sums, the
 * activation and the product taken from them unrounded, h rounded once.  gate
 * and up, if not NULL, receive g and u rounded, for the backward pass. */
typedef struct opt8_gated_ffn {
  const void* x;
  const void* w_gate;
  const void* w_up;
  void* h;
  void* gate;          /* both or neither                                             */
  void* up;
  int64_t rows, d, f;  /* rows >= 0 (0 queues nothing); d, f > 0                      */
  int64_t ldx, ldw;    /* >= d; both weights share ldw                                */
  int64_t ldh, ldg;    /* >= f; gate and up share ldg                                 */
  int32_t type;        /* OPT8_TYPE_BF16 or FP16, of every matrix                     */
  int32_t act;         /* opt8_act                                                    */
} opt8_gated_ffn;
int opt8_gated_ffn_forward(const opt8_gated_ffn* ffn, void* hip_stream);

/* Its backward pass, from dh and the stored g and u:
 *   dg = dh * u * act'(g), du = dh * act(g)     (fp32, rounded once to the type)
 *   dx = dg w_gate + du w_up, dw_gate = dg^T x, dw_up = du^T x
 * with fp32 sums, each result rounded once.  dx, or both dw, may be NULL.
 * dw_gate and dw_up are dense bf16/fp16 [f, d] with lddw (bf16: the gradients
 * that opt8_adamw_step reads); rows == 0 stores zeros in them. */
typedef struct opt8_gated_ffn_grad {
  const void* dh;
  const void* x;
  const void* w_gate;
  const void* w_up;
  const void* gate;
  const void* up;
  void* dx;
  void* dw_gate;
  void* dw_up;
  void* workspace;     /* 16-byte aligned; contents need not be kept.  The call writes it:
                          calls that may run at once (on two streams, as replays of two
                          captured graphs) take one each                              */
  int64_t workspace_bytes;
  int64_t rows, d, f;
  int64_t ldx, ldw;
  int64_t lddh, ldg;
  int64_t lddx, lddw;
  int32_t type;
  int32_t act;
} opt8_gated_ffn_grad;
int opt8_gated_ffn_backward(const opt8_gated_ffn_grad* grad, void* hip_stream);

/* Bytes of workspace that opt8_gated_ffn_backward needs for these sizes (a pure
 * function; negative sizes give 0). */
int64_t opt8_gated_ffn_workspace(int64_t rows, int64_t d, int64_t f);

#ifdef __cplusplus
}
#endif

#endif /* OPT8_PRODUCTS_H_ */
