/*
 * opt8_layers.h -- C ABI of the operators around a language model's matrix
 * products, for AMD Instinct MI355X (gfx950): token embeddings (lookup and
 * gradient), the root-mean-square norm (with the residual's addition and 8-bit
 * codes for opt8_fp8_matmul; backward pass), and the norm and clipping of a list
 * of gradients, before the optimizer's step reads them.  Library: libopt8.so.
 * Status codes, error channel and conventions are those of opt8.h and
 * opt8_products.h: device pointers on the current HIP device, owned by the caller
 * and valid until the work queued on hip_stream has finished; arguments checked
 * before anything is queued (on a validation error nothing is queued or
 * modified); calls are asynchronous to the host.  No call allocates, copies from
 * the host, keeps anything for a later one or needs opt8_init_codebooks; every
 * call may be captured into a graph, and gives the same bits for the same input.
 * Calls that may run at once (on two streams, as replays of two captured graphs)
 * must not share an output or a workspace; a workspace's contents need not be kept
 * between calls.
 *
 * Matrices are row-major with `ld` elements from one row to the next; they need
 * their element's own alignment only and are faster on 16 bytes (8-bit codes:
 * 16-byte rows, as in opt8_products.h).  What lies behind a row's end is neither
 * read nor written.  No count of rows exceeds 2^22, none of columns 2^20, no matrix
 * 2^34 elements, no ld 2^38.  An output may not overlap another buffer of the call,
 * except where a call says that it may be the same one.
 *
 * Status codes of these calls: OPT8_E_NULL (a required pointer), OPT8_E_SIZE
 * (counts, ld, workspace), OPT8_E_MODE (an unknown type, or one where it does not
 * belong), OPT8_E_HPARAM (scale, eps, max_norm), OPT8_E_ALIGN, OPT8_E_ALIAS,
 * OPT8_E_NOMEM (opt8_grad_table) and OPT8_E_HIP (a launch failed; with more than
 * one launch those before it are queued).
 */
#ifndef OPT8_LAYERS_H_
#define OPT8_LAYERS_H_

#include "opt8_products.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  OPT8_ID_INT32 = 0,
  OPT8_ID_INT64 = 1
} opt8_id_type;

/* y[i] = scale * table[ids[i]] + place_table[place_ids[i]]: in fp32, rounded once
 * for the product with scale and once for the sum, then to the type.  An id that is
 * no row of its table (a padding of -1) stands for a row of zeros.  place_ids and
 * place_table are NULL where there are no places.  A table without rows may be NULL. */
typedef struct opt8_embedding {
  const void* ids;           /* [tokens]                                             */
  const void* table;         /* [vocab, d]                                           */
  const void* place_ids;     /* [tokens], of the same type as ids                    */
  const void* place_table;   /* [places, d]                                          */
  void* y;                   /* [tokens, d]                                          */
  int64_t tokens, vocab, places, d;   /* >= 0; tokens == 0 or d == 0 queues nothing     */
  int64_t ldtable, ldplace, ldy;
  float scale;               /* finite                                               */
  int32_t type;              /* of the tables and y: OPT8_TYPE_BF16, FP16 or FP32    */
  int32_t id_type;           /* opt8_id_type                                         */
} opt8_embedding;
int opt8_embedding_forward(const opt8_embedding* embedding, void* hip_stream);

/* dtable[v] = scale * (sum of dy[i] over the tokens i whose id is v), summed in an
 * order that depends on the ids alone (in fp32 up to 128 tokens, in 64 bits what such
 * parts of more give), rounded once.  Tokens whose id is no
 * row of the table are left out, whatever their dy.  accumulate == 0: every row of
 * dtable is written, those without a token with zeros (bf16: the gradient that
 * opt8_adamw_step reads).  accumulate != 0: the sum is added to what the row holds,
 * and rows without a token are neither read nor written.  The gradient of
 * place_table is the same call with the places for ids. */
typedef struct opt8_embedding_grad {
  const void* ids;           /* [tokens]                                             */
  const void* dy;            /* [tokens, d]                                          */
  void* dtable;              /* [vocab, d]                                           */
  void* workspace;           /* 16-byte aligned                                      */
  int64_t workspace_bytes;   /* >= opt8_embedding_workspace(tokens, vocab, d)        */
  int64_t tokens, vocab, d;  /* >= 0; vocab == 0 or d == 0 queues nothing            */
  int64_t lddy, lddtable;
  float scale;               /* finite                                               */
  int32_t type;              /* of dy: OPT8_TYPE_BF16, FP16 or FP32                  */
  int32_t dtable_type;       /* the same, or OPT8_TYPE_FP32                          */
  int32_t id_type;           /* opt8_id_type                                         */
  int32_t accumulate;
} opt8_embedding_grad;
int opt8_embedding_backward(const opt8_embedding_grad* grad, void* hip_stream);

/* Bytes of workspace that opt8_embedding_backward needs for these sizes (a pure
 * function; sizes outside the limits give 0). */
int64_t opt8_embedding_workspace(int64_t tokens, int64_t vocab, int64_t d);

/* With t = x + residual (in fp32; t = x without one) of a row of d values:
 *   rstd = 1 / sqrt(mean(t^2) + eps),   n = (t * rstd) * weight
 * and any of these outputs, each computed from the unrounded t and n:
 *   sum   t, rounded once: the residual of the next block, and x of the backward pass
 *   y     n, rounded once
 *   q, scale   codes of n and their scales, as opt8_fp8_quantize gives them by rows
 *         (OPT8_FP8_BLOCK_ROW; scale [ceil(d/128), rows]): operand a of opt8_fp8_matmul
 *   rstd  fp32 [rows], for the backward pass
 * The squares are added up in 64 bits and rstd is rounded once, so a row of finite t
 * has its formula's values also where its squares leave fp32.  With eps == 0 a row of
 * zeros has an infinite rstd, and so has one whose rstd fp32 cannot hold (a root below
 * 2^-128); a root above 2^126 has a subnormal rstd, of fewer bits.  sum may be the same
 * matrix as residual or x (the same address and ld). */
typedef struct opt8_rms_norm {
  const void* x;             /* [rows, d]                                            */
  const void* residual;      /* [rows, d], or NULL                                   */
  const void* weight;        /* [d]                                                  */
  void* sum;                 /* [rows, d], or NULL; only with residual               */
  void* y;                   /* [rows, d], or NULL                                   */
  void* q;                   /* [rows, d], or NULL                                   */
  float* scale;              /* with q                                               */
  float* rstd;               /* [rows], or NULL                                      */
  int64_t rows, d;           /* rows >= 0 (0 queues nothing), d > 0                  */
  int64_t ldx, ldresidual, ldsum, ldy;
  int64_t ldq;               /* a multiple of 16                                     */
  float eps;                 /* >= 0, finite                                         */
  int32_t type;              /* of x, residual, sum and y: BF16, FP16 or FP32        */
  int32_t weight_type;       /* the same, or OPT8_TYPE_FP32                          */
  int32_t q_type;            /* OPT8_TYPE_E4M3 or E5M2; read with q only             */
} opt8_rms_norm;
int opt8_rms_norm_forward(const opt8_rms_norm* norm, void* hip_stream);

/* Its backward pass, from dy (of y), the normalised rows' x (the forward pass's sum
 * where it had a residual) and rstd.  With h = x * rstd and g = dy * weight, in fp32:
 *   dx = rstd * (g - h * mean(g * h)) + dsum      (dsum: gradient that reaches x by
 *                                                 the residual's own way, or NULL)
 *   dweight = sum over rows of dy * h
 * each rounded once.  dx or dweight may be NULL, not both; dx may be the same matrix
 * as dy or dsum (the same address and ld).  rows == 0 stores zeros in dweight. */
typedef struct opt8_rms_norm_grad {
  const void* dy;            /* [rows, d]                                            */
  const void* x;             /* [rows, d]                                            */
  const void* weight;        /* [d]; read for dx                                     */
  const float* rstd;         /* [rows]                                               */
  const void* dsum;          /* [rows, d], or NULL; read for dx                      */
  void* dx;                  /* [rows, d]                                            */
  void* dweight;             /* [d]                                                  */
  void* workspace;           /* 16-byte aligned; read for dweight                    */
  int64_t workspace_bytes;   /* >= opt8_rms_norm_workspace(rows, d)                  */
  int64_t rows, d;
  int64_t lddy, ldx, lddsum, lddx;
  int32_t type;              /* of dy, x, dsum and dx: BF16, FP16 or FP32            */
  int32_t weight_type;       /* the same, or OPT8_TYPE_FP32                          */
  int32_t dweight_type;      /* the same, or OPT8_TYPE_FP32                          */
} opt8_rms_norm_grad;
int opt8_rms_norm_backward(const opt8_rms_norm_grad* grad, void* hip_stream);

/* Bytes of workspace that opt8_rms_norm_backward needs for dweight (a pure function;
 * sizes outside the limits give 0). */
int64_t opt8_rms_norm_workspace(int64_t rows, int64_t d);

/* One gradient of a list, and where its clipped values go: to `out` (of any type),
 * or back into `grad` where out is NULL or the same address (of the same type). */
typedef struct opt8_grad {
  void* grad;                /* numel adjacent values, aligned to them               */
  void* out;
  int64_t numel;             /* >= 0, <= 2^37                                        */
  int32_t type;              /* OPT8_TYPE_BF16, FP16 or FP32                         */
  int32_t out_type;          /* likewise; read where out is not NULL                 */
} opt8_grad;

/* The list as the kernels read it: 24 bytes, and 24 for each piece of at most 8192
 * values of a gradient.
 * opt8_grad_table_bytes gives its size (or a negative status) and opt8_grad_table
 * writes it to HOST memory; the caller copies it to the device, and passes that copy
 * as often as it likes while the gradients stay at their addresses.  No two buffers
 * of a list may overlap (but a gradient and its own out, which are the same).
 * n <= 2^22 gradients and 2^26 pieces. */
#define OPT8_GRAD_PIECE 8192
#define OPT8_GRAD_PIECE_BYTES 24
int64_t opt8_grad_table_bytes(const opt8_grad* grads, int32_t n);
int opt8_grad_table(const opt8_grad* grads, int32_t n, void* host_table, int64_t bytes);

#define OPT8_GRAD_WORKSPACE 16384   /* bytes of workspace that opt8_grad_norm needs   */

typedef struct opt8_grads {
  const void* table;         /* device copy of a list's table, 8-byte aligned         */
  int64_t table_bytes;       /* of that copy: what opt8_grad_table_bytes gave, or more
                                (what lies behind the list's pieces is not read)     */
  double* squares;           /* [1]                                                  */
  float* norm;               /* [1], or NULL                                         */
  void* workspace;           /* 16-byte aligned                                      */
  int64_t workspace_bytes;   /* >= OPT8_GRAD_WORKSPACE                               */
  double max_norm;           /* >= 0, finite; of the clipping                        */
} opt8_grads;

/* squares = sum of the squares of all values of the list (each exact, the sum in 64
 * bits), norm = sqrt(squares) in fp32.  Where ranks hold parts of one model's
 * gradients, they add up `squares` between this call and the clipping. */
int opt8_grad_norm(const opt8_grads* grads, void* hip_stream);

/* From `squares`: norm = sqrt(squares), factor = min(1, max_norm / (norm + 1e-6))
 * (64 bits, rounded once to fp32), and every gradient's out = grad * factor (rounded
 * to fp32 and then to out's type).  A factor of 1 leaves gradients without an own out
 * as they are, unread.  A norm of NaN makes NaN of every value, an infinite one zeros
 * of the finite ones. */
int opt8_grad_clip(const opt8_grads* grads, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* OPT8_LAYERS_H_ */
