// Argument checks and C entry points of the operators in opt8_products.h.
#include "operand_checks.h"
#include "products_internal.h"

namespace opt8 {
namespace {

int check_block(int block) {
  if (block != OPT8_FP8_BLOCK_ROW && block != OPT8_FP8_BLOCK_TILE)
    return refuse(OPT8_E_MODE, "unknown block %d", block);
  return OPT8_OK;
}

int check_ffn_type(int type, int act) {
  if (type != OPT8_TYPE_BF16 && type != OPT8_TYPE_FP16)
    return refuse(OPT8_E_MODE, "the block is bf16 or fp16 (got type %d)", type);
  if (act != OPT8_ACT_SILU && act != OPT8_ACT_GELU && act != OPT8_ACT_GELU_TANH)
    return refuse(OPT8_E_MODE, "unknown act %d", act);
  return OPT8_OK;
}

int quantize(const opt8_fp8_quant* a, void* hip_stream) {
  clear_last_error();
  if (!a) return refuse(OPT8_E_NULL, "quant is NULL");
  int rc;
  if ((rc = check_count("rows", a->rows, 0, kMaxCount)) || (rc = check_count("cols", a->cols, 0, kMaxCount))) return rc;
  if (a->x_type != OPT8_TYPE_BF16 && a->x_type != OPT8_TYPE_FP16 && a->x_type != OPT8_TYPE_FP32)
    return refuse(OPT8_E_MODE, "x is bf16, fp16 or fp32 (got type %d)", a->x_type);
  if (a->q_type != OPT8_TYPE_E4M3 && a->q_type != OPT8_TYPE_E5M2)
    return refuse(OPT8_E_MODE, "codes are e4m3 or e5m2 (got type %d)", a->q_type);
  if ((rc = check_block(a->block))) return rc;
  if (a->rows == 0 || a->cols == 0) return OPT8_OK;
  if (!a->q && !a->qt) return refuse(OPT8_E_NULL, "q and qt are both NULL");
  if (!a->q != !a->scale) return refuse(OPT8_E_NULL, "q and scale go together");
  if (!a->qt != !a->scale_t) return refuse(OPT8_E_NULL, "qt and scale_t go together");
  if (!a->x) return refuse(OPT8_E_NULL, "x is NULL");
  const bool tile = a->block == OPT8_FP8_BLOCK_TILE;
  const int64_t across = tile ? blocks(a->rows) : a->rows, across_t = tile ? blocks(a->cols) : a->cols;
  const Matrix list[] = {
      {"x", a->x, a->rows, a->cols, a->ldx, type_bytes(a->x_type), false, false},
      {"q", a->q, a->rows, a->cols, a->ldq, 1, true, true},
      {"scale", a->scale, blocks(a->cols), across, across, 4, true, false},
      {"qt", a->qt, a->cols, a->rows, a->ldt, 1, true, true},
      {"scale_t", a->scale_t, blocks(a->rows), across_t, across_t, 4, true, false},
  };
  if ((rc = check_matrices(list, 5))) return rc;
  return launched(launch_fp8_quantize(*a, static_cast<hipStream_t>(hip_stream)), "opt8_fp8_quantize");
}

int matmul(const opt8_fp8_product* a, void* hip_stream) {
  clear_last_error();
  if (!a) return refuse(OPT8_E_NULL, "product is NULL");
  int rc;
  if ((rc = check_count("m", a->m, 0, kMaxCount)) || (rc = check_count("n", a->n, 0, kMaxCount)) ||
      (rc = check_count("k", a->k, 0, kMaxCount)))
    return rc;
  if (a->a_type != OPT8_TYPE_E4M3 && a->a_type != OPT8_TYPE_E5M2)
    return refuse(OPT8_E_MODE, "a is e4m3 or e5m2 (got type %d)", a->a_type);
  if (a->b_type != OPT8_TYPE_E4M3) return refuse(OPT8_E_MODE, "b is e4m3 (got type %d)", a->b_type);
  if (a->c_type != OPT8_TYPE_BF16 && a->c_type != OPT8_TYPE_FP16)
    return refuse(OPT8_E_MODE, "c is bf16 or fp16 (got type %d)", a->c_type);
  if ((rc = check_block(a->block_b))) return rc;
  if (a->m == 0 || a->n == 0) return OPT8_OK;
  if (!a->c) return refuse(OPT8_E_NULL, "c is NULL");
  if (a->k > 0 && (!a->a || !a->scale_a || !a->b || !a->scale_b))
    return refuse(OPT8_E_NULL, "a, scale_a, b or scale_b is NULL");
  const int64_t across = a->block_b == OPT8_FP8_BLOCK_TILE ? blocks(a->n) : a->n;
  const Matrix list[] = {
      {"c", a->c, a->m, a->n, a->ldc, 2, true, false},
      {"a", a->k ? a->a : nullptr, a->m, a->k, a->lda, 1, false, true},
      {"scale_a", a->k ? a->scale_a : nullptr, blocks(a->k), a->m, a->m, 4, false, false},
      {"b", a->k ? a->b : nullptr, a->n, a->k, a->ldb, 1, false, true},
      {"scale_b", a->k ? a->scale_b : nullptr, blocks(a->k), across, across, 4, false, false},
  };
  if ((rc = check_matrices(list, 5))) return rc;
  return launched(launch_fp8_matmul(*a, static_cast<hipStream_t>(hip_stream)), "opt8_fp8_matmul");
}

int gated_forward(const opt8_gated_ffn* a, void* hip_stream) {
  clear_last_error();
  if (!a) return refuse(OPT8_E_NULL, "ffn is NULL");
  int rc;
  if ((rc = check_count("rows", a->rows, 0, kMaxCount)) || (rc = check_count("d", a->d, 1, kMaxWidth)) ||
      (rc = check_count("f", a->f, 1, kMaxWidth)) || (rc = check_ffn_type(a->type, a->act)))
    return rc;
  if (a->rows == 0) return OPT8_OK;
  if (!a->gate != !a->up) return refuse(OPT8_E_NULL, "gate and up go together");
  if (!a->x || !a->w_gate || !a->w_up || !a->h) return refuse(OPT8_E_NULL, "x, w_gate, w_up or h is NULL");
  const Matrix list[] = {
      {"x", a->x, a->rows, a->d, a->ldx, 2, false, true},
      {"w_gate", a->w_gate, a->f, a->d, a->ldw, 2, false, true},
      {"w_up", a->w_up, a->f, a->d, a->ldw, 2, false, true},
      {"h", a->h, a->rows, a->f, a->ldh, 2, true, false},
      {"gate", a->gate, a->rows, a->f, a->ldg, 2, true, false},
      {"up", a->up, a->rows, a->f, a->ldg, 2, true, false},
  };
  if ((rc = check_matrices(list, 6))) return rc;
  return launched(launch_gated_ffn_forward(*a, static_cast<hipStream_t>(hip_stream)), "opt8_gated_ffn_forward");
}

int gated_backward(const opt8_gated_ffn_grad* a, void* hip_stream) {
  clear_last_error();
  if (!a) return refuse(OPT8_E_NULL, "grad is NULL");
  int rc;
  if ((rc = check_count("rows", a->rows, 0, kMaxCount)) || (rc = check_count("d", a->d, 1, kMaxWidth)) ||
      (rc = check_count("f", a->f, 1, kMaxWidth)) || (rc = check_ffn_type(a->type, a->act)))
    return rc;
  if (!a->dw_gate != !a->dw_up) return refuse(OPT8_E_NULL, "dw_gate and dw_up go together");
  const bool some = a->rows > 0;
  if (!some && !a->dw_gate) return OPT8_OK;
  if (!a->dx && !a->dw_gate) return refuse(OPT8_E_NULL, "dx and both dw are NULL");
  if (some && (!a->dh || !a->gate || !a->up || !a->workspace || (a->dx && (!a->w_gate || !a->w_up)) || (a->dw_gate && !a->x)))
    return refuse(OPT8_E_NULL, "dh, gate, up, workspace, the weights (for dx) or x (for the dw) is NULL");
  const int64_t need = opt8_gated_ffn_workspace(a->rows, a->d, a->f);
  if (some && a->workspace_bytes < need)
    return refuse(OPT8_E_SIZE, "workspace holds %lld bytes, %lld are needed", static_cast<long long>(a->workspace_bytes),
                  static_cast<long long>(need));
  const void* dx = some ? a->dx : nullptr;
  const Matrix list[] = {
      {"dh", some ? a->dh : nullptr, a->rows, a->f, a->lddh, 2, false, true},
      {"x", some && a->dw_gate ? a->x : nullptr, a->rows, a->d, a->ldx, 2, false, true},
      {"w_gate", dx ? a->w_gate : nullptr, a->f, a->d, a->ldw, 2, false, true},
      {"w_up", dx ? a->w_up : nullptr, a->f, a->d, a->ldw, 2, false, true},
      {"gate", some ? a->gate : nullptr, a->rows, a->f, a->ldg, 2, false, true},
      {"up", some ? a->up : nullptr, a->rows, a->f, a->ldg, 2, false, true},
      {"dx", dx, a->rows, a->d, a->lddx, 2, true, false},
      {"dw_gate", a->dw_gate, a->f, a->d, a->lddw, 2, true, false},
      {"dw_up", a->dw_up, a->f, a->d, a->lddw, 2, true, false},
      {"workspace", some ? a->workspace : nullptr, need / 16, 1, 1, 16, true, true},    // pieces of 16 bytes
  };
  if ((rc = check_matrices(list, 10))) return rc;
  return launched(launch_gated_ffn_backward(*a, static_cast<hipStream_t>(hip_stream)), "opt8_gated_ffn_backward");
}

}  // namespace
}  // namespace opt8

extern "C" int opt8_fp8_quantize(const opt8_fp8_quant* quant, void* hip_stream) {
  return opt8::quantize(quant, hip_stream);
}

extern "C" int opt8_fp8_matmul(const opt8_fp8_product* product, void* hip_stream) {
  return opt8::matmul(product, hip_stream);
}

extern "C" int opt8_gated_ffn_forward(const opt8_gated_ffn* ffn, void* hip_stream) {
  return opt8::gated_forward(ffn, hip_stream);
}

extern "C" int opt8_gated_ffn_backward(const opt8_gated_ffn_grad* grad, void* hip_stream) {
  return opt8::gated_backward(grad, hip_stream);
}

extern "C" int64_t opt8_gated_ffn_workspace(int64_t rows, int64_t d, int64_t f) {
  if (rows < 0 || d < 0 || f < 0 || rows > opt8::kMaxCount || d > opt8::kMaxWidth || f > opt8::kMaxWidth) return 0;
  return opt8::gated_workspace(rows, d, f);
}
