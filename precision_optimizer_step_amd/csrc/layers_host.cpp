// Argument checks and C entry points of the operators in opt8_layers.h.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "layers_internal.h"
#include "operand_checks.h"

namespace opt8 {
namespace {

// 512 columns of a row to a wave of 64: 2^34 elements are 2^31 threads (rows of fewer
// columns, at most 2^22, take a wave each).
constexpr int64_t kMaxLayerElements = int64_t{1} << 34;

bool wide_type(int type) { return type == OPT8_TYPE_BF16 || type == OPT8_TYPE_FP16 || type == OPT8_TYPE_FP32; }

int check_type(const char* what, int type) {
  if (!wide_type(type)) return refuse(OPT8_E_MODE, "%s: bf16, fp16 or fp32 (got type %d)", what, type);
  return OPT8_OK;
}

// Weights and their gradients: of the rows' type or of 32 bits.
int check_type_beside(const char* what, int type, int rows_type) {
  if (type != rows_type && type != OPT8_TYPE_FP32)
    return refuse(OPT8_E_MODE, "%s: of the rows' type or fp32 (got type %d)", what, type);
  return OPT8_OK;
}

int check_ids(int id_type) {
  if (id_type != OPT8_ID_INT32 && id_type != OPT8_ID_INT64) return refuse(OPT8_E_MODE, "unknown id type %d", id_type);
  return OPT8_OK;
}

int id_bytes(int id_type) { return id_type == OPT8_ID_INT32 ? 4 : 8; }

// The matrices of one call.
int check_layers(const Matrix* list, int n) {
  for (int i = 0; i < n; ++i)
    if (list[i].p && list[i].rows * list[i].cols > kMaxLayerElements)
      return refuse(OPT8_E_SIZE, "%s: over 2^34 elements", list[i].name);
  return check_matrices(list, n);
}

bool same_place(const void* a, int64_t lda, const void* b, int64_t ldb) { return a && a == b && lda == ldb; }

int check_workspace(const void* p, int64_t bytes, int64_t need) {
  if (need > 0 && !p) return refuse(OPT8_E_NULL, "workspace is NULL");
  if (bytes < need)
    return refuse(OPT8_E_SIZE, "workspace holds %lld bytes, %lld are needed", static_cast<long long>(bytes),
                  static_cast<long long>(need));
  return OPT8_OK;
}

// A workspace's bytes as a matrix of pieces of 16, for the check of overlaps.
Matrix workspace_of(const void* p, int64_t bytes) { return {"workspace", p, bytes / 16, 1, 1, 16, true, true}; }

int embedding_forward(const opt8_embedding* a, void* hip_stream) {
  clear_last_error();
  if (!a) return refuse(OPT8_E_NULL, "embedding is NULL");
  int rc;
  if ((rc = check_count("tokens", a->tokens, 0, kMaxCount)) || (rc = check_count("vocab", a->vocab, 0, kMaxCount)) ||
      (rc = check_count("d", a->d, 0, kMaxWidth)) || (rc = check_type("embedding", a->type)) || (rc = check_ids(a->id_type)))
    return rc;
  if (!std::isfinite(a->scale)) return refuse(OPT8_E_HPARAM, "scale is not finite");
  if (a->tokens == 0 || a->d == 0) return OPT8_OK;
  if (a->place_ids && (rc = check_count("places", a->places, 0, kMaxCount))) return rc;
  if (a->place_ids ? !a->place_table && a->places > 0 : a->place_table != nullptr)
    return refuse(OPT8_E_NULL, "place_ids and place_table go together");
  if (!a->ids || !a->y || (a->vocab > 0 && !a->table)) return refuse(OPT8_E_NULL, "ids, table or y is NULL");
  const int size = type_bytes(a->type), id = id_bytes(a->id_type);
  const Matrix list[] = {
      {"ids", a->ids, a->tokens, 1, 1, id, false, false},
      {"table", a->vocab > 0 ? a->table : nullptr, a->vocab, a->d, a->ldtable, size, false, false},
      {"place_ids", a->place_ids, a->tokens, 1, 1, id, false, false},
      {"place_table", a->place_ids && a->places > 0 ? a->place_table : nullptr, a->places, a->d, a->ldplace, size, false, false},
      {"y", a->y, a->tokens, a->d, a->ldy, size, true, false},
  };
  if ((rc = check_layers(list, 5))) return rc;
  return launched(launch_embedding_forward(*a, static_cast<hipStream_t>(hip_stream)), "opt8_embedding_forward");
}

int embedding_backward(const opt8_embedding_grad* a, void* hip_stream) {
  clear_last_error();
  if (!a) return refuse(OPT8_E_NULL, "grad is NULL");
  int rc;
  if ((rc = check_count("tokens", a->tokens, 0, kMaxCount)) || (rc = check_count("vocab", a->vocab, 0, kMaxCount)) ||
      (rc = check_count("d", a->d, 0, kMaxWidth)) || (rc = check_type("dy", a->type)) ||
      (rc = check_type_beside("dtable", a->dtable_type, a->type)) || (rc = check_ids(a->id_type)))
    return rc;
  if (!std::isfinite(a->scale)) return refuse(OPT8_E_HPARAM, "scale is not finite");
  if (a->vocab == 0 || a->d == 0 || (a->accumulate && a->tokens == 0)) return OPT8_OK;
  if (!a->dtable || (a->tokens > 0 && (!a->ids || !a->dy))) return refuse(OPT8_E_NULL, "ids, dy or dtable is NULL");
  const int64_t need = opt8_embedding_workspace(a->tokens, a->vocab, a->d);
  if ((rc = check_workspace(a->workspace, a->workspace_bytes, need))) return rc;
  const bool some = a->tokens > 0;
  const Matrix list[] = {
      {"ids", some ? a->ids : nullptr, a->tokens, 1, 1, id_bytes(a->id_type), false, false},
      {"dy", some ? a->dy : nullptr, a->tokens, a->d, a->lddy, type_bytes(a->type), false, false},
      {"dtable", a->dtable, a->vocab, a->d, a->lddtable, type_bytes(a->dtable_type), true, false},
      workspace_of(a->workspace, need),
  };
  if ((rc = check_layers(list, 4))) return rc;
  return launched(launch_embedding_backward(*a, static_cast<hipStream_t>(hip_stream)), "opt8_embedding_backward");
}

int rms_norm_forward(const opt8_rms_norm* a, void* hip_stream) {
  clear_last_error();
  if (!a) return refuse(OPT8_E_NULL, "norm is NULL");
  int rc;
  if ((rc = check_count("rows", a->rows, 0, kMaxCount)) || (rc = check_count("d", a->d, 1, kMaxWidth)) ||
      (rc = check_type("x", a->type)) || (rc = check_type_beside("weight", a->weight_type, a->type)))
    return rc;
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps)) return refuse(OPT8_E_HPARAM, "eps must be finite and not below 0");
  if (a->q && a->q_type != OPT8_TYPE_E4M3 && a->q_type != OPT8_TYPE_E5M2)
    return refuse(OPT8_E_MODE, "codes are e4m3 or e5m2 (got type %d)", a->q_type);
  if (a->rows == 0) return OPT8_OK;
  if (!a->x || !a->weight) return refuse(OPT8_E_NULL, "x or weight is NULL");
  if (!a->q != !a->scale) return refuse(OPT8_E_NULL, "q and scale go together");
  if (a->sum && !a->residual) return refuse(OPT8_E_NULL, "sum goes with a residual");
  if (!a->sum && !a->y && !a->q && !a->rstd) return refuse(OPT8_E_NULL, "no output: sum, y, q and rstd are all NULL");
  const int size = type_bytes(a->type);
  // a sum that takes its operand's place is checked as that one, which is then an output
  const bool on_x = same_place(a->sum, a->ldsum, a->x, a->ldx), on_r = same_place(a->sum, a->ldsum, a->residual, a->ldresidual);
  const Matrix list[] = {
      {"x", on_x ? nullptr : a->x, a->rows, a->d, a->ldx, size, false, false},
      {"residual", on_r ? nullptr : a->residual, a->rows, a->d, a->ldresidual, size, false, false},
      {"weight", a->weight, 1, a->d, a->d, type_bytes(a->weight_type), false, false},
      {"sum", a->sum, a->rows, a->d, a->ldsum, size, true, false},
      {"y", a->y, a->rows, a->d, a->ldy, size, true, false},
      {"q", a->q, a->rows, a->d, a->ldq, 1, true, true},
      {"scale", a->scale, blocks(a->d), a->rows, a->rows, 4, true, false},
      {"rstd", a->rstd, 1, a->rows, a->rows, 4, true, false},
  };
  if ((rc = check_layers(list, 8))) return rc;
  return launched(launch_rms_norm_forward(*a, static_cast<hipStream_t>(hip_stream)), "opt8_rms_norm_forward");
}

int rms_norm_backward(const opt8_rms_norm_grad* a, void* hip_stream) {
  clear_last_error();
  if (!a) return refuse(OPT8_E_NULL, "grad is NULL");
  int rc;
  if ((rc = check_count("rows", a->rows, 0, kMaxCount)) || (rc = check_count("d", a->d, 1, kMaxWidth)) ||
      (rc = check_type("dy", a->type)) || (rc = check_type_beside("weight", a->weight_type, a->type)) ||
      (rc = check_type_beside("dweight", a->dweight_type, a->type)))
    return rc;
  const bool some = a->rows > 0;
  if (!some && !a->dweight) return OPT8_OK;
  if (!a->dx && !a->dweight) return refuse(OPT8_E_NULL, "dx and dweight are both NULL");
  if (some && (!a->dy || !a->x || !a->rstd || (a->dx && !a->weight)))
    return refuse(OPT8_E_NULL, "dy, x, rstd or weight (for dx) is NULL");
  const int64_t need = a->dweight ? opt8_rms_norm_workspace(a->rows, a->d) : 0;
  if ((rc = check_workspace(a->workspace, a->workspace_bytes, need))) return rc;
  const int size = type_bytes(a->type);
  const void* dx = some ? a->dx : nullptr;
  const void* dsum = dx ? a->dsum : nullptr;
  const bool on_dy = same_place(dx, a->lddx, a->dy, a->lddy), on_dsum = same_place(dx, a->lddx, dsum, a->lddsum);
  const Matrix list[] = {
      {"dy", some && !on_dy ? a->dy : nullptr, a->rows, a->d, a->lddy, size, false, false},
      {"x", some ? a->x : nullptr, a->rows, a->d, a->ldx, size, false, false},
      {"weight", dx ? a->weight : nullptr, 1, a->d, a->d, type_bytes(a->weight_type), false, false},
      {"rstd", some ? a->rstd : nullptr, 1, a->rows, a->rows, 4, false, false},
      {"dsum", on_dsum ? nullptr : dsum, a->rows, a->d, a->lddsum, size, false, false},
      {"dx", dx, a->rows, a->d, a->lddx, size, true, false},
      {"dweight", a->dweight, 1, a->d, a->d, type_bytes(a->dweight_type), true, false},
      workspace_of(need > 0 ? a->workspace : nullptr, need),
  };
  if ((rc = check_layers(list, 8))) return rc;
  opt8_rms_norm_grad call = *a;
  call.dsum = dsum;    // without dx it was not checked, and nothing comes of it
  return launched(launch_rms_norm_backward(call, static_cast<hipStream_t>(hip_stream)), "opt8_rms_norm_backward");
}

// ---------------------------------------------------------------- lists of gradients
constexpr int32_t kMaxGrads = 1 << 22;
constexpr int64_t kMaxPieces = int64_t{1} << 26;

// Pieces of a list, or a status.
int64_t grad_pieces(const opt8_grad* grads, int32_t n) {
  if (n < 0 || n > kMaxGrads) return refuse(OPT8_E_SIZE, "n must be 0 to 2^22 (got %d)", n);
  if (n > 0 && !grads) return refuse(OPT8_E_NULL, "grads is NULL");
  int64_t pieces = 0;
  for (int32_t i = 0; i < n; ++i) {
    const opt8_grad& g = grads[i];
    if (g.numel < 0 || g.numel > kMaxElements)
      return refuse(OPT8_E_SIZE, "gradient %d: numel must be 0 to 2^37 (got %lld)", i, static_cast<long long>(g.numel));
    if (!wide_type(g.type) || (g.out && !wide_type(g.out_type)))
      return refuse(OPT8_E_MODE, "gradient %d: bf16, fp16 or fp32", i);
    if (g.numel == 0) continue;
    if (!g.grad) return refuse(OPT8_E_NULL, "gradient %d is NULL", i);
    if (g.out == g.grad && g.out_type != g.type) return refuse(OPT8_E_MODE, "gradient %d: its own place has another type", i);
    if (reinterpret_cast<uintptr_t>(g.grad) % static_cast<uintptr_t>(type_bytes(g.type)) ||
        (g.out && reinterpret_cast<uintptr_t>(g.out) % static_cast<uintptr_t>(type_bytes(g.out_type))))
      return refuse(OPT8_E_ALIGN, "gradient %d: not aligned to its elements", i);
    pieces += pieces_of(g.numel, OPT8_GRAD_PIECE);
    if (pieces > kMaxPieces) return refuse(OPT8_E_SIZE, "the list has over 2^26 pieces of 8192 values");
  }
  return pieces;
}

struct GradSpan {
  uintptr_t begin, end;
  int32_t index;
  bool operator<(const GradSpan& o) const { return begin < o.begin; }
};

int grad_table(const opt8_grad* grads, int32_t n, void* table, int64_t bytes) {
  const int64_t pieces = grad_pieces(grads, n);
  if (pieces < 0) return static_cast<int>(pieces);
  const int64_t need = (pieces + 1) * OPT8_GRAD_PIECE_BYTES;
  if (bytes < need)
    return refuse(OPT8_E_SIZE, "the table holds %lld bytes, %lld are needed", static_cast<long long>(bytes),
                  static_cast<long long>(need));
  if (!table) return refuse(OPT8_E_NULL, "the table is NULL");
  try {
    std::vector<GradSpan> spans;
    spans.reserve(2 * static_cast<size_t>(n));
    auto add = [&](const void* p, int64_t count, int type, int32_t i) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      spans.push_back({at, at + static_cast<uintptr_t>(count) * type_bytes(type), i});
    };
    for (int32_t i = 0; i < n; ++i) {
      const opt8_grad& g = grads[i];
      if (g.numel == 0) continue;
      add(g.grad, g.numel, g.type, i);
      if (g.out && g.out != g.grad) add(g.out, g.numel, g.out_type, i);
    }
    if (!std::is_sorted(spans.begin(), spans.end())) std::sort(spans.begin(), spans.end());
    for (size_t i = 1; i < spans.size(); ++i)
      if (spans[i].begin < spans[i - 1].end)
        return refuse(OPT8_E_ALIAS, "buffers of gradients %d and %d overlap", spans[i - 1].index, spans[i].index);
  } catch (const std::bad_alloc&) {
    return refuse(OPT8_E_NOMEM, "out of host memory");
  }
  char* at = static_cast<char*>(table) + sizeof(GradHead);
  GradHead head{pieces, 0, 0};
  for (const bool own : {true, false}) {
    for (int32_t i = 0; i < n; ++i) {
      const opt8_grad& g = grads[i];
      if (own != (g.out && g.out != g.grad)) continue;
      char* from = static_cast<char*>(g.grad);
      char* to = static_cast<char*>(own ? g.out : g.grad);
      const int32_t to_type = own ? g.out_type : g.type;
      const int64_t size = type_bytes(g.type), to_size = type_bytes(to_type);
      for (int64_t first = 0; first < g.numel; first += OPT8_GRAD_PIECE) {
        GradPiece piece;
        piece.from = from + first * size;
        piece.to = to + first * to_size;
        piece.count = static_cast<int32_t>(std::min<int64_t>(OPT8_GRAD_PIECE, g.numel - first));
        piece.type = static_cast<int16_t>(g.type);
        piece.to_type = static_cast<int16_t>(to_type);
        std::memcpy(at, &piece, sizeof piece);
        at += sizeof piece;
        head.own += own;
      }
    }
  }
  std::memcpy(table, &head, sizeof head);
  return OPT8_OK;
}

int check_grads(const opt8_grads* a, bool norm) {
  clear_last_error();
  if (!a) return refuse(OPT8_E_NULL, "grads is NULL");
  int rc;
  if (a->table_bytes < OPT8_GRAD_PIECE_BYTES || a->table_bytes % OPT8_GRAD_PIECE_BYTES ||
      a->table_bytes > (kMaxPieces + 1) * OPT8_GRAD_PIECE_BYTES)
    return refuse(OPT8_E_SIZE, "a table has 24 bytes and 24 for each piece (got %lld)", static_cast<long long>(a->table_bytes));
  if (!norm && (!(a->max_norm >= 0.0) || !std::isfinite(a->max_norm)))
    return refuse(OPT8_E_HPARAM, "max_norm must be finite and not below 0");
  if (!a->squares || !a->table) return refuse(OPT8_E_NULL, "table or squares is NULL");
  if (norm && (rc = check_workspace(a->workspace, a->workspace_bytes, OPT8_GRAD_WORKSPACE))) return rc;
  if (reinterpret_cast<uintptr_t>(a->table) % 8) return refuse(OPT8_E_ALIGN, "table: not aligned to 8 bytes");
  const Matrix list[] = {
      {"table", a->table, a->table_bytes, 1, 1, 1, false, false},
      {"squares", a->squares, 1, 1, 1, 8, norm, false},
      {"norm", a->norm, 1, 1, 1, 4, true, false},
      workspace_of(norm ? a->workspace : nullptr, OPT8_GRAD_WORKSPACE),
  };
  return check_layers(list, 4);
}

}  // namespace
}  // namespace opt8

extern "C" int opt8_embedding_forward(const opt8_embedding* embedding, void* hip_stream) {
  return opt8::embedding_forward(embedding, hip_stream);
}

extern "C" int opt8_embedding_backward(const opt8_embedding_grad* grad, void* hip_stream) {
  return opt8::embedding_backward(grad, hip_stream);
}

extern "C" int64_t opt8_embedding_workspace(int64_t tokens, int64_t vocab, int64_t d) {
  if (tokens < 0 || vocab < 0 || d < 0 || tokens > opt8::kMaxCount || vocab > opt8::kMaxCount || d > opt8::kMaxWidth) return 0;
  return opt8::embedding_space(tokens, vocab, d).bytes;
}

extern "C" int opt8_rms_norm_forward(const opt8_rms_norm* norm, void* hip_stream) {
  return opt8::rms_norm_forward(norm, hip_stream);
}

extern "C" int opt8_rms_norm_backward(const opt8_rms_norm_grad* grad, void* hip_stream) {
  return opt8::rms_norm_backward(grad, hip_stream);
}

extern "C" int64_t opt8_rms_norm_workspace(int64_t rows, int64_t d) {
  if (rows < 0 || d < 1 || rows > opt8::kMaxCount || d > opt8::kMaxWidth) return 0;
  return opt8::norm_grad_space(rows, d);
}

extern "C" int64_t opt8_grad_table_bytes(const opt8_grad* grads, int32_t n) {
  opt8::clear_last_error();
  const int64_t pieces = opt8::grad_pieces(grads, n);
  return pieces < 0 ? pieces : (pieces + 1) * OPT8_GRAD_PIECE_BYTES;
}

extern "C" int opt8_grad_table(const opt8_grad* grads, int32_t n, void* host_table, int64_t bytes) {
  opt8::clear_last_error();
  return opt8::grad_table(grads, n, host_table, bytes);
}

extern "C" int opt8_grad_norm(const opt8_grads* grads, void* hip_stream) {
  const int rc = opt8::check_grads(grads, true);
  if (rc) return rc;
  return opt8::launched(opt8::launch_grad_norm(*grads, static_cast<hipStream_t>(hip_stream)), "opt8_grad_norm");
}

extern "C" int opt8_grad_clip(const opt8_grads* grads, void* hip_stream) {
  const int rc = opt8::check_grads(grads, false);
  if (rc) return rc;
  return opt8::launched(opt8::launch_grad_clip(*grads, static_cast<hipStream_t>(hip_stream)), "opt8_grad_clip");
}
