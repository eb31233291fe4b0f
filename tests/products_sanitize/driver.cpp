// products_host.cpp with recording stand-ins for the launches and the error
// channel: random arguments through every entry point.  A launch may happen only
// where no output shares a byte with another buffer (checked byte by byte on
// small matrices), every buffer holds its rows, and the refusal code is one of the
// documented ones.
#include <cstdio>
#include <cstring>
#include <random>
#include <set>
#include <string>
#include <vector>

#include "opt8_error.h"
#include "products_internal.h"

namespace opt8 {
static std::string g_error;
static int g_launches = 0;
static hipError_t g_result = hipSuccess;
void clear_last_error() { g_error.clear(); }
int set_last_error(int code, const char* message) {
  g_error = message;
  return code;
}
hipError_t launch_fp8_quantize(const opt8_fp8_quant&, hipStream_t) { ++g_launches; return g_result; }
hipError_t launch_fp8_matmul(const opt8_fp8_product&, hipStream_t) { ++g_launches; return g_result; }
hipError_t launch_gated_ffn_forward(const opt8_gated_ffn&, hipStream_t) { ++g_launches; return g_result; }
hipError_t launch_gated_ffn_backward(const opt8_gated_ffn_grad&, hipStream_t) { ++g_launches; return g_result; }
}  // namespace opt8

extern "C" const char* hipGetErrorString(hipError_t) { return "stand-in error"; }

namespace {

std::mt19937_64 rng(1);
int64_t upto(int64_t n) { return static_cast<int64_t>(rng() % static_cast<uint64_t>(n + 1)); }

struct Buffer {
  uintptr_t p;
  int64_t rows, cols, ld;
  int size;
  bool output;
};

std::set<uintptr_t> bytes_of(const Buffer& b) {
  std::set<uintptr_t> s;
  for (int64_t r = 0; r < b.rows; ++r)
    for (int64_t c = 0; c < b.cols * b.size; ++c) s.insert(b.p + r * b.ld * b.size + c);
  return s;
}

bool shared(const std::vector<Buffer>& list) {
  for (size_t i = 0; i < list.size(); ++i) {
    if (!list[i].output || !list[i].p) continue;
    const auto a = bytes_of(list[i]);
    for (size_t j = 0; j < list.size(); ++j) {
      if (i == j || !list[j].p) continue;
      for (uintptr_t x : bytes_of(list[j]))
        if (a.count(x)) return true;
    }
  }
  return false;
}

int failures = 0, accepted = 0, aliases = 0;

void check(int rc, int launches, const std::vector<Buffer>& list, const char* what) {
  const bool ran = opt8::g_launches > launches;
  if (ran) {
    ++accepted;
    if (shared(list)) { std::printf("%s: launched with shared bytes\n", what); ++failures; }
    for (const Buffer& b : list)
      if (b.p && b.ld < b.cols) { std::printf("%s: launched with ld below cols\n", what); ++failures; }
  }
  if (rc == OPT8_E_ALIAS) ++aliases;
  if (rc != OPT8_OK && opt8::g_error.empty()) { std::printf("%s: a refusal without a message\n", what); ++failures; }
  if (rc < OPT8_E_NOMEM || rc > OPT8_OK) { std::printf("%s: unknown status %d\n", what, rc); ++failures; }
}

template <class T>
T* at(uintptr_t p) { return reinterpret_cast<T*>(p); }

// Addresses close together (a few hundred bytes), so that many calls overlap.
uintptr_t place() { return 0x100000 + 16 * static_cast<uintptr_t>(upto(60)); }

void ffn(int round) {
  opt8_gated_ffn a;
  std::memset(&a, 0, sizeof a);
  const uintptr_t far = 0x200000;
  a.x = at<void>(far);
  a.w_gate = at<void>(far + 0x100000);
  a.w_up = at<void>(far + 0x200000);
  a.rows = 1 + upto(3);
  a.d = 1 + upto(7);
  a.f = 1 + upto(11);
  a.ldx = a.ldw = 8;
  a.ldg = a.f + upto(12);
  a.ldh = round % 2 ? a.ldg : a.f + upto(12);
  const uintptr_t h = place(), g = place(), u = round % 3 ? place() : g + 2 * static_cast<uintptr_t>(upto(20));
  a.h = at<void>(h);
  a.gate = at<void>(g);
  a.up = at<void>(u);
  a.type = static_cast<int32_t>(upto(2));
  a.act = static_cast<int32_t>(upto(3));
  const int before = opt8::g_launches;
  const int rc = opt8_gated_ffn_forward(&a, nullptr);
  check(rc, before, {{h, a.rows, a.f, a.ldh, 2, true}, {g, a.rows, a.f, a.ldg, 2, true}, {u, a.rows, a.f, a.ldg, 2, true}},
        "gated_ffn_forward");
}

void quant(int round) {
  opt8_fp8_quant a;
  std::memset(&a, 0, sizeof a);
  a.rows = 1 + upto(3);
  a.cols = 1 + upto(20);
  a.ldx = a.cols + upto(8);
  a.ldq = 16 * (1 + upto(2));
  a.ldt = 16 * (1 + upto(1));
  a.x_type = static_cast<int32_t>(upto(3));
  a.q_type = OPT8_TYPE_E4M3 + static_cast<int32_t>(upto(1));
  a.block = static_cast<int32_t>(upto(1));
  const int xs = a.x_type == OPT8_TYPE_FP32 ? 4 : 2;
  const uintptr_t x = place(), q = place(), s = place(), qt = round % 2 ? place() : 0, st = qt ? place() : 0;
  a.x = at<void>(x);
  a.q = at<void>(q);
  a.scale = at<float>(s);
  a.qt = at<void>(qt);
  a.scale_t = at<float>(st);
  const bool tile = a.block == OPT8_FP8_BLOCK_TILE;
  const int64_t na = tile ? 1 : a.rows, nt = tile ? 1 : a.cols;
  const int before = opt8::g_launches;
  const int rc = opt8_fp8_quantize(&a, nullptr);
  check(rc, before, {{x, a.rows, a.cols, a.ldx, xs, false}, {q, a.rows, a.cols, a.ldq, 1, true}, {s, 1, na, na, 4, true},
                     {qt, a.cols, a.rows, a.ldt, 1, true}, {st, 1, nt, nt, 4, true}}, "fp8_quantize");
}

void product(int) {
  opt8_fp8_product a;
  std::memset(&a, 0, sizeof a);
  a.m = upto(4);
  a.n = upto(6);
  a.k = upto(40);
  a.lda = 16 * (1 + upto(3));
  a.ldb = 16 * (1 + upto(3));
  a.ldc = a.n + upto(4);
  a.a_type = OPT8_TYPE_E4M3;
  a.b_type = OPT8_TYPE_E4M3;
  a.c_type = static_cast<int32_t>(upto(1));
  a.block_b = static_cast<int32_t>(upto(1));
  const uintptr_t pa = place(), sa = place(), pb = place(), sb = place(), c = place() + static_cast<uintptr_t>(upto(3));
  a.a = at<void>(pa);
  a.scale_a = at<float>(sa);
  a.b = at<void>(pb);
  a.scale_b = at<float>(sb);
  a.c = at<void>(c);
  const int64_t nb = a.block_b == OPT8_FP8_BLOCK_TILE ? (a.n + 127) / 128 : a.n, kb = (a.k + 127) / 128;
  const int before = opt8::g_launches;
  const int rc = opt8_fp8_matmul(&a, nullptr);
  check(rc, before, {{c, a.m, a.n, a.ldc, 2, true}, {pa, a.k ? a.m : 0, a.k, a.lda, 1, false}, {sa, kb, a.m, a.m, 4, false},
                     {pb, a.k ? a.n : 0, a.k, a.ldb, 1, false}, {sb, kb, nb, nb, 4, false}}, "fp8_matmul");
}

void grad(int) {
  opt8_gated_ffn_grad a;
  std::memset(&a, 0, sizeof a);
  a.rows = upto(3);
  a.d = 1 + upto(7);
  a.f = 1 + upto(7);
  a.ldx = a.ldw = a.lddh = a.ldg = 8;
  a.lddx = a.d + upto(3);
  a.lddw = a.d + upto(3);
  const uintptr_t far = 0x200000;
  a.dh = at<void>(far);
  a.x = at<void>(far + 0x1000);
  a.w_gate = at<void>(far + 0x2000);
  a.w_up = at<void>(far + 0x3000);
  a.gate = at<void>(far + 0x4000);
  a.up = at<void>(far + 0x5000);
  a.workspace = at<void>(far + 0x100000);
  a.workspace_bytes = opt8_gated_ffn_workspace(a.rows, a.d, a.f) - (upto(9) == 0);
  const uintptr_t dx = upto(5) ? place() : 0, dg = upto(5) ? place() : 0, du = dg ? place() : 0;
  a.dx = at<void>(dx);
  a.dw_gate = at<void>(dg);
  a.dw_up = at<void>(du);
  const int before = opt8::g_launches;
  const int rc = opt8_gated_ffn_backward(&a, nullptr);
  check(rc, before, {{dx, a.rows, a.d, a.lddx, 2, true}, {dg, a.f, a.d, a.lddw, 2, true}, {du, a.f, a.d, a.lddw, 2, true}},
        "gated_ffn_backward");
}

}  // namespace

int main() {
  for (int i = 0; i < 20000; ++i) {
    ffn(i);
    quant(i);
    product(i);
    grad(i);
  }
  // sizes at and past their limits: no arithmetic on them overflows
  for (int64_t v : {int64_t{0}, int64_t{1}, int64_t{1} << 20, int64_t{1} << 22, (int64_t{1} << 22) + 1, INT64_MAX, INT64_MIN}) {
    for (int64_t w : {int64_t{1}, int64_t{1} << 22, int64_t{1} << 40, INT64_MAX, INT64_MIN}) {
      opt8_fp8_quant q{at<void>(1 << 20), at<void>(2 << 20), at<float>(3 << 20), nullptr, nullptr, v, w, w, w, 0, 0, 3, 0};
      (void)opt8_fp8_quantize(&q, nullptr);
      opt8_fp8_product p{at<void>(1 << 20), at<float>(2 << 20), at<void>(3 << 20), at<float>(4 << 20), at<void>(5 << 20), v, w, v,
                         w, w, w, 3, 3, 0, 1};
      (void)opt8_fp8_matmul(&p, nullptr);
      opt8_gated_ffn f{at<void>(1 << 20), at<void>(2 << 20), at<void>(3 << 20), at<void>(4 << 20), nullptr, nullptr, v, w, v, w, w,
                       w, w, 0, 0};
      (void)opt8_gated_ffn_forward(&f, nullptr);
      (void)opt8_gated_ffn_workspace(v, w, v);
      (void)opt8_gated_ffn_workspace(w, v, v);
    }
  }
  // the widest row distances beside the most rows: a matrix's span stays in 64 bits
  for (int64_t ld : {int64_t{1} << 38, (int64_t{1} << 38) + 1, int64_t{1} << 40}) {
    const int before = opt8::g_launches;
    opt8_fp8_quant q{at<void>(1 << 20), at<void>(int64_t{1} << 62), at<float>(3 << 20), nullptr, nullptr, int64_t{1} << 22, 1, ld, 16, 0,
                     OPT8_TYPE_FP32, OPT8_TYPE_E4M3, OPT8_FP8_BLOCK_TILE};
    const int rc = opt8_fp8_quantize(&q, nullptr);
    if (rc == OPT8_OK || opt8::g_launches != before) {
      std::printf("ld %lld: scale lies in x's span, not refused\n", static_cast<long long>(ld));
      ++failures;
    }
  }
  // a launch that fails is reported
  opt8::g_result = hipErrorInvalidConfiguration;
  opt8_fp8_quant q{at<void>(1 << 20), at<void>(2 << 20), at<float>(3 << 20), nullptr, nullptr, 4, 16, 16, 16, 0, 0, 3, 0};
  if (opt8_fp8_quantize(&q, nullptr) != OPT8_E_HIP || opt8::g_error.find("stand-in") == std::string::npos) {
    std::printf("a failed launch was not reported\n");
    ++failures;
  }
  std::printf("%d launched, %d refused as overlapping\n", accepted, aliases);
  if (accepted < 1000 || aliases < 1000) ++failures;
  if (failures) return 1;
  std::printf("all checks passed\n");
  return 0;
}
