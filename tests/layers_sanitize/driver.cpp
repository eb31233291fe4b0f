// layers_host.cpp with recording stand-ins for the launches and the error
// channel: random arguments through every entry point.  A launch may happen only
// where no output shares a byte with another buffer (checked byte by byte on
// small matrices), except for the places that a call may take; a list's table
// holds every value of every gradient once; the refusal code is one of the
// documented ones; a host allocation that fails is OPT8_E_NOMEM.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <random>
#include <set>
#include <string>
#include <vector>

#include "layers_internal.h"
#include "opt8_error.h"

static bool g_no_memory = false;
void* operator new(std::size_t n) {
  if (g_no_memory) throw std::bad_alloc();
  if (void* p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

namespace opt8 {
static char g_error[600];
static int g_launches = 0;
static hipError_t g_result = hipSuccess;
void clear_last_error() { g_error[0] = 0; }
int set_last_error(int code, const char* message) {
  std::snprintf(g_error, sizeof g_error, "%s", message);
  return code;
}
hipError_t launch_embedding_forward(const opt8_embedding&, hipStream_t) { ++g_launches; return g_result; }
hipError_t launch_embedding_backward(const opt8_embedding_grad&, hipStream_t) { ++g_launches; return g_result; }
hipError_t launch_rms_norm_forward(const opt8_rms_norm&, hipStream_t) { ++g_launches; return g_result; }
hipError_t launch_rms_norm_backward(const opt8_rms_norm_grad&, hipStream_t) { ++g_launches; return g_result; }
hipError_t launch_grad_norm(const opt8_grads&, hipStream_t) { ++g_launches; return g_result; }
hipError_t launch_grad_clip(const opt8_grads&, hipStream_t) { ++g_launches; return g_result; }
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
  if (opt8::g_launches > launches) {
    ++accepted;
    if (shared(list)) { std::printf("%s: launched with shared bytes\n", what); ++failures; }
    for (const Buffer& b : list)
      if (b.p && b.rows > 0 && b.ld < b.cols) { std::printf("%s: launched with ld below cols\n", what); ++failures; }
  }
  if (rc == OPT8_E_ALIAS) ++aliases;
  if (rc != OPT8_OK && !opt8::g_error[0]) { std::printf("%s: a refusal without a message\n", what); ++failures; }
  if (rc < OPT8_E_NOMEM || rc > OPT8_OK) { std::printf("%s: unknown status %d\n", what, rc); ++failures; }
}

template <class T>
T* at(uintptr_t p) { return reinterpret_cast<T*>(p); }
uintptr_t place() { return 0x100000 + 16 * static_cast<uintptr_t>(upto(80)); }
constexpr uintptr_t kFar = 0x200000;

void embed(int) {
  opt8_embedding a;
  std::memset(&a, 0, sizeof a);
  a.tokens = upto(4);
  a.vocab = upto(5);
  a.places = upto(3);
  a.d = upto(9);
  a.ldtable = a.d + upto(3) - 1;
  a.ldplace = a.d + upto(3);
  a.ldy = a.d + upto(3);
  a.scale = 1.0f;
  a.type = static_cast<int32_t>(upto(3));
  a.id_type = static_cast<int32_t>(upto(1));
  const uintptr_t ids = place(), t = place(), pi = upto(2) ? place() : 0, pt = pi ? place() : 0, y = place() + 2 * static_cast<uintptr_t>(upto(2));
  a.ids = at<void>(ids);
  a.table = at<void>(t);
  a.place_ids = at<void>(pi);
  a.place_table = at<void>(pt);
  a.y = at<void>(y);
  const int size = a.type == OPT8_TYPE_FP32 ? 4 : 2, id = a.id_type ? 8 : 4;
  const int before = opt8::g_launches;
  const int rc = opt8_embedding_forward(&a, nullptr);
  check(rc, before, {{ids, a.tokens, 1, 1, id, false}, {t, a.vocab, a.d, a.ldtable, size, false}, {pi, a.tokens, 1, 1, id, false},
                     {pt, a.places, a.d, a.ldplace, size, false}, {y, a.tokens, a.d, a.ldy, size, true}}, "embedding_forward");
}

void embed_grad(int) {
  opt8_embedding_grad a;
  std::memset(&a, 0, sizeof a);
  a.tokens = upto(4);
  a.vocab = upto(5);
  a.d = upto(9);
  a.lddy = a.d + upto(3);
  a.lddtable = a.d + upto(3);
  a.type = static_cast<int32_t>(upto(2));
  a.dtable_type = upto(1) ? a.type : OPT8_TYPE_FP32;
  a.id_type = static_cast<int32_t>(upto(2));
  a.accumulate = static_cast<int32_t>(upto(1));
  const uintptr_t ids = place(), dy = place(), dt = place();
  a.ids = at<void>(ids);
  a.dy = at<void>(dy);
  a.dtable = at<void>(dt);
  const int64_t need = opt8_embedding_workspace(a.tokens, a.vocab, a.d);
  a.workspace = at<void>(upto(20) ? kFar : kFar - static_cast<uintptr_t>(need));
  a.workspace_bytes = need - (upto(9) == 0);
  const int before = opt8::g_launches;
  const int rc = opt8_embedding_backward(&a, nullptr);
  if (rc == OPT8_OK && opt8::g_launches > before && a.workspace_bytes < need) { std::printf("a short workspace\n"); ++failures; }
  check(rc, before, {{ids, a.tokens, 1, 1, a.id_type ? 8 : 4, false}, {dy, a.tokens, a.d, a.lddy, a.type == OPT8_TYPE_FP32 ? 4 : 2, false},
                     {dt, a.vocab, a.d, a.lddtable, a.dtable_type == OPT8_TYPE_FP32 ? 4 : 2, true}}, "embedding_backward");
}

void norm(int round) {
  opt8_rms_norm a;
  std::memset(&a, 0, sizeof a);
  a.rows = upto(3);
  a.d = 1 + upto(9);
  a.ldx = a.d + upto(2);
  a.ldresidual = a.d + upto(2);
  a.ldsum = a.d + upto(2);
  a.ldy = a.d + upto(2);
  a.ldq = 16 * (1 + upto(1));
  a.type = static_cast<int32_t>(upto(2));
  a.weight_type = upto(1) ? a.type : OPT8_TYPE_FP32;
  a.q_type = OPT8_TYPE_E4M3;
  const int size = a.type == OPT8_TYPE_FP32 ? 4 : 2;
  const uintptr_t x = place(), r = upto(3) ? place() : 0, w = place(), y = upto(2) ? place() : 0, q = upto(2) ? place() : 0, sc = q ? place() : 0;
  const uintptr_t rs = upto(2) ? place() : 0;
  uintptr_t s = r && upto(2) ? place() : 0;
  if (s && round % 3 == 0) s = x, a.ldsum = upto(3) ? a.ldx : a.ldsum;
  if (s && round % 3 == 1) s = r, a.ldsum = upto(3) ? a.ldresidual : a.ldsum;
  a.x = at<void>(x);
  a.residual = at<void>(r);
  a.weight = at<void>(w);
  a.sum = at<void>(s);
  a.y = at<void>(y);
  a.q = at<void>(q);
  a.scale = at<float>(sc);
  a.rstd = at<float>(rs);
  const bool on_x = s && s == x && a.ldsum == a.ldx, on_r = s && s == r && a.ldsum == a.ldresidual;
  const int before = opt8::g_launches;
  const int rc = opt8_rms_norm_forward(&a, nullptr);
  check(rc, before, {{on_x ? 0 : x, a.rows, a.d, a.ldx, size, false}, {on_r ? 0 : r, a.rows, a.d, a.ldresidual, size, false},
                     {w, 1, a.d, a.d, a.weight_type == OPT8_TYPE_FP32 ? 4 : 2, false}, {s, a.rows, a.d, a.ldsum, size, true},
                     {y, a.rows, a.d, a.ldy, size, true}, {q, a.rows, a.d, a.ldq, 1, true}, {sc, 1, a.rows, a.rows, 4, true},
                     {rs, 1, a.rows, a.rows, 4, true}}, "rms_norm_forward");
}

void norm_grad(int round) {
  opt8_rms_norm_grad a;
  std::memset(&a, 0, sizeof a);
  a.rows = upto(3);
  a.d = 1 + upto(9);
  a.lddy = a.d + upto(2);
  a.ldx = a.d + upto(2);
  a.lddsum = a.d + upto(2);
  a.lddx = a.d + upto(2);
  a.type = static_cast<int32_t>(upto(2));
  a.weight_type = a.type;
  a.dweight_type = OPT8_TYPE_FP32;
  const int size = a.type == OPT8_TYPE_FP32 ? 4 : 2;
  const uintptr_t dy = place(), x = place(), w = place(), rs = place(), ds = upto(2) ? place() : 0, dw = upto(3) ? place() : 0;
  uintptr_t dx = upto(3) ? place() : 0;
  if (dx && round % 3 == 0) dx = dy, a.lddx = upto(3) ? a.lddy : a.lddx;
  if (dx && ds && round % 3 == 1) dx = ds, a.lddx = upto(3) ? a.lddsum : a.lddx;
  a.dy = at<void>(dy);
  a.x = at<void>(x);
  a.weight = at<void>(w);
  a.rstd = at<float>(rs);
  a.dsum = at<void>(ds);
  a.dx = at<void>(dx);
  a.dweight = at<void>(dw);
  a.workspace = at<void>(kFar);
  a.workspace_bytes = opt8_rms_norm_workspace(a.rows, a.d) - (upto(9) == 0);
  const bool on_dy = dx && dx == dy && a.lddx == a.lddy, on_ds = dx && dx == ds && a.lddx == a.lddsum;
  const int before = opt8::g_launches;
  const int rc = opt8_rms_norm_backward(&a, nullptr);
  check(rc, before, {{on_dy ? 0 : dy, a.rows, a.d, a.lddy, size, false}, {x, a.rows, a.d, a.ldx, size, false}, {dx ? w : 0, a.rows ? 1 : 0, a.d, a.d, size, false},
                     {rs, a.rows ? 1 : 0, a.rows, a.rows, 4, false}, {dx && !on_ds ? ds : 0, a.rows, a.d, a.lddsum, size, false},
                     {dx, a.rows, a.d, a.lddx, size, true}, {dw, 1, a.d, a.d, 4, true}}, "rms_norm_backward");
}

void list(int) {
  std::vector<opt8_grad> g(static_cast<size_t>(upto(6)));
  uintptr_t next = 0x100000;
  bool apart = true;
  std::set<uintptr_t> bytes;
  for (auto& e : g) {
    e.type = static_cast<int32_t>(upto(2));
    e.out_type = static_cast<int32_t>(upto(2));
    e.numel = upto(5) ? upto(40) : 8192 * upto(2) + upto(3);
    e.grad = at<void>(upto(20) ? next : 0x100000);
    next += 4 * static_cast<uintptr_t>(e.numel) + 16;
    e.out = upto(1) ? at<void>(next) : nullptr;
    next += 4 * static_cast<uintptr_t>(e.numel) + 16;
    if (e.out && upto(3) == 0) e.out = e.grad, e.out_type = e.type;
    auto add = [&](void* p, int type) {
      for (int64_t i = 0; i < e.numel * (type == OPT8_TYPE_FP32 ? 4 : 2); ++i) apart &= bytes.insert(reinterpret_cast<uintptr_t>(p) + i).second;
    };
    add(e.grad, e.type);
    if (e.out && e.out != e.grad) add(e.out, e.out_type);
  }
  const int64_t size = opt8_grad_table_bytes(g.data(), static_cast<int32_t>(g.size()));
  if (size < 24) { std::printf("table_bytes %lld: %s\n", static_cast<long long>(size), opt8::g_error); ++failures; return; }
  std::vector<char> table(static_cast<size_t>(size));
  const int rc = opt8_grad_table(g.data(), static_cast<int32_t>(g.size()), table.data(), size);
  if ((rc == OPT8_OK) != apart || (rc != OPT8_OK && rc != OPT8_E_ALIAS)) { std::printf("list: status %d, apart %d\n", rc, apart); ++failures; }
  if (rc != OPT8_OK) { ++aliases; return; }
  ++accepted;
  opt8::GradHead head;
  std::memcpy(&head, table.data(), sizeof head);
  if (size != 24 * (head.pieces + 1)) { std::printf("list: %lld pieces\n", static_cast<long long>(head.pieces)); ++failures; }
  int64_t values = 0, want = 0;
  for (int64_t i = 0; i < head.pieces; ++i) {
    opt8::GradPiece p;
    std::memcpy(&p, table.data() + 24 * (i + 1), sizeof p);
    values += p.count;
    if ((p.from != p.to) != (i < head.own) || p.count < 1 || p.count > 8192) { std::printf("list: piece %lld\n", static_cast<long long>(i)); ++failures; }
    for (int k = 0; k < p.count * (p.type == OPT8_TYPE_FP32 ? 4 : 2); ++k)
      if (!bytes.erase(reinterpret_cast<uintptr_t>(p.from) + k)) { std::printf("list: a byte twice\n"); ++failures; break; }
    if (p.from != p.to)
      for (int k = 0; k < p.count * (p.to_type == OPT8_TYPE_FP32 ? 4 : 2); ++k)
        if (!bytes.erase(reinterpret_cast<uintptr_t>(p.to) + k)) { std::printf("list: a byte twice\n"); ++failures; break; }
  }
  for (auto& e : g) want += e.numel;
  if (values != want || !bytes.empty()) { std::printf("list: %lld of %lld values\n", static_cast<long long>(values), static_cast<long long>(want)); ++failures; }
}

}  // namespace

int main() {
  for (int i = 0; i < 20000; ++i) {
    embed(i);
    embed_grad(i);
    norm(i);
    norm_grad(i);
    if (i % 20 == 0) list(i);
  }
  // sizes at and past their limits: no arithmetic on them overflows
  const int64_t ends[] = {INT64_MIN, -1, 0, 1, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, 1 << 22, (1 << 22) + 1, int64_t{1} << 38, INT64_MAX};
  for (int64_t a : ends)
    for (int64_t b : ends)
      for (int64_t c : ends) {
        if (opt8_embedding_workspace(a, b, c) < 0 || opt8_rms_norm_workspace(a, c) < 0) { std::printf("a negative workspace\n"); ++failures; }
        opt8_embedding_grad e;
        std::memset(&e, 0, sizeof e);
        e.ids = at<void>(0x1000);
        e.dy = at<void>(uintptr_t{1} << 50);
        e.dtable = at<void>(uintptr_t{1} << 51);
        e.workspace = at<void>(uintptr_t{1} << 52);
        e.workspace_bytes = INT64_MAX;
        e.tokens = a;
        e.vocab = b;
        e.d = c;
        e.lddy = c;
        e.lddtable = b;
        (void)opt8_embedding_backward(&e, nullptr);
        opt8_rms_norm n;
        std::memset(&n, 0, sizeof n);
        n.x = at<void>(uintptr_t{1} << 50);
        n.weight = at<void>(0x1000);
        n.y = at<void>(uintptr_t{1} << 52);
        n.rows = a;
        n.d = b;
        n.ldx = n.ldy = c;
        (void)opt8_rms_norm_forward(&n, nullptr);
        opt8_grad g;
        std::memset(&g, 0, sizeof g);
        g.grad = at<void>(0x1000);
        g.numel = a;
        (void)opt8_grad_table_bytes(&g, 1);
        opt8_grads l;
        std::memset(&l, 0, sizeof l);
        l.table = l.squares = static_cast<double*>(at<void>(0x1000));
        l.table_bytes = a;
        (void)opt8_grad_clip(&l, nullptr);
      }
  opt8::g_result = hipErrorInvalidValue;
  opt8_grads l;
  std::memset(&l, 0, sizeof l);
  l.table = at<void>(0x1000);
  l.table_bytes = 24;
  l.squares = at<double>(0x2000);
  if (opt8_grad_clip(&l, nullptr) != OPT8_E_HIP || !std::strstr(opt8::g_error, "stand-in")) { std::printf("a failed launch\n"); ++failures; }
  opt8_grad g;
  std::memset(&g, 0, sizeof g);
  g.grad = at<void>(0x1000);
  g.numel = 5;
  char table[48];
  g_no_memory = true;
  const int rc = opt8_grad_table(&g, 1, table, sizeof table);
  g_no_memory = false;
  if (rc != OPT8_E_NOMEM) { std::printf("no memory: %d\n", rc); ++failures; }
  if (accepted < 1000 || aliases < 1000) { std::printf("accepted %d, aliases %d\n", accepted, aliases); ++failures; }
  if (failures) return 1;
  std::printf("all checks passed (%d accepted, %d refused for overlaps)\n", accepted, aliases);
  return 0;
}
