// layers_host.cpp with stand-ins for the launches that keep what they are given: a
// pointer that the checks left out, because the call has no use for it, must not
// reach a kernel.
#include <cstdio>
#include <cstring>

#include "layers_internal.h"
#include "opt8_error.h"

namespace opt8 {
static char g_error[600];
static opt8_rms_norm_grad g_grad;
static int g_launches = 0;
void clear_last_error() { g_error[0] = 0; }
int set_last_error(int code, const char* message) {
  std::snprintf(g_error, sizeof g_error, "%s", message);
  return code;
}
hipError_t launch_embedding_forward(const opt8_embedding&, hipStream_t) { return hipSuccess; }
hipError_t launch_embedding_backward(const opt8_embedding_grad&, hipStream_t) { return hipSuccess; }
hipError_t launch_rms_norm_forward(const opt8_rms_norm&, hipStream_t) { return hipSuccess; }
hipError_t launch_rms_norm_backward(const opt8_rms_norm_grad& a, hipStream_t) {
  g_grad = a;
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_grad_norm(const opt8_grads&, hipStream_t) { return hipSuccess; }
hipError_t launch_grad_clip(const opt8_grads&, hipStream_t) { return hipSuccess; }
}  // namespace opt8

extern "C" const char* hipGetErrorString(hipError_t) { return "stand-in error"; }

template <class T>
static T* at(uintptr_t p) { return reinterpret_cast<T*>(p); }

int main() {
  opt8_rms_norm_grad a;
  std::memset(&a, 0, sizeof a);
  a.dy = at<void>(0x100000);
  a.x = at<void>(0x200000);
  a.weight = at<void>(0x300000);
  a.rstd = at<float>(0x400000);
  a.dx = at<void>(0x500000);
  a.dweight = at<void>(0x600000);
  a.workspace = at<void>(0x700000);
  a.rows = 3;
  a.d = 10;
  a.workspace_bytes = opt8_rms_norm_workspace(a.rows, a.d);
  a.lddy = a.ldx = a.lddx = a.lddsum = 10;
  a.type = a.weight_type = a.dweight_type = OPT8_TYPE_BF16;
  int failures = 0;
  auto run = [&](const char* what, int rc, bool dsum) {
    const int before = opt8::g_launches;
    const int got = opt8_rms_norm_backward(&a, nullptr);
    if (got != rc) { std::printf("%s: status %d (%s)\n", what, got, opt8::g_error); ++failures; }
    if ((opt8::g_launches > before) != (rc == OPT8_OK)) { std::printf("%s: launches\n", what); ++failures; }
    if (rc == OPT8_OK && (opt8::g_grad.dsum == a.dsum) != dsum) { std::printf("%s: dsum reached the kernel: %d\n", what, !dsum); ++failures; }
    if (rc == OPT8_OK && !dsum && opt8::g_grad.dsum) { std::printf("%s: an unchecked dsum reached the kernel\n", what); ++failures; }
  };
  a.dsum = at<void>(0x800000);
  run("dx with dsum", OPT8_OK, true);
  a.lddsum = 9;
  run("dx with a short lddsum", OPT8_E_SIZE, false);
  a.lddsum = 10;
  a.dsum = at<void>(0x800001);
  run("dx with a misaligned dsum", OPT8_E_ALIGN, false);
  a.dx = nullptr;
  run("no dx and a misaligned dsum", OPT8_OK, false);
  a.lddsum = -5;
  run("no dx and a stale lddsum", OPT8_OK, false);
  a.dx = at<void>(0x500000);
  a.rows = 0;
  run("no rows", OPT8_OK, false);
  if (failures) return 1;
  std::printf("all checks passed\n");
  return 0;
}
