// The argument checks of the training-step operators under AddressSanitizer
// and UBSan, on the CPU: train_api.cpp against launchers that only record that
// they were reached.  Many draws of sizes, strides, pointers and types, valid
// and not; pointers are numbers that nothing dereferences.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <string>

#include "dion.h"
#include "train_internal.h"

static long reached = 0, refused = 0;
static std::string last;

namespace dion {
int set_error(int code, const std::string& msg) {
  last = msg;
  return code;
}
int run_phase(const char*, const char*, double flops, double bytes, hipStream_t, const std::function<void()>& launch) {
  if (!(flops >= 0) || !(bytes >= 0)) std::abort();
  launch();
  return 0;
}
int norm_back_parts(int64_t rows, int, int) { return rows < 512 ? (int)rows : 512; }
size_t int8_linear_scratch(const Int8Args& g) { return (size_t)((g.m + g.n) % 7) * 1024; }
size_t distill_scratch(int64_t rows, int, int k, int, bool) { return ((size_t)rows + (size_t)k) % 3 * 512; }
void launch_rmsnorm(int, int, bool, const NormArgs& a, hipStream_t) {
  if (!a.x || !a.y || !a.stat || a.rows <= 0 || a.cols <= 0 || a.ldx < a.cols) std::abort();
  ++reached;
}
void launch_int8_dequantize(int, const int8_t*, int64_t, const float*, void*, int64_t, int64_t, int, hipStream_t) { ++reached; }
void launch_rmsnorm_backward(int, int, const NormBackArgs& a, hipStream_t) {
  if (!a.partial || !a.dweight || a.parts != norm_back_parts(a.rows, a.cols, 0)) std::abort();
  ++reached;
}
void launch_int8_linear(Int8Args a, hipStream_t) {
  if (!a.out || (int8_linear_scratch(a) > 256 && !a.partial)) std::abort();
  ++reached;
}
void launch_distill_forward(int, const DistillArgs& a, hipStream_t) {
  if (!a.loss || !a.stats || (distill_scratch(a.rows, a.vocab, a.k, 0, false) > 256 && !a.parts)) std::abort();
  ++reached;
}
void launch_distill_backward(int, const DistillArgs& a, hipStream_t) {
  if (!a.dz || !a.stats) std::abort();
  ++reached;
}
void launch_distill_step(int, const DistillArgs& a, hipStream_t) {
  if (!a.dz || !a.loss || (distill_scratch(a.rows, a.vocab, a.k, 0, true) > 256 && !a.parts)) std::abort();
  ++reached;
}
}  // namespace dion

static unsigned long long state = 88172645463325252ull;
static unsigned next_u() {  // xorshift64
  state ^= state << 13;
  state ^= state >> 7;
  state ^= state << 17;
  return (unsigned)(state >> 11);
}
static long long pick(const long long* v, int n) { return v[next_u() % (unsigned)n]; }
#define PICK(...) [] { static const long long v[] = {__VA_ARGS__}; return pick(v, (int)(sizeof(v) / sizeof(v[0]))); }()

static char* ptr() {   // mostly far apart and aligned, sometimes NULL, close or odd
  static unsigned long long base = 0x100000000000ull;
  base += 0x1000000000000ull / 4096;
  const unsigned r = next_u() % 40;
  if (r == 0) return nullptr;
  if (r == 1) return (char*)(base | 1);
  if (r == 2) return (char*)0x100000001000ull;
  return (char*)base;
}
static void count(int rc) {
  if (rc == 0) return;
  if (rc != -1 && rc != -2 && rc != -3) std::abort();
  if (last.empty()) std::abort();
  ++refused;
}

int main() {
  for (int it = 0; it < 60000; ++it) {
    const long long rows = PICK(0, 1, 2, 5, 100, 4096, -1, 1ll << 40, 0x7fffffffffffffffll);
    const int cols = (int)PICK(1, 2, 64, 777, 65536, 65537, 0, -5, 0x7fffffff);
    const long long ld = PICK(64, 777, 65536, 1ll << 20, 1ll << 31, 0, -1, 0x7fffffffffffffffll);
    const int dt = (int)PICK(0, 0, 1, 2, 3, -1), wdt = (int)PICK(0, 1, 2, 7), k = (int)PICK(0, 1, 8, 1024, 1025, -1);
    const float eps = (float)PICK(0, 1, -1), temp = (float)PICK(1, 2, 0, -1);
    const size_t have = (size_t)PICK(0, 255, 4096, 1ll << 30);
    count(dion_rmsnorm(ptr(), ld, ptr(), ld, ptr(), ptr(), ld, ptr(), ld, (float*)ptr(), rows, cols, dt, wdt, eps, nullptr));
    count(dion_rmsnorm_int8(ptr(), ld, nullptr, 0, ptr(), nullptr, 0, (int8_t*)ptr(), ld, (float*)ptr(), rows, cols, dt, wdt, eps, nullptr));
    count(dion_int8_quantize(ptr(), ld, (int8_t*)ptr(), ld, (float*)ptr(), rows, cols, dt, nullptr));
    count(dion_int8_dequantize((int8_t*)ptr(), ld, (float*)ptr(), ptr(), ld, rows, cols, dt, nullptr));
    (void)dion_rmsnorm_backward_workspace_size(rows, cols, dt);
    count(dion_rmsnorm_backward(ptr(), ld, ptr(), ld, ptr(), (float*)ptr(), ptr(), ld, ptr(), ld, ptr(), rows, cols, dt, wdt, ptr(), have, nullptr));
    (void)dion_int8_linear_workspace_size((int8_t*)ptr(), ld, (int8_t*)ptr(), ld, rows, cols, k);
    count(dion_int8_linear((int8_t*)ptr(), ld, (float*)ptr(), (int8_t*)ptr(), ld, (float*)ptr(), ptr(), wdt, ptr(), ld, rows, cols, k, dt, ptr(), have, nullptr));
    (void)dion_distill_topk_workspace_size(rows, cols, k, dt, 1);
    count(dion_distill_topk(ptr(), ld, ptr(), ptr(), (float*)ptr(), (float*)ptr(), rows, cols, k, dt, wdt, (int)PICK(4, 8, 2), temp, ptr(), have, nullptr));
    count(dion_distill_topk_backward((float*)ptr(), ptr(), ld, (float*)ptr(), ptr(), ptr(), ptr(), ld, rows, cols, k, dt, wdt, (int)PICK(4, 8), temp, nullptr));
    count(dion_distill_topk_step(ptr(), ld, ptr(), ptr(), (float*)ptr(), (float*)ptr(), ptr(), ld, rows, cols, k, dt, wdt, (int)PICK(4, 8), temp, ptr(), have, nullptr));
  }
  if (reached < 1000 || refused < 1000) std::abort();
  std::printf("train host check: %ld launches, %ld refusals\n", reached, refused);
  return 0;
}
