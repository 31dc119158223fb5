// The argument checks of the layer norm, the 4-bit operators and the log
// probabilities under AddressSanitizer and UBSan, on the CPU: model_api.cpp
// against launchers that only record that they were reached, with what the
// kernels rely on.  Many draws of sizes, strides, pointers and types, valid and
// not; pointers are numbers that nothing dereferences.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <string>

#include "dion.h"
#include "model_internal.h"
#include "train_internal.h"

static long reached = 0, refused = 0;
static size_t scratch = 0;
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
int layernorm_back_parts(int64_t rows, int, int) { return rows < 512 ? (int)rows : 512; }
size_t mxfp4_linear_scratch(const MxArgs&) { return scratch; }
static void need(bool ok) {
  if (!ok) std::abort();
  ++reached;
}
void launch_layernorm(int, int, const LayerNormArgs& a, hipStream_t) {
  need(a.x && a.y && a.weight && a.mean && a.rstd && a.rows > 0 && a.cols > 0 && a.ldx >= a.cols);
}
void launch_layernorm_backward(int, int, const LayerNormBackArgs& a, hipStream_t) {
  need(a.partial && a.dweight && (a.rows == 0 || (a.mean && a.rstd)) && a.parts == layernorm_back_parts(a.rows, a.cols, 0));
}
void launch_mxfp4_quantize(int, const MxCodesArgs& a, hipStream_t) {
  need(a.x && a.q && a.s && a.rows > 0 && a.ldq >= (a.cols + 1LL) / 2 && a.lds >= (a.cols + 31LL) / 32);
}
void launch_mxfp4_dequantize(int f, const MxCodesArgs& a, hipStream_t s) { launch_mxfp4_quantize(f, a, s); }
void launch_mxfp4_linear(MxArgs a, hipStream_t) {
  need(a.out && a.m > 0 && a.n > 0 && (scratch == 0) == (a.partial == nullptr) &&
       (a.kb == 0 || (a.lda >= a.kb && a.ldb >= a.kb)));
}
size_t logprob_scratch(int64_t, int, int, int) { return scratch; }
void launch_token_logprobs(int, const LogprobArgs& a, hipStream_t) {
  need(a.z && a.entropy && (!a.tok || a.logprob) && (a.k == 0 || (a.top && a.index)) && a.k <= kLogprobMaxTop &&
       (a.k == 0 || a.vocab <= kLogprobMaxTopVocab) && a.temp > 0 && (scratch == 0) == (a.parts == nullptr));
}
void launch_token_logprobs_backward(int, const LogprobArgs& a, hipStream_t) { need(a.z && a.dz && a.stats && a.temp > 0); }
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
static uint8_t* u8() { return (uint8_t*)ptr(); }
static float* f32() { return (float*)ptr(); }

int main() {
  for (int it = 0; it < 60000; ++it) {
    const long long rows = PICK(0, 1, 2, 5, 100, 4096, -1, 1ll << 40, 0x7fffffffffffffffll);
    const int cols = (int)PICK(1, 2, 64, 777, 65536, 65537, 0, -5, 0x7fffffff, 1 << 19, 1 << 22);
    const long long ld = PICK(64, 777, 65536, 1ll << 20, 1ll << 31, 0, -1, 0x7fffffffffffffffll);
    const int dt = (int)PICK(0, 0, 1, 2, 3, -1), wdt = (int)PICK(0, 1, 2, 7), k = (int)PICK(0, 1, 8, 64, 1024, 1025, -1, 4096);
    const float eps = (float)PICK(0, 1, -1), temp = (float)PICK(1, 2, 0, -1);
    const size_t have = (size_t)PICK(0, 255, 4096, 1ll << 30);
    scratch = (size_t)PICK(0, 0, 1, 256, 4096);
    count(dion_layernorm(ptr(), ld, ptr(), ld, ptr(), ptr(), ptr(), ld, ptr(), ld, f32(), f32(), rows, cols, dt, wdt, eps, nullptr));
    (void)dion_layernorm_backward_workspace_size(rows, cols, dt);
    count(dion_layernorm_backward(ptr(), ld, ptr(), ld, ptr(), f32(), f32(), ptr(), ld, ptr(), ld, ptr(), ptr(), rows, cols, dt, wdt, ptr(), have, nullptr));
    count(dion_mxfp4_quantize(ptr(), ld, u8(), ld, u8(), ld, rows, cols, dt, nullptr));
    count(dion_mxfp4_dequantize(u8(), ld, u8(), ld, ptr(), ld, rows, cols, dt, nullptr));
    (void)dion_mxfp4_linear_workspace_size(u8(), ld, u8(), ld, u8(), ld, u8(), ld, rows, cols, k);
    count(dion_mxfp4_linear(u8(), ld, u8(), ld, u8(), ld, u8(), ld, ptr(), wdt, ptr(), ld, rows, cols, k, dt, ptr(), have, nullptr));
    (void)dion_token_logprobs_workspace_size(rows, cols, k, dt);
    count(dion_token_logprobs(ptr(), ld, ptr(), f32(), f32(), f32(), f32(), (int64_t*)ptr(), rows, cols, k, dt, (int)PICK(4, 8, 2), temp, ptr(), have, nullptr));
    count(dion_token_logprobs_backward(f32(), f32(), ptr(), ld, f32(), ptr(), ptr(), ld, rows, cols, dt, (int)PICK(4, 8), temp, nullptr));
  }
  if (reached < 1000 || refused < 1000) std::abort();
  std::printf("model host check: %ld launches, %ld refusals\n", reached, refused);
  return 0;
}
