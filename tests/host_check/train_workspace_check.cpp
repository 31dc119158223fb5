// Workspaces of the training-step operators on the CPU, under AddressSanitizer
// and UBSan: train_api.cpp against launchers whose scratch is any number of
// bytes, the smallest among them.  A call that needs some gets no further
// without a checked workspace of that size, a call that needs none is handed
// none, whatever it was given.  Pointers are numbers that nothing dereferences.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <string>

#include "dion.h"
#include "train_internal.h"

static size_t scratch = 0;   // what the operators need
static long reached = 0;
static const void* got = nullptr;

namespace dion {
int set_error(int code, const std::string&) { return code; }
int run_phase(const char*, const char*, double, double, hipStream_t, const std::function<void()>& launch) {
  launch();
  return 0;
}
int norm_back_parts(int64_t, int, int) { return 1; }
size_t int8_linear_scratch(const Int8Args&) { return scratch; }
size_t distill_scratch(int64_t, int, int, int, bool) { return scratch; }
void launch_rmsnorm(int, int, bool, const NormArgs&, hipStream_t) {}
void launch_int8_dequantize(int, const int8_t*, int64_t, const float*, void*, int64_t, int64_t, int, hipStream_t) {}
void launch_rmsnorm_backward(int, int, const NormBackArgs&, hipStream_t) {}
void launch_int8_linear(Int8Args a, hipStream_t) { ++reached, got = a.partial; }
void launch_distill_forward(int, const DistillArgs& a, hipStream_t) { ++reached, got = a.parts; }
void launch_distill_backward(int, const DistillArgs&, hipStream_t) {}
void launch_distill_step(int, const DistillArgs& a, hipStream_t) { ++reached, got = a.parts; }
}  // namespace dion

static char* at(int i) { return (char*)(0x100000000000ull + 0x1000000000ull * i); }
#define CHECK(x)                                          \
  do {                                                    \
    if (!(x)) {                                           \
      std::printf("line %d, scratch %zu: %s\n", __LINE__, scratch, #x); \
      std::exit(1);                                       \
    }                                                     \
  } while (0)

int main() {
  const size_t sizes[] = {0, 1, 4, 100, 255, 256, 257, 511, 512, 513, 768, 100000};
  for (size_t s : sizes) {
    scratch = s;
    for (int op = 0; op < 3; ++op) {
      const auto size = [&]() {
        if (op == 0) return dion_int8_linear_workspace_size((int8_t*)at(0), 64, (int8_t*)at(1), 64, 4, 8, 64);
        return dion_distill_topk_workspace_size(4, 64, 3, DION_BF16, op == 2);
      };
      const auto call = [&](char* ws, size_t have) {
        if (op == 0)
          return dion_int8_linear((int8_t*)at(0), 64, (float*)at(2), (int8_t*)at(1), 64, (float*)at(3), nullptr, 0, at(4), 8,
                                  4, 8, 64, DION_BF16, ws, have, nullptr);
        if (op == 1)
          return dion_distill_topk(at(0), 64, at(1), at(2), (float*)at(3), (float*)at(4), 4, 64, 3, DION_BF16, DION_FP32,
                                   8, 1.f, ws, have, nullptr);
        return dion_distill_topk_step(at(0), 64, at(1), at(2), nullptr, (float*)at(3), at(4), 64, 4, 64, 3, DION_BF16,
                                      DION_FP32, 8, 1.f, ws, have, nullptr);
      };
      const size_t need = size();
      const long before = reached;
      if (s == 0) {
        CHECK(need == 256);
        CHECK(call(nullptr, 0) == 0 && !got);
        CHECK(call(at(9) + 3, 1) == 0 && !got);
        CHECK(call(at(9), 1 << 20) == 0 && !got);
        CHECK(reached == before + 3);
      } else {
        CHECK(need > 256 && need >= s && need % 256 == 0);
        CHECK(call(nullptr, 0) == DION_E_WORKSPACE);
        CHECK(call(nullptr, need) == DION_E_WORKSPACE);
        CHECK(call(at(9), 0) == DION_E_WORKSPACE);
        CHECK(call(at(9), need - 1) == DION_E_WORKSPACE);
        CHECK(call(at(9) + 8, need) == DION_E_WORKSPACE);
        CHECK(call(at(4), need) == DION_E_INVAL);
        CHECK(reached == before);
        CHECK(call(at(9), need) == 0 && got == at(9) && reached == before + 1);
      }
    }
  }
  std::printf("train workspace check: %ld launches\n", reached);
  return 0;
}
