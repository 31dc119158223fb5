// Internal declarations of the training-step operators (RMS norm, 8-bit
// product, distillation loss): argument blocks shared by the host checks
// (train_api.cpp) and the kernels, and the launchers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <functional>
#include <string>

namespace dion {

// Error reporting and per-phase profiling of the C ABI (dion_api.cpp).
int set_error(int code, const std::string& msg);
// Runs `launch` as one profiled phase of `stream` (events around it while
// profiling is enabled) and reports a failed launch as DION_E_HIP.
int run_phase(const char* name, const char* kernel, double flops, double bytes, hipStream_t stream,
              const std::function<void()>& launch);

// Element formats: the values of dion_dtype (0 bf16, 1 fp32, 2 fp16).
struct NormArgs {
  const void* x;
  const void* residual;   // may be NULL
  const void* weight;     // NULL: the rows are quantised as they are (no norm)
  void* h;                // may be NULL: x + residual is not kept
  void* y;                // 16/32-bit output, or int8 codes
  float* stat;            // rstd (16/32-bit output) or the row's scale (int8)
  int64_t ldx, ldr, ldh, ldy;
  int64_t rows;
  int cols;
  float eps;
};

struct NormBackArgs {
  const void* dy;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* dh;         // may be NULL
  void* dx;
  void* dweight;
  float* partial;         // [parts][cols] partial sums of dweight
  int64_t lddy, ldh, lddh, lddx;
  int64_t rows;
  int cols;
  int parts;
};

struct Int8Args {
  const int8_t* a;        // m x k
  const int8_t* b;        // n x k
  const float* sa;        // m
  const float* sb;        // n
  const void* bias;       // n, may be NULL
  void* out;              // m x n
  int64_t lda, ldb, ldo;
  int64_t m, n;
  int k;
  int bias_fmt, out_fmt;
  int* partial;           // scratch: splits x m x n sums, then aligned copies
};

struct DistillArgs {
  const void* z;          // rows x vocab student logits
  const void* t;          // rows x k teacher's top logits
  const void* idx;        // rows x k their indices (32 or 64 bits)
  const float* gl;        // rows: gradient of each row's loss (NULL: 1)
  float* loss;            // rows
  float2* stats;          // rows: (a reference m near the largest logit, sum of exp((z - m) / T)); NULL: not kept
  void* dz;               // rows x vocab
  int64_t ldz, ldd;
  int64_t rows;
  int vocab, k;
  int t_fmt, idx64;
  float temp;
  float2* parts;          // scratch of a few rows in shares: rows x shares statistics,
  float* zi;              // and rows x k logits at the entries; NULL otherwise
  int shares;
};

// rows of one dweight partial sum (fixed by the sizes alone, so that the
// order of the sum is too)
int norm_back_parts(int64_t rows, int cols, int fmt);
constexpr int kNormMaxCols = 65536;
constexpr int kDistillMaxK = 1024;

void launch_rmsnorm(int fmt, int wfmt, bool int8_out, const NormArgs& a, hipStream_t s);
void launch_int8_dequantize(int fmt, const int8_t* q, int64_t ldq, const float* scale, void* y, int64_t ldy,
                            int64_t rows, int cols, hipStream_t s);
void launch_rmsnorm_backward(int fmt, int wfmt, const NormBackArgs& a, hipStream_t s);
// bytes of Int8Args::partial that this product needs (its sizes, strides and
// the alignment of a and b)
size_t int8_linear_scratch(const Int8Args& a);
void launch_int8_linear(Int8Args a, hipStream_t s);
// bytes of scratch (DistillArgs::parts) that the loss, or the loss with its gradient, needs
size_t distill_scratch(int64_t rows, int vocab, int k, int fmt, bool gradient);
void launch_distill_forward(int fmt, const DistillArgs& a, hipStream_t s);
void launch_distill_backward(int fmt, const DistillArgs& a, hipStream_t s);
void launch_distill_step(int fmt, const DistillArgs& a, hipStream_t s);

}  // namespace dion
