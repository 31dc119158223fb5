// Internal declarations of the operators of models in a training step (layer
// norm, microscaled 4-bit floating point, log probabilities): argument blocks
// shared by the host checks (model_api.cpp) and the kernels, and the launchers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace dion {

// Element formats: the values of dion_dtype (0 bf16, 1 fp32, 2 fp16).
struct LayerNormArgs {
  const void* x;
  const void* residual;   // may be NULL
  const void* weight;
  const void* bias;       // may be NULL; of the weight's type
  void* h;                // may be NULL: x + residual is not kept
  void* y;
  float* mean;
  float* rstd;
  int64_t ldx, ldr, ldh, ldy;
  int64_t rows;
  int cols;
  float eps;
};

struct LayerNormBackArgs {
  const void* dy;
  const void* h;
  const void* weight;
  const float* mean;
  const float* rstd;
  const void* dh;         // may be NULL
  void* dx;
  void* dweight;          // NULL: dx alone, no partial sums
  void* dbias;            // may be NULL, and is without dweight
  float* partial;         // [parts][cols] partial sums of dweight, then the same of dbias
  int64_t lddy, ldh, lddh, lddx;
  int64_t rows;
  int cols;
  int parts;
};

// 4-bit codes: rows of ceil(cols / 2) bytes, the even element in the low half;
// scales: rows of ceil(cols / 32) bytes, 2^(s - 127), 255 = NaN.
struct MxCodesArgs {
  void* x;                // values: read by the quantisation, written by the reading back
  uint8_t* q;
  uint8_t* s;
  int64_t ldx, ldq, lds;
  int64_t rows;
  int cols;
};

struct MxArgs {
  const uint8_t* a;       // m x k
  const uint8_t* sa;
  const uint8_t* b;       // n x k
  const uint8_t* sb;
  const void* bias;       // n, may be NULL
  void* out;              // m x n
  int64_t lda, ldsa, ldb, ldsb, ldo;
  int64_t m, n;
  int kb;                 // bytes of codes in a row: k / 2
  int bias_fmt, out_fmt;
  float* partial;         // scratch: splits x m x n sums, then aligned copies
};

struct LogprobArgs {
  const void* z;          // rows x vocab logits
  const void* tok;        // rows tokens (32 or 64 bits), NULL: none
  float* logprob;         // rows, with tokens
  float* entropy;         // rows
  float4* stats;          // rows: (largest logit, sum of exponentials, entropy, log of the sum); NULL: not kept
  float* top;             // rows x k log probabilities
  int64_t* index;         // rows x k their tokens
  const float* gl;        // backward: gradients of logprob and of the entropy (NULL: 0)
  const float* ge;
  void* dz;               // rows x vocab
  int64_t ldz, ldd;
  int64_t rows;
  int vocab, k;
  int tok64;
  float temp;
  float4* parts;          // scratch of a few rows in shares: rows x shares sums,
  uint64_t* list;         // and rows x shares x k alternatives; NULL otherwise
  int shares, per;        // shares of a row, logits in one
};

constexpr int kLayerNormMaxCols = 65536;
constexpr int kLogprobMaxTop = 1024;
constexpr int kLogprobMaxTopVocab = 1 << 19;   // largest vocabulary with alternatives

// partial sums of dweight and dbias (fixed by the sizes alone, so that the
// order of the sums is too)
int layernorm_back_parts(int64_t rows, int cols, int fmt);
void launch_layernorm(int fmt, int wfmt, const LayerNormArgs& a, hipStream_t s);
void launch_layernorm_backward(int fmt, int wfmt, const LayerNormBackArgs& a, hipStream_t s);

void launch_mxfp4_quantize(int fmt, const MxCodesArgs& a, hipStream_t s);
void launch_mxfp4_dequantize(int fmt, const MxCodesArgs& a, hipStream_t s);
// bytes of MxArgs::partial that this product needs (its sizes, strides and the
// alignment of its operands)
size_t mxfp4_linear_scratch(const MxArgs& a);
void launch_mxfp4_linear(MxArgs a, hipStream_t s);

// bytes of scratch (LogprobArgs::parts) that the log probabilities need
size_t logprob_scratch(int64_t rows, int vocab, int k, int fmt);
void launch_token_logprobs(int fmt, const LogprobArgs& a, hipStream_t s);
void launch_token_logprobs_backward(int fmt, const LogprobArgs& a, hipStream_t s);

}  // namespace dion
