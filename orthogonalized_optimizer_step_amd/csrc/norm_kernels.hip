// RMS norm with the residual's addition: forward with an output in the
// input's type or in 8 bits with a scale for each row, and backward; and the
// 8-bit codes of rows without a norm.
//
//   s = x + residual (fp32)      h = s rounded to the input's type
//   rstd = 1 / sqrt(mean(s^2) + eps)      y = s rstd w, rounded once
//   8 bits: a = max |y|, scale = a / 127, q = rint(y (127 / a)) (ties to even)
//   backward, with g = dy w and c = rstd^2 mean(g h):
//     dx = rstd (g - h c) + dh        dw_j = sum over rows of dy_j h_j rstd
#include "train_device.h"
#include "train_internal.h"

namespace dion {

namespace {

constexpr int NT = 256;

// A row whose largest |y| is below 2^-119 has scale 0 and codes 0 (127 / a
// would come near overflow); a row with an infinity or a NaN has scale NaN, so
// that what is computed from its codes shows it.
__device__ __forceinline__ void row_scale(float a, float& scale, float& inv) {
  const bool bad = !(a <= 3.402823466e+38f), tiny = a < 0x1p-119f;
  scale = bad ? __builtin_nanf("") : (tiny ? 0.f : a / 127.f);
  inv = bad || tiny ? 0.f : 127.f / a;
}

template <typename T, typename W, bool INT8>
__global__ __launch_bounds__(NT) void k_rmsnorm(NormArgs a) {
  __shared__ float red[NT / 64];
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.ldx;
  const T* r = a.residual ? (const T*)a.residual + row * a.ldr : nullptr;
  const W* w = (const W*)a.weight;
  T* h = a.h ? (T*)a.h + row * a.ldh : nullptr;
  auto value = [&](int j) {
    float s = to_f(x[j]);
    if (r) s += to_f(r[j]);
    return s;
  };
  float rstd = 1.f;
  if (w) {
    float ss = 0.f;
    for (int j = threadIdx.x; j < a.cols; j += NT) {
      const float s = value(j);
      ss += s * s;
    }
    rstd = 1.f / sqrtf(block_sum<NT>(ss, red) / (float)a.cols + a.eps);
  }
  auto out = [&](int j, float s) { return w ? s * rstd * to_f(w[j]) : s; };
  float scale = 0.f, inv = 0.f;
  if (INT8) {
    float m = 0.f;
    for (int j = threadIdx.x; j < a.cols; j += NT) m = max_nan(m, fabsf(out(j, value(j))));
    row_scale(block_max<NT>(m, red), scale, inv);
  }
  for (int j = threadIdx.x; j < a.cols; j += NT) {
    const float s = value(j), y = out(j, s);
    if (h) h[j] = from_f<T>(s);
    if (INT8) ((int8_t*)a.y)[row * a.ldy + j] = (int8_t)(int)rintf(inv == 0.f ? 0.f : y * inv);
    else ((T*)a.y)[row * a.ldy + j] = from_f<T>(y);
  }
  if (threadIdx.x == 0) a.stat[row] = INT8 ? scale : rstd;
}

template <typename T>
__global__ __launch_bounds__(NT) void k_int8_dequantize(const int8_t* q, int64_t ldq, const float* scale, T* y,
                                                        int64_t ldy, int cols) {
  const int64_t row = blockIdx.x;
  const float s = scale[row];
  for (int j = threadIdx.x; j < cols; j += NT) y[row * ldy + j] = from_f<T>((float)q[row * ldq + j] * s);
}

template <typename T, typename W>
__global__ __launch_bounds__(NT) void k_rmsnorm_dx(NormBackArgs a) {
  __shared__ float red[NT / 64];
  const int64_t row = blockIdx.x;
  const T* dy = (const T*)a.dy + row * a.lddy;
  const T* h = (const T*)a.h + row * a.ldh;
  const T* dh = a.dh ? (const T*)a.dh + row * a.lddh : nullptr;
  const W* w = (const W*)a.weight;
  const float rstd = a.rstd[row];
  float d = 0.f;
  for (int j = threadIdx.x; j < a.cols; j += NT) d += to_f(dy[j]) * to_f(w[j]) * to_f(h[j]);
  const float c = block_sum<NT>(d, red) / (float)a.cols * rstd * rstd;
  for (int j = threadIdx.x; j < a.cols; j += NT) {
    float v = rstd * (to_f(dy[j]) * to_f(w[j]) - to_f(h[j]) * c);
    if (dh) v += to_f(dh[j]);
    ((T*)a.dx)[row * a.lddx + j] = from_f<T>(v);
  }
}

// partial[p][j]: the rows of part p in order
template <typename T>
__global__ __launch_bounds__(NT) void k_rmsnorm_dw_part(NormBackArgs a) {
  const int j = blockIdx.x * NT + threadIdx.x;
  if (j >= a.cols) return;
  const int64_t chunk = (a.rows + a.parts - 1) / a.parts, r0 = blockIdx.y * chunk;
  const int64_t r1 = r0 + chunk < a.rows ? r0 + chunk : a.rows;
  float d = 0.f;
  for (int64_t r = r0; r < r1; ++r)
    d += to_f(((const T*)a.dy)[r * a.lddy + j]) * to_f(((const T*)a.h)[r * a.ldh + j]) * a.rstd[r];
  a.partial[(int64_t)blockIdx.y * a.cols + j] = d;
}

template <typename W>
__global__ __launch_bounds__(NT) void k_rmsnorm_dw(NormBackArgs a) {
  const int j = blockIdx.x * NT + threadIdx.x;
  if (j >= a.cols) return;
  float d = 0.f;
  for (int p = 0; p < a.parts; ++p) d += a.partial[(int64_t)p * a.cols + j];
  ((W*)a.dweight)[j] = from_f<W>(d);
}

template <typename T, typename W>
void launch_norm(bool int8_out, const NormArgs& a, hipStream_t s) {
  const dim3 g((unsigned)a.rows);
  if (int8_out) hipLaunchKernelGGL((k_rmsnorm<T, W, true>), g, dim3(NT), 0, s, a);
  else hipLaunchKernelGGL((k_rmsnorm<T, W, false>), g, dim3(NT), 0, s, a);
}

template <typename T, typename W>
void launch_back(const NormBackArgs& a, hipStream_t s) {
  const unsigned gx = (unsigned)((a.cols + NT - 1) / NT);
  // dweight first: dx may overwrite dy or dh
  if (a.parts) hipLaunchKernelGGL((k_rmsnorm_dw_part<T>), dim3(gx, (unsigned)a.parts), dim3(NT), 0, s, a);
  hipLaunchKernelGGL((k_rmsnorm_dw<W>), dim3(gx), dim3(NT), 0, s, a);
  if (a.rows) hipLaunchKernelGGL((k_rmsnorm_dx<T, W>), dim3((unsigned)a.rows), dim3(NT), 0, s, a);
}

}  // namespace

int norm_back_parts(int64_t rows, int cols) {
  (void)cols;
  return (int)(rows < 64 ? (rows > 0 ? 1 : 0) : rows / 64 < 256 ? rows / 64 : 256);
}

#define DION_FMT2(F, fmt, wfmt, ...)                                         \
  do {                                                                       \
    if (fmt == 1) F<float, float>(__VA_ARGS__);                              \
    else if (fmt == 0 && wfmt == 1) F<bf16_t, float>(__VA_ARGS__);           \
    else if (fmt == 0) F<bf16_t, bf16_t>(__VA_ARGS__);                       \
    else if (wfmt == 1) F<fp16_t, float>(__VA_ARGS__);                       \
    else F<fp16_t, fp16_t>(__VA_ARGS__);                                     \
  } while (0)

void launch_rmsnorm(int fmt, int wfmt, bool int8_out, const NormArgs& a, hipStream_t s) {
  DION_FMT2(launch_norm, fmt, wfmt, int8_out, a, s);
}

void launch_rmsnorm_backward(int fmt, int wfmt, const NormBackArgs& a, hipStream_t s) {
  DION_FMT2(launch_back, fmt, wfmt, a, s);
}

void launch_int8_dequantize(int fmt, const int8_t* q, int64_t ldq, const float* scale, void* y, int64_t ldy,
                            int64_t rows, int cols, hipStream_t s) {
  const dim3 g((unsigned)rows), b(NT);
  if (fmt == 1) hipLaunchKernelGGL((k_int8_dequantize<float>), g, b, 0, s, q, ldq, scale, (float*)y, ldy, cols);
  else if (fmt == 0) hipLaunchKernelGGL((k_int8_dequantize<bf16_t>), g, b, 0, s, q, ldq, scale, (bf16_t*)y, ldy, cols);
  else hipLaunchKernelGGL((k_int8_dequantize<fp16_t>), g, b, 0, s, q, ldq, scale, (fp16_t*)y, ldy, cols);
}

}  // namespace dion
