// Distillation loss on a teacher's top logits, and its gradient.
//
// Row by row, with student logits z (vocab values), teacher logits t_k at
// indices i_k and temperature T:
//   p = softmax of t / T over the present entries (index inside the
//   vocabulary, t_k > -inf);  log q_j = (z_j - m) / T - ls with m = max z and
//   ls = log sum exp((z - m) / T)
//   loss = T^2 sum_k p_k (log p_k - log q_{i_k})   (terms with p_k = 0 are 0)
//   dz_j = gl T (q_j - sum over k with i_k = j of p_k)
// A row with no present entry has loss 0 and gradient 0, whatever z holds; a
// row whose loss has gradient gl = 0 has gradient 0.
#include "train_device.h"
#include "train_internal.h"

namespace dion {

namespace {

constexpr int NT = 256;

// The teacher's distribution of one row in LDS.
struct Teacher {
  float logp[kDistillMaxK];   // log p_k, -inf where p_k = 0 or the entry is absent
  int idx[kDistillMaxK];      // -1 where absent
  float red[NT / 64];
};

__device__ __forceinline__ int64_t teacher_index(const DistillArgs& a, int64_t i) {
  return a.idx64 ? ((const int64_t*)a.idx)[i] : (int64_t)((const int32_t*)a.idx)[i];
}

// Fills T for `row`; returns whether any entry is present.
__device__ bool teacher_row(const DistillArgs& a, int64_t row, Teacher& T) {
  float top = -__builtin_inff();
  for (int k = threadIdx.x; k < a.k; k += NT) {
    const int64_t i = teacher_index(a, row * a.k + k);
    const float t = load_fmt(a.t, row * a.k + k, a.t_fmt);
    const bool ok = i >= 0 && i < a.vocab && t != -__builtin_inff();
    T.idx[k] = ok ? (int)i : -1;
    T.logp[k] = t;
    if (ok) top = max_nan(top, t);
  }
  top = block_max<NT>(top, T.red);
  if (top == -__builtin_inff()) return false;
  float s = 0.f;
  for (int k = threadIdx.x; k < a.k; k += NT) {
    const float u = T.idx[k] >= 0 ? (T.logp[k] - top) / a.temp : -__builtin_inff();
    T.logp[k] = u;
    s += expf(u);
  }
  const float ls = logf(block_sum<NT>(s, T.red));
  for (int k = threadIdx.x; k < a.k; k += NT) {
    const float lp = T.logp[k] - ls;
    T.logp[k] = expf(lp) == 0.f ? -__builtin_inff() : lp;
  }
  __syncthreads();
  return true;
}

template <typename Z> __global__ __launch_bounds__(NT) void k_distill_forward(DistillArgs a) {
  __shared__ Teacher T;
  const int64_t row = blockIdx.x;
  const Z* z = (const Z*)a.z + row * a.ldz;
  if (!teacher_row(a, row, T)) {
    if (threadIdx.x == 0) {
      if (a.loss) a.loss[row] = 0.f;
      a.stats[row] = make_float2(0.f, 0.f);
    }
    return;
  }
  float m = -__builtin_inff();
  for (int j = threadIdx.x; j < a.vocab; j += NT) m = max_nan(m, to_f(z[j]));
  m = block_max<NT>(m, T.red);
  float s = 0.f;
  for (int j = threadIdx.x; j < a.vocab; j += NT) s += expf((to_f(z[j]) - m) / a.temp);
  const float ls = logf(block_sum<NT>(s, T.red));
  float l = 0.f;
  for (int k = threadIdx.x; k < a.k; k += NT) {
    const float lp = T.logp[k];
    if (lp != -__builtin_inff()) l += expf(lp) * (lp - ((to_f(z[T.idx[k]]) - m) / a.temp - ls));
  }
  l = block_sum<NT>(l, T.red);
  if (threadIdx.x == 0) {
    if (a.loss) a.loss[row] = a.temp * a.temp * l;
    a.stats[row] = make_float2(m, ls);
  }
}

template <typename Z> __global__ __launch_bounds__(NT) void k_distill_backward(DistillArgs a) {
  __shared__ Teacher T;
  const int64_t row = blockIdx.x;
  const Z* z = (const Z*)a.z + row * a.ldz;
  Z* dz = (Z*)a.dz + row * a.ldd;
  const float g = a.gl ? a.gl[row] : 1.f;
  const bool live = teacher_row(a, row, T);
  if (!live || g == 0.f) {
    for (int j = threadIdx.x; j < a.vocab; j += NT) dz[j] = from_f<Z>(0.f);
    return;
  }
  const float2 st = a.stats[row];
  const float gt = g * a.temp;
  // the teacher's entries first: dz may be z itself
  float own[kDistillMaxK / NT];
#pragma unroll
  for (int i = 0; i < kDistillMaxK / NT; ++i) {
    const int k = threadIdx.x + i * NT;
    if (k < a.k && T.idx[k] >= 0) {
      float p = 0.f;
      for (int o = 0; o < a.k; ++o)
        if (T.idx[o] == T.idx[k]) p += expf(T.logp[o]);
      own[i] = gt * (expf((to_f(z[T.idx[k]]) - st.x) / a.temp - st.y) - p);
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < a.vocab; j += NT)
    dz[j] = from_f<Z>(gt * expf((to_f(z[j]) - st.x) / a.temp - st.y));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kDistillMaxK / NT; ++i) {
    const int k = threadIdx.x + i * NT;
    if (k < a.k && T.idx[k] >= 0) dz[T.idx[k]] = from_f<Z>(own[i]);
  }
}

}  // namespace

void launch_distill_forward(int fmt, const DistillArgs& a, hipStream_t s) {
  const dim3 g((unsigned)a.rows), b(NT);
  if (fmt == 1) hipLaunchKernelGGL((k_distill_forward<float>), g, b, 0, s, a);
  else if (fmt == 0) hipLaunchKernelGGL((k_distill_forward<bf16_t>), g, b, 0, s, a);
  else hipLaunchKernelGGL((k_distill_forward<fp16_t>), g, b, 0, s, a);
}

void launch_distill_backward(int fmt, const DistillArgs& a, hipStream_t s) {
  const dim3 g((unsigned)a.rows), b(NT);
  if (fmt == 1) hipLaunchKernelGGL((k_distill_backward<float>), g, b, 0, s, a);
  else if (fmt == 0) hipLaunchKernelGGL((k_distill_backward<bf16_t>), g, b, 0, s, a);
  else hipLaunchKernelGGL((k_distill_backward<fp16_t>), g, b, 0, s, a);
}

}  // namespace dion
