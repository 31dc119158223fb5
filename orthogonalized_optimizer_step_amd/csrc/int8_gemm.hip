// Product of 8-bit integers with a scale for each token and channel:
//   out[i][j] = round(float(sum_k a[i][k] b[j][k]) * sa[i] * sb[j] + bias[j])
// The sum is exact in int32 (k < 2^17), so the only roundings are the fp32
// conversion of the sum, the scales' products and the output's own.
//
// v_mfma_i32_16x16x64_i8: lane l holds 16 consecutive k of row l % 16 (k block
// l / 16) of each operand; result element e of lane l is row 4 (l / 16) + e of
// the first operand and row l % 16 of the second.
#include "train_device.h"
#include "train_internal.h"

namespace dion {

namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

constexpr int TILE = 64, BK = 64, LD = BK + 16;

__global__ __launch_bounds__(256) void k_int8_tile(Int8Args g) {
  __shared__ __attribute__((aligned(16))) int8_t sA[TILE * LD], sB[TILE * LD];
  const int64_t m0 = (int64_t)blockIdx.y * TILE, n0 = (int64_t)blockIdx.x * TILE;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  intx4 acc[2][2] = {};
  for (int k0 = 0; k0 < g.k; k0 += BK) {
    __syncthreads();
    for (int i = tid; i < TILE * BK; i += 256) {
      const int r = i / BK, c = i % BK, k = k0 + c;
      sA[r * LD + c] = m0 + r < g.m && k < g.k ? g.a[(m0 + r) * g.lda + k] : 0;
      sB[r * LD + c] = n0 + r < g.n && k < g.k ? g.b[(n0 + r) * g.ldb + k] : 0;
    }
    __syncthreads();
    const int kc = (lane >> 4) * 16;
    intx4 fa[2], fb[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      fa[f] = *(const intx4*)(sA + (wm + f * 16 + (lane & 15)) * LD + kc);
      fb[f] = *(const intx4*)(sB + (wn + f * 16 + (lane & 15)) * LD + kc);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t r = m0 + wm + i * 16 + (lane >> 4) * 4 + e, c = n0 + wn + j * 16 + (lane & 15);
        if (r < g.m && c < g.n) {
          float v = (float)acc[i][j][e] * g.sa[r] * g.sb[c];
          if (g.bias) v += load_fmt(g.bias, c, g.bias_fmt);
          store_fmt(g.out, r * g.ldo + c, g.out_fmt, v);
        }
      }
}

}  // namespace

void launch_int8_linear(const Int8Args& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + TILE - 1) / TILE), (unsigned)((a.m + TILE - 1) / TILE));
  hipLaunchKernelGGL(k_int8_tile, grid, dim3(256), 0, s, a);
}

}  // namespace dion
