// RMS norm with the residual's addition: forward with an output in the
// input's type or in 8 bits with a scale for each row, and backward; and the
// 8-bit codes of rows without a norm.
//
//   s = x + residual (fp32)      h = s rounded to the input's type
//   rstd = 1 / sqrt(mean(s^2) + eps)      y = s rstd w, rounded once
//   8 bits: a = max |y|, scale = a / 127, q = rint(y (127 (1 / a))) (ties to even)
//   backward, with g = dy w and c = rstd^2 mean(g h):
//     dx = rstd (g - h c) + dh        dw_j = sum over rows of dy_j h_j rstd
//
// A row is read once into registers, CH 16-byte chunks by each of its NT (16
// to 1024) threads (chunk i of thread t at element (i NT + t) N), and everything is
// formed from there.  All of it is bound by memory; what it takes at 8192 x
// 4096 and the like stands at the launch rules below.
#include <algorithm>

#include "norm_device.h"
#include "train_internal.h"

namespace dion {

namespace {

// A row whose largest |y| is below 2^-119 has scale 0 and codes 0 (127 / a
// would come near overflow); a row with an infinity or a NaN has scale NaN, so
// that what is computed from its codes shows it.
__device__ __forceinline__ void row_scale(float a, float& scale, float& inv) {
  const bool bad = !(a <= 3.402823466e+38f), tiny = a < 0x1p-119f;
  scale = bad ? __builtin_nanf("") : (tiny ? 0.f : a / 127.f);
  inv = bad || tiny ? 0.f : 127.f * (1.f / a);
}

// N codes from element j on: rint(y inv).  |y inv| <= 127.5, so that adding
// 1.5 2^23 rounds it to the integer in the sum's low bits.
template <int N> __device__ __forceinline__ void store_codes(int8_t* q, int j, int n, const float* y, float inv) {
#pragma clang fp contract(off)   // the product is rounded first
  uint32_t p[N / 4];
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    uint32_t u[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) u[b] = __float_as_uint(y[e + b] * inv + 12582912.f);
    p[e / 4] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[3], u[2], 0x0c0c0400u),
                                     __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u), 0x05040100u);
    if (inv == 0.f) p[e / 4] = 0;   // whatever y holds
  }
  if (j + N <= n) {
    __builtin_memcpy(q + j, p, N);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (j + e < n) q[j + e] = (int8_t)(p[e / 4] >> (8 * (e % 4)));
  }
}

// Forward.  Without a weight (codes of plain rows) y = s.
template <typename T, bool INT8, int NT, int CH>
__global__ __launch_bounds__(block_of(NT)) void k_rmsnorm(NormArgs a, bool w32) {
  typedef Chunk<T> C;
  constexpr int N = C::N, RPB = block_of(NT) / NT;
  __shared__ float red[3][16];
  const int t = threadIdx.x % NT;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / NT; row < a.rows; row += (int64_t)gridDim.x * RPB) {
    const T* x = (const T*)a.x + row * a.ldx;
    const T* r = a.residual ? (const T*)a.residual + row * a.ldr : nullptr;
    T* h = a.h ? (T*)a.h + row * a.ldh : nullptr;
    float s[CH][N];
    {
      uintx4 vx[CH], vr[CH];   // every load of the row ahead of its use
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int j = (i * NT + t) * N;
        if (j < a.cols) {
          vx[i] = C::load(x, j, a.cols, 0.f);
          if (r) vr[i] = C::load(r, j, a.cols, 0.f);
        }
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < N; ++e) s[i][e] = 0.f;
        if ((i * NT + t) * N < a.cols) {
          C::unpack(vx[i], s[i]);
          if (r) add<T>(vr[i], s[i]);
        }
      }
    }
    float rstd = 1.f;
    if (a.weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) ss += s[i][e] * s[i][e];
      ss = row_join<NT>(ss, red[turn ^= 1], Add());
      rstd = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = (i * NT + t) * N;
      if (j >= a.cols) continue;
      if (h) C::store_near(h, j, a.cols, s[i]);
      if (a.weight) {
        float w[N];
        load_weight<T>(a.weight, w32, j, a.cols, w);
#pragma unroll
        for (int e = 0; e < N; ++e) s[i][e] = s[i][e] * rstd * w[e];
      }
      if (!INT8) C::store_near((T*)a.y + row * a.ldy, j, a.cols, s[i]);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (INT8) m = MaxAbs()(m, s[i][e]);
    }
    float scale = 0.f, inv = 0.f;
    if (INT8) {
      if (!a.weight) turn ^= 1;   // the only join of the row
      row_scale(row_join<NT>(m, a.weight ? red[2] : red[turn], MaxAbs()), scale, inv);
      int8_t* q = (int8_t*)a.y + row * a.ldy;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int j = (i * NT + t) * N;
        if (j >= a.cols) continue;
        store_codes<N>(q, j, a.cols, s[i], inv);
      }
    }
    if (t == 0) a.stat[row] = INT8 ? scale : rstd;
  }
}

// Rows too long to be held: read again for each step, from the caches.
template <typename T, bool INT8>
__global__ __launch_bounds__(1024) void k_rmsnorm_long(NormArgs a, bool w32) {
  typedef Chunk<T> C;
  constexpr int N = C::N;
  __shared__ float red[3][16];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ldx;
    const T* r = a.residual ? (const T*)a.residual + row * a.ldr : nullptr;
    T* h = a.h ? (T*)a.h + row * a.ldh : nullptr;
    auto sum = [&](int j, float* s) {
      C::unpack(C::load(x, j, a.cols, 0.f), s);
      if (r) add<T>(C::load(r, j, a.cols, 0.f), s);
    };
    float rstd = 1.f;
    if (a.weight) {
      float ss = 0.f;
      for (int j = threadIdx.x * N; j < a.cols; j += 1024 * N) {
        float s[N];
        sum(j, s);
#pragma unroll
        for (int e = 0; e < N; ++e) ss += s[e] * s[e];
      }
      rstd = 1.f / sqrtf(block_reduce<1024>(ss, 0.f, red[turn ^= 1], Add()) / (float)a.cols + a.eps);
    }
    auto norm = [&](int j, float* s) {
      if (!a.weight) return;
      float w[N];
      load_weight<T>(a.weight, w32, j, a.cols, w);
#pragma unroll
      for (int e = 0; e < N; ++e) s[e] = s[e] * rstd * w[e];
    };
    float scale = 0.f, inv = 0.f;
    if (INT8) {
      float m = 0.f;
      for (int j = threadIdx.x * N; j < a.cols; j += 1024 * N) {
        float s[N];
        sum(j, s);
        norm(j, s);
#pragma unroll
        for (int e = 0; e < N; ++e) m = MaxAbs()(m, s[e]);
      }
      if (!a.weight) turn ^= 1;   // the only join of the row
      row_scale(block_reduce<1024>(m, 0.f, a.weight ? red[2] : red[turn], MaxAbs()), scale, inv);
    }
    for (int j = threadIdx.x * N; j < a.cols; j += 1024 * N) {
      float s[N];
      sum(j, s);
      if (h) C::store_near(h, j, a.cols, s);
      norm(j, s);
      if (INT8) store_codes<N>((int8_t*)a.y + row * a.ldy, j, a.cols, s, inv);
      else C::store_near((T*)a.y + row * a.ldy, j, a.cols, s);
    }
    if (threadIdx.x == 0) a.stat[row] = INT8 ? scale : rstd;
  }
}

// y = q scale, 16 codes a thread.  A row's blocks lie along y and z of the grid,
// which have 65536 at most each; offsets are taken from the thread's first
// element, where they stay small at any length of row.
template <typename T>
__global__ __launch_bounds__(256) void k_int8_dequantize(const int8_t* q, int64_t ldq, const float* scale, T* y,
                                                         int64_t ldy, int64_t rows, int cols) {
  typedef Chunk<T> C;
  const int64_t j = (((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 256 + threadIdx.x) * 16;
  if (j >= cols) return;
  const int left = cols - (int)j;   // of the row
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int8_t* src = q + row * ldq + j;
    const float s = scale[row];
    int8_t c[16];
    if (left >= 16) {
      __builtin_memcpy(c, src, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) c[e] = e < left ? src[e] : 0;
    }
    float f[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = (float)c[e] * s;
#pragma unroll
    for (int e = 0; e < 16; e += C::N)
      if (e < left) C::store_near(y + row * ldy + j, e, left, f + e);
  }
}

// Backward.  A row's threads take rows gridDim.x RPB apart; the next row's
// chunks are asked for before this row's dx is written, and dweight's terms
// stay in registers until the end: one partial sum for each block, in the
// order of its rows, joined over blocks by k_rmsnorm_dw.
template <typename T, int NT, int CH>
__global__ __launch_bounds__(block_of(NT)) void k_rmsnorm_backward(NormBackArgs a, bool w32) {
  typedef Chunk<T> C;
  constexpr int N = C::N, RPB = block_of(NT) / NT;
  __shared__ float red[2][16];
  int turn = 0;
  __shared__ float joined[RPB > 1 ? RPB * NT * CH * N : 1];
  const int t = threadIdx.x % NT, slot = threadIdx.x / NT;
  float w[CH][N], dw[CH][N];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int j = (i * NT + t) * N;
#pragma unroll
    for (int e = 0; e < N; ++e) w[i][e] = dw[i][e] = 0.f;
    if (j < a.cols) load_weight<T>(a.weight, w32, j, a.cols, w[i]);
  }
  uintx4 vy[CH], vh[CH], vd[CH];
  float rs = 0.f;
  auto fetch = [&](int64_t row, uintx4* y, uintx4* h, uintx4* d, float& r) {
    if (row >= a.rows) return;
    r = a.rstd[row];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = (i * NT + t) * N;
      if (j >= a.cols) continue;
      y[i] = C::load((const T*)a.dy + row * a.lddy, j, a.cols, 0.f);
      h[i] = C::load((const T*)a.h + row * a.ldh, j, a.cols, 0.f);
      if (a.dh) d[i] = C::load((const T*)a.dh + row * a.lddh, j, a.cols, 0.f);
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + slot;
  fetch(row, vy, vh, vd, rs);
  for (; row < a.rows; row += step) {
    float dy[CH][N], h[CH][N], dot = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if ((i * NT + t) * N < a.cols) {
        C::unpack(vy[i], dy[i]);
        C::unpack(vh[i], h[i]);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          dw[i][e] += dy[i][e] * h[i][e] * rs;
          dy[i][e] *= w[i][e];
          dot += dy[i][e] * h[i][e];
        }
      }
    }
    uintx4 ny[CH], nh[CH], nd[CH];
    float nr = 0.f;
    fetch(row + step, ny, nh, nd, nr);
    const float c = row_join<NT>(dot, red[turn ^= 1], Add()) / (float)a.cols * rs * rs;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = (i * NT + t) * N;
      if (j >= a.cols) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) dy[i][e] = rs * (dy[i][e] - h[i][e] * c);
      if (a.dh) {
        float d[N];
        C::unpack(vd[i], d);
#pragma unroll
        for (int e = 0; e < N; ++e) dy[i][e] += d[e];
      }
      C::store_near((T*)a.dx + row * a.lddx, j, a.cols, dy[i]);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      vy[i] = ny[i];
      vh[i] = nh[i];
      vd[i] = nd[i];
    }
    rs = nr;
  }
  float* out = a.partial + (int64_t)blockIdx.x * a.cols;
  if (RPB > 1) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) joined[slot * NT * CH * N + (i * NT + t) * N + e] = dw[i][e];
    __syncthreads();
    for (int j = threadIdx.x; j < a.cols; j += block_of(NT)) {
      float v = 0.f;
#pragma unroll
      for (int r = 0; r < RPB; ++r) v += joined[r * NT * CH * N + j];
      out[j] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int j = (i * NT + t) * N + e;
        if (j < a.cols) out[j] = dw[i][e];
      }
  }
}

// Rows too long to be held with their weights and sums: dx with a second read
// of the row, dweight's partial sums by columns.
template <typename T>
__global__ __launch_bounds__(1024) void k_rmsnorm_dx_long(NormBackArgs a, bool w32) {
  typedef Chunk<T> C;
  constexpr int N = C::N;
  __shared__ float red[2][16];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* dy = (const T*)a.dy + row * a.lddy;
    const T* h = (const T*)a.h + row * a.ldh;
    const T* dh = a.dh ? (const T*)a.dh + row * a.lddh : nullptr;
    const float rstd = a.rstd[row];
    float dot = 0.f;
    for (int j = threadIdx.x * N; j < a.cols; j += 1024 * N) {
      float y[N], v[N], w[N];
      C::unpack(C::load(dy, j, a.cols, 0.f), y);
      C::unpack(C::load(h, j, a.cols, 0.f), v);
      load_weight<T>(a.weight, w32, j, a.cols, w);
#pragma unroll
      for (int e = 0; e < N; ++e) dot += y[e] * w[e] * v[e];
    }
    const float c = block_reduce<1024>(dot, 0.f, red[turn ^= 1], Add()) / (float)a.cols * rstd * rstd;
    for (int j = threadIdx.x * N; j < a.cols; j += 1024 * N) {
      float y[N], v[N], w[N];
      C::unpack(C::load(dy, j, a.cols, 0.f), y);
      C::unpack(C::load(h, j, a.cols, 0.f), v);
      load_weight<T>(a.weight, w32, j, a.cols, w);
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = rstd * (y[e] * w[e] - v[e] * c);
      if (dh) {
        float d[N];
        C::unpack(C::load(dh, j, a.cols, 0.f), d);
#pragma unroll
        for (int e = 0; e < N; ++e) y[e] += d[e];
      }
      C::store_near((T*)a.dx + row * a.lddx, j, a.cols, y);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_rmsnorm_dw_long(NormBackArgs a) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= a.cols) return;
  const int64_t r0 = a.rows * blockIdx.y / a.parts, r1 = a.rows * (blockIdx.y + 1) / a.parts;
  float d = 0.f;
  for (int64_t r = r0; r < r1; ++r)
    d += to_f(((const T*)a.dy)[r * a.lddy + j]) * to_f(((const T*)a.h)[r * a.ldh + j]) * a.rstd[r];
  a.partial[(int64_t)blockIdx.y * a.cols + j] = d;
}

// dweight from the parts' sums: 32 columns a block, the parts shared by 32
// groups of threads, whose sums meet in LDS.
template <typename W> __global__ __launch_bounds__(1024) void k_rmsnorm_dw(NormBackArgs a) {
  __shared__ float sum[32][33];
  const int x = threadIdx.x & 31, g = threadIdx.x >> 5, j = blockIdx.x * 32 + x;
  float d = 0.f;
  if (j < a.cols) {
#pragma unroll 8
    for (int p = g; p < a.parts; p += 32) d += a.partial[(int64_t)p * a.cols + j];
  }
  sum[g][x] = d;
  __syncthreads();
  // thread (g, x) now holds part x of column g: a half wave joins a column
  d = sum[x][g];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor(d, o, 32);
  const int c = blockIdx.x * 32 + g;
  if (x == 0 && c < a.cols) ((W*)a.dweight)[c] = from_f<W>(d);
}

template <typename T, bool INT8, int NT, int CH>
void launch_forward(const NormArgs& a, bool w32, hipStream_t s) {
  constexpr int RPB = block_of(NT) / NT;
  const unsigned grid = (unsigned)std::min<int64_t>((a.rows + RPB - 1) / RPB, 1 << 20);
  hipLaunchKernelGGL((k_rmsnorm<T, INT8, NT, CH>), dim3(grid), dim3(block_of(NT)), 0, s, a, w32);
}

constexpr int kHeldChunks = 2048;   // longest row that is held, in 16-byte chunks

// Threads and chunks of a row, for 2^25 elements of bf16 with a residual to 8
// bits (us): a row of 4096 41 on 512 threads, 46 on 256; of 8192 49 on 512
// threads, 61 on 1024; of 16384 54 on 1024 threads, 65 on 512.  Many threads
// with little each hide memory best, until the waves of a row wait for one
// another at its two joins.  2^24 elements in rows of 64: 30 on 16 threads, 106
// on 64; in rows of 256: 23 on 32, 31 on 64.
template <typename T, bool INT8>
void launch_norm(const NormArgs& a, bool w32, hipStream_t s) {
  const int chunks = (a.cols + Chunk<T>::N - 1) / Chunk<T>::N;
  if (chunks <= 16) launch_forward<T, INT8, 16, 1>(a, w32, s);
  else if (chunks <= 32) launch_forward<T, INT8, 32, 1>(a, w32, s);
  else if (chunks <= 64) launch_forward<T, INT8, 64, 1>(a, w32, s);
  else if (chunks <= 128) launch_forward<T, INT8, 64, 2>(a, w32, s);
  else if (chunks <= 256) launch_forward<T, INT8, 256, 1>(a, w32, s);
  else if (chunks <= 512) launch_forward<T, INT8, 512, 1>(a, w32, s);
  else if (chunks <= 1024) launch_forward<T, INT8, 512, 2>(a, w32, s);
  else if (chunks <= kHeldChunks) launch_forward<T, INT8, 1024, 2>(a, w32, s);
  else
    hipLaunchKernelGGL((k_rmsnorm_long<T, INT8>), dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)), dim3(1024), 0, s, a,
                       w32);
}

template <typename T, int NT, int CH>
void launch_backward(const NormBackArgs& a, bool w32, hipStream_t s) {
  hipLaunchKernelGGL((k_rmsnorm_backward<T, NT, CH>), dim3((unsigned)a.parts), dim3(block_of(NT)), 0, s, a, w32);
}

template <typename T>
void launch_back(const NormBackArgs& a, bool w32, hipStream_t s) {
  const int chunks = (a.cols + Chunk<T>::N - 1) / Chunk<T>::N;
  if (a.rows > 0) {
    if (chunks <= 16) launch_backward<T, 16, 1>(a, w32, s);
    else if (chunks <= 32) launch_backward<T, 32, 1>(a, w32, s);
    else if (chunks <= 64) launch_backward<T, 64, 1>(a, w32, s);
    else if (chunks <= 128) launch_backward<T, 64, 2>(a, w32, s);
    else if (chunks <= 256) launch_backward<T, 256, 1>(a, w32, s);
    else if (chunks <= 512) launch_backward<T, 512, 1>(a, w32, s);
    else if (chunks <= 1024) launch_backward<T, 1024, 1>(a, w32, s);
    else if (chunks <= kHeldChunks) launch_backward<T, 1024, 2>(a, w32, s);
    else {
      const unsigned gx = (unsigned)((a.cols + 255) / 256);
      // dweight first: dx may be written over dy or dh
      hipLaunchKernelGGL((k_rmsnorm_dw_long<T>), dim3(gx, (unsigned)a.parts), dim3(256), 0, s, a);
      hipLaunchKernelGGL((k_rmsnorm_dx_long<T>), dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)), dim3(1024), 0, s, a,
                         w32);
    }
  }
  const dim3 gw((unsigned)((a.cols + 31) / 32));
  if (w32) hipLaunchKernelGGL((k_rmsnorm_dw<float>), gw, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((k_rmsnorm_dw<T>), gw, dim3(1024), 0, s, a);
}

}  // namespace

// Blocks of the backward pass, each with a partial sum of dweight: as many for
// every CU, which counts more than as many rows for every block.  More blocks hide memory better; fewer have less
// to write and read again (4 bytes a column each).  2^24 elements, 256 / 512 /
// 1024 blocks (us): bf16 rows of 256 30.2 / 25.4 / 25.7, of 1024 26.7 / 26.0 /
// 28.7, of 2048 33.4 / 28.3 / 30.2, of 4096 27.6 / 29.0 / 33.9; fp32 rows of 64
// 88 / 56 / 46, of 1024 80 / 59 / 49, of 2048 63 / 48 / 49, of 4096 44 / 46 / 52.  bf16 rows of
// 768, four to a block: 43.6 on 768 blocks with the forward pass, 45.5 on 512.
// One row to a block whose threads it does not fill, 512 / 1024: bf16 16000 x
// 1066 67 / 45, fp32 83 / 60.  Rows that start inside 16 bytes wait longer for
// memory, 256 / 512: bf16 4000 x 4001 45 / 39, fp32 57 / 50.
int norm_back_parts(int64_t rows, int cols, int fmt) {
  const int chunks = (cols + (fmt == 1 ? 3 : 7)) / (fmt == 1 ? 4 : 8);
  if (chunks > kHeldChunks) return (int)std::min<int64_t>(256, (rows + 31) / 32);
  const bool whole = cols % (fmt == 1 ? 4 : 8) == 0;
  const int64_t most = cols <= (fmt == 1 ? 1536 : 512)               ? 1024
                       : chunks <= 128                               ? 768
                       : cols <= 1536                                ? 1024
                       : cols <= 2048 || (cols <= 4096 && !whole)    ? 512
                                                                     : 256;
  const int64_t per = chunks <= 16 ? 16 : chunks <= 32 ? 8 : chunks <= 128 ? 4 : 1;   // rows at once
  return (int)std::min(most, (rows + per - 1) / per);
}

void launch_rmsnorm(int fmt, int wfmt, bool int8_out, const NormArgs& a, hipStream_t s) {
  const bool w32 = wfmt == 1;
  if (int8_out) {
    if (fmt == 1) launch_norm<float, true>(a, w32, s);
    else if (fmt == 0) launch_norm<bf16_t, true>(a, w32, s);
    else launch_norm<fp16_t, true>(a, w32, s);
  } else {
    if (fmt == 1) launch_norm<float, false>(a, w32, s);
    else if (fmt == 0) launch_norm<bf16_t, false>(a, w32, s);
    else launch_norm<fp16_t, false>(a, w32, s);
  }
}

void launch_rmsnorm_backward(int fmt, int wfmt, const NormBackArgs& a, hipStream_t s) {
  const bool w32 = wfmt == 1;
  if (fmt == 1) launch_back<float>(a, w32, s);
  else if (fmt == 0) launch_back<bf16_t>(a, w32, s);
  else launch_back<fp16_t>(a, w32, s);
}

void launch_int8_dequantize(int fmt, const int8_t* q, int64_t ldq, const float* scale, void* y, int64_t ldy,
                            int64_t rows, int cols, hipStream_t s) {
  const int64_t blocks = ((int64_t)cols + 4095) / 4096, gy = std::min<int64_t>(blocks, 1 << 15);
  const dim3 g((unsigned)std::min<int64_t>(rows, 1 << 20), (unsigned)gy, (unsigned)((blocks + gy - 1) / gy)), b(256);
  if (fmt == 1) hipLaunchKernelGGL((k_int8_dequantize<float>), g, b, 0, s, q, ldq, scale, (float*)y, ldy, rows, cols);
  else if (fmt == 0) hipLaunchKernelGGL((k_int8_dequantize<bf16_t>), g, b, 0, s, q, ldq, scale, (bf16_t*)y, ldy, rows, cols);
  else hipLaunchKernelGGL((k_int8_dequantize<fp16_t>), g, b, 0, s, q, ldq, scale, (fp16_t*)y, ldy, rows, cols);
}

}  // namespace dion
