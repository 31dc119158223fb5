// Layer norm with the residual's addition, forward and backward.
//
//   s = x + residual (fp32)      h = s rounded to the input's type
//   mean = sum s / n      rstd = 1 / sqrt(sum (s - mean)^2 / n + eps)
//   y = (s - mean) rstd w + b, rounded once
//   backward, with u = (h - mean) rstd and g = dy w:
//     dx = rstd (g - mean(g) - u mean(g u)) + dh
//     dw_j = sum over rows of dy_j u_j        db_j = sum over rows of dy_j
//
// The squares are summed about the mean of the first sum, and what that mean
// was off by (the mean of the differences, of the size of its rounding) is
// taken out of both: rows far from zero lose no more than their own rounding.
//
// A row is read once into registers, CH 16-byte chunks by each of its NT (16
// to 1024) threads (chunk i of thread t at element (i NT + t) N), as the RMS
// norm's are.  All of it is bound by memory: 16384 x 768 bf16 with the residual
// takes 23 us (4.4 TB/s; a copy on the card reaches 6.2), back 19 (4.0) and 3.9
// for the join of the columns' sums; 8192 x 4096 46 to 49 (5.6) and 57.
#include <algorithm>

#include "model_internal.h"
#include "norm_device.h"

namespace dion {

namespace {

// Two values over the NT threads of a row in one join; `red`: 32 floats.
template <int NT> __device__ __forceinline__ void row_sum2(float& a, float& b, float* red) {
  if constexpr (NT <= 64) {
    a = row_join<NT>(a, red, Add());
    b = row_join<NT>(b, red, Add());
  } else {
    constexpr int W = NT / 64;
    a = wave_sum(a);
    b = wave_sum(b);
    const int lane = threadIdx.x & 63;
    if (lane == 0) *(float2*)(red + 2 * (threadIdx.x >> 6)) = make_float2(a, b);
    lds_barrier();
    const float2 v = lane < W ? *(const float2*)(red + 2 * lane) : make_float2(0.f, 0.f);
    a = row_reduce<W>(v.x, 0.f, Add());
    b = row_reduce<W>(v.y, 0.f, Add());
  }
}

// Sums of v and v^2 with v = s - mean over the elements of a chunk that lie in the row.
template <int N> __device__ __forceinline__ void centre(float* s, float mean, int left, float& sum, float& sq) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    s[e] -= mean;
    const float v = left >= N || e < left ? s[e] : 0.f;
    sum += v;
    sq += v * v;
  }
}

// sq: the mean of the squares about a mean that was off by `off`.  Squares
// beyond fp32 leave 0: infinity less off's own, which is not rounded and so not
// infinite with them.  NaN stays.
__device__ __forceinline__ float rstd_of(float sq, float off, float eps) {
  const float var = fmaf(-off, off, sq);
  return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);
}

template <typename T, int NT, int CH>
__global__ __launch_bounds__(block_of(NT), NT >= 256 && CH == 1 ? 8 : 4) void k_layernorm(LayerNormArgs a, bool w32) {
  typedef Chunk<T> C;
  constexpr int N = C::N, RPB = block_of(NT) / NT;
  __shared__ __attribute__((aligned(8))) float red[2][32];
  const int t = threadIdx.x % NT;
  const float inv = 1.f / (float)a.cols;
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / NT; row < a.rows; row += (int64_t)gridDim.x * RPB) {
    const T* x = (const T*)a.x + row * a.ldx;
    const T* r = a.residual ? (const T*)a.residual + row * a.ldr : nullptr;
    T* h = a.h ? (T*)a.h + row * a.ldh : nullptr;
    float s[CH][N], sum = 0.f;
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
#pragma unroll
        for (int e = 0; e < N; ++e) sum += s[i][e];
      }
    }
    const float mean = row_join<NT>(sum, red[0], Add()) * inv;
    float off = 0.f, sq = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = (i * NT + t) * N;
      if (j >= a.cols) continue;
      if (h) C::store_near(h, j, a.cols, s[i]);
      centre<N>(s[i], mean, a.cols - j, off, sq);
    }
    row_sum2<NT>(off, sq, red[1]);
    off *= inv;
    const float rstd = rstd_of(sq * inv, off, a.eps);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = (i * NT + t) * N;
      if (j >= a.cols) continue;
      float w[N], b[N] = {};
      load_weight<T>(a.weight, w32, j, a.cols, w);
      if (a.bias) load_weight<T>(a.bias, w32, j, a.cols, b);
#pragma unroll
      for (int e = 0; e < N; ++e) s[i][e] = (s[i][e] - off) * rstd * w[e] + b[e];
      C::store_near((T*)a.y + row * a.ldy, j, a.cols, s[i]);
    }
    if (t == 0) {
      a.mean[row] = mean + off;
      a.rstd[row] = rstd;
    }
  }
}

// Rows too long to be held: read again for each step, from the caches.
template <typename T>
__global__ __launch_bounds__(1024) void k_layernorm_long(LayerNormArgs a, bool w32) {
  typedef Chunk<T> C;
  constexpr int N = C::N;
  __shared__ __attribute__((aligned(8))) float red[2][32];
  const float inv = 1.f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ldx;
    const T* r = a.residual ? (const T*)a.residual + row * a.ldr : nullptr;
    T* h = a.h ? (T*)a.h + row * a.ldh : nullptr;
    auto load = [&](int j, float* s) {
      C::unpack(C::load(x, j, a.cols, 0.f), s);
      if (r) add<T>(C::load(r, j, a.cols, 0.f), s);
    };
    float sum = 0.f, off = 0.f, sq = 0.f;
    for (int j = threadIdx.x * N; j < a.cols; j += 1024 * N) {
      float s[N];
      load(j, s);
#pragma unroll
      for (int e = 0; e < N; ++e) sum += s[e];
    }
    const float mean = row_join<1024>(sum, red[0], Add()) * inv;
    for (int j = threadIdx.x * N; j < a.cols; j += 1024 * N) {
      float s[N];
      load(j, s);
      centre<N>(s, mean, a.cols - j, off, sq);
    }
    row_sum2<1024>(off, sq, red[1]);
    off *= inv;
    const float rstd = rstd_of(sq * inv, off, a.eps);
    for (int j = threadIdx.x * N; j < a.cols; j += 1024 * N) {
      float s[N], w[N], b[N] = {};
      load(j, s);
      if (h) C::store_near(h, j, a.cols, s);
      load_weight<T>(a.weight, w32, j, a.cols, w);
      if (a.bias) load_weight<T>(a.bias, w32, j, a.cols, b);
#pragma unroll
      for (int e = 0; e < N; ++e) s[e] = (s[e] - mean - off) * rstd * w[e] + b[e];
      C::store_near((T*)a.y + row * a.ldy, j, a.cols, s);
    }
    if (threadIdx.x == 0) {
      a.mean[row] = mean + off;
      a.rstd[row] = rstd;
    }
  }
}

// Backward.  A row's threads take rows gridDim.x RPB apart; the next row's
// chunks are asked for before this row's dx is written, and the terms of
// dweight and dbias stay in registers until the end: one partial sum of each
// for each block, in the order of its rows, joined over blocks by
// k_layernorm_join (not where no dweight is asked for).  64 threads with two
// chunks each hold more than 128 registers, and spill at the bound of the others.
template <typename T, int NT, int CH>
__global__ __launch_bounds__(block_of(NT), NT == 64 && CH == 2 ? 1 : 4) void k_layernorm_backward(LayerNormBackArgs a, bool w32) {
  typedef Chunk<T> C;
  constexpr int N = C::N, RPB = block_of(NT) / NT;
  __shared__ __attribute__((aligned(8))) float red[2][32];
  int turn = 0;
  __shared__ float joined[RPB > 1 ? RPB * NT * CH * N : 1];
  const int t = threadIdx.x % NT, slot = threadIdx.x / NT;
  const float inv = 1.f / (float)a.cols;
  float w[CH][N], dw[CH][N], db[CH][N];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int j = (i * NT + t) * N;
#pragma unroll
    for (int e = 0; e < N; ++e) w[i][e] = dw[i][e] = db[i][e] = 0.f;
    if (j < a.cols) load_weight<T>(a.weight, w32, j, a.cols, w[i]);
  }
  uintx4 vy[CH], vh[CH], vd[CH];
  float rs = 0.f, mean = 0.f;
  auto fetch = [&](int64_t row, uintx4* y, uintx4* h, uintx4* d, float& r, float& m) {
    if (row >= a.rows) return;
    r = a.rstd[row];
    m = a.mean[row];
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
  fetch(row, vy, vh, vd, rs, mean);
  for (; row < a.rows; row += step) {
    float g[CH][N], u[CH][N], sg = 0.f, sgu = 0.f;   // past the row's end dy and w are 0
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if ((i * NT + t) * N < a.cols) {
        C::unpack(vy[i], g[i]);
        C::unpack(vh[i], u[i]);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          u[i][e] = (u[i][e] - mean) * rs;
          dw[i][e] += g[i][e] * u[i][e];
          db[i][e] += g[i][e];
          g[i][e] *= w[i][e];
          sg += g[i][e];
          sgu += g[i][e] * u[i][e];
        }
      }
    }
    uintx4 ny[CH], nh[CH], nd[CH];
    float nr = 0.f, nm = 0.f;
    fetch(row + step, ny, nh, nd, nr, nm);
    row_sum2<NT>(sg, sgu, red[turn ^= 1]);
    sg *= inv;
    sgu *= inv;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = (i * NT + t) * N;
      if (j >= a.cols) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) g[i][e] = rs * (g[i][e] - sg - u[i][e] * sgu);
      if (a.dh) {
        float d[N];
        C::unpack(vd[i], d);
#pragma unroll
        for (int e = 0; e < N; ++e) g[i][e] += d[e];
      }
      C::store_near((T*)a.dx + row * a.lddx, j, a.cols, g[i]);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      vy[i] = ny[i];
      vh[i] = nh[i];
      vd[i] = nd[i];
    }
    rs = nr;
    mean = nm;
  }
  auto write = [&](const float (*v)[N], float* out) {
    if (RPB > 1) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) joined[slot * NT * CH * N + (i * NT + t) * N + e] = v[i][e];
      __syncthreads();
      for (int j = threadIdx.x; j < a.cols; j += block_of(NT)) {
        float d = 0.f;
#pragma unroll
        for (int r = 0; r < RPB; ++r) d += joined[r * NT * CH * N + j];
        out[j] = d;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int j = (i * NT + t) * N + e;
          if (j < a.cols) out[j] = v[i][e];
        }
    }
  };
  if (a.dweight) write(dw, a.partial + (int64_t)blockIdx.x * a.cols);
  if (a.dbias) write(db, a.partial + (int64_t)(a.parts + blockIdx.x) * a.cols);
}

// Rows too long to be held with their weights and sums: dx with a second read
// of the row, the partial sums by columns.
template <typename T>
__global__ __launch_bounds__(1024) void k_layernorm_dx_long(LayerNormBackArgs a, bool w32) {
  typedef Chunk<T> C;
  constexpr int N = C::N;
  __shared__ __attribute__((aligned(8))) float red[2][32];
  int turn = 0;
  const float inv = 1.f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* dy = (const T*)a.dy + row * a.lddy;
    const T* h = (const T*)a.h + row * a.ldh;
    const T* dh = a.dh ? (const T*)a.dh + row * a.lddh : nullptr;
    const float rstd = a.rstd[row], mean = a.mean[row];
    auto load = [&](int j, float* g, float* u) {
      float w[N];
      C::unpack(C::load(dy, j, a.cols, 0.f), g);
      C::unpack(C::load(h, j, a.cols, 0.f), u);
      load_weight<T>(a.weight, w32, j, a.cols, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        g[e] *= w[e];
        u[e] = (u[e] - mean) * rstd;
      }
    };
    float sg = 0.f, sgu = 0.f;
    for (int j = threadIdx.x * N; j < a.cols; j += 1024 * N) {
      float g[N], u[N];
      load(j, g, u);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        sg += g[e];
        sgu += g[e] * u[e];
      }
    }
    row_sum2<1024>(sg, sgu, red[turn ^= 1]);
    sg *= inv;
    sgu *= inv;
    for (int j = threadIdx.x * N; j < a.cols; j += 1024 * N) {
      float g[N], u[N];
      load(j, g, u);
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] = rstd * (g[e] - sg - u[e] * sgu);
      if (dh) add<T>(C::load(dh, j, a.cols, 0.f), g);
      C::store_near((T*)a.dx + row * a.lddx, j, a.cols, g);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_layernorm_dw_long(LayerNormBackArgs a) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= a.cols) return;
  const int64_t r0 = a.rows * blockIdx.y / a.parts, r1 = a.rows * (blockIdx.y + 1) / a.parts;
  float dw = 0.f, db = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float g = to_f(((const T*)a.dy)[r * a.lddy + j]);
    dw += g * ((to_f(((const T*)a.h)[r * a.ldh + j]) - a.mean[r]) * a.rstd[r]);
    db += g;
  }
  a.partial[(int64_t)blockIdx.y * a.cols + j] = dw;
  if (a.dbias) a.partial[(int64_t)(a.parts + blockIdx.y) * a.cols + j] = db;
}

// dweight (blockIdx.y 0) and dbias (1) from the parts' sums: 32 columns a
// block, the parts shared by 32 groups of threads, whose sums meet in LDS.
template <typename W> __global__ __launch_bounds__(1024) void k_layernorm_join(LayerNormBackArgs a) {
  __shared__ float sum[32][33];
  const int x = threadIdx.x & 31, g = threadIdx.x >> 5, j = blockIdx.x * 32 + x;
  const float* part = a.partial + (int64_t)blockIdx.y * a.parts * a.cols;
  float d = 0.f;
  if (j < a.cols) {
#pragma unroll 8
    for (int p = g; p < a.parts; p += 32) d += part[(int64_t)p * a.cols + j];
  }
  sum[g][x] = d;
  __syncthreads();
  // thread (g, x) now holds part x of column g: a half wave joins a column
  d = sum[x][g];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor(d, o, 32);
  const int c = blockIdx.x * 32 + g;
  if (x == 0 && c < a.cols) ((W*)(blockIdx.y ? a.dbias : a.dweight))[c] = from_f<W>(d);
}

template <typename T, int NT, int CH>
void launch_forward(const LayerNormArgs& a, bool w32, hipStream_t s) {
  constexpr int RPB = block_of(NT) / NT;
  const unsigned grid = (unsigned)std::min<int64_t>((a.rows + RPB - 1) / RPB, 1 << 20);
  hipLaunchKernelGGL((k_layernorm<T, NT, CH>), dim3(grid), dim3(block_of(NT)), 0, s, a, w32);
}

constexpr int kHeldChunks = 2048;   // longest row that is held, in 16-byte chunks

// Threads and chunks of a row: many threads with little each hide memory best,
// and 64 registers (eight waves a SIMD) where a row is more than a wave's.  2^25
// elements of bf16 with a residual (us): rows of 4096 46 to 49 on 512 threads; of
// 8192 52 on 1024 threads and 64 registers, 61 with 62 to 71, 69 on 512 with two chunks;
// of 16384 63 on 1024 with two.
template <typename T> void launch_norm(const LayerNormArgs& a, bool w32, hipStream_t s) {
  const int chunks = (a.cols + Chunk<T>::N - 1) / Chunk<T>::N;
  if (chunks <= 16) launch_forward<T, 16, 1>(a, w32, s);
  else if (chunks <= 32) launch_forward<T, 32, 1>(a, w32, s);
  else if (chunks <= 64) launch_forward<T, 64, 1>(a, w32, s);
  else if (chunks <= 128) launch_forward<T, 64, 2>(a, w32, s);
  else if (chunks <= 256) launch_forward<T, 256, 1>(a, w32, s);
  else if (chunks <= 512) launch_forward<T, 512, 1>(a, w32, s);
  else if (chunks <= 1024) launch_forward<T, 1024, 1>(a, w32, s);
  else if (chunks <= kHeldChunks) launch_forward<T, 1024, 2>(a, w32, s);
  else
    hipLaunchKernelGGL((k_layernorm_long<T>), dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)), dim3(1024), 0, s, a, w32);
}

template <typename T, int NT, int CH>
void launch_backward(const LayerNormBackArgs& a, bool w32, hipStream_t s) {
  hipLaunchKernelGGL((k_layernorm_backward<T, NT, CH>), dim3((unsigned)a.parts), dim3(block_of(NT)), 0, s, a, w32);
}

constexpr int kHeldBackChunks = 2048;   // the same of the backward pass

template <typename T> void launch_back(const LayerNormBackArgs& a, bool w32, hipStream_t s) {
  const int chunks = (a.cols + Chunk<T>::N - 1) / Chunk<T>::N;
  if (a.rows > 0) {
    if (chunks <= 16) launch_backward<T, 16, 1>(a, w32, s);
    else if (chunks <= 32) launch_backward<T, 32, 1>(a, w32, s);
    else if (chunks <= 64) launch_backward<T, 64, 1>(a, w32, s);
    else if (chunks <= 128) launch_backward<T, 64, 2>(a, w32, s);
    else if (chunks <= 256) launch_backward<T, 256, 1>(a, w32, s);
    else if (chunks <= 512) launch_backward<T, 512, 1>(a, w32, s);
    else if (chunks <= 1024) launch_backward<T, 1024, 1>(a, w32, s);
    else if (chunks <= kHeldBackChunks) launch_backward<T, 1024, 2>(a, w32, s);
    else {
      const unsigned gx = (unsigned)((a.cols + 255) / 256);
      // the sums first: dx may be written over dy or dh
      if (a.dweight) hipLaunchKernelGGL((k_layernorm_dw_long<T>), dim3(gx, (unsigned)a.parts), dim3(256), 0, s, a);
      hipLaunchKernelGGL((k_layernorm_dx_long<T>), dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)), dim3(1024), 0, s, a,
                         w32);
    }
  }
  if (!a.dweight) return;
  const dim3 grid((unsigned)((a.cols + 31) / 32), a.dbias ? 2 : 1);
  if (w32) hipLaunchKernelGGL((k_layernorm_join<float>), grid, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((k_layernorm_join<T>), grid, dim3(1024), 0, s, a);
}

}  // namespace

// As the RMS norm's, whose measurements hold for two sums as well: 16000 x 1066
// bf16 84 -> 57 us, 262144 x 64 42 -> 31, 16384 x 768 27 -> 25 against 512 blocks
// for every size.  Four rows in turn where that leaves 256 blocks: with fewer the
// blocks' sums are written and joined for little (1000 x 1066 bf16 20.6 -> 14.0,
// 2048 x 768 fp32 13.2 -> 11.9, 1021 x 1601 fp32 16.1 -> 14.0).
int layernorm_back_parts(int64_t rows, int cols, int fmt) {
  const int chunks = (cols + (fmt == 1 ? 3 : 7)) / (fmt == 1 ? 4 : 8);
  if (chunks > kHeldBackChunks) return (int)std::min<int64_t>(256, (rows + 31) / 32);
  const bool whole = cols % (fmt == 1 ? 4 : 8) == 0;
  const int64_t most = cols <= (fmt == 1 ? 1536 : 512)               ? 1024
                       : chunks <= 128                               ? 768
                       : cols <= 1536                                ? 1024
                       : cols <= 2048 || (cols <= 4096 && !whole)    ? 512
                                                                     : 256;
  const int64_t per = chunks <= 16 ? 16 : chunks <= 32 ? 8 : chunks <= 128 ? 4 : 1;   // rows at once
  const int64_t four = std::max<int64_t>(256, (rows + 4 * per - 1) / (4 * per));
  return (int)std::min({most, four, (rows + per - 1) / per});
}

void launch_layernorm(int fmt, int wfmt, const LayerNormArgs& a, hipStream_t s) {
  const bool w32 = wfmt == 1;
  if (fmt == 1) launch_norm<float>(a, w32, s);
  else if (fmt == 0) launch_norm<bf16_t>(a, w32, s);
  else launch_norm<fp16_t>(a, w32, s);
}

void launch_layernorm_backward(int fmt, int wfmt, const LayerNormBackArgs& a, hipStream_t s) {
  const bool w32 = wfmt == 1;
  if (fmt == 1) launch_back<float>(a, w32, s);
  else if (fmt == 0) launch_back<bf16_t>(a, w32, s);
  else launch_back<fp16_t>(a, w32, s);
}

}  // namespace dion
