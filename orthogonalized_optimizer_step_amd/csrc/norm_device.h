// What the norms' kernels share: a row's threads and their joins, the weights'
// loads.
#pragma once

#include "train_device.h"

namespace dion {

// Threads of a block: rows of up to a wave share one.
constexpr int block_of(int nt) { return nt <= 64 ? 256 : nt; }

// Over the NT threads of a row; `red`: 16 floats, one array for each of two
// uses in turn.
template <int NT, typename Op> __device__ __forceinline__ float row_join(float v, float* red, Op op) {
  if constexpr (NT == 16) return row16_reduce(v, op);
  else if constexpr (NT == 32) return pair_reduce(row16_reduce(v, op), op);
  else if constexpr (NT == 64) return wave_reduce(v, 0.f, op);
  else return block_reduce<NT>(v, 0.f, red, op);
}

// N weights from element j on, 0 past the row's end
template <typename T>
__device__ __forceinline__ void load_weight(const void* w, bool w32, int j, int n, float* f) {
  constexpr int N = Chunk<T>::N;
  if (sizeof(T) == 4 || !w32) {
    Chunk<T>::unpack(Chunk<T>::load((const T*)w, j, n, 0.f), f);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) Chunk<float>::unpack(Chunk<float>::load((const float*)w, j + i, n, 0.f), f + i);
  }
}

template <typename T> __device__ __forceinline__ void add(const uintx4& v, float* f) {
  float g[Chunk<T>::N];
  Chunk<T>::unpack(v, g);
#pragma unroll
  for (int e = 0; e < Chunk<T>::N; ++e) f[e] += g[e];
}

}  // namespace dion
