// Product of 8-bit integers with a scale for each token and channel:
//   out[i][j] = round(float(sum_k a[i][k] b[j][k]) * sa[i] * sb[j] + bias[j])
// The sum is exact in int32 (k < 2^17), so the only roundings are the fp32
// conversion of the sum, the scales' products, the bias' addition and the
// output's own, and the result does not depend on how the sum is split or on
// which kernel takes it.
//
// v_mfma_i32_32x32x32_i8: lane l holds 16 consecutive k of row l % 32 (k block
// l / 32) of each operand; result element e of lane l is row
// 8 (e / 4) + 4 (l / 32) + e % 4 of the first operand and row l % 32 of the
// second.  b goes first, so that a lane holds four consecutive channels of one
// token.
#include <algorithm>

#include "mma_device.h"
#include "train_internal.h"

namespace dion {

namespace {

// 32 bytes at p + shift (p at a whole dword, shift 0 .. 3) from the 36 at p
typedef intx4 intx4d __attribute__((aligned(4)));
__device__ __forceinline__ void load_shifted(const int8_t* p, uint32_t shift, intx4& lo, intx4& hi) {
  const intx4 u = *(const intx4d*)p, v = *(const intx4d*)(p + 16);
  const int w = *(const int*)(p + 32);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = (int)__builtin_amdgcn_alignbyte((uint32_t)(i < 3 ? u[(i + 1) & 3] : v[0]), (uint32_t)u[i], shift);
    hi[i] = (int)__builtin_amdgcn_alignbyte((uint32_t)(i < 3 ? v[(i + 1) & 3] : w), (uint32_t)v[i], shift);
  }
}

// An output before its rounding.  The bias is added to the rounded product
// everywhere: fused in some kernels alone, a token's last bit would depend on
// how many others come with it.
__device__ __forceinline__ float scaled(int sum, float sa, float sb, bool biased, float bias) {
#pragma clang fp contract(off)
  const float v = (float)sum * sa * sb;
  return biased ? v + bias : v;
}
__device__ __forceinline__ float scaled(const Int8Args& g, int64_t row, int64_t col, int sum) {
  return scaled(sum, g.sa[row], g.sb[col], g.bias, g.bias ? load_fmt(g.bias, col, g.bias_fmt) : 0.f);
}

// One BM x BN tile of the output by WM x WN waves, S stages of BK bytes in
// LDS, copied straight there S - 1 stages ahead (a and b in rows at multiples
// of 16 bytes).  Each wave holds two sets of fragments: those of the next 32
// bytes are read from LDS while the present ones are multiplied, across the
// stage's end too.
template <int BM, int BN, int WM, int WN, int S, typename O>
__global__ __launch_bounds__(64 * WM * WN) void k_int8_mma(Int8Args g, int* partial) {
  constexpr int W = WM * WN, NT = 64 * W;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;   // wave tile, its fragments
  constexpr int STAGE = (BM + BN) * BK;
  constexpr int NP = STAGE / 1024 / W;            // 1 KB pieces of a stage per wave
  constexpr int PR = 1024 / BK, CR = BK / 16;     // rows of a piece, chunks of a row
  constexpr int OV = OutVec<O>::N, SROW = TN + OV;   // staged output row
  constexpr int STAGED = W * 32 * SROW * (int)sizeof(O);
  constexpr int LDS = S * STAGE > STAGED ? S * STAGE : STAGED;
  // Copies of the stage S - 1 ahead: all at once after the turn, or (the
  // largest tile, with one block per CU) spread over the products of two steps.
  constexpr int KS = BK / 32;
  constexpr bool SPREAD = BM * BN >= 256 * 256;
  constexpr int PW = NP / 2, EVERY = SPREAD ? FM * FN / PW : 1;
  static_assert(!SPREAD || (PW * 2 == NP && EVERY * PW == FM * FN), "the copies divide the products");
  static_assert(S <= 4 && NP * W * 1024 == STAGE && BM % PR == 0, "whole pieces");
  __shared__ __attribute__((aligned(1024))) int8_t smem[LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int ti, tj;
  tile_of_block((int)((g.m + BM - 1) / BM), (int)((g.n + BN - 1) / BN), ti, tj);
  const int64_t m0 = (int64_t)ti * BM, n0 = (int64_t)tj * BN;
  const int rm = (int)min((int64_t)BM, g.m - m0), rn = (int)min((int64_t)BN, g.n - n0);   // valid rows of the tile
  const int8_t* A = g.a + m0 * g.lda;
  const int8_t* B = g.b + n0 * g.ldb;
  // this split's stages
  const int all = (g.k + BK - 1) / BK;
  const int kt0 = (int)((int64_t)all * blockIdx.y / gridDim.y);
  const int nk = (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y) - kt0;
  const uint32_t lds0 = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) int8_t*)smem);

  // piece q = wave + i W of a stage: rows PR q .. of a, then of b; lane l has
  // row l / CR and the chunk whose place is l % CR
  uint32_t voff[NP];
  int vk[NP];
  const intx4 ra = raw_buffer(A, (uint32_t)((rm - 1) * g.lda + g.k)), rb = raw_buffer(B, (uint32_t)((rn - 1) * g.ldb + g.k));
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int q = wave + i * W;
    const bool isa = q < BM / PR;
    const int r = (isa ? q : q - BM / PR) * PR + lane / CR;
    vk[i] = swz(r, lane % CR) * 16;
    voff[i] = r < (isa ? rm : rn) ? (uint32_t)(r * (isa ? g.lda : g.ldb)) + vk[i] : OUT_OF_RANGE;
  }
  auto issue = [&](int kt, int i) {   // piece i of stage kt
    const int k0 = (kt0 + kt) * BK, q = wave + i * W;
    const uint32_t v = k0 + vk[i] < g.k ? voff[i] : OUT_OF_RANGE;
    dma16(v, q < BM / PR ? ra : rb, (uint32_t)k0,
          (uint32_t)__builtin_amdgcn_readfirstlane(lds0 + (kt % S) * STAGE + q * 1024));
  };

  intx16 acc[FM][FN] = {};
  intx4 fa[2][FM], fb[2][FN];
  const int r = lane & 31;
  auto fetch = [&](int kt, int ks, int set) {
    const int8_t* s = smem + (kt % S) * STAGE + swz(r, ks * 2 + (lane >> 5)) * 16;
#pragma unroll
    for (int f = 0; f < FM; ++f) fa[set][f] = *(const intx4*)(s + (wm * TM + f * 32 + r) * BK);
#pragma unroll
    for (int f = 0; f < FN; ++f) fb[set][f] = *(const intx4*)(s + (BM + wn * TN + f * 32 + r) * BK);
  };
  // the stage that is needed next has landed, and every wave is done with the one before it
  auto turn = [&](int kt) {
    const int later = min(nk - 1, kt + S - 2) - kt;   // stages issued after kt
    if (S >= 4 && later >= 2) wait_vmcnt<2 * NP>();
    else if (S >= 3 && later >= 1) wait_vmcnt<NP>();
    else wait_vmcnt<0>();
    lds_barrier();
    if (!SPREAD && kt + S - 1 < nk) {
#pragma unroll
      for (int i = 0; i < NP; ++i) issue(kt + S - 1, i);
    }
  };
  if (nk > 0) {
#pragma unroll
    for (int t = 0; t < S - 1; ++t)
      if (t < nk) {
#pragma unroll
        for (int i = 0; i < NP; ++i) issue(t, i);
      }
    turn(0);
    if (SPREAD && S - 1 < nk) {
#pragma unroll
      for (int i = 0; i < PW; ++i) issue(S - 1, i);
    }
    fetch(0, 0, 0);
    for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (ks + 1 < KS) {
          fetch(kt, ks + 1, (ks + 1) & 1);
        } else if (kt + 1 < nk) {
          turn(kt + 1);
          fetch(kt + 1, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);   // the reads above go out before the products, not beside their use
        // spread copies, one after every EVERY products: half of a stage's
        // right after its turn, half beside the next step's products
        const int w = (ks + 1) % KS, st = ks + 1 < KS ? kt + S - 1 : kt + S;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[ks & 1][j], fa[ks & 1][i], acc[i][j], 0, 0, 0);
            const int t = i * FN + j;
            if (SPREAD && w < 2 && t % EVERY == EVERY - 1) {
              __builtin_amdgcn_sched_barrier(0);
              if (st < nk) issue(st, w * PW + t / EVERY);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (partial) {   // several splits: the sums as they are, for k_int8_join
    int* out = partial + (int64_t)blockIdx.y * g.m * g.n;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t row = m0 + wm * TM + i * 32 + r;
      if (row >= g.m) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t col = n0 + wn * TN + j * 32 + q * 8 + (lane >> 5) * 4;
          int* o = out + row * g.n + col;
          const intx4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          if (col + 4 <= g.n) *(intx4u*)o = v;
          else
            for (int e = 0; e < 4; ++e)
              if (col + e < g.n) o[e] = v[e];
        }
    }
    return;
  }
  __syncthreads();   // the stages are free: each wave stages 32 rows of its output at a time

  O* st = (O*)smem + wave * 32 * SROW;
  const int64_t cbase = n0 + wn * TN;
  constexpr int CPR = TN / OV;   // 16-byte pieces of a staged row
  // the lane's channels' scales and biases, once for all its rows (past the
  // last channel the last one's: not written)
  float sb[FN][16], bias[FN][16];
#pragma unroll
  for (int j = 0; j < FN; ++j)
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int64_t col = min(cbase + j * 32 + (q >> 2) * 8 + (lane >> 5) * 4 + (q & 3), g.n - 1);
      sb[j][q] = g.sb[col];
      bias[j][q] = g.bias ? load_fmt(g.bias, col, g.bias_fmt) : 0.f;
    }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t row = m0 + wm * TM + i * 32 + r;
    const float sa = g.sa[min(row, g.m - 1)];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        typedef O Ox4 __attribute__((ext_vector_type(4)));
        Ox4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = from_f<O>(scaled(acc[i][j][q * 4 + e], sa, sb[j][q * 4 + e], g.bias, bias[j][q * 4 + e]));
        }
        *(Ox4*)(st + r * SROW + j * 32 + q * 8 + (lane >> 5) * 4) = v;
      }
    asm volatile("" : : : "memory");   // a wave's LDS accesses execute in order
#pragma unroll
    for (int q0 = 0; q0 < 32 * CPR; q0 += 64) {
      const int q = q0 + lane, rr = q / CPR, c = (q % CPR) * OV;
      const int64_t orow = m0 + wm * TM + i * 32 + rr, col = cbase + c;
      if (orow < g.m && col < g.n) {
        const O* s = st + rr * SROW + c;
        O* o = (O*)g.out + orow * g.ldo + col;
        if (col + OV <= g.n) *(intx4u*)o = *(const intx4*)s;
        else
          for (int e = 0; col + e < g.n; ++e) o[e] = s[e];
      }
    }
    asm volatile("" : : : "memory");
  }
}

// The splits' sums, scaled.  Tokens lie along y and z of the grid, which have
// 65536 blocks at most each.
template <typename O> __global__ __launch_bounds__(256) void k_int8_join(Int8Args g, const int* partial, int splits) {
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
  if (col >= g.n || row >= g.m) return;
  int v = 0;
  for (int s = 0; s < splits; ++s) v += partial[((int64_t)s * g.m + row) * g.n + col];
  ((O*)g.out)[row * g.ldo + col] = from_f<O>(scaled(g, row, col, v));
}

void launch_join(const Int8Args& a, int splits, hipStream_t s) {
  const int64_t y = std::min<int64_t>(a.m, 1 << 15);
  const dim3 grid((unsigned)((a.n + 255) / 256), (unsigned)y, (unsigned)((a.m + y - 1) / y));
  if (a.out_fmt == 1) hipLaunchKernelGGL((k_int8_join<float>), grid, dim3(256), 0, s, a, a.partial, splits);
  else if (a.out_fmt == 0) hipLaunchKernelGGL((k_int8_join<bf16_t>), grid, dim3(256), 0, s, a, a.partial, splits);
  else hipLaunchKernelGGL((k_int8_join<fp16_t>), grid, dim3(256), 0, s, a, a.partial, splits);
}

template <int BM, int BN, int WM, int WN, int S>
void launch_mma(const Int8Args& a, int splits, hipStream_t s) {
  const int64_t tiles = (a.m + BM - 1) / BM * ((a.n + BN - 1) / BN);
  const dim3 grid((unsigned)tiles, splits), block(64 * WM * WN);
  int* part = splits > 1 ? a.partial : nullptr;
  if (a.out_fmt == 1) hipLaunchKernelGGL((k_int8_mma<BM, BN, WM, WN, S, float>), grid, block, 0, s, a, part);
  else if (a.out_fmt == 0) hipLaunchKernelGGL((k_int8_mma<BM, BN, WM, WN, S, bf16_t>), grid, block, 0, s, a, part);
  else hipLaunchKernelGGL((k_int8_mma<BM, BN, WM, WN, S, fp16_t>), grid, block, 0, s, a, part);
  if (part) launch_join(a, splits, s);
}

// Up to 16 tokens: the block takes 16 NW channels; its waves take 16 of them
// and every KW-th 128-byte piece of the split's share of k each, and the sums
// of the KW meet in LDS.  Fragments go from global memory to registers
// (v_mfma_i32_16x16x64_i8: lane l holds 16 consecutive k of row l % 16, k
// block l / 16; result element e of lane l is row 4 (l / 16) + e of the first
// operand and row l % 16 of the second), at any alignment.  Rows past the end
// repeat the last one and are not written.
//
// SHIFT: rows that start inside a dword, in matrices that start at one.
// Loads of 16 bytes inside dwords take twice the time (6 x 14336 x 12277: 98
// us; 56 this way, and rows of 12284 53 on the plain loads); so whole dwords are
// loaded and moved together, 32 bytes of k a lane.  They hold up to three bytes before the lane's own (of the row
// before, or the gap) and four after, which the loop keeps inside the row.
template <int NW, int KW, bool SHIFT, typename O>
__global__ __launch_bounds__(64 * NW * KW) void k_int8_rows(Int8Args g, int* partial) {
  __shared__ __attribute__((aligned(16))) int sum[KW * NW * 256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nw = wave % NW, kw = wave / NW;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NW);
  const int r = lane & 15, kc = (lane >> 4) * 16;
  const int8_t* b = g.b + min(n0 + nw * 16 + r, g.n - 1) * g.ldb;
  const int8_t* a = g.a + min((int64_t)r, g.m - 1) * g.lda;
  intx4 acc = {0, 0, 0, 0};
  const int pieces = (g.k + 127) / 128;
  const int p0 = (int)((int64_t)pieces * blockIdx.y / gridDim.y);
  const int kend = min(g.k, (int)((int64_t)pieces * (blockIdx.y + 1) / gridDim.y) * 128);
  int k0 = (p0 + kw) * 128;
  if (SHIFT) {
    const uint32_t sa = (uint32_t)(uintptr_t)a & 3, sb = (uint32_t)(uintptr_t)b & 3;
    const int8_t *aw = a - sa + 2 * kc, *bw = b - sb + 2 * kc;
#pragma unroll 4
    for (; k0 + 128 <= kend && k0 + 132 <= g.k; k0 += KW * 128) {
      intx4 a0, a1, b0, b1;
      load_shifted(bw + k0, sb, b0, b1);
      load_shifted(aw + k0, sa, a0, a1);
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(b0, a0, acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(b1, a1, acc, 0, 0, 0);
    }
  }
#pragma unroll 4
  for (; !SHIFT && k0 + 128 <= kend; k0 += KW * 128) {
#pragma unroll
    for (int h = 0; h < 128; h += 64)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(*(const intx4u*)(b + k0 + kc + h), *(const intx4u*)(a + k0 + kc + h),
                                                  acc, 0, 0, 0);
  }
  if (k0 < kend) {   // the last piece, in part or up to the row's end
    for (int h = 0; h < 128; h += 64)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(load_chunk(b, k0 + kc + h, kend), load_chunk(a, k0 + kc + h, kend),
                                                  acc, 0, 0, 0);
  }
  // [kw][token][channel of the block]
  *(intx4*)(sum + (kw * 16 + r) * (16 * NW) + nw * 16 + (lane >> 4) * 4) = acc;
  __syncthreads();
  for (int i = tid; i < NW * 256; i += 64 * NW * KW) {
    int v = 0;
#pragma unroll
    for (int w = 0; w < KW; ++w) v += sum[w * NW * 256 + i];
    const int64_t row = i / (16 * NW), col = n0 + i % (16 * NW);
    if (row < g.m && col < g.n) {
      if (partial) partial[((int64_t)blockIdx.y * g.m + row) * g.n + col] = v;
      else ((O*)g.out)[row * g.ldo + col] = from_f<O>(scaled(g, row, col, v));
    }
  }
}

template <int NW, int KW, bool SHIFT>
void launch_rows_as(const Int8Args& a, int splits, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + 16 * NW - 1) / (16 * NW)), splits), block(64 * NW * KW);
  int* part = splits > 1 ? a.partial : nullptr;
  if (a.out_fmt == 1) hipLaunchKernelGGL((k_int8_rows<NW, KW, SHIFT, float>), grid, block, 0, s, a, part);
  else if (a.out_fmt == 0) hipLaunchKernelGGL((k_int8_rows<NW, KW, SHIFT, bf16_t>), grid, block, 0, s, a, part);
  else hipLaunchKernelGGL((k_int8_rows<NW, KW, SHIFT, fp16_t>), grid, block, 0, s, a, part);
  if (part) launch_join(a, splits, s);
}

template <int NW, int KW>
void launch_rows(const Int8Args& a, int splits, hipStream_t s) {
  const bool inside = (a.m > 1 && a.lda % 4) || (a.n > 1 && a.ldb % 4);   // a dword
  const bool start = ((uintptr_t)a.a | (uintptr_t)a.b) % 4 == 0;
  if (inside && start) launch_rows_as<NW, KW, true>(a, splits, s);
  else launch_rows_as<NW, KW, false>(a, splits, s);
}

// Rows of a and b at multiples of 16 bytes, zeros past k: 16 bytes a thread.
// Blocks lie along x and y of the grid: one dimension has less than 2^32
// threads, and 2^36 bytes of a have as many pieces.
__global__ __launch_bounds__(256) void k_int8_align(Int8Args g, int8_t* a, int8_t* b, int pitch) {
  const int per = pitch / 16;
  const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x, na = a ? g.m * per : 0, nb = b ? g.n * per : 0;
  if (i < na) {
    const int64_t r = i / per;
    const int c = (int)(i % per) * 16;
    *(intx4*)(a + r * pitch + c) = load_chunk(g.a + r * g.lda, c, g.k);
  } else if (i < na + nb) {
    const int64_t r = (i - na) / per;
    const int c = (int)((i - na) % per) * 16;
    *(intx4*)(b + r * pitch + c) = load_chunk(g.b + r * g.ldb, c, g.k);
  }
}

// Which kernel takes a product, by its sizes alone (us on an MI355X, bf16
// output).
//  - Up to 16 tokens the rows kernel: its traffic is the weights', read once,
//    at any alignment.  Four channel groups to a block where that leaves most
//    CUs a block (1 x 14336 x 4096: 11.4 against 13.0 with one, and 5.0 TB/s);
//    one where it would not (1 x 4096 x 4096: 5.2 against 11.1), and k split
//    over blocks when there are few channels and each wave would still have
//    some pieces of k (8 x 512 x 14336: 7.5 against 12.0).  Beyond 16 tokens
//    its fragments of a cost more than they save (20 x 14336 x 4096: 20.7
//    against the 64 x 64 tile's 13.8).
//  - Otherwise the tile and the split of k with the least of the sum of the
//    rounds over the 256 CUs at a stage's time (128 bytes of k), a tile's
//    fixed time, and the time of writing and joining the splits' sums.  A
//    stage takes 1.31 for 256 x 256, one block per CU (8192 x 14336 x 4096:
//    490, 128 x 128: 590); 1.28 for 128 x 128 two to a CU, 0.70 alone (2048 x
//    4096 x 4096: 43, 256 x 256: 54); 0.55 and 0.30 for 64 x 64 (512 x 4096 x
//    4096: 18, 128 x 128: 28).  24 x 4096 x 14336 on 64 x 64: 14.3 in four
//    splits, 35.3 in one.
struct Int8Plan {
  enum { ROWS1, ROWS4, TILE64, TILE128, TILE256 } kind;
  int splits;
};

Int8Plan int8_plan(int64_t m, int64_t n, int k) {
  const int stages = (k + 127) / 128;
  if (m <= 16) {
    if (n >= 64 * 208) return {Int8Plan::ROWS4, 1};
    const int64_t blocks = (n + 15) / 16;
    return {Int8Plan::ROWS1, (int)std::max<int64_t>(1, std::min<int64_t>(256 / blocks, stages / 28))};
  }
  const auto tiles = [&](int64_t t) { return (m + t - 1) / t * ((n + t - 1) / t); };
  Int8Plan best{Int8Plan::TILE64, 1};
  double least = 1e30;
  const auto consider = [&](decltype(Int8Plan::TILE64) kind, int64_t t, double alone, double two, double fixed) {
    for (int s = 1; s <= 16; ++s) {
      if (s > 1 && stages / s < 4) break;
      const int64_t blocks = tiles(t) * s;
      const double round = two > 0 ? (blocks <= 256 ? alone : two * (double)((blocks + 511) / 512))
                                   : alone * (double)((blocks + 255) / 256);
      const double us = round * ((stages + s - 1) / s) + fixed + (s > 1 ? 3.0 + 8e-6 * s * (double)m * (double)n / 4.0 : 0.0);
      if (us < least) {
        least = us;
        best = {kind, s};
      }
    }
  };
  consider(Int8Plan::TILE256, 256, 1.31, 0, 9);
  consider(Int8Plan::TILE128, 128, 0.70, 1.28, 5);
  consider(Int8Plan::TILE64, 64, 0.30, 0.55, 3);
  return best;
}

// Scratch of a call: the splits' sums, then aligned copies of what is not
// aligned (copies straight into LDS need rows at multiples of 16 bytes and
// 31-bit offsets inside a tile; k padded to whole 16 bytes).
struct Int8Layout {
  Int8Plan plan;
  size_t partial, a, b;   // bytes
  int pitch;
};

Int8Layout int8_layout(const Int8Args& g) {
  Int8Layout l{int8_plan(g.m, g.n, g.k), 0, 0, 0, (g.k + 15) / 16 * 16};
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  if (l.plan.splits > 1) l.partial = up((size_t)l.plan.splits * g.m * g.n * 4);
  if (l.plan.kind == Int8Plan::ROWS1 || l.plan.kind == Int8Plan::ROWS4 || g.k == 0) return l;
  const auto bad = [&](const int8_t* p, int64_t ld) {
    return ((uintptr_t)p | (uint64_t)ld | (uint64_t)g.k) % 16 != 0 || ld >= (1 << 22);
  };
  if (bad(g.a, g.lda)) l.a = up((size_t)g.m * l.pitch);
  if (bad(g.b, g.ldb)) l.b = up((size_t)g.n * l.pitch);
  return l;
}

}  // namespace

size_t int8_linear_scratch(const Int8Args& g) {
  const Int8Layout l = int8_layout(g);
  return l.partial + l.a + l.b;
}

void launch_int8_linear(Int8Args g, hipStream_t s) {
  const Int8Layout l = int8_layout(g);
  if (l.a || l.b) {
    int8_t* a = l.a ? (int8_t*)g.partial + l.partial : nullptr;
    int8_t* b = l.b ? (int8_t*)g.partial + l.partial + l.a : nullptr;
    const int64_t chunks = ((a ? g.m : 0) + (b ? g.n : 0)) * (l.pitch / 16);
    const int64_t blocks = (chunks + 255) / 256, x = std::min<int64_t>(blocks, 1 << 20);
    hipLaunchKernelGGL(k_int8_align, dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)), dim3(256), 0, s, g, a, b, l.pitch);
    if (a) g.a = a, g.lda = l.pitch;
    if (b) g.b = b, g.ldb = l.pitch;
    g.k = l.pitch;   // the zeros of at least one of the two factors fill the rest
    // (k is a multiple of 16 already where only one of them was copied)
  }
  switch (l.plan.kind) {
    case Int8Plan::ROWS1: return launch_rows<1, 16>(g, l.plan.splits, s);
    case Int8Plan::ROWS4: return launch_rows<4, 4>(g, l.plan.splits, s);
    case Int8Plan::TILE64: return launch_mma<64, 64, 2, 2, 4>(g, l.plan.splits, s);
    case Int8Plan::TILE128: return launch_mma<128, 128, 2, 2, 2>(g, l.plan.splits, s);
    case Int8Plan::TILE256: return launch_mma<256, 256, 2, 4, 2>(g, l.plan.splits, s);
  }
}

}  // namespace dion
