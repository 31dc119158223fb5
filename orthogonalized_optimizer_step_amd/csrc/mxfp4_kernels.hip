// Microscaled 4-bit floating point: codes of rows, the values they stand for,
// and the product of two such matrices.
//
// A code is a sign, two bits of exponent and one of mantissa: 0, 0.5, 1, 1.5,
// 2, 3, 4, 6.  Each 32 consecutive elements of a row share a scale 2^(s - 127).
//   e = the least (from -127 on) with max|x| < 7 2^e      s = e + 127
//   code = the nearest to x 2^-e, ties to the even code
// 7 is where 6 and the next value of the same grid, 8, are equally near: below
// it nothing is off by more than half a step of the grid.  (Relative error of
// normal values 0.112 so; 0.115 with 8, by which what lies between 7 and 8 is cut to 6, and
// with 6, by which more is left to the small steps.)  A block with an infinity or a NaN has
// the scale 255, which stands for NaN.
//
//   out[i][j] = sum_k a[i][k] b[j][k] + bias[j]
// by v_mfma_scale_f32_32x32x64_f8f6f4 and 16x16x128: lane l holds 32
// consecutive k (16 bytes) of row l % 32 (l % 16), block l / 32 (l / 16) of
// each operand, and their scale; result element e of lane l of the first is
// row 8 (e / 4) + 4 (l / 32) + e % 4 of the first operand and row l % 32 of
// the second, of the other row 4 (l / 16) + e and row l % 16.  b goes first,
// so that a lane holds four consecutive channels of one token.  Products are
// exact, sums are fp32; their order depends on the sizes and on whether rows
// lie at multiples of 16 bytes.
//
// Codes and values are bound by memory: 8192 x 4096 bf16 take 17 to 20 us each
// (4.3 to 5.0 TB/s).  Large products are bound by the matrix cores' turns with
// LDS: 8192 x 14336 x 4096 262 to 286 us (3.4 to 3.7 PFLOP/s), small ones by the
// weights' bytes: 1 x 14336 x 4096 9.4 (3.3 TB/s).
#include <algorithm>

#include "mma_device.h"
#include "model_internal.h"

namespace dion {

namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef floatx4 floatx4u __attribute__((aligned(4)));

constexpr int MX = 32;   // elements of a scale

// The largest over the 4 or 8 neighbouring lanes of a block.
template <int LANES> __device__ __forceinline__ uint32_t block_max(uint32_t v) {
  const auto move = [&](uint32_t x) { v = max(v, x); };
  move(__builtin_amdgcn_update_dpp(v, v, 0xb1, 0xf, 0xf, false));   // lane xor 1
  move(__builtin_amdgcn_update_dpp(v, v, 0x4e, 0xf, 0xf, false));   // lane xor 2
  if (LANES == 8) move(__builtin_amdgcn_update_dpp(v, v, 0x141, 0xf, 0xf, false));   // the other half of 8
  return v;
}

// Blocks of 256 threads, tx of them along a row; a thread takes 16 bytes of
// values in each of ROWS rows, all asked for before the first is used.  Grid:
// rows along x, the rest of long rows along y.  8192 x 4096 bf16 (us): codes in
// ROWS = 2 19.8, in 4 21.6, in 1 20.0; values in 4 16.7 past the caches, 21.5
// through them.
template <typename T>
__global__ __launch_bounds__(256) void k_mxfp4_quantize(MxCodesArgs a, int tx) {
  typedef Chunk<T> C;
  constexpr int N = C::N, L = MX / N, ROWS = 2;
  const int t = threadIdx.x % tx, per = (a.cols + MX - 1) / MX * L;
  const int64_t step = (int64_t)gridDim.x * (256 / tx);
  for (int64_t row = (int64_t)blockIdx.x * (256 / tx) + threadIdx.x / tx; row < a.rows; row += ROWS * step)
    for (int64_t p = (int64_t)blockIdx.y * tx + t; p < per; p += (int64_t)gridDim.y * tx) {
      const int64_t j = p * N;   // may lie behind the row's end, where values are 0
      uintx4 v[ROWS];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        v[u] = uintx4{0, 0, 0, 0};
        if (row + u * step < a.rows && j < a.cols)
          v[u] = C::load((const T*)a.x + (row + u * step) * a.ldx, (int)j, a.cols, 0.f);
      }
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const int64_t r = row + u * step;
        if (r >= a.rows) break;
        float f[N];
        C::unpack(v[u], f);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
        top = block_max<L>(top);
        const bool bad = top >= 0x7f800000u;
        const int s = bad ? 255 : max(0, (int)((top + 0x200000u) >> 23) - 2);   // 7 = 1.75 2^2: a carry from there on
        const float inv = __uint_as_float((uint32_t)(254 - min(s, 253)) << 23);   // 2^-e
        uint32_t q = 0;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float x = f[i] * inv, y = f[i + 1] * inv;
          if (i == 0) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x, y, 1.f, 0);
          if (i == 2) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x, y, 1.f, 1);
          if (i == 4) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x, y, 1.f, 2);
          if (i == 6) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x, y, 1.f, 3);
        }
        if (bad) q = 0;
        uint8_t* o = a.q + r * a.ldq + j / 2;
        if (j + N <= a.cols) __builtin_memcpy(o, &q, N / 2);
        else
          for (int i = 0; 2 * i < N; ++i)
            if (j + 2 * i < a.cols) o[i] = (uint8_t)(q >> (8 * i));
        // the scales of four blocks from the first one's lane, where the row has four more
        uint8_t* sc = a.s + r * a.lds + p / L;
        if (L == 4 && (p / 16 + 1) * 16 <= per) {
          int all = s;
          all |= __builtin_amdgcn_update_dpp(0, s, 0x104, 0xf, 0xf, false) << 8;    // from lane + 4, 8, 12
          all |= __builtin_amdgcn_update_dpp(0, s, 0x108, 0xf, 0xf, false) << 16;
          all |= __builtin_amdgcn_update_dpp(0, s, 0x10c, 0xf, 0xf, false) << 24;
          if (t % 16 == 0) __builtin_memcpy(sc, &all, 4);
        } else if (t % L == 0) {
          *sc = (uint8_t)s;
        }
      }
    }
}

// The values: the same shares of the rows.
template <typename T>
__global__ __launch_bounds__(256) void k_mxfp4_dequantize(MxCodesArgs a, int tx) {
  typedef Chunk<T> C;
  constexpr int N = C::N, L = MX / N, ROWS = 4;
  const int t = threadIdx.x % tx, per = (a.cols + N - 1) / N;
  const int64_t step = (int64_t)gridDim.x * (256 / tx);
  for (int64_t row = (int64_t)blockIdx.x * (256 / tx) + threadIdx.x / tx; row < a.rows; row += ROWS * step)
    for (int64_t p = (int64_t)blockIdx.y * tx + t; p < per; p += (int64_t)gridDim.y * tx) {
      const int64_t j = p * N;
      uint32_t q[ROWS];
      int s[ROWS];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const int64_t r = row + u * step;
        q[u] = 0, s[u] = 0;
        if (r >= a.rows) break;
        const uint8_t* c = a.q + r * a.ldq + j / 2;
        if (j + N <= a.cols) __builtin_memcpy(&q[u], c, N / 2);
        else
          for (int i = 0; 2 * i < N; ++i)
            if (j + 2 * i < a.cols) q[u] |= (uint32_t)c[i] << (8 * i);
        s[u] = a.s[r * a.lds + p / L];
      }
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const int64_t r = row + u * step;
        if (r >= a.rows) break;
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t code = q[u] >> (4 * i) & 7;
          // 0, 0.5 and the others, whose bits are an exponent's and a mantissa's
          const float v = code < 2 ? 0.5f * code : __uint_as_float((code << 22) + (126u << 23));
          f[i] = s[u] == 255 ? __builtin_nanf("") : ldexpf(q[u] >> (4 * i) & 8 ? -v : v, s[u] - 127);
        }
        C::store((T*)a.x + r * a.ldx, (int)j, a.cols, f);
      }
    }
}

// Threads along a row: a power of two that covers it, a row of lanes at least.
int along(int64_t pieces) {
  int tx = 16;
  while (tx < 256 && tx < pieces) tx *= 2;
  return tx;
}
// A row to a thread while there are no more than fill the CUs, `rows` otherwise.
dim3 codes_grid(const MxCodesArgs& a, int64_t pieces, int tx, int rows) {
  const int64_t x = (a.rows + 256 / tx - 1) / (256 / tx), y = std::min<int64_t>((pieces + tx - 1) / tx, 1 << 15);
  return dim3((unsigned)std::min<int64_t>(x * y <= 2048 ? x : (x + rows - 1) / rows, 1 << 20), (unsigned)y);
}

template <typename T> void launch_quantize(const MxCodesArgs& a, hipStream_t s) {
  const int64_t pieces = ((int64_t)a.cols + MX - 1) / MX * (MX / Chunk<T>::N);
  const int tx = along(pieces);
  hipLaunchKernelGGL((k_mxfp4_quantize<T>), codes_grid(a, pieces, tx, 2), dim3(256), 0, s, a, tx);
}
template <typename T> void launch_dequantize(const MxCodesArgs& a, hipStream_t s) {
  const int64_t pieces = ((int64_t)a.cols + Chunk<T>::N - 1) / Chunk<T>::N;
  const int tx = along(pieces);
  hipLaunchKernelGGL((k_mxfp4_dequantize<T>), codes_grid(a, pieces, tx, 4), dim3(256), 0, s, a, tx);
}

// ------------------------------------------------------------------ product
__device__ __forceinline__ intx8 wide(intx4 v) { return intx8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// The scales' bytes ks of sb and sa; 4: 4-bit floating point.
__device__ __forceinline__ floatx16 mma32(intx4 b, intx4 a, floatx16 c, int sb, int sa, int ks) {
  const intx8 x = wide(b), y = wide(a);
  if (ks == 0) return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 0, sb, 0, sa);
  if (ks == 1) return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 1, sb, 1, sa);
  if (ks == 2) return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 2, sb, 2, sa);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 3, sb, 3, sa);
}
__device__ __forceinline__ floatx4 mma16(intx4 b, intx4 a, floatx4 c, int sb, int sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(b), wide(a), c, 4, 4, 0, sb, 0, sa);
}

__device__ __forceinline__ float biased(const MxArgs& g, int64_t col, float v) {
  return g.bias ? v + load_fmt(g.bias, col, g.bias_fmt) : v;
}

// One BM x BN tile of the output by WM x WN waves, as the 8-bit product's: S
// stages of BK bytes of codes (256 k) in LDS, copied straight there S - 1
// stages ahead, fragments of the next 32 bytes read while the present ones are
// multiplied.  The scales come along 32 bytes of a row at once, those of G =
// 4 stages, into two places of their own in turn, and a stage ahead of the
// codes, so that a stage's are read from LDS in the middle of the one before; a
// lane's four (blocks l / 32, 2 + l / 32, ..) are picked into one register.
// (8192 x 14336 x 4096: 297 us with 16 bytes at once, read at the turn.)  Codes
// and scales lie in rows at multiples of 16 bytes, whole chunks of them.
template <int BM, int BN, int WM, int WN, int S, typename O>
__global__ __launch_bounds__(64 * WM * WN) void k_mxfp4_mma(MxArgs g, float* partial) {
  constexpr int W = WM * WN, NT = 64 * W;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;   // wave tile, its fragments
  constexpr int STAGE = (BM + BN) * BK;
  constexpr int NP = STAGE / 1024 / W;            // 1 KB pieces of a stage per wave
  constexpr int PR = 1024 / BK, CR = BK / 16;     // rows of a piece, chunks of a row
  constexpr int G = 4, SCALES = (BM + BN) * 8 * G, SP = SCALES / 1024 / W;   // pieces of a group's scales per wave
  constexpr int OV = OutVec<O>::N, SROW = TN + OV;   // staged output row
  constexpr int STAGED = W * 32 * SROW * (int)sizeof(O);
  constexpr int HELD = S * STAGE + 2 * SCALES, LDS = HELD > STAGED ? HELD : STAGED;
  constexpr int KS = BK / 32;
  constexpr bool SPREAD = BM * BN >= 256 * 256;
  constexpr int PW = NP / 2, EVERY = SPREAD ? FM * FN / PW : 1;
  static_assert(!SPREAD || (PW * 2 == NP && EVERY * PW == FM * FN), "the copies divide the products");
  static_assert(S <= 4 && NP * W * 1024 == STAGE && BM % PR == 0 && SP * W * 1024 == SCALES && S <= G, "whole pieces");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int ti, tj;
  tile_of_block((int)((g.m + BM - 1) / BM), (int)((g.n + BN - 1) / BN), ti, tj);
  const int64_t m0 = (int64_t)ti * BM, n0 = (int64_t)tj * BN;
  const int rm = (int)min((int64_t)BM, g.m - m0), rn = (int)min((int64_t)BN, g.n - n0);   // valid rows of the tile
  // this split's stages
  const int all = (g.kb + BK - 1) / BK, sb16 = (g.kb + 255) / 256 * 16;   // (bytes of a row of scales, whole chunks)
  const int kt0 = (int)((int64_t)all * blockIdx.y / gridDim.y);
  const int nk = (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y) - kt0;
  const uint32_t lds0 = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)smem);

  // piece q = wave + i W of a stage: rows PR q .. of a, then of b; lane l has
  // row l / CR and the chunk whose place is l % CR (the same chunk in all of
  // its pieces: W PR is a multiple of 16).  Rows past the tile's last are
  // behind the descriptors' ends.
  static_assert(W * PR % 16 == 0 && BM / PR % W == 0, "a piece index is of one matrix and one swizzle");
  const intx4 ra = raw_buffer(g.a + m0 * g.lda, (uint32_t)((rm - 1) * g.lda + g.kb));
  const intx4 rb = raw_buffer(g.b + n0 * g.ldb, (uint32_t)((rn - 1) * g.ldb + g.kb));
  const intx4 rsa = raw_buffer(g.sa + m0 * g.ldsa, (uint32_t)((rm - 1) * g.ldsa + sb16));
  const intx4 rsb = raw_buffer(g.sb + n0 * g.ldsb, (uint32_t)((rn - 1) * g.ldsb + sb16));
  const int prow = wave * PR + lane / CR, vk = swz(prow, lane % CR) * 16;
  const uint32_t va = (uint32_t)(prow * (int)g.lda + vk), vb = (uint32_t)(prow * (int)g.ldb + vk);
  // piece q = wave + i W of a group's scales: rows 32 q .. of a, then of b, two lanes to a row
  const int schunk = (lane & 1) * 16;
  auto issue = [&](int kt, int i) {   // piece i of stage kt
    constexpr int A = BM / PR / W;   // pieces of a
    const int k0 = (kt0 + kt) * BK, q = wave + i * W;
    const uint32_t v = i < A ? va + (uint32_t)(i * W * PR * (int)g.lda) : vb + (uint32_t)((i - A) * W * PR * (int)g.ldb);
    dma16(k0 + vk < g.kb ? v : OUT_OF_RANGE, i < A ? ra : rb, (uint32_t)k0,
          (uint32_t)__builtin_amdgcn_readfirstlane(lds0 + (kt % S) * STAGE + q * 1024));
  };
  auto issue_scales = [&](int kt) {   // with the first of a group's stages
    const uint32_t group = (uint32_t)(kt0 + kt) / G;
    if ((uint32_t)(kt0 + kt) % G != 0 && kt > 0) return;
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      const int q = wave + i * W, row = q * 32 + lane / 2;
      const bool isa = q < BM / 32;
      const uint32_t v = (uint32_t)(isa ? row * (int)g.ldsa : (row - BM) * (int)g.ldsb) + schunk;
      dma16((int)(group * 8 * G) + schunk < sb16 ? v : OUT_OF_RANGE, isa ? rsa : rsb, group * 8 * G,
            (uint32_t)__builtin_amdgcn_readfirstlane(lds0 + S * STAGE + group % 2 * SCALES + q * 1024));
    }
  };

  floatx16 acc[FM][FN] = {};
  intx4 fa[2][FM], fb[2][FN];
  int sa[FM], sb[FN];       // the scales of this stage
  uint2 na[FM], nb[FN];     // of the next, all eight of a row
  const int r = lane & 31;
  const uint32_t pick = lane < 32 ? 0x06040200u : 0x07050301u;
  auto fetch = [&](int kt, int ks, int set) {
    const uint8_t* s = smem + (kt % S) * STAGE + swz(r, ks * 2 + (lane >> 5)) * 16;
#pragma unroll
    for (int f = 0; f < FM; ++f) fa[set][f] = *(const intx4*)(s + (wm * TM + f * 32 + r) * BK);
#pragma unroll
    for (int f = 0; f < FN; ++f) fb[set][f] = *(const intx4*)(s + (BM + wn * TN + f * 32 + r) * BK);
  };
  auto fetch_scales = [&](int kt) {
    const uint32_t at = (uint32_t)(kt0 + kt);
    const uint8_t* s = smem + S * STAGE + at / G % 2 * SCALES + at % G * 8;
#pragma unroll
    for (int f = 0; f < FM; ++f) na[f] = *(const uint2*)(s + (wm * TM + f * 32 + r) * 8 * G);
#pragma unroll
    for (int f = 0; f < FN; ++f) nb[f] = *(const uint2*)(s + (BM + wn * TN + f * 32 + r) * 8 * G);
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = (int)__builtin_amdgcn_perm(na[f].y, na[f].x, pick);
#pragma unroll
    for (int f = 0; f < FN; ++f) sb[f] = (int)__builtin_amdgcn_perm(nb[f].y, nb[f].x, pick);
  };
  // the stage that is needed next has landed, and every wave is done with the one before it
  auto turn = [&](int kt) {
    const int later = min(nk - 1, kt + S - 2) - kt;   // stages issued after kt, NP copies each or one more
    if (S >= 4 && later >= 2) wait_vmcnt<2 * NP>();
    else if (S >= 3 && later >= 1) wait_vmcnt<NP>();
    else wait_vmcnt<0>();
    lds_barrier();
    if (kt + S < nk) issue_scales(kt + S);
    if (!SPREAD && kt + S - 1 < nk) {
#pragma unroll
      for (int i = 0; i < NP; ++i) issue(kt + S - 1, i);
    }
  };
  if (nk > 0) {
#pragma unroll
    for (int t = 0; t < S; ++t)
      if (t < nk) issue_scales(t);
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
    fetch_scales(0);
    take_scales();
    for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (ks + 1 < KS) {
          fetch(kt, ks + 1, (ks + 1) & 1);
          if (ks == 1 && kt + 1 < nk) fetch_scales(kt + 1);
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
            acc[i][j] = mma32(fb[ks & 1][j], fa[ks & 1][i], acc[i][j], sb[j], sa[i], ks);
            // here: the compiler would move products behind later branches
            if constexpr (SPREAD) asm volatile("" : "+v"(acc[i][j]));
            else asm volatile("" : "+a"(acc[i][j]));
            const int t = i * FN + j;
            if (SPREAD && w < 2 && t % EVERY == EVERY - 1) {
              __builtin_amdgcn_sched_barrier(0);
              if (st < nk) issue(st, w * PW + t / EVERY);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
        __builtin_amdgcn_sched_barrier(0);
      }
      take_scales();
    }
  }
  if (partial) {   // several splits: the sums as they are, for k_mxfp4_join
    float* out = partial + (int64_t)blockIdx.y * g.m * g.n;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t row = m0 + wm * TM + i * 32 + r;
      if (row >= g.m) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t col = n0 + wn * TN + j * 32 + q * 8 + (lane >> 5) * 4;
          float* o = out + row * g.n + col;
          const floatx4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          if (col + 4 <= g.n) *(floatx4u*)o = v;
          else
            for (int e = 0; e < 4; ++e)
              if (col + e < g.n) o[e] = v[e];
        }
    }
    return;
  }
  // The stages are free: each wave stages 32 rows of its output at a time, and
  // writes them past the caches, which the operands and the next call's inputs
  // have more use for (8192 x 14336 x 4096 with a's codes before it: 308 us
  // through them, 288 past them; 2048 x 4096 x 4096 with a norm of it behind 38.6
  // and 37.9).
  __syncthreads();

  O* st = (O*)smem + wave * 32 * SROW;
  const int64_t cbase = n0 + wn * TN;
  constexpr int CPR = TN / OV;   // 16-byte pieces of a staged row
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        typedef O Ox4 __attribute__((ext_vector_type(4)));
        Ox4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // past the last channel its bias: not written
          const int64_t col = min(cbase + j * 32 + q * 8 + (lane >> 5) * 4 + e, g.n - 1);
          v[e] = from_f<O>(biased(g, col, acc[i][j][q * 4 + e]));
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
        if (col + OV <= g.n) __builtin_nontemporal_store(*(const intx4*)s, (intx4u*)o);
        else
          for (int e = 0; col + e < g.n; ++e) o[e] = s[e];
      }
    }
    asm volatile("" : : : "memory");
  }
}

// The splits' sums, in their order.  Tokens lie along y and z of the grid,
// which have 65536 blocks at most each.
template <typename O> __global__ __launch_bounds__(256) void k_mxfp4_join(MxArgs g, const float* partial, int splits) {
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
  if (col >= g.n || row >= g.m) return;
  float v = 0.f;
  for (int s = 0; s < splits; ++s) v += partial[((int64_t)s * g.m + row) * g.n + col];
  ((O*)g.out)[row * g.ldo + col] = from_f<O>(biased(g, col, v));
}

void launch_join(const MxArgs& a, int splits, hipStream_t s) {
  const int64_t y = std::min<int64_t>(a.m, 1 << 15);
  const dim3 grid((unsigned)((a.n + 255) / 256), (unsigned)y, (unsigned)((a.m + y - 1) / y));
  if (a.out_fmt == 1) hipLaunchKernelGGL((k_mxfp4_join<float>), grid, dim3(256), 0, s, a, a.partial, splits);
  else if (a.out_fmt == 0) hipLaunchKernelGGL((k_mxfp4_join<bf16_t>), grid, dim3(256), 0, s, a, a.partial, splits);
  else hipLaunchKernelGGL((k_mxfp4_join<fp16_t>), grid, dim3(256), 0, s, a, a.partial, splits);
}

template <int BM, int BN, int WM, int WN, int S>
void launch_mma(const MxArgs& a, int splits, hipStream_t s) {
  const int64_t tiles = (a.m + BM - 1) / BM * ((a.n + BN - 1) / BN);
  const dim3 grid((unsigned)tiles, splits), block(64 * WM * WN);
  float* part = splits > 1 ? a.partial : nullptr;
  if (a.out_fmt == 1) hipLaunchKernelGGL((k_mxfp4_mma<BM, BN, WM, WN, S, float>), grid, block, 0, s, a, part);
  else if (a.out_fmt == 0) hipLaunchKernelGGL((k_mxfp4_mma<BM, BN, WM, WN, S, bf16_t>), grid, block, 0, s, a, part);
  else hipLaunchKernelGGL((k_mxfp4_mma<BM, BN, WM, WN, S, fp16_t>), grid, block, 0, s, a, part);
  if (part) launch_join(a, splits, s);
}

// Up to 16 tokens: the block takes 16 channels; each of its KW waves every
// KW-th 128-byte piece of the split's share of k, and the sums of the KW meet
// in LDS.  Codes and scales go from global memory to registers, at any
// alignment.  Rows past the end repeat the last one and are not written.
constexpr int KW = 16;
template <typename O> __global__ __launch_bounds__(64 * KW) void k_mxfp4_rows(MxArgs g, float* partial) {
  __shared__ __attribute__((aligned(16))) float sum[KW * 256];
  const int tid = threadIdx.x, lane = tid & 63, kw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int r = lane & 15, kc = lane >> 4;   // row, block of 32 in its 128
  const int64_t rb = min(n0 + r, g.n - 1), ra = min((int64_t)r, g.m - 1);
  const uint8_t *b = g.b + rb * g.ldb, *a = g.a + ra * g.lda, *sb = g.sb + rb * g.ldsb, *sa = g.sa + ra * g.ldsa;
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  const int pieces = (g.kb + 127) / 128, nb = (g.kb + 15) / 16;
  const int p0 = (int)((int64_t)pieces * blockIdx.y / gridDim.y);
  const int kend = min(g.kb, (int)((int64_t)pieces * (blockIdx.y + 1) / gridDim.y) * 128);
  int k0 = (p0 + kw) * 128;
#pragma unroll 4
  for (; k0 + 128 <= kend; k0 += KW * 128) {
    uint2 vb, va;   // the scales of 128 bytes
    __builtin_memcpy(&vb, sb + k0 / 16, 8);
    __builtin_memcpy(&va, sa + k0 / 16, 8);
    acc = mma16(*(const intx4u*)(b + k0 + kc * 16), *(const intx4u*)(a + k0 + kc * 16), acc, (int)(vb.x >> (8 * kc)),
                (int)(va.x >> (8 * kc)));
    acc = mma16(*(const intx4u*)(b + k0 + kc * 16 + 64), *(const intx4u*)(a + k0 + kc * 16 + 64), acc,
                (int)(vb.y >> (8 * kc)), (int)(va.y >> (8 * kc)));
  }
  if (k0 < kend) {   // the last piece, in part
    for (int h = 0; h < 128; h += 64) {
      const int k = k0 + kc * 16 + h, blk = k / 16;
      const int xb = blk < nb ? sb[blk] : 0, xa = blk < nb ? sa[blk] : 0;
      acc = mma16(load_chunk((const int8_t*)b, k, kend), load_chunk((const int8_t*)a, k, kend), acc, xb, xa);
    }
  }
  *(floatx4*)(sum + (kw * 16 + r) * 16 + kc * 4) = acc;   // [kw][token][channel of the block]
  __syncthreads();
  if (tid < 256) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) v += sum[w * 256 + tid];
    const int64_t row = tid / 16, col = n0 + tid % 16;
    if (row < g.m && col < g.n) {
      if (partial) partial[((int64_t)blockIdx.y * g.m + row) * g.n + col] = v;
      else ((O*)g.out)[row * g.ldo + col] = from_f<O>(biased(g, col, v));
    }
  }
}

void launch_rows(const MxArgs& a, int splits, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + 15) / 16), splits), block(64 * KW);
  float* part = splits > 1 ? a.partial : nullptr;
  if (a.out_fmt == 1) hipLaunchKernelGGL((k_mxfp4_rows<float>), grid, block, 0, s, a, part);
  else if (a.out_fmt == 0) hipLaunchKernelGGL((k_mxfp4_rows<bf16_t>), grid, block, 0, s, a, part);
  else hipLaunchKernelGGL((k_mxfp4_rows<fp16_t>), grid, block, 0, s, a, part);
  if (part) launch_join(a, splits, s);
}

// Rows at multiples of 16 bytes, zeros past their ends, of up to four matrices
// of bytes: 16 a thread.  Blocks lie along x and y of the grid.
struct AlignJob {
  const uint8_t* from;   // NULL: not copied
  uint8_t* to;
  int64_t ld, rows;
  int bytes, pitch;
};
struct AlignJobs { AlignJob of[4]; };
__global__ __launch_bounds__(256) void k_mxfp4_align(AlignJobs jobs) {
  int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const AlignJob& job = jobs.of[q];
    if (!job.from) continue;
    const int per = job.pitch / 16;
    const int64_t n = job.rows * per;
    if (i >= 0 && i < n) {
      const int64_t r = i / per;
      const int c = (int)(i % per) * 16;
      *(intx4*)(job.to + r * job.pitch + c) = load_chunk((const int8_t*)job.from + r * job.ld, c, job.bytes);
    }
    i -= n;
  }
}

// Which kernel takes a product, by its sizes, and whether its operands lie as
// the tiles need them (us on an MI355X, bf16 output).
//  - Up to 16 tokens the rows kernel, which reads the weights once at any
//    alignment, in rounds of 16 channels for each of the 256 CUs, against the tiles
//    of 64 channels, which fill the CUs in one round up to 16384 and whose copies
//    straight into LDS keep more of memory busy, where nothing has to be copied for
//    them.  The tiles from the fourth round on (1 token, k = 4096, rows and tiles: n =
//    4096 4.7 and 8.7, 8192 7.1 and 9.3, 12288 9.7 and 9.6, 12352 11.0 and 9.7, 14336
//    11.1 and 9.7, 32768 20 and 17, 131072 71 and 57; k = 14336: 12288 20.4 and 23.5,
//    12352 24.3 and 23.5, 131072 177 and 165), and from the third on for more than
//    8 tokens, of which each costs the rows kernel reads of its own (k = 4096: 16
//    tokens at n = 8192 9.0 and 9.4; at 8256 4 tokens 9.5 and 9.5, 8 10.1 and 9.5, 16
//    11.3 and 9.5; k = 14336, n = 9216: 4 tokens 21.0 and 23.0, 8 23.4 and 23.1, 12
//    25.7 and 23.2).
//    The rows kernel has k split over blocks where there are few channels and more
//    than 32 stages of it, 14 at least to a block: the join costs 1 to 2 (1 token, one,
//    two, four and eight splits: 512 x 4096 4.1, 5.3, 5.3, 6.2; 512 x 8192 6.0, 6.3,
//    6.3, 6.7; 64 x 14336 7.2, 6.4, 5.6, 6.1; 1024 x 14336 7.9, 7.5, 6.8, 7.8; 2048 x
//    14336 8.8, 8.4, 8.9, 11.0; 512 x 28672 14.4, 10.9, 8.6, 7.9; 512 x 65536 31, 20, 13,
//    11).
//  - Otherwise the tile and the split of k with the least of the sum of the
//    rounds over the 256 CUs at a stage's time (256 k), a tile's fixed time, and
//    the time of writing and joining the splits' sums.  A stage takes 2.0 for
//    256 x 256, one block per CU, and 1.3 while half of the CUs have none (1024 x
//    14336 x 4096: 39, 128 x 128: 51); 1.3 for 128 x 128 two to a CU, 0.8 and
//    0.58 alone (2048 x 4096 x 4096: 27; 512 x 14336 x 4096: 26, 256 x 256: 33);
//    0.6, 0.36 and 0.31 for 64 x 64 (512 x 4096 x 4096: 13; 256 x 14336 x 4096:
//    23.5, 128 x 128: 20.7).  24 x 4096 x 14336 on 64 x 64: 12.6 in four splits, 21
//    in one.
struct MxPlan {
  enum { ROWS, TILE64, TILE128, TILE256 } kind;
  int splits;
};

MxPlan mx_plan(int64_t m, int64_t n, int kb, bool aligned) {
  const int stages = (kb + 127) / 128;
  if (m <= 16) {
    const int64_t blocks = (n + 15) / 16;
    if (aligned && blocks > (m > 8 ? 2 : 3) * 256) return {MxPlan::TILE64, 1};
    return {MxPlan::ROWS, stages <= 32 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(256 / blocks, stages / 14))};
  }
  const auto tiles = [&](int64_t t) { return (m + t - 1) / t * ((n + t - 1) / t); };
  MxPlan best{MxPlan::TILE64, 1};
  double least = 1e30;
  const auto consider = [&](decltype(MxPlan::TILE64) kind, int64_t t, double half, double alone, double two, double fixed) {
    for (int s = 1; s <= 16; ++s) {
      if (s > 1 && stages / s < 4) break;
      const int64_t blocks = tiles(t) * s;
      const double round = blocks <= 128          ? half
                           : blocks <= 256        ? alone
                           : two > 0              ? two * (double)((blocks + 511) / 512)
                                                  : alone * (double)((blocks + 255) / 256);
      const double us = round * ((stages + s - 1) / s) + fixed + (s > 1 ? 3.0 + 8e-6 * s * (double)m * (double)n / 4.0 : 0.0);
      if (us < least) {
        least = us;
        best = {kind, s};
      }
    }
  };
  consider(MxPlan::TILE256, 256, 1.3, 2.0, 0, 7);
  consider(MxPlan::TILE128, 128, 0.58, 0.82, 1.3, 6.7);
  consider(MxPlan::TILE64, 64, 0.31, 0.36, 0.6, 4);
  return best;
}

// Scratch of a call: the splits' sums, then aligned copies of what is not
// aligned (copies straight into LDS need rows of whole 16 bytes at multiples
// of 16, and 31-bit offsets inside a tile).
struct MxLayout {
  MxPlan plan;
  size_t partial, copy[4];   // bytes: sums; a, its scales, b, its scales
  int pitch[2];              // of codes, of scales
};

MxLayout mx_layout(const MxArgs& g) {
  const int nb = (g.kb + 15) / 16;
  const auto bad = [&](const uint8_t* p, int64_t ld, int bytes) {
    return ((uintptr_t)p | (uint64_t)ld | (uint64_t)bytes) % 16 != 0 || ld >= (1 << 22);
  };
  const bool copies[4] = {bad(g.a, g.lda, g.kb), bad(g.sa, g.ldsa, nb), bad(g.b, g.ldb, g.kb), bad(g.sb, g.ldsb, nb)};
  const bool aligned = !(copies[0] || copies[1] || copies[2] || copies[3]);
  MxLayout l{mx_plan(g.m, g.n, g.kb, aligned), 0, {}, {nb * 16, (nb + 15) / 16 * 16}};
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  if (l.plan.splits > 1) l.partial = up((size_t)l.plan.splits * g.m * g.n * 4);
  if (l.plan.kind == MxPlan::ROWS || g.kb == 0) return l;
  for (int q = 0; q < 4; ++q)
    if (copies[q]) l.copy[q] = up((size_t)(q < 2 ? g.m : g.n) * l.pitch[q % 2]);
  return l;
}

}  // namespace

size_t mxfp4_linear_scratch(const MxArgs& g) {
  const MxLayout l = mx_layout(g);
  return l.partial + l.copy[0] + l.copy[1] + l.copy[2] + l.copy[3];
}

void launch_mxfp4_linear(MxArgs g, hipStream_t s) {
  const MxLayout l = mx_layout(g);
  const int nb = (g.kb + 15) / 16;
  const uint8_t** at[4] = {&g.a, &g.sa, &g.b, &g.sb};
  int64_t* ld[4] = {&g.lda, &g.ldsa, &g.ldb, &g.ldsb};
  AlignJobs jobs{};
  uint8_t* to = (uint8_t*)g.partial + l.partial;
  int64_t chunks = 0;
  for (int q = 0; q < 4; ++q) {
    if (!l.copy[q]) continue;
    AlignJob& job = jobs.of[q];
    job = {*at[q], to, *ld[q], q < 2 ? g.m : g.n, q % 2 ? nb : g.kb, l.pitch[q % 2]};
    chunks += job.rows * (job.pitch / 16);
    *at[q] = to;
    *ld[q] = job.pitch;
    to += l.copy[q];
  }
  if (chunks) {
    const int64_t blocks = (chunks + 255) / 256, x = std::min<int64_t>(blocks, 1 << 20);
    hipLaunchKernelGGL(k_mxfp4_align, dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)), dim3(256), 0, s, jobs);
    if (l.copy[0] || l.copy[2]) g.kb = l.pitch[0];   // the zeros of at least one of the two factors fill the rest
  }
  switch (l.plan.kind) {
    case MxPlan::ROWS: return launch_rows(g, l.plan.splits, s);
    case MxPlan::TILE64: return launch_mma<64, 64, 2, 2, 4>(g, l.plan.splits, s);
    case MxPlan::TILE128: return launch_mma<128, 128, 2, 2, 2>(g, l.plan.splits, s);
    case MxPlan::TILE256: return launch_mma<256, 256, 2, 4, 2>(g, l.plan.splits, s);
  }
}

void launch_mxfp4_quantize(int fmt, const MxCodesArgs& a, hipStream_t s) {
  if (fmt == 1) launch_quantize<float>(a, s);
  else if (fmt == 0) launch_quantize<bf16_t>(a, s);
  else launch_quantize<fp16_t>(a, s);
}

void launch_mxfp4_dequantize(int fmt, const MxCodesArgs& a, hipStream_t s) {
  if (fmt == 1) launch_dequantize<float>(a, s);
  else if (fmt == 0) launch_dequantize<bf16_t>(a, s);
  else launch_dequantize<fp16_t>(a, s);
}

}  // namespace dion
