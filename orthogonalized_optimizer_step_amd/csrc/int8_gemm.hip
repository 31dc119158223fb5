// Product of 8-bit integers with a scale for each token and channel:
//   out[i][j] = round(float(sum_k a[i][k] b[j][k]) * sa[i] * sb[j] + bias[j])
// The sum is exact in int32 (k < 2^17), so the only roundings are the fp32
// conversion of the sum, the scales' products and the output's own, and the
// result does not depend on how the sum is split.
//
// v_mfma_i32_32x32x32_i8: lane l holds 16 consecutive k of row l % 32 (k block
// l / 32) of each operand; result element e of lane l is row
// 8 (e / 4) + 4 (l / 32) + e % 4 of the first operand and row l % 32 of the
// second.  b goes first, so that a lane holds four consecutive channels of one
// token.
#include "train_device.h"
#include "train_internal.h"

namespace dion {

namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx16 __attribute__((ext_vector_type(16)));
// sixteen bytes at any alignment
typedef intx4 intx4u __attribute__((aligned(1)));

constexpr int BK = 128;   // bytes of k in a stage: one cache line of each row

// Position of 16-byte chunk c of row r in its 128-byte LDS row: any 8
// consecutive rows reading one chunk touch all 128 bytes, any 16 touch both
// halves of 256, so the fragment reads meet no bank twice.
__device__ __forceinline__ int swz(int r, int c) { return c ^ ((r ^ ((r >> 3) & 1)) & 7); }

// One 16-byte copy per lane from global memory straight into LDS: lane l's
// bytes land at lds_addr + 16 l; lanes whose offset is past the descriptor's
// range get zeros.  Counted by vmcnt, waited for explicitly.
__device__ __forceinline__ void dma16(uint32_t voff, intx4 rsrc, uint32_t soff, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds_addr)
               : "memory", "m0");
}
template <int N> __device__ __forceinline__ void wait_vmcnt() { asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory"); }
// a barrier that waits for the wave's LDS accesses but not for copies in flight
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

constexpr uint32_t OUT_OF_RANGE = 0x80000000u;

// Descriptor of `bytes` bytes from p (raw: offsets in bytes, past the end reads zero).
__device__ __forceinline__ intx4 raw_buffer(const void* p, uint32_t bytes) {
  const uint64_t u = (uint64_t)p;
  intx4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32) & 0xffff);
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000;
  return r;
}

// 16 bytes of a row from k on, zeros from `ks` on
__device__ __forceinline__ intx4 load_chunk(const int8_t* row, int k, int ks) {
  if (k + 16 <= ks) return *(const intx4u*)(row + k);
  intx4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (k + i < ks) v[i >> 2] |= (int)(uint8_t)row[k + i] << (8 * (i & 3));
  return v;
}

template <typename O> struct OutVec;   // 16 bytes of output elements
template <> struct OutVec<float> { static constexpr int N = 4; };
template <> struct OutVec<bf16_t> { static constexpr int N = 8; };
template <> struct OutVec<fp16_t> { static constexpr int N = 8; };

// Tile (ti, tj) of block b: blocks are dealt to the 8 XCDs round-robin; each
// XCD takes a contiguous run of the tiles in bands of eight tile rows walked
// column by column, so that the tiles it works on at once share operand panels
// in its L2.
__device__ __forceinline__ void tile_of_block(int TM, int TN, int& ti, int& tj) {
  const int total = TM * TN, x = blockIdx.x & 7, per = total / 8, more = total % 8;
  int t = (blockIdx.x >> 3) + x * per + min(x, more);
  const int band = t / (8 * TN), r0 = band * 8, rows = min(8, TM - r0);
  t -= band * 8 * TN;
  tj = t / rows;
  ti = r0 + t % rows;
}

// One BM x BN tile of the output by WM x WN waves, S stages of BK bytes in
// LDS.  DMA: the stages are copied straight into LDS S - 1 stages ahead (rows
// at multiples of 16 bytes); otherwise they pass through registers (any
// alignment).  Each wave holds two sets of fragments: those of the next 32
// bytes are read from LDS while the present ones are multiplied, across the
// stage's end too.
template <int BM, int BN, int WM, int WN, int S, bool DMA, typename O>
__global__ __launch_bounds__(64 * WM * WN) void k_int8_mma(Int8Args g) {
  constexpr int W = WM * WN, NT = 64 * W;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;   // wave tile, its fragments
  constexpr int STAGE = (BM + BN) * BK;
  constexpr int NP = STAGE / 1024 / W;            // 1 KB pieces (8 rows) of a stage per wave
  constexpr int OV = OutVec<O>::N, SROW = TN + OV;   // staged output row
  constexpr int STAGED = W * 32 * SROW * (int)sizeof(O);
  constexpr int LDS = S * STAGE > STAGED ? S * STAGE : STAGED;
  static_assert(NP * W * 1024 == STAGE && BM % 8 == 0, "whole pieces");
  __shared__ __attribute__((aligned(1024))) int8_t smem[LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int ti, tj;
  tile_of_block((int)((g.m + BM - 1) / BM), (int)((g.n + BN - 1) / BN), ti, tj);
  const int64_t m0 = (int64_t)ti * BM, n0 = (int64_t)tj * BN;
  const int rm = (int)min((int64_t)BM, g.m - m0), rn = (int)min((int64_t)BN, g.n - n0);   // valid rows of the tile
  const int8_t* A = g.a + m0 * g.lda;
  const int8_t* B = g.b + n0 * g.ldb;
  const int nk = (g.k + BK - 1) / BK;
  const uint32_t lds0 = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) int8_t*)smem);

  // piece q = wave + i W of a stage: rows 8 q .. 8 q + 7 (a's, then b's), lane
  // l row l / 8 and the chunk whose place is l % 8
  uint32_t voff[NP];
  int vk[NP];
  const intx4 ra = raw_buffer(A, (uint32_t)((rm - 1) * g.lda + g.k)), rb = raw_buffer(B, (uint32_t)((rn - 1) * g.ldb + g.k));
  intx4 reg[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int q = wave + i * W;
    const bool isa = q < BM / 8;
    const int r = (isa ? q : q - BM / 8) * 8 + (lane >> 3);
    vk[i] = swz(r, lane & 7) * 16;
    voff[i] = r < (isa ? rm : rn) ? (uint32_t)(r * (isa ? g.lda : g.ldb)) + vk[i] : OUT_OF_RANGE;
  }
  auto issue = [&](int kt) {
    const int k0 = kt * BK;
    const bool whole = k0 + BK <= g.k;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int q = wave + i * W;
      const bool isa = q < BM / 8;
      if (DMA) {
        const uint32_t v = whole || k0 + vk[i] < g.k ? voff[i] : OUT_OF_RANGE;
        dma16(v, isa ? ra : rb, (uint32_t)k0,
              (uint32_t)__builtin_amdgcn_readfirstlane(lds0 + (kt % S) * STAGE + q * 1024));
      } else {
        const int8_t* p = (isa ? A : B) + (int64_t)((isa ? q : q - BM / 8) * 8 + (lane >> 3)) * (isa ? g.lda : g.ldb);
        reg[i] = voff[i] != OUT_OF_RANGE ? load_chunk(p, k0 + vk[i], g.k) : intx4{0, 0, 0, 0};
      }
    }
  };
  auto store = [&](int kt) {   // registers to LDS
#pragma unroll
    for (int i = 0; i < NP; ++i) *(intx4*)(smem + (kt % S) * STAGE + (wave + i * W) * 1024 + lane * 16) = reg[i];
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
    if (DMA) {
      const int later = min(nk - 1, kt + S - 2) - kt;   // stages issued after kt
      if (S >= 4 && later >= 2) wait_vmcnt<2 * NP>();
      else if (S >= 3 && later >= 1) wait_vmcnt<NP>();
      else wait_vmcnt<0>();
    } else {
      store(kt);
    }
    lds_barrier();
    if (DMA) {
      if (kt + S - 1 < nk) issue(kt + S - 1);
    } else {
      if (kt + 1 < nk) issue(kt + 1);
    }
  };
  if (nk > 0) {
    if (DMA) {
#pragma unroll
      for (int i = 0; i < S - 1; ++i)
        if (i < nk) issue(i);
    } else {
      issue(0);
    }
    turn(0);
    fetch(0, 0, 0);
    for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
      for (int ks = 0; ks < BK / 32; ++ks) {
        if (ks + 1 < BK / 32) {
          fetch(kt, ks + 1, (ks + 1) & 1);
        } else if (kt + 1 < nk) {
          turn(kt + 1);
          fetch(kt + 1, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[ks & 1][j], fa[ks & 1][i], acc[i][j], 0, 0, 0);
      }
    }
  }
  __syncthreads();   // the stages are free: each wave stages 32 rows of its output at a time

  O* st = (O*)smem + wave * 32 * SROW;
  const int64_t cbase = n0 + wn * TN;
  constexpr int CPR = TN / OV;   // 16-byte pieces of a staged row
  const O* outp = (const O*)g.out;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t row = m0 + wm * TM + i * 32 + r;
    const float sa = row < g.m ? g.sa[row] : 0.f;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = j * 32 + q * 8 + (lane >> 5) * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t col = cbase + c + e;
          float v = 0.f;
          if (col < g.n) {
            v = (float)acc[i][j][q * 4 + e] * sa * g.sb[col];
            if (g.bias) v += load_fmt(g.bias, col, g.bias_fmt);
          }
          st[r * SROW + c + e] = from_f<O>(v);
        }
      }
    asm volatile("" : : : "memory");   // a wave's LDS accesses execute in order
#pragma unroll
    for (int q0 = 0; q0 < 32 * CPR; q0 += 64) {
      const int q = q0 + lane, rr = q / CPR, c = (q % CPR) * OV;
      const int64_t orow = m0 + wm * TM + i * 32 + rr, col = cbase + c;
      if (orow < g.m && col < g.n) {
        const O* s = st + rr * SROW + c;
        O* o = (O*)outp + orow * g.ldo + col;
        if (col + OV <= g.n) *(intx4u*)o = *(const intx4*)s;
        else
          for (int e = 0; col + e < g.n; ++e) o[e] = s[e];
      }
    }
    asm volatile("" : : : "memory");
  }
}

template <int BM, int BN, int WM, int WN, int S, bool DMA>
void launch_mma(const Int8Args& a, hipStream_t s) {
  const int64_t tiles = (a.m + BM - 1) / BM * ((a.n + BN - 1) / BN);
  const dim3 grid((unsigned)tiles), block(64 * WM * WN);
  if (a.out_fmt == 1) hipLaunchKernelGGL((k_int8_mma<BM, BN, WM, WN, S, DMA, float>), grid, block, 0, s, a);
  else if (a.out_fmt == 0) hipLaunchKernelGGL((k_int8_mma<BM, BN, WM, WN, S, DMA, bf16_t>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_int8_mma<BM, BN, WM, WN, S, DMA, fp16_t>), grid, block, 0, s, a);
}

}  // namespace

void launch_int8_linear(const Int8Args& a, hipStream_t s) {
  // copies straight into LDS need rows at multiples of 16 bytes, whole 16-byte
  // chunks and 31-bit offsets inside a tile
  const bool dma = ((uintptr_t)a.a | (uintptr_t)a.b | (uint64_t)a.lda | (uint64_t)a.ldb | (uint64_t)a.k) % 16 == 0 &&
                   a.lda < (1 << 22) && a.ldb < (1 << 22);
  const auto tiles = [&](int64_t t) { return (a.m + t - 1) / t * ((a.n + t - 1) / t); };
  if (!dma) launch_mma<128, 128, 2, 2, 2, false>(a, s);
  else if (tiles(256) >= 256) launch_mma<256, 256, 2, 2, 2, true>(a, s);
  else if (tiles(128) >= 128) launch_mma<128, 128, 2, 2, 2, true>(a, s);
  else launch_mma<64, 64, 2, 2, 4, true>(a, s);
}

}  // namespace dion
