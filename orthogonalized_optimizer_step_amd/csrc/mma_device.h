// What the products on narrow operands (8-bit integers, 4-bit floating point)
// share: copies straight into LDS and the order of their bytes there, loads at
// a row's end, the tiles' order.
#pragma once

#include "train_device.h"

namespace dion {

typedef int intx16 __attribute__((ext_vector_type(16)));
// sixteen bytes at any alignment
typedef intx4 intx4u __attribute__((aligned(1)));

constexpr int BK = 128;   // bytes of k in a stage: one cache line of each row

// Position of 16-byte chunk c of row r in its 128-byte LDS row: any 8
// consecutive rows reading one chunk touch all 128 bytes, any 16 both halves
// of 256, so the fragment reads meet no bank twice.
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

// 16 bytes of a row from k on, zeros from `ks` on: at the row's end its last
// 16 bytes, moved down
__device__ __forceinline__ intx4 load_chunk(const int8_t* row, int k, int ks) {
  if (k + 16 <= ks) return *(const intx4u*)(row + k);
  intx4 v = {0, 0, 0, 0};
  if (k >= ks) return v;
  if (ks >= 16) {
    union { intx4 v; uint64_t u[2]; } c;
    c.v = *(const intx4u*)(row + ks - 16);
    const int bits = 8 * (k + 16 - ks);   // 8 .. 120
    if (bits < 64) c.u[0] = c.u[0] >> bits | c.u[1] << (64 - bits);
    else c.u[0] = c.u[1] >> (bits - 64);
    c.u[1] = bits < 64 ? c.u[1] >> bits : 0;
    return c.v;
  }
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

}  // namespace dion
