// Layouts and splits that the low-rank kernels share (adapters.hip, block.hip).
#pragma once

#include "host.h"

namespace qnf4 {

// v as hi + mid + lo in bf16 (24 bits: products with it are as exact as fp32 ones).
__device__ __forceinline__ void split3(float v, uint16_t* o) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t h = pack_bf16x2(v, 0.0f) & 0xffffu;
    o[i] = (uint16_t)h;
    v = __fsub_rn(v, __uint_as_float(h << 16));
  }
}

// The 16-byte chunks of an LDS row of 2·NJ or 6·NJ of them (ranks) XORed by bits
// of the row, so that the 4 rows of a transposing read lie on different banks.
template <int NJ>
__device__ __forceinline__ int rank_swz(int row) {
  return NJ == 4 ? (row & 3) << 1 : NJ == 2 ? row & 2 : 0;
}
// Byte of 16-byte chunk `chunk` of a row of 128 bytes (64 reduction elements).
__device__ __forceinline__ int dswz(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }
// Byte of column col (a multiple of 4) of a row of 128 columns: chunk c at
// c ^ ((row & 3) << 1), the 4 rows of a transposing read on different banks.
__device__ __forceinline__ int gswz(int row, int col) {
  return row * 256 + (((col >> 3) ^ ((row & 3) << 1)) << 4) + 2 * (col & 7);
}

// Eight products of bf16 pairs added to acc.
__device__ __forceinline__ float dot8(const u32x4_t a, const u32x4_t b, float acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = __builtin_fmaf(bf16lo(a[i]), bf16lo(b[i]), acc);
    acc = __builtin_fmaf(bf16hi(a[i]), bf16hi(b[i]), acc);
  }
  return acc;
}

}  // namespace qnf4
