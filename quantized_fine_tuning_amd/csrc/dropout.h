// Dropout of an adapter's input from a counter-based generator: Philox4x32-10 of
// Salmon, Moraes, Dror and Shaw (2011), whose 128 bits for the key `seed` and the
// counter (i / 8, offset) are the eight 16-bit pieces of elements 8(i/8) .. +7 of
// a tensor.  Element i is kept where its piece is at least `out` of 65,536.  The
// mask is computed where it is needed and stored nowhere.
#pragma once

#include "host.h"

namespace qnf4 {

// The dropout of a kernel's run, its offset as of now.
__device__ __forceinline__ DropView drawn(DropView d) {
  if (d.step) {
    const uint64_t o = ((uint64_t)d.off1 << 32 | d.off0) + *d.step;
    d.off0 = (uint32_t)o;
    d.off1 = (uint32_t)(o >> 32);
  }
  return d;
}

// One call is 20 widening multiplications (v_mad_u64_u32, a quarter of the rate) and
// as many pairs of xors: 108 ns of a SIMD for a wave's 512 elements, 153 with their
// eight comparisons (keep8).  With the two halves of each product found apart 143.
__device__ __forceinline__ u32x4_t philox(const DropView& d, uint32_t chunk) {
  uint32_t c0 = chunk, c1 = 0u, c2 = d.off0, c3 = d.off1, k0 = d.key0, k1 = d.key1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{c0, c1, c2, c3};
}

// Eight 16-bit values with zeros in the place of those that the generator's bits
// of their chunk drop (whatever those are: NaN and infinities go too).
__device__ __forceinline__ u32x4_t drop8(const DropView& d, u32x4_t bits, u32x4_t v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t low = (bits[i] & 0xffffu) >= d.out ? 0xffffu : 0u;
    v[i] &= low | (bits[i] >> 16 >= d.out ? 0xffff0000u : 0u);
  }
  return v;
}

// Bit e: whether element e of the chunk is kept.
__device__ __forceinline__ uint32_t keep8(const DropView& d, uint32_t chunk) {
  const u32x4_t bits = philox(d, chunk);
  const uint32_t out = d.out << 16;
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m |= (bits[i] << 16 >= out ? 1u << (2 * i) : 0u) | (bits[i] >= out ? 2u << (2 * i) : 0u);
  return m;
}

}  // namespace qnf4
