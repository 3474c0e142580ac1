// One step of the sum of split-reduction partials (see splitk.hip).
#pragma once

#include "common.h"

namespace qnf4 {

// out[4i .. 4i + 3] = P[0] + P[1] + ..., added in split order in fp32.
template <bool F16>
__device__ __forceinline__ void splitk_sum4(const f32x4_t* __restrict__ P, int splits, int64_t n4, int64_t i,
                                            void* __restrict__ out, int out16) {
  f32x4_t a = __builtin_nontemporal_load(P + i);
  // the loads of four partials are issued before their adds
  for (int s = 1; s < splits; s += 4) {
    f32x4_t b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // an existing partial whatever q, so that the loads are unconditional
      const int sq = s + q < splits ? s + q : splits - 1;
      b[q] = __builtin_nontemporal_load(P + (int64_t)sq * n4 + i);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (s + q < splits) {
        a[0] = a[0] + b[q][0];
        a[1] = a[1] + b[q][1];
        a[2] = a[2] + b[q][2];
        a[3] = a[3] + b[q][3];
      }
  }
  if (out16) {
    u32x2_t o;
    o[0] = pack16<F16>(a[0], a[1]);
    o[1] = pack16<F16>(a[2], a[3]);
    static_cast<u32x2_t*>(out)[i] = o;
  } else {
    static_cast<f32x4_t*>(out)[i] = a;
  }
}

}  // namespace qnf4
