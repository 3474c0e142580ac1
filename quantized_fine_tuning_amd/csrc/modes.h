// What the dequant-in-tile GEMMs (fwd.hip, dx.hip) run for, beside the plain
// layer: tokens that carry different adapters, one layer whose adapter's input
// has dropout, or the two layers of a gated block.
#pragma once

#include <type_traits>

#include "host.h"

namespace qnf4 {

constexpr int kPlain = 0, kMulti = 1, kBlock1 = 2, kBlock2 = 3;
template <int MODE>
using ModeArgs = std::conditional_t<MODE == kMulti, AdapterGemmArgs,
                                    std::conditional_t<MODE == kPlain, NoAdapters, BlockGemmArgs>>;

// The weight of the first or the second layer.
template <typename Args>
__device__ __forceinline__ Nf4View layer(const Nf4View& W, const Args& a, bool second) {
  if constexpr (std::is_same_v<Args, BlockGemmArgs>)
    return second ? a.W2 : W;
  else
    return W;
}

}  // namespace qnf4
