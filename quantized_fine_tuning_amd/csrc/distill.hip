// Distillation from a teacher's top logits, gfx950.  Per token, with z the
// student's logits over V columns, t the teacher's logits at the columns c_i:
//   p = softmax(t/tau) over the entries, q = softmax(z/tau) over the columns,
//   loss = w·tau²·Σ_i p_i·(log p_i − log q_{c_i}),
//   dZ[v] = ∂loss/∂z_v = w·tau·(q_v − Σ_{i: c_i = v} p_i).
// An entry whose column lies outside [0, V) is no entry; a token without
// entries, or of weight 0, has loss 0 and a zero gradient.
//
// A logit of −infinity (a masked column) has q = 0; a row whose largest logit
// lies below −1e30 (every column masked) has loss 0 and a zero gradient.
//
// One workgroup per token, everything in fp32.  With the row's maximum at
// hand the exponent is (z − max)·(log2 e/tau), off by two ulps of itself.
// From a saved log-sum-exp it is z/tau − lse, whose quotient is formed as a
// product with 1/tau in two parts: a rounded quotient would be off by an ulp
// of z/tau.
#include <algorithm>

#include "host.h"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;

enum { kF32 = 0, kBf16 = 1, kF16 = 2 };

template <int TYPE>
__device__ __forceinline__ float load_as_f32(const void* p, int64_t i) {
  if constexpr (TYPE == kF32) return static_cast<const float*>(p)[i];
  const uint16_t v = static_cast<const uint16_t*>(p)[i];
  return widen16<TYPE == kF16>(v);
}
template <int TYPE>
__device__ __forceinline__ void store_rounded(void* p, int64_t i, float v) {
  if constexpr (TYPE == kF32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = (uint16_t)(pack16<TYPE == kF16>(v, 0.f) & 0xffffu);
}

struct MaxOp {
  __device__ static float of(float a, float b) { return fmaxf(a, b); }
};
struct SumOp {
  __device__ static float of(float a, float b) { return a + b; }
};
// The same value in every thread; the waves' results combined in wave order.
template <typename OP>
__device__ __forceinline__ float block_reduce(float v, float* s) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = OP::of(v, __shfl_xor(v, o, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = s[0];
  for (int w = 1; w < (int)blockDim.x / 64; ++w) v = OP::of(v, s[w]);
  return v;
}

constexpr float kMasked = -1e30f;
constexpr float kLog2e = 1.44269504f;

// Exponentials of one row: e(z) = exp(z/tau − reference).
struct RowExp {
  bool saved;          // reference: the saved log-sum-exp, else the maximum
  float ref, c;        // c = log2(e)/tau
  float ihi, ilo;      // 1/tau in two parts
  __device__ __forceinline__ float operator()(float z) const {
    if (!saved) return __builtin_amdgcn_exp2f((z - ref) * c);
    z = fmaxf(z, kMasked);  // (−infinity would give inf − inf below)
    const float hi = __fmul_rn(z, ihi);
    const float lo = __builtin_fmaf(z, ilo, __builtin_fmaf(z, ihi, -hi));
    return __builtin_amdgcn_exp2f(((hi - ref) + lo) * kLog2e);
  }
};

template <int ZT, int TT>
__global__ __launch_bounds__(kThreads) void distill_kernel(DistillArgs a, float c, float ihi, float ilo) {
  __shared__ float s_p[kMaxTop];
  __shared__ float s_z[kMaxTop];
  __shared__ int s_c[kMaxTop];
  __shared__ float s_red[kThreads / 64];
  const int tid = threadIdx.x;
  const int64_t m = blockIdx.x;
  const int64_t row = m * a.ldz;
  // the entries
  float t_max = -INFINITY;
  for (int i = tid; i < a.k; i += kThreads) {
    const int col = a.at[m * a.k + i];
    const bool ok = col >= 0 && col < a.V;
    const float t = ok ? load_as_f32<TT>(a.top, m * a.k + i) / a.tau : -INFINITY;
    s_c[i] = ok ? col : -1;
    s_z[i] = ok ? load_as_f32<ZT>(a.Z, row + col) : 0.f;
    s_p[i] = t;
    t_max = fmaxf(t_max, t);
  }
  t_max = block_reduce<MaxOp>(t_max, s_red);
  const bool entries = t_max > -INFINITY;
  float t_sum = 0.f;
  for (int i = tid; i < a.k; i += kThreads) t_sum += entries ? expf(s_p[i] - t_max) : 0.f;
  t_sum = block_reduce<SumOp>(t_sum, s_red);
  const float w = a.weight ? a.weight[m] : 1.0f;

  // the row's reference and the sum of its exponentials
  RowExp e{a.lse_in != nullptr, 0.f, c, ihi, ilo};
  float inv = 1.0f, lse;
  bool columns = true;
  if (e.saved) {
    e.ref = lse = a.lse_in[m];
    columns = lse > -INFINITY;
  } else {
    float z_max = -INFINITY;
    for (int64_t v = tid; v < a.V; v += kThreads) z_max = fmaxf(z_max, load_as_f32<ZT>(a.Z, row + v));
    e.ref = z_max = block_reduce<MaxOp>(z_max, s_red);
    columns = z_max > kMasked;
    float sum = 0.f;
    for (int64_t v = tid; v < a.V; v += kThreads) sum += e(load_as_f32<ZT>(a.Z, row + v));
    sum = block_reduce<SumOp>(sum, s_red);
    inv = 1.0f / sum;
    lse = columns ? z_max / a.tau + logf(sum) : -INFINITY;
    if (a.lse && tid == 0) a.lse[m] = lse;
  }
  const bool live = entries && columns && w != 0.f;
  if (a.loss) {
    const float log_sum = live ? logf(t_sum) : 0.f;
    float loss = 0.f;
    if (live)
      for (int i = tid; i < a.k; i += kThreads) {
        const float p = expf(s_p[i] - t_max) / t_sum;
        if (p > 0.f) loss += p * (s_p[i] - t_max - log_sum - (s_z[i] / a.tau - lse));
      }
    loss = block_reduce<SumOp>(loss, s_red);
    if (tid == 0) a.loss[m] = live ? w * a.tau * a.tau * loss : 0.f;
  }
  if (!a.dZ) return;
  const float g = w * a.tau;
  for (int64_t v = tid; v < a.ldz; v += kThreads) {
    float d = 0.f;
    if (live && v < a.V) d = g * (e(load_as_f32<ZT>(a.Z, row + v)) * inv);
    store_rounded<ZT>(a.dZ, row + v, d);
  }
  if (!live) return;
  // the entries' columns once more, the teacher's share taken off (the first
  // of several entries of one column takes all of theirs)
  __threadfence_block();
  __syncthreads();
  for (int i = tid; i < a.k; i += kThreads) {
    const int col = s_c[i];
    bool first = col >= 0;
    float p = 0.f;
    for (int o = 0; o < a.k; ++o)
      if (s_c[o] == col) {
        if (o < i) first = false;
        p += expf(s_p[o] - t_max) / t_sum;
      }
    if (first) store_rounded<ZT>(a.dZ, row + col, g * (e(s_z[i]) * inv - p));
  }
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, int z_type, int t_type, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  const double i = 1.0 / (double)a.tau;
  const float c = (float)(1.4426950408889634 * i), ihi = (float)i, ilo = (float)(i - (double)ihi);
#define QNF4_DISTILL(ZT, TT) \
  if (z_type == ZT && t_type == TT) distill_kernel<ZT, TT><<<(unsigned)a.M, kThreads, 0, st>>>(a, c, ihi, ilo);
  QNF4_DISTILL(kF32, kF32)
  QNF4_DISTILL(kF32, kBf16)
  QNF4_DISTILL(kF32, kF16)
  QNF4_DISTILL(kBf16, kF32)
  QNF4_DISTILL(kBf16, kBf16)
  QNF4_DISTILL(kBf16, kF16)
  QNF4_DISTILL(kF16, kF32)
  QNF4_DISTILL(kF16, kBf16)
  QNF4_DISTILL(kF16, kF16)
#undef QNF4_DISTILL
  return hipGetLastError();
}

}  // namespace qnf4
