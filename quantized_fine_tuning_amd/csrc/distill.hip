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
//
// Bound by HBM: a row is read once and its gradient written once.  The row
// stays in registers between the two (VECS 16-byte chunks a thread, the
// loads of all of them in flight together), so maximum, sum and gradient
// need no second read; a row of more than 16,384 chunks is read once for an
// online maximum and sum and once more (from the caches) for the gradient.
// Chunks are those of the tensor's own 16-byte grid, so that rows of any
// alignment load and store whole chunks except at their two ends.  The
// entries are wave 0's work, beside the row's loads: it leaves the
// probabilities in LDS and keeps the loss to itself, so a row costs three
// barriers.
#include <algorithm>

#include "host.h"

namespace qnf4 {
namespace {

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

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// The elements of one 16-byte chunk.
template <int TYPE>
struct Chunk {
  static constexpr int N = TYPE == kF32 ? 4 : 8;
  __device__ __forceinline__ static float get(const u32x4_t& v, int i) {
    if constexpr (TYPE == kF32)
      return __uint_as_float(v[i]);
    else if constexpr (TYPE == kF16)
      return widen16<true>(i & 1 ? v[i >> 1] >> 16 : v[i >> 1] & 0xffffu);
    else
      return i & 1 ? bf16hi(v[i >> 1]) : bf16lo(v[i >> 1]);
  }
  __device__ __forceinline__ static u32x4_t pack(const float* f) {
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kF32)
        o[i] = __float_as_uint(f[i]);
      else
        o[i] = pack16<TYPE == kF16>(f[2 * i], f[2 * i + 1]);
    }
    return o;
  }
};

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

// VECS > 0: the row's chunks in registers, VECS per thread of T; VECS == 0:
// any number of chunks, read again for the gradient.  SAVED: the row's
// log-sum-exp is given.
template <int ZT, int TT, int T, int VECS, bool SAVED>
__global__ __launch_bounds__(T) void distill_kernel(DistillArgs a, float c, float ihi, float ilo) {
  using C = Chunk<ZT>;
  constexpr int kWaves = T / 64, kPer = kMaxTop / 64;
  constexpr int64_t kSize = ZT == kF32 ? 4 : 2;
  __shared__ float s_p[kMaxTop], s_z[kMaxTop];
  __shared__ __attribute__((aligned(16))) int s_c[kMaxTop];
  __shared__ float s_max[kWaves], s_sum[kWaves], s_entry[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t m = blockIdx.x;
  // the row on the tensor's 16-byte grid: `head` elements of its first chunk
  // belong to the row before
  const int64_t row = m * a.ldz;
  const int head = (int)(row & (C::N - 1));
  const char* const zc = static_cast<const char*>(a.Z) + (row - head) * kSize;
  const int V = (int)a.V, ld = (int)a.ldz;
  // (up to a whole dword: one that reaches past the end would read as zero
  // altogether; the dword's other half is never used)
  const rsrc_t rz = make_rsrc(zc, round_up((a.M * a.ldz - (row - head)) * kSize, 4));
  const int chunks = (head + V + C::N - 1) / C::N;       // that hold columns
  const int chunks_out = (head + ld + C::N - 1) / C::N;  // that hold the padding too
  auto load = [&](int i) __attribute__((always_inline)) {
    return buf_load16(rz, i < chunks ? (uint32_t)i * 16u : 0x7fffffffu, 0u);
  };
  // element e of chunk i is a column of this row
  auto whole = [&](int i) __attribute__((always_inline)) {
    return i * C::N >= head && (i + 1) * C::N <= head + V;
  };
  auto column = [&](int i, int e) __attribute__((always_inline)) {
    const int v = i * C::N + e - head;
    return v >= 0 && v < V;
  };
  constexpr int NV = VECS > 0 ? VECS : 1;
  u32x4_t z[NV];
  if constexpr (VECS > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) z[j] = load(tid + j * T);
  }

  // the entries (wave 0; entry 64q + lane)
  float t_max = -INFINITY, t_sum = 0.f;
  float t[kPer], zt[kPer];
  if (wave == 0) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = 64 * q + lane;
      t[q] = -INFINITY;
      zt[q] = 0.f;
      if (64 * q < a.k && i < a.k) {
        const int col = a.at[m * a.k + i];
        const bool ok = col >= 0 && col < V;
        if (ok) {
          t[q] = load_as_f32<TT>(a.top, m * a.k + i) / a.tau;
          zt[q] = load_as_f32<ZT>(a.Z, row + col);
        }
        s_c[i] = ok ? col : -1;
        s_z[i] = zt[q];
      }
      t_max = fmaxf(t_max, t[q]);
    }
    t_max = wave_max(t_max);
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (64 * q < a.k) t_sum += t_max > -INFINITY ? expf(t[q] - t_max) : 0.f;
    t_sum = wave_sum(t_sum);
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (64 * q + lane < a.k) s_p[64 * q + lane] = t_max > -INFINITY ? expf(t[q] - t_max) / t_sum : 0.f;
    if (lane == 0) s_entry[0] = t_max;
  }

  // the row's reference and the sum of its exponentials
  RowExp e{SAVED, 0.f, c, ihi, ilo};
  float inv = 1.0f, lse;
  bool columns;
  if constexpr (SAVED) {
    e.ref = lse = a.lse_in[m];
    columns = lse > -INFINITY;
    __syncthreads();
  } else {
    float z_max = -INFINITY, sum = 0.f;
    if constexpr (VECS > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = tid + j * T;
        if (whole(i)) {
#pragma unroll
          for (int k = 0; k < C::N; ++k) z_max = fmaxf(z_max, C::get(z[j], k));
        } else {
#pragma unroll
          for (int k = 0; k < C::N; ++k) z_max = fmaxf(z_max, column(i, k) ? C::get(z[j], k) : -INFINITY);
        }
      }
    } else {
      // running maximum and sum of this thread's chunks
      for (int i = tid; i < chunks; i += T) {
        const u32x4_t v = load(i);
        float f[C::N], high = -INFINITY;
#pragma unroll
        for (int k = 0; k < C::N; ++k) {
          f[k] = column(i, k) ? C::get(v, k) : -INFINITY;
          high = fmaxf(high, f[k]);
        }
        if (high > z_max) {
          sum *= z_max > kMasked ? __builtin_amdgcn_exp2f((z_max - high) * c) : 0.f;
          z_max = high;
        }
        e.ref = z_max;
        if (z_max > kMasked) {
#pragma unroll
          for (int k = 0; k < C::N; ++k) sum += e(f[k]);
        }
      }
    }
    const float own_max = z_max;
    z_max = wave_max(z_max);
    if (lane == 0) s_max[wave] = z_max;
    __syncthreads();
    z_max = s_max[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) z_max = fmaxf(z_max, s_max[w]);
    e.ref = z_max;
    columns = z_max > kMasked;
    if constexpr (VECS > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = tid + j * T;
        if (whole(i)) {
#pragma unroll
          for (int k = 0; k < C::N; ++k) sum += e(C::get(z[j], k));
        } else {
#pragma unroll
          for (int k = 0; k < C::N; ++k) sum += column(i, k) ? e(C::get(z[j], k)) : 0.f;
        }
      }
    } else {
      sum *= own_max > kMasked ? e(own_max) : 0.f;
    }
    sum = wave_sum(sum);
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    sum = s_sum[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += s_sum[w];
    inv = 1.0f / sum;
    lse = columns ? z_max / a.tau + logf(sum) : -INFINITY;
    if (a.lse && tid == 0) a.lse[m] = lse;
  }
  const float w = a.weight ? a.weight[m] : 1.0f;
  const bool live = columns && w != 0.f && s_entry[0] > -INFINITY;
  if (a.loss && wave == 0) {
    const float log_sum = logf(t_sum);
    float loss = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = 64 * q + lane;
      if (i < a.k && live) {
        const float p = s_p[i];
        if (p > 0.f) loss += p * (t[q] - t_max - log_sum - (zt[q] / a.tau - lse));
      }
    }
    loss = wave_sum(loss);
    if (lane == 0) a.loss[m] = live ? w * a.tau * a.tau * loss : 0.f;
  }
  if (!a.dZ) return;

  const float g = w * a.tau, gi = g * inv;
  char* const dc = static_cast<char*>(a.dZ) + (row - head) * kSize;
  auto store = [&](int i, const u32x4_t& v) __attribute__((always_inline)) {
    float f[C::N];
    if (whole(i)) {
#pragma unroll
      for (int k = 0; k < C::N; ++k) f[k] = live ? gi * e(C::get(v, k)) : 0.f;
      *reinterpret_cast<u32x4_t*>(dc + (int64_t)i * 16) = C::pack(f);
    } else {
      // an end of the row: element by element, zeros in the padding
#pragma unroll
      for (int k = 0; k < C::N; ++k) {
        const int col = i * C::N + k - head;
        if (col >= 0 && col < ld) store_rounded<ZT>(a.dZ, row + col, live && col < V ? gi * e(C::get(v, k)) : 0.f);
      }
    }
  };
  if constexpr (VECS > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (tid + j * T < chunks) store(tid + j * T, z[j]);
  } else {
    for (int i = tid; i < chunks; i += T) store(i, load(i));
  }
  for (int i = chunks + tid; i < chunks_out; i += T) store(i, u32x4_t{0u, 0u, 0u, 0u});
  if (!live) return;
  // the entries' columns once more, the teacher's share taken off (the first
  // of several entries of one column takes all of theirs)
  __threadfence_block();
  __syncthreads();
  for (int i = tid; i < a.k; i += T) {
    const int col = s_c[i];
    bool first = col >= 0;
    float p = 0.f;
    for (int o = 0; o < a.k; ++o)
      if (s_c[o] == col) {
        if (o < i) first = false;
        p += s_p[o];
      }
    if (first) store_rounded<ZT>(a.dZ, row + col, g * (e(s_z[i]) * inv - p));
  }
}

template <int ZT, int TT, bool SAVED>
void launch(const DistillArgs& a, float c, float ihi, float ilo, hipStream_t st) {
  constexpr int N = Chunk<ZT>::N;
  const int64_t chunks = (a.V + 2 * (N - 1)) / N;  // whatever the row's alignment
  const unsigned grid = (unsigned)a.M;
  // 512 threads and as few chunks a thread as hold the row; from 8,192 chunks
  // on 1,024 threads
#define QNF4_ROW(T, VECS) distill_kernel<ZT, TT, T, VECS, SAVED><<<grid, T, 0, st>>>(a, c, ihi, ilo)
  if (chunks <= 512)
    QNF4_ROW(512, 1);
  else if (chunks <= 1024)
    QNF4_ROW(512, 2);
  else if (chunks <= 2048)
    QNF4_ROW(512, 4);
  else if (chunks <= 4096)
    QNF4_ROW(512, 8);
  else if (chunks <= 8192)
    QNF4_ROW(512, 16);
  else if (chunks <= 16384)
    QNF4_ROW(1024, 16);
  else
    QNF4_ROW(1024, 0);
#undef QNF4_ROW
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, int z_type, int t_type, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  const double i = 1.0 / (double)a.tau;
  const float c = (float)(1.4426950408889634 * i), ihi = (float)i, ilo = (float)(i - (double)ihi);
#define QNF4_DISTILL(ZT, TT)                     \
  if (z_type == ZT && t_type == TT) {            \
    if (a.lse_in)                                \
      launch<ZT, TT, true>(a, c, ihi, ilo, st);  \
    else                                         \
      launch<ZT, TT, false>(a, c, ihi, ilo, st); \
  }
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
