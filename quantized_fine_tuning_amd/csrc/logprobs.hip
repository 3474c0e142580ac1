// Log-probabilities of given tokens, entropies, the most likely tokens, and
// their gradient, gfx950.  Per token, with z its logits over V columns and t the
// given column:
//   q = softmax(z/tau),  logp = log q_t,  H = −Σ_v q_v·log q_v,
//   dZ[v] = (g·([v = t] − q_v) − h·q_v·(log q_v + H))/tau
// for the gradients g of logp and h of H.  A column outside [0, V) is no token:
// logp 0, and g counts as 0.
//
// Masks and NaN are the distillation kernels': a logit of −infinity has q = 0; a
// row whose largest logit lies below −1e30 has no columns (logp, H and the
// gradient 0, lse −infinity); NaN passes through maxima unseen and shows in the
// sums.  A logit below −1e30 is no alternative among the most likely.
//
// Everything in fp32, exponents in base 2 with c = log2(e)/tau: x = (z − max)·c, S =
// Σ 2^x, W = Σ x·2^x; then
//   logp = x_t·ln 2 − ln S,  H = ln S − ln 2·W/S.
// The difference comes first, so that x is 0 at the maximum wherever the row lies.
// A row in registers takes x = fma(z, c, −rc) with rc = fl(max·c), one operation in place
// of two (values and entropy of 4096 x 32000 bf16 40.0 us against 41.0): every x and log2 S
// are off alike by what rc was rounded by, and no result sees it, 2^-6 at most below
// |rc| = 2^19 (`far` is what lies beyond, a mask of −1e10, say).  In far rows of 16-bit
// logits none but the maximum has a share that fp32 holds: the next lies 2^-11 of |max|
// or more below, 256 and more times 1/c.  There c becomes the power of two that puts
// |rc| into [2^19, 2^20), so that rc is exact, x 0 at the maximum and −256 or less
// elsewhere.  Far rows of 32 bits take the maximum off their registers first.  Of far
// rows log q is found from the difference.  Rows too long for registers have the
// difference throughout.
//
// Forward, with or without the gradient: one workgroup per token, the row in
// registers between its passes (or, too long for that, read again from the
// caches).  4096 x 32000 bf16 with the gradient 100 us, 524 MB at 5.2 TB/s, more than a
// large copy's rate; the values alone 40.  Few rows are latency: 32 x 32000 4.5 us, with
// 20 alternatives and entropy 9.0.
//
// The k most likely columns, equal logits by their index: every thread's largest
// logit is known from the maximum, and the k-th largest of those is a bound that
// at least k columns reach and few more do.  Those go to a list in LDS whose
// order is then found by counting, so that it does not depend on who came first.
// Where a wave has more of them than its part of the list holds (equal logits, or
// likely columns side by side, as where logits fall with the index), the k-th largest
// is found bit by bit, and so is the last index among its equals, in 62 passes over
// the row (32 x 32000, k = 64, such logits 242 us, independent ones 11).
//
// Gradient from a saved log-sum-exp (and entropy): no sums over the row, so rows
// are cut into parts of 2,048 chunks, a workgroup each; log2 q takes z·c −
// lse·log2(e) in two parts each (rounded ones would be off by an ulp of z/tau).  777 x
// 50001 fp32 66 us, 311 MB at 4.7 TB/s.
#include <type_traits>

#include "host.h"
#include "rows.h"

namespace qnf4 {
namespace {

constexpr float kLn2 = 0.693147182f;

// An order of floats as unsigned numbers (−0 and +0 equal; NaN lowest).
__device__ __forceinline__ uint32_t order_of(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// the lowest that is an alternative: the float above kMasked
constexpr uint32_t kLowest = ~0xf149f2cau + 1u;

constexpr int kCandidates = 2048;
struct Candidates {
  alignas(16) uint32_t key[kCandidates + 8];
  alignas(16) int col[kCandidates + 8];
  int n;
  uint32_t bound;
  int count[16];
  // what each wave found, before it is put together
  uint32_t wave_key[kCandidates];
  int wave_col[kCandidates];
};

// Σ over the workgroup of a per-thread count.
template <int T>
__device__ __forceinline__ int block_count(int n, int* s) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = n;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < T / 64; ++w) all += s[w];
  return all;
}

// Fills `s` with the columns among which the k first are (those alone, or all there
// are if fewer than k).  `each` calls its argument with (logit, column) of this
// thread's columns, every lane of a wave together, in chunks where some lane reaches
// the bound; `again` with (order, column) of every column, read from memory (for the
// rare row: it takes no registers).  The bound is found to the order's 14 high bits
// (sign, exponent, five of the mantissa): lower by 3 % at most, a few columns more.
// Twice as many maxima as columns asked for bound them nearly as well as all, in fewer
// comparisons (k = 20 of 32 rows of 32000 8.9 us against 9.8).
// Every wave lists what it finds by itself: with one counter for all, each of its
// columns waited for an atomic (32 rows of 32000, k = 20: 11.3 us, then 9.8).
template <int T, typename Each, typename Again>
__device__ __forceinline__ void find_top(Candidates& s, int k, float own_max, Each&& each, Again&& again) {
  constexpr int kWaves = T / 64, kOwn = kCandidates / kWaves;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  s.key[tid] = order_of(own_max);
  __syncthreads();
  if (tid < 64) {
    uint32_t own[T / 64], bound = 0u;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) own[i] = s.key[lane + 64 * i];
    // the maxima of 64·G groups of threads
    auto search = [&](auto groups) __attribute__((always_inline)) {
      constexpr int G = decltype(groups)::value < T / 64 ? decltype(groups)::value : T / 64;
      uint32_t most[G] = {};
#pragma unroll
      for (int i = 0; i < T / 64; ++i) most[i % G] = most[i % G] > own[i] ? most[i % G] : own[i];
      for (int b = 31; b >= 18; --b) {
        const uint32_t next = bound | 1u << b;
        int n = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) n += __popcll(__ballot(most[i] >= next));
        if (n >= k) bound = next;
      }
    };
    if (k <= 32)
      search(std::integral_constant<int, 1>());
    else if (k <= 64)
      search(std::integral_constant<int, 2>());
    else
      search(std::integral_constant<int, 16>());
    if (lane == 0) s.bound = bound > kLowest ? bound : kLowest;
  }
  __syncthreads();
  const float bound = of_order(s.bound);
  int found = 0;
  each(bound, [&](float v, int col) __attribute__((always_inline)) {
    const bool in = v >= bound;
    const uint64_t mask = __ballot(in);
    if (mask == 0) return;
    const int at = found + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
    if (in && at < kOwn) {
      s.wave_key[wave * kOwn + at] = order_of(v);
      s.wave_col[wave * kOwn + at] = col;
    }
    found += __popcll(mask);
  });
  if (lane == 0) s.count[wave] = found;
  __syncthreads();
  int before = 0, all = 0;
  bool fits = true;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int n = s.count[w];
    before += w < wave ? n : 0;
    all += n;
    fits = fits && n <= kOwn;
  }
  if (fits) {
    for (int i = lane; i < found; i += 64) {
      s.key[before + i] = s.wave_key[wave * kOwn + i];
      s.col[before + i] = s.wave_col[wave * kOwn + i];
    }
    if (tid == 0) s.n = all;
    __syncthreads();
    return;
  }
  auto put = [&](uint32_t key, int col) __attribute__((always_inline)) {
    const int at = atomicAdd(&s.n, 1);
    if (at < kCandidates) {
      s.key[at] = key;
      s.col[at] = col;
    }
  };
  // the k-th largest, then the last index of those equal to it that are taken
  uint32_t kth = 0u;
  for (int b = 31; b >= 0; --b) {
    const uint32_t next = kth | 1u << b;
    int n = 0;
    again([&](uint32_t key, int) __attribute__((always_inline)) { n += key >= next; });
    if (block_count<T>(n, s.count) >= k) kth = next;
  }
  int n = 0;
  again([&](uint32_t key, int) __attribute__((always_inline)) { n += key > kth; });
  int need = k - block_count<T>(n, s.count);
  if (kth < kLowest) {  // fewer than k in all: everything above
    kth = kLowest - 1;
    need = 0;
  }
  int last = need > 0 ? 0 : -1;  // the least bound below which `need` of them lie
  for (int b = 28; b >= 0; --b) {
    const int next = last | 1 << b;
    n = 0;
    again([&](uint32_t key, int col) __attribute__((always_inline)) { n += key == kth && col < next; });
    if (block_count<T>(n, s.count) < need) last = next;
  }
  __syncthreads();
  if (tid == 0) s.n = 0;
  __syncthreads();
  again([&](uint32_t key, int col) __attribute__((always_inline)) {
    if (key > kth || (key == kth && col <= last)) put(key, col);
  });
  __syncthreads();
}

// VECS > 0: the row's chunks in registers, VECS per thread of T; VECS == 0: any
// number of chunks, two in flight per thread, read again for every further pass.
// DOT: with W, for the entropy or its gradient; TOP: with the most likely columns.
// (Registers of one variant would halve the workgroups that the others have
// resident: 4096 x 32000 bf16 with gradient took 155 us with all in one kernel.)
template <int ZT, int T, int VECS, bool DOT, bool TOP>
__global__ __launch_bounds__(T, T == 1024 && (ZT != kF32 || VECS == 0) && !TOP ? 8 : 1) void logprobs_kernel(
    LogprobsArgs a, float c) {
  using C = Chunk<ZT>;
  constexpr int kWaves = T / 64;
  __shared__ float s_max[kWaves], s_sum[kWaves], s_dot[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t m = blockIdx.x;
  const Row<ZT> R(a.Z, a.dZ, a.M, a.V, a.ldz, m);
  constexpr int NV = VECS > 0 ? VECS : 2;
  u32x4_t z[NV];
  if constexpr (VECS > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) z[j] = R.load(tid + j * T);
  }
  const int target = a.target[m];
  const bool has = target >= 0 && target < R.V;
  const float zt = load_as_f32<ZT>(a.Z, R.row + (has ? target : 0));

  auto chunk_max = [&](const u32x4_t& v, float high) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < C::N; k += 2) high = max3(high, C::get(v, k), C::get(v, k + 1));
    return high;
  };
  // (ref: the maximum, 0 while every column is masked; cr, rc, far: as above)
  float ref = 0.f, cr = c, rc = 0.f, sum = 0.f, dot = 0.f;
  bool far = VECS == 0;
  // the exponent of a logit, and of one of the registers'
  auto x_of = [&](float v) __attribute__((always_inline)) {
    return VECS == 0 || (ZT == kF32 && far) ? (v - ref) * c : __builtin_fmaf(v, cr, -rc);
  };
  auto x = [&](float v) __attribute__((always_inline)) { return VECS == 0 ? (v - ref) * c : __builtin_fmaf(v, cr, -rc); };
  // (a masked column's x is −infinity, which times its 2^x of 0 would be NaN)
  auto chunk_sum = [&](const u32x4_t& v) __attribute__((always_inline)) {
    if constexpr (DOT) {
#pragma unroll
      for (int k = 0; k < C::N; ++k) {
        const float xk = x(C::get(v, k)), e = __builtin_amdgcn_exp2f(xk);
        sum += e;
        dot = __builtin_fmaf(fmaxf(xk, kMasked), e, dot);
      }
    } else {
#pragma unroll
      for (int k = 0; k < C::N; ++k) sum += __builtin_amdgcn_exp2f(x(C::get(v, k)));
    }
  };
  // the sums over ref as sums over v
  auto rescale = [&](bool some, float v) __attribute__((always_inline)) {
    const float before = ref;
    ref = v > kMasked ? v : 0.f;
    const float down = fmaxf((before - ref) * c, kMasked), f = some ? __builtin_amdgcn_exp2f(down) : 0.f;
    if constexpr (DOT) dot = some ? f * __builtin_fmaf(down, sum, dot) : 0.f;
    sum *= f;
  };
  float z_max = -INFINITY;
  if constexpr (VECS > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      z[j] = R.only_columns(tid + j * T, z[j]);
      z_max = chunk_max(z[j], z_max);
    }
  } else {
    // running maximum and sums of this thread's chunks
    for (int i0 = tid; i0 < R.chunks; i0 += NV * T) {
#pragma unroll
      for (int j = 0; j < NV; ++j) z[j] = R.load(i0 + j * T);
      float high = z_max;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        z[j] = R.only_columns(i0 + j * T, z[j]);
        high = chunk_max(z[j], high);
      }
      if (high > z_max) {
        rescale(z_max > kMasked, high);
        z_max = high;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) chunk_sum(opaque(z[j]));
    }
  }
  const float own_max = z_max;
  z_max = wave_max(z_max);
  if (lane == 0) s_max[wave] = z_max;
  __syncthreads();
  z_max = s_max[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) z_max = fmaxf(z_max, s_max[w]);
  const bool masked = !(z_max > kMasked);
  if constexpr (VECS > 0) {
    ref = uniform(masked ? 0.f : z_max);
    rc = __fmul_rn(ref, c);
    far = fabsf(rc) >= kFarRow;
    if constexpr (ZT != kF32) {
      cr = uniform(far ? far_scale(ref) : c);
      rc = __fmul_rn(ref, cr);
    } else if (far) {
      rc = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[j][k] = __float_as_uint(__uint_as_float(z[j][k]) - ref);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) chunk_sum(z[j] = opaque(z[j]));
  } else {
    rescale(own_max > kMasked, z_max);  // (a NaN among masked columns stays in the sum)
  }
  sum = wave_sum(sum);
  if constexpr (DOT) dot = wave_sum(dot);
  if (lane == 0) {
    s_sum[wave] = sum;
    if constexpr (DOT) s_dot[wave] = dot;
  }
  __syncthreads();
  sum = s_sum[0];
  if constexpr (DOT) dot = s_dot[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    sum += s_sum[w];
    if constexpr (DOT) dot += s_dot[w];
  }
  // (maxima pass over NaN: where they say that every column is masked the sum has
  // the last word, zero for masked columns, NaN where one is NaN)
  const bool columns = !masked || sum != 0.f;
  const float log_sum = logf(sum), inv = 1.0f / sum;
  const float entropy = columns ? log_sum - kLn2 * (dot * inv) : 0.f;
  auto log_q = [&](float v) __attribute__((always_inline)) {
    return far ? (v - ref) * (c * kLn2) - log_sum : __builtin_fmaf(x_of(v), kLn2, -log_sum);
  };
  if (tid == 0) {
    if (a.logp) a.logp[m] = has && columns ? log_q(zt) : 0.f;
    if (a.lse) a.lse[m] = columns ? z_max / a.tau + (log_sum - kLn2 * x_of(z_max)) : -INFINITY;
    if (a.entropy) a.entropy[m] = entropy;
  }
  auto again = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll 1
    for (int i = tid; i < R.chunks; i += T) {
      const u32x4_t v = R.only_columns(i, R.load(i));
#pragma unroll
      for (int k = 0; k < C::N; ++k) f(order_of(C::get(v, k)), i * C::N + k - R.head);
    }
  };
  auto each = [&](float least, auto&& f) __attribute__((always_inline)) {
    auto chunk = [&](int i, const u32x4_t& v) __attribute__((always_inline)) {
      if (__ballot(chunk_max(v, -INFINITY) >= least) == 0) return;
#pragma unroll
      for (int k = 0; k < C::N; ++k) f(C::get(v, k), i * C::N + k - R.head);
    };
    // (registers that no longer hold the logits themselves: from memory)
    if (VECS > 0 && !(ZT == kF32 && far)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) chunk(tid + j * T, z[j] = opaque(z[j]));
    } else {
#pragma unroll 1
      for (int i = tid; i - tid < R.chunks; i += T) chunk(i, R.only_columns(i, R.load(i)));
    }
  };
  if constexpr (TOP) {
    __shared__ Candidates s_top;
    find_top<T>(s_top, a.k, own_max, each, again);
    const int n = s_top.n;
    // (a last eight that come after every candidate)
    if (tid < 8) {
      s_top.key[n + tid] = 0u;
      s_top.col[n + tid] = 0x7fffffff;
    }
    __syncthreads();
    for (int i = tid; i < n; i += T) {
      const uint32_t key = s_top.key[i];
      const int col = s_top.col[i];
      int rank = 0;
      for (int j = 0; j < n; j += 8) {
        const u32x4_t k0 = *reinterpret_cast<const u32x4_t*>(s_top.key + j), k1 = *reinterpret_cast<const u32x4_t*>(s_top.key + j + 4);
        const int4 c0 = *reinterpret_cast<const int4*>(s_top.col + j), c1 = *reinterpret_cast<const int4*>(s_top.col + j + 4);
        const int cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t o = q < 4 ? k0[q] : k1[q - 4];
          rank += o > key || (o == key && cs[q] < col);
        }
      }
      if (rank < a.k) {
        a.top_logp[m * a.k + rank] = log_q(of_order(key));
        a.top_index[m * a.k + rank] = col;
      }
    }
    for (int i = n + tid; i < a.k; i += T) {
      a.top_logp[m * a.k + i] = -INFINITY;
      a.top_index[m * a.k + i] = -1;
    }
  }
  if (!a.dZ) return;
  const float g = (has && a.d_logp ? a.d_logp[m] : 0.f) / a.tau, h = (a.d_entropy ? a.d_entropy[m] : 0.f) / a.tau;
  const bool live = columns && (g != 0.f || h != 0.f);
  const float gi = -g * inv, hi = -h * inv, qt = uniform(__builtin_amdgcn_exp2f(x_of(zt)) * inv);
  const float log_qt = DOT ? uniform(log_q(zt)) : 0.f;
  auto grad = [&](float v) __attribute__((always_inline)) {
    if (!live) return 0.f;
    const float xv = x(v), e = __builtin_amdgcn_exp2f(xv);
    if constexpr (!DOT) return gi * e;
    // (fmaxf: a masked column's log q is −infinity, its q 0; a NaN row is NaN by inv)
    return e * __builtin_fmaf(hi, fmaxf(__builtin_fmaf(xv, kLn2, -log_sum), kMasked) + entropy, gi);
  };
  // the given token's own element once more, by the thread that wrote its chunk
  auto store = [&](int i, const u32x4_t& v) __attribute__((always_inline)) {
    R.store(a.dZ, i, v, grad);
    if (live && has && g != 0.f && (target + R.head) / C::N == i) {
      const float e = DOT && qt > 0.f ? h * qt * (log_qt + entropy) : 0.f;
      store_rounded<ZT>(a.dZ, R.row + target, g * (1.f - qt) - e);
    }
  };
  if constexpr (VECS > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (tid + j * T < R.chunks) store(tid + j * T, z[j] = opaque(z[j]));
  } else {
    for (int i0 = tid; i0 < R.chunks; i0 += NV * T) {
#pragma unroll
      for (int j = 0; j < NV; ++j) z[j] = R.load(i0 + j * T);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (i0 + j * T < R.chunks) store(i0 + j * T, R.only_columns(i0 + j * T, z[j]));
    }
  }
  for (int i = R.chunks + tid; i < R.chunks_out; i += T)
    R.store(a.dZ, i, u32x4_t{0u, 0u, 0u, 0u}, [](float) { return 0.f; });
}

// The gradient of 2,048 chunks of one row from what the forward pass saved; of a far
// row's (kFarLse) first part all of it, for in place the other parts' logits are needed
// until its sum is known (4096 x 32000 bf16, all rows far, 185 us, near 107).  Rows without
// a gradient are read like any other.
constexpr int kPartThreads = 256, kPartVecs = 8, kPart = kPartThreads * kPartVecs;
template <int ZT>
__global__ __launch_bounds__(kPartThreads) void logprobs_gradient_kernel(LogprobsArgs a, float chi, float clo) {
  using C = Chunk<ZT>;
  const int tid = threadIdx.x;
  const int64_t m = blockIdx.x;
  const Row<ZT> R(a.Z, a.dZ, a.M, a.V, a.ldz, m);
  const int i0 = kPart * (int)blockIdx.y + tid;
  u32x4_t z[kPartVecs];
#pragma unroll
  for (int j = 0; j < kPartVecs; ++j) z[j] = R.load(i0 + j * kPartThreads);
  const int target = a.target[m];
  const bool has = target >= 0 && target < R.V;
  const float lse = a.lse_in[m];
  const float g = (has && a.d_logp ? a.d_logp[m] : 0.f) / a.tau, h = (a.d_entropy ? a.d_entropy[m] : 0.f) / a.tau;
  const float entropy = a.d_entropy ? a.entropy_in[m] : 0.f;
  bool live = lse != -INFINITY && (g != 0.f || h != 0.f);
  // chunk i of the gradient, from log2 q
  auto write = [&](int i, const u32x4_t& v, auto&& log2_q) __attribute__((always_inline)) {
    auto value = [&](float v, float own) __attribute__((always_inline)) {
      const float l = log2_q(v), q = __builtin_amdgcn_exp2f(l);
      float d = own - g * q;
      if (h != 0.f) d -= h * q * (__builtin_fmaf(l, kLn2, entropy));
      return d;
    };
    R.store(a.dZ, i, v, [&](float v) __attribute__((always_inline)) { return live ? value(v, 0.f) : 0.f; });
    // the given token's own element once more, by the thread that wrote its chunk
    if (live && has && (target + R.head) / C::N == i) {
      float zt = 0.f;
#pragma unroll
      for (int k = 0; k < C::N; ++k)
        if (i * C::N + k - R.head == target) zt = C::get(v, k);
      store_rounded<ZT>(a.dZ, R.row + target, value(zt, g));
    }
  };
  if (live && fabsf(lse) >= kFarLse) {
    if (blockIdx.y > 0) return;
    const RowSum S = sum_row<ZT, kPartThreads>(R, chi);
    live = S.sum != 0.f;
    const float log2_s = log2f(S.sum);
    auto log2_q = [&](float v) __attribute__((always_inline)) {
      const float l = (v - S.ref) * chi - log2_s;
      return l < kMasked ? kMasked : l;  // (times a q of 0; NaN stays)
    };
#pragma unroll 1
    for (int i = tid; i < R.chunks_out; i += kPartThreads) write(i, R.only_columns(i, R.load(i)), log2_q);
    return;
  }
  // lse·log2(e) in two parts
  const float rhi = __fmul_rn(lse, 1.44269502f);
  const float rlo = __builtin_fmaf(lse, 1.92596303e-8f, __builtin_fmaf(lse, 1.44269502f, -rhi));
  auto log2_q = [&](float v) __attribute__((always_inline)) {
    v = v < kMasked ? kMasked : v;  // (−infinity·clo might be +infinity; NaN stays)
    return __builtin_fmaf(v, chi, -rhi) + __builtin_fmaf(v, clo, -rlo);
  };
#pragma unroll
  for (int j = 0; j < kPartVecs; ++j) {
    const int i = i0 + j * kPartThreads;
    if (i < R.chunks_out) write(i, R.only_columns(i, z[j]), log2_q);
  }
}

template <int ZT>
void launch(const LogprobsArgs& a, hipStream_t st) {
  constexpr int N = Chunk<ZT>::N;
  const double c = 1.4426950408889634 / (double)a.tau;
  const float chi = (float)c, clo = (float)(c - (double)chi);
  const unsigned grid = (unsigned)a.M;
  if (a.lse_in) {
    const int64_t parts = ((a.ldz + 2 * (N - 1)) / N + kPart - 1) / kPart;  // whatever the row's alignment
    logprobs_gradient_kernel<ZT><<<dim3(grid, (unsigned)parts), kPartThreads, 0, st>>>(a, chi, clo);
    return;
  }
  const int64_t chunks = (a.V + 2 * (N - 1)) / N;
  // 512 threads and as few chunks a thread as hold the row; from 4,096 chunks on
  // 1,024 threads; above 8,192 the running form
  const bool dot = a.entropy || a.d_entropy, top = a.k > 0;
#define QNF4_ROW(T, VECS)                                               \
  if (dot && top)                                                       \
    logprobs_kernel<ZT, T, VECS, true, true><<<grid, T, 0, st>>>(a, chi);  \
  else if (dot)                                                         \
    logprobs_kernel<ZT, T, VECS, true, false><<<grid, T, 0, st>>>(a, chi); \
  else if (top)                                                         \
    logprobs_kernel<ZT, T, VECS, false, true><<<grid, T, 0, st>>>(a, chi); \
  else                                                                  \
    logprobs_kernel<ZT, T, VECS, false, false><<<grid, T, 0, st>>>(a, chi);
  if (chunks <= 512) {
    QNF4_ROW(512, 1)
  } else if (chunks <= 1024) {
    QNF4_ROW(512, 2)
  } else if (chunks <= 2048) {
    QNF4_ROW(512, 4)
  } else if (chunks <= 4096) {
    QNF4_ROW(512, 8)
  } else if (chunks <= 8192) {
    QNF4_ROW(1024, 8)
  } else {
    QNF4_ROW(1024, 0)
  }
#undef QNF4_ROW
}

}  // namespace

hipError_t launch_logprobs(const LogprobsArgs& a, int z_type, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  if (z_type == kF32)
    launch<kF32>(a, st);
  else if (z_type == kBf16)
    launch<kBf16>(a, st);
  else
    launch<kF16>(a, st);
  return hipGetLastError();
}

}  // namespace qnf4
