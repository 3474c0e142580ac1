// Distillation from a teacher's top logits, gfx950.  Per token, with z the
// student's logits over V columns, t the teacher's logits at the columns c_i:
//   p = softmax(t/tau) over the entries, q = softmax(z/tau) over the columns,
//   loss = w·tau²·Σ_i p_i·(log p_i − log q_{c_i}),
//   dZ[v] = ∂loss/∂z_v = w·tau·(q_v − Σ_{i: c_i = v} p_i).
// An entry whose column lies outside [0, V) is no entry; a token without
// entries, or of weight 0, has loss 0 and a zero gradient.
//
// A logit of −infinity (a masked column) has q = 0; a row whose largest logit
// lies below −1e30 (every column masked) has loss 0 and a zero gradient.  NaN is
// no mask: it passes through maxima unseen and shows in the sums.
//
// Everything in fp32, exponents in base 2 with c = log2(e)/tau.
//
// Forward (with or without the gradient): one workgroup per token.  With ref
// the row's maximum and rc = fl(ref·c) an exponent is fma(z, c, −rc), off by
// an ulp of itself; what rc was rounded by is the same factor for the whole
// row and comes back into the log-sum-exp alone.  Bound by HBM: a row is read
// once and its gradient written once.  The row stays in registers between
// the two (VECS 16-byte chunks a thread, the loads of all of them in flight
// together); a row too long for that is read once for a running maximum and
// sum (and once more, from the caches, for its gradient).  Chunks are those of
// the tensor's own 16-byte grid, so that rows of any alignment load and store
// whole chunks except at their two ends.  The entries are wave 0's work, beside the row's loads, so a row
// costs three barriers.  (4096 x 32000 bf16, k = 64: 115 us, 4.6 TB/s, a large
// copy reaching 4.6; 509 x 32003 fp32: 33 us; the loss alone of 1024 x 128000
// bf16: 48 us.  A row of 32000 bf16 alone takes 8 us: one workgroup's three
// passes of latency.)
//
// Gradient from a saved log-sum-exp: no sums over the row, so rows are cut
// into parts of 2,048 chunks, a workgroup each.  Its exponent z·c − lse·log2(e)
// takes both products in two parts: rounded ones would be off by an ulp of
// z/tau.  (777 x 50001 fp16, k = 128: 44 us on the same inputs over and over,
// 50 on changing ones; the kernel 43, 4.8 TB/s.)
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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;  // (fmaxf would first quiet each operand that comes from bits)
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}

// The row's place on the tensor's 16-byte grid: `head` elements of its first
// chunk belong to the row before.
template <int ZT>
struct Row {
  using C = Chunk<ZT>;
  static constexpr int64_t kSize = ZT == kF32 ? 4 : 2;
  int64_t row;
  int head, V, ld, chunks, chunks_out;  // chunks that hold columns, and the padding too
  rsrc_t rz;
  char* out;
  __device__ __forceinline__ Row(const DistillArgs& a, int64_t m) {
    row = m * a.ldz;
    head = (int)(row & (C::N - 1));
    V = (int)a.V;
    ld = (int)a.ldz;
    // (up to a whole dword: one that reaches past the end would read as zero
    // altogether; the dword's other half is never used)
    rz = make_rsrc(static_cast<const char*>(a.Z) + (row - head) * kSize,
                   round_up((a.M * a.ldz - (row - head)) * kSize, 4));
    out = static_cast<char*>(a.dZ) + (row - head) * kSize;
    chunks = (head + V + C::N - 1) / C::N;
    chunks_out = (head + ld + C::N - 1) / C::N;
  }
  __device__ __forceinline__ u32x4_t load(int i) const {
    return buf_load16(rz, i < chunks ? (uint32_t)i * 16u : 0x7fffffffu, 0u);
  }
  __device__ __forceinline__ bool whole(int i) const { return i * C::N >= head && (i + 1) * C::N <= head + V; }
  // chunk i with −infinity in the place of what is no column of this row
  // (exponentials of 0; another row's elements at the ends, padding)
  __device__ __forceinline__ u32x4_t only_columns(int i, u32x4_t v) const {
    if (!whole(i)) {
#pragma unroll
      for (int k = 0; k < C::N; ++k) {
        const int col = i * C::N + k - head;
        if (col >= 0 && col < V) continue;
        if constexpr (ZT == kF32)
          v[k] = 0xff800000u;
        else if (k & 1)
          v[k >> 1] = (v[k >> 1] & 0xffffu) | (ZT == kF16 ? 0xfc000000u : 0xff800000u);
        else
          v[k >> 1] = (v[k >> 1] & 0xffff0000u) | (ZT == kF16 ? 0xfc00u : 0xff80u);
      }
    }
    return v;
  }
  // value(z) for chunk i's columns, zeros in the padding (not value(−infinity):
  // a row that is not a number has NaN there)
  template <typename F>
  __device__ __forceinline__ void store(void* dZ, int i, const u32x4_t& v, F&& value) const {
    if (whole(i)) {
      float f[C::N];
#pragma unroll
      for (int k = 0; k < C::N; ++k) f[k] = value(C::get(v, k));
      *reinterpret_cast<u32x4_t*>(out + (int64_t)i * 16) = C::pack(f);
    } else {
#pragma unroll
      for (int k = 0; k < C::N; ++k) {
        const int col = i * C::N + k - head;
        if (col >= 0 && col < ld) store_rounded<ZT>(dZ, row + col, col < V ? value(C::get(v, k)) : 0.f);
      }
    }
  }
};

// The entries of one row: columns, logits, student logits and probabilities,
// for wave 0 to fill.  tau divides differences of logits: a logit's own quotient
// may pass what fp32 holds.
struct Entries {
  int c[kMaxTop];
  float t[kMaxTop], z[kMaxTop], p[kMaxTop];
  float t_max, t_log;  // maximum of t, log Σ exp((t − t_max)/tau)
  bool any;            // whether there is an entry (one of logit −infinity is none)
};
template <int ZT, int TT>
__device__ __forceinline__ void load_entries(Entries& s, const DistillArgs& a, int64_t m, int64_t row, int lane) {
  for (int i = lane; i < a.k; i += 64) {
    const int col = a.at[m * a.k + i];
    const bool ok = col >= 0 && col < a.V;
    const float t = load_as_f32<TT>(a.top, m * a.k + i);
    const float z = load_as_f32<ZT>(a.Z, row + (ok ? col : 0));
    s.c[i] = ok ? col : -1;
    s.z[i] = ok ? z : 0.f;
    s.t[i] = ok ? t : -INFINITY;
  }
}
__device__ __forceinline__ void entry_softmax(Entries& s, int k, float tau, int lane) {
  float t_max = -INFINITY, t_sum = 0.f;
  for (int i = lane; i < k; i += 64) t_max = fmaxf(t_max, s.t[i]);
  t_max = wave_max(t_max);
  // (maxima pass over NaN, the sum does not: entries of NaN are entries)
  for (int i = lane; i < k; i += 64) {
    s.p[i] = s.t[i] != -INFINITY ? expf((s.t[i] - t_max) / tau) : 0.f;
    t_sum += s.p[i];
  }
  t_sum = wave_sum(t_sum);
  const bool any = t_sum != 0.f;
  const float inv = any ? 1.0f / t_sum : 0.f;
  for (int i = lane; i < k; i += 64)
    if (s.t[i] != -INFINITY) s.p[i] *= inv;  // (else 0, beside a NaN too)
  if (lane == 0) {
    s.t_max = t_max;
    s.t_log = any ? logf(t_sum) : 0.f;
    s.any = any;
  }
}
// The teacher's share taken off the columns [v0, v1), once their exponentials
// are written: the first of several entries of one column takes all of theirs.
template <int ZT, typename F>
__device__ __forceinline__ void take_entries(const Entries& s, const DistillArgs& a, int64_t row, int v0, int v1,
                                             float g, F&& q) {
  __threadfence_block();
  __syncthreads();
  for (int i = threadIdx.x; i < a.k; i += blockDim.x) {
    const int col = s.c[i];
    bool first = col >= v0 && col < v1;
    float p = 0.f;
    for (int o = 0; o < a.k; ++o)
      if (s.c[o] == col) {
        if (o < i) first = false;
        p += s.p[o];
      }
    if (first) store_rounded<ZT>(a.dZ, row + col, g * (q(s.z[i]) - p));
  }
}

// VECS > 0: the row's chunks in registers, VECS per thread of T; VECS == 0:
// any number of chunks, two in flight per thread, read again for the gradient.
// (8 waves a SIMD for the 1,024-thread forms: a second workgroup loads its row
// while the first computes; 777 rows of 50,001 fp16 columns took 60 us without
// it and 54 with.  Four-byte logits spill at that and go without.)
template <int ZT, int TT, int T, int VECS>
__global__ __launch_bounds__(T, T == 1024 && (ZT != kF32 || VECS == 0) ? 8 : 1) void distill_kernel(DistillArgs a, float c) {
  using C = Chunk<ZT>;
  constexpr int kWaves = T / 64;
  __shared__ Entries s;
  __shared__ float s_max[kWaves], s_sum[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t m = blockIdx.x;
  const Row<ZT> R(a, m);
  constexpr int NV = VECS > 0 ? VECS : 2;
  u32x4_t z[NV];
  if constexpr (VECS > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) z[j] = R.load(tid + j * T);
  }
  if (wave == 0) {
    load_entries<ZT, TT>(s, a, m, R.row, lane);
    entry_softmax(s, a.k, a.tau, lane);
  }

  // (Each pass widens the 16-bit values anew, from an opaque copy of the chunk:
  // kept widened from one pass to the next they would take twice its registers.)
  // the largest column of a chunk, beside `high`
  auto chunk_max = [&](const u32x4_t& v, float high) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < C::N; k += 2) high = max3(high, C::get(v, k), C::get(v, k + 1));
    return high;
  };
  float rc = 0.f;
  auto e = [&](float x) __attribute__((always_inline)) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(x, c, -rc));
  };
  auto chunk_sum = [&](const u32x4_t& v, float sum) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < C::N; ++k) sum += e(C::get(v, k));
    return sum;
  };
  float z_max = -INFINITY, sum = 0.f;
  if constexpr (VECS > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      z[j] = R.only_columns(tid + j * T, z[j]);
      z_max = chunk_max(z[j], z_max);
    }
  } else {
    // running maximum and sum of this thread's chunks (as long as it has met
    // masked columns alone, rc is 0 and they add zeros, a NaN itself)
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
        const float before = rc;
        rc = high > kMasked ? __fmul_rn(high, c) : 0.f;
        sum *= z_max > kMasked ? __builtin_amdgcn_exp2f(before - rc) : 0.f;
        z_max = high;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) sum = chunk_sum(opaque(z[j]), sum);
    }
  }
  const float own_max = z_max, own_rc = rc;
  z_max = wave_max(z_max);
  if (lane == 0) s_max[wave] = z_max;
  __syncthreads();
  z_max = s_max[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) z_max = fmaxf(z_max, s_max[w]);
  // (maxima pass over NaN: where they say that every column is masked the sum
  // has the last word, zero for masked columns, NaN where one is NaN)
  const bool masked = !(z_max > kMasked);
  rc = masked ? 0.f : __fmul_rn(z_max, c);
  if constexpr (VECS > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) sum = chunk_sum(z[j] = opaque(z[j]), sum);
  } else {
    sum *= own_max > kMasked ? __builtin_amdgcn_exp2f(own_rc - rc) : 0.f;
  }
  sum = wave_sum(sum);
  if (lane == 0) s_sum[wave] = sum;
  __syncthreads();
  sum = s_sum[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += s_sum[w];
  const float w = a.weight ? a.weight[m] : 1.0f;
  const bool columns = !masked || sum != 0.f;
  const bool live = columns && w != 0.f && s.any;
  if (wave == 0) {
    const float log_sum = logf(sum) - 0.693147182f * __builtin_fmaf(z_max, c, -rc);
    const float lse = columns ? z_max / a.tau + log_sum : -INFINITY;
    if (a.lse && lane == 0) a.lse[m] = lse;
    float loss = 0.f;
    if (live)
      for (int i = lane; i < a.k; i += 64)
        if (s.p[i] != 0.f) loss += s.p[i] * ((s.t[i] - s.t_max) / a.tau - s.t_log - (s.z[i] / a.tau - lse));
    loss = wave_sum(loss);
    if (lane == 0) a.loss[m] = live ? w * a.tau * a.tau * loss : 0.f;
  }
  if (!a.dZ) return;
  const float g = w * a.tau, inv = 1.0f / sum, gi = g * inv;
  auto grad = [&](float x) __attribute__((always_inline)) { return live ? gi * e(x) : 0.f; };
  if constexpr (VECS > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (tid + j * T < R.chunks) R.store(a.dZ, tid + j * T, opaque(z[j]), grad);
  } else {
    for (int i0 = tid; i0 < R.chunks; i0 += NV * T) {
#pragma unroll
      for (int j = 0; j < NV; ++j) z[j] = R.load(i0 + j * T);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (i0 + j * T < R.chunks) R.store(a.dZ, i0 + j * T, R.only_columns(i0 + j * T, z[j]), grad);
    }
  }
  for (int i = R.chunks + tid; i < R.chunks_out; i += T)
    R.store(a.dZ, i, u32x4_t{0u, 0u, 0u, 0u}, [](float) { return 0.f; });
  if (live) take_entries<ZT>(s, a, R.row, 0, R.V, g, [&](float x) { return e(x) * inv; });
}

// The gradient of 2,048 chunks of one row from its saved log-sum-exp.
constexpr int kPartThreads = 256, kPartVecs = 8, kPart = kPartThreads * kPartVecs;
template <int ZT, int TT>
__global__ __launch_bounds__(kPartThreads) void distill_gradient_kernel(DistillArgs a, float chi, float clo) {
  using C = Chunk<ZT>;
  __shared__ Entries s;
  const int tid = threadIdx.x;
  const int64_t m = blockIdx.x;
  const Row<ZT> R(a, m);
  const int i0 = kPart * (int)blockIdx.y + tid;
  u32x4_t z[kPartVecs];
#pragma unroll
  for (int j = 0; j < kPartVecs; ++j) z[j] = R.load(i0 + j * kPartThreads);
  const float lse = a.lse_in[m], w = a.weight ? a.weight[m] : 1.0f;
  const bool in_place = a.dZ == a.Z;
  // (in place the entries' logits have to be read before any is overwritten;
  // otherwise the first wave sees to the entries while the others write)
  if (in_place) {
    if (tid < 64) load_entries<ZT, TT>(s, a, m, R.row, tid);
    __syncthreads();
  }
  bool live = lse != -INFINITY && w != 0.f;  // (a NaN lse, of a row with a NaN or an infinity, is no masked row's)
  const float g = w * a.tau;
  // lse·log2(e) in two parts
  const float rhi = __fmul_rn(lse, 1.44269502f);
  const float rlo = __builtin_fmaf(lse, 1.92596303e-8f, __builtin_fmaf(lse, 1.44269502f, -rhi));
  auto q = [&](float x) __attribute__((always_inline)) {
    x = x < kMasked ? kMasked : x;  // (−infinity·clo might be +infinity; NaN stays)
    return __builtin_amdgcn_exp2f(__builtin_fmaf(x, chi, -rhi) + __builtin_fmaf(x, clo, -rlo));
  };
  auto grad = [&](float x) __attribute__((always_inline)) { return live ? g * q(x) : 0.f; };
#pragma unroll
  for (int j = 0; j < kPartVecs; ++j)
    if (i0 + j * kPartThreads < R.chunks_out) {
      z[j] = R.only_columns(i0 + j * kPartThreads, z[j]);
      R.store(a.dZ, i0 + j * kPartThreads, z[j], grad);
    }
  // (the exponentials are written before the entries are waited for; a row
  // without entries gets its zeros now)
  if (tid < 64) {
    if (!in_place) load_entries<ZT, TT>(s, a, m, R.row, tid);
    entry_softmax(s, a.k, a.tau, tid);
  }
  __syncthreads();
  if (live && !s.any) {
    live = false;
#pragma unroll
    for (int j = 0; j < kPartVecs; ++j)
      if (i0 + j * kPartThreads < R.chunks_out) R.store(a.dZ, i0 + j * kPartThreads, z[j], grad);
  }
  const int v0 = kPart * (int)blockIdx.y * C::N - R.head;
  if (live) take_entries<ZT>(s, a, R.row, std::max(v0, 0), std::min(v0 + kPart * C::N, R.V), g, q);
}

template <int ZT, int TT>
void launch(const DistillArgs& a, hipStream_t st) {
  constexpr int N = Chunk<ZT>::N;
  const double c = 1.4426950408889634 / (double)a.tau;
  const float chi = (float)c, clo = (float)(c - (double)chi);
  const unsigned grid = (unsigned)a.M;
  if (a.lse_in) {
    const int64_t parts = ((a.ldz + 2 * (N - 1)) / N + kPart - 1) / kPart;  // whatever the row's alignment
    distill_gradient_kernel<ZT, TT><<<dim3(grid, (unsigned)parts), kPartThreads, 0, st>>>(a, chi, clo);
    return;
  }
  const int64_t chunks = (a.V + 2 * (N - 1)) / N;
  // 512 threads and as few chunks a thread as hold the row; from 4,096 chunks
  // on 1,024 threads; above 8,192 the running form.  (By the row alone, not by
  // whether its gradient is asked for: the loss is the same to the bit.)
#define QNF4_ROW(T, VECS) distill_kernel<ZT, TT, T, VECS><<<grid, T, 0, st>>>(a, chi)
  if (chunks <= 512)
    QNF4_ROW(512, 1);
  else if (chunks <= 1024)
    QNF4_ROW(512, 2);
  else if (chunks <= 2048)
    QNF4_ROW(512, 4);
  else if (chunks <= 4096)
    QNF4_ROW(512, 8);
  else if (chunks <= 8192)
    QNF4_ROW(1024, 8);
  else
    QNF4_ROW(1024, 0);
#undef QNF4_ROW
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, int z_type, int t_type, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
#define QNF4_DISTILL(ZT, TT) \
  if (z_type == ZT && t_type == TT) launch<ZT, TT>(a, st);
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
