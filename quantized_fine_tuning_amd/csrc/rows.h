// Rows of logits on the tensor's 16-byte grid, for the kernels that go over a
// vocabulary (distill.hip, logprobs.hip), gfx950.
#pragma once

#include "host.h"

namespace qnf4 {

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
  __device__ __forceinline__ Row(const void* Z, void* dZ, int64_t M, int64_t cols, int64_t ldz, int64_t m) {
    row = m * ldz;
    head = (int)(row & (C::N - 1));
    V = (int)cols;
    ld = (int)ldz;
    // (up to a whole dword: one that reaches past the end would read as zero
    // altogether; the dword's other half is never used)
    rz = make_rsrc(static_cast<const char*>(Z) + (row - head) * kSize,
                   round_up((M * ldz - (row - head)) * kSize, 4));
    out = static_cast<char*>(dZ) + (row - head) * kSize;
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

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// What |max·log2(e)/tau| a row is far from zero from, and for one of 16-bit logits the power
// of two that max times is in [2^19, 2^20) (logprobs.hip).
constexpr float kFarRow = 0x1p19f;
__device__ __forceinline__ float far_scale(float max) {
  return __uint_as_float((273u - (__float_as_uint(max) >> 23 & 255u)) << 23);
}

// A log-sum-exp of this size and more is held in steps of 2^-7 and more (1,024 at
// 1e10), no measure for the exponents of its row: a gradient from it takes the sum
// again, by differences from the row's maximum.
constexpr float kFarLse = 65536.f;

// A row's maximum (0 if every column is masked) and Σ 2^((z − it)·c), for every thread
// of a workgroup of T that reads the row twice.
struct RowSum {
  float ref, sum;
};
template <int ZT, int T>
__device__ __forceinline__ RowSum sum_row(const Row<ZT>& R, float c) {
  using C = Chunk<ZT>;
  __shared__ float s_row[2][T / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float high = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int i = threadIdx.x; i < R.chunks; i += T) {
    const u32x4_t v = R.only_columns(i, R.load(i));
#pragma unroll
    for (int k = 0; k < C::N; k += 2) high = max3(high, C::get(v, k), C::get(v, k + 1));
  }
  high = wave_max(high);
  if (lane == 0) s_row[0][wave] = high;
  __syncthreads();
  for (int w = 0; w < T / 64; ++w) high = fmaxf(high, s_row[0][w]);
  const float ref = high > kMasked ? high : 0.f;
#pragma unroll 1
  for (int i = threadIdx.x; i < R.chunks; i += T) {
    const u32x4_t v = R.only_columns(i, R.load(i));
#pragma unroll
    for (int k = 0; k < C::N; ++k) sum += __builtin_amdgcn_exp2f((C::get(v, k) - ref) * c);
  }
  sum = wave_sum(sum);
  if (lane == 0) s_row[1][wave] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < T / 64; ++w) sum += s_row[1][w];
  return {ref, sum};
}

}  // namespace qnf4
