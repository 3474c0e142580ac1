// Low-rank adapters of many requests beside one quantized weight, gfx950:
//   Y[m] = X[m]·Ŵᵀ + s_a·(X[m]·A_aᵀ)·B_aᵀ,  a = a(m) the adapter of token m,
// and its gradients, with T = X[m]·A_aᵀ and U = dY[m]·B_a:
//   dX[m] = dY[m]·Ŵ + s_a·U[m]·A_a,
//   dA_a = s_a·Σ_{m: a(m) = a} U[m]ᵀ·X[m],  dB_a = s_a·Σ_{m: a(m) = a} dY[m]ᵀ·T[m].
// The base product runs in the dequant-in-tile GEMMs, whose fp32 results go
// to the workspace; the adapter products below are added to them in fp32 and
// the sum is rounded once.
#include <algorithm>

#include "host.h"

namespace qnf4 {

hipError_t launch_dx_gemm(const Nf4View& W, const uint16_t* dY, int64_t M, const uint16_t* sU,
                          const uint16_t* AT2, int64_t Rp, void* dX, bool dx16, int splits, float* P, bool f16,
                          hipStream_t st);
hipError_t launch_fwd_gemm(const Nf4View& W, const uint16_t* X, int64_t M, const uint16_t* sT,
                           const uint16_t* B2, int64_t Rp, void* Y, bool y16, int splits, float* P, bool f16,
                           hipStream_t st);
int fwd_gemm_splits(int64_t M, int64_t N, int64_t K, size_t cap);
int dx_gemm_splits(int64_t M, int64_t N, int64_t K, size_t cap);

namespace {

unsigned cdiv(int64_t a, int64_t b) { return (unsigned)((a + b - 1) / b); }

// ---------------------------------------------------------------------------
// Plan: the tokens sorted by adapter (stable, so that the sums over an
// adapter's tokens run in token order).  One workgroup of 16 waves, each over
// its own run of tokens: counts per wave and adapter, their prefix sums over
// adapters and waves, then every token's position.  A token's rank among the
// equal adapters of its 64-token chunk comes from one ballot per bit of the
// adapter's number.
// ---------------------------------------------------------------------------
constexpr int kPlanWaves = 16;
__global__ __launch_bounds__(64 * kPlanWaves) void adapters_plan_kernel(const int32_t* __restrict__ index, int64_t M,
                                                                        int count, PlanView pl) {
  extern __shared__ int32_t hist[];  // [16][count + 1]; column `count`: no adapter
  __shared__ int32_t s_wave[2][kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cols = count + 1;
  for (int i = tid; i < kPlanWaves * cols; i += 64 * kPlanWaves) hist[i] = 0;
  __syncthreads();
  const int64_t per = (M + kPlanWaves * 64 - 1) / (kPlanWaves * 64) * 64;
  const int64_t m_end = std::min<int64_t>(M, per * (wave + 1));
  int32_t* const mine = hist + wave * cols;
  for (int64_t m = per * wave + lane; m < m_end; m += 64) {
    const int32_t a = index[m];
    const int32_t o = a >= 0 && a < count ? a : -1;
    pl.owner[m] = o;
    atomicAdd(&mine[o < 0 ? count : o], 1);  // integer counts: any order gives the same
  }
  __syncthreads();
  // thread a: adapter a's tokens, then exclusive sums over the adapters of
  // the tokens and of "carries any token"
  int total = 0;
  if (tid < count)
    for (int w = 0; w < kPlanWaves; ++w) total += hist[w * cols + tid];
  const int used = total > 0 ? 1 : 0;
  int st = total, su = used;
  for (int o = 1; o < 64; o <<= 1) {
    const int a = __shfl_up(st, o, 64), b = __shfl_up(su, o, 64);
    if (lane >= o) {
      st += a;
      su += b;
    }
  }
  if (lane == 63) {
    s_wave[0][wave] = st;
    s_wave[1][wave] = su;
  }
  __syncthreads();
  int bt = 0, bu = 0, all = 0, nact = 0;
  for (int w = 0; w < kPlanWaves; ++w) {
    if (w < wave) {
      bt += s_wave[0][w];
      bu += s_wave[1][w];
    }
    all += s_wave[0][w];
    nact += s_wave[1][w];
  }
  st += bt - total;
  su += bu - used;
  __syncthreads();
  if (tid < count) {
    pl.slot[tid] = used ? su : -1;
    if (used) {
      pl.id[su] = tid;
      pl.start[su] = st;
    }
    int run = st;
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = hist[w * cols + tid];
      hist[w * cols + tid] = run;
      run += c;
    }
  }
  if (tid == 0) {
    pl.head[0] = nact;
    pl.head[1] = all;
    pl.start[nact] = all;
    int run = all;
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = hist[w * cols + count];
      hist[w * cols + count] = run;
      run += c;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz((unsigned)count);
  for (int64_t m0 = per * wave; m0 < m_end; m0 += 64) {
    const int64_t m = m0 + lane;
    const bool ok = m < m_end;
    int a = count;
    if (ok) {
      const int32_t v = index[m];
      a = v >= 0 && v < count ? v : count;
    }
    uint64_t same = __ballot(ok);
    for (int b = 0; b < bits; ++b) {
      const uint64_t one = __ballot((a >> b) & 1);
      same &= ((a >> b) & 1) ? one : ~one;
    }
    if (ok) {
      const int at = mine[a];
      const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
      pl.perm[at + before] = (int32_t)m;
    }
    // (a wave's LDS accesses run in order: every lane has read its count)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (ok && (same >> lane) == 1) mine[a] += __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  __threadfence_block();
  __syncthreads();
  for (int64_t p = tid; p < M; p += 64 * kPlanWaves) {
    const int32_t m = pl.perm[p];
    const int32_t v = index[m];
    pl.group[p] = v >= 0 && v < count ? pl.slot[v] : nact;
  }
}

// ---------------------------------------------------------------------------
// T[m][j] = X[m]·A_a[j] (zeros for a token without an adapter): a wave per
// (token, 4 ranks), 8 reduction elements per lane and step.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float dot8(const u32x4_t a, const u32x4_t b, float acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = __builtin_fmaf(bf16lo(a[i]), bf16lo(b[i]), acc);
    acc = __builtin_fmaf(bf16hi(a[i]), bf16hi(b[i]), acc);
  }
  return acc;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__global__ __launch_bounds__(256) void adapters_down_kernel(const uint16_t* __restrict__ X, int64_t K, AdapterView ad,
                                                            PlanView pl, float* __restrict__ T) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = blockIdx.x;
  const int j0 = 16 * (int)blockIdx.y + 4 * wave;
  if (j0 >= ad.r) return;
  const int a = pl.owner[m];
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (a >= 0 && a < ad.count) {
    const uint16_t* x = X + m * K;
    const uint16_t* w = ad.A + ((int64_t)a * ad.r + j0) * K;
    for (int64_t k = 8 * lane; k < K; k += 512) {
      const u32x4_t xv = *reinterpret_cast<const u32x4_t*>(x + k);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[j] = dot8(xv, *reinterpret_cast<const u32x4_t*>(w + j * K + k), acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float t = wave_sum(acc[j]);
    if (lane == 0) T[m * ad.r + j0 + j] = t;
  }
}

// U[m][j] = Σ_n dY[m][n]·B_a[n][j]: a workgroup per (token, 16 ranks), thread
// (n slice tid / 16, rank tid % 16), the 16 slices summed in order.
__global__ __launch_bounds__(256) void adapters_gradient_down_kernel(const uint16_t* __restrict__ dY, int64_t N,
                                                                     AdapterView ad, PlanView pl,
                                                                     float* __restrict__ U) {
  __shared__ float s[16][17];
  const int jj = threadIdx.x & 15, nn = threadIdx.x >> 4;
  const int64_t m = blockIdx.x;
  const int j = 16 * (int)blockIdx.y + jj;
  const int a = pl.owner[m];
  float acc = 0.f;
  if (a >= 0 && a < ad.count && j < ad.r) {
    const uint16_t* b = ad.B + (int64_t)a * N * ad.r + j;
    for (int64_t n = nn; n < N; n += 16)
      acc = __builtin_fmaf(bf16_to_f32(dY[m * N + n]), bf16_to_f32(b[n * ad.r]), acc);
  }
  s[nn][jj] = acc;
  __syncthreads();
  if (nn == 0 && j < ad.r) {
    float t = 0.f;
    for (int i = 0; i < 16; ++i) t += s[i][jj];
    U[m * ad.r + j] = t;
  }
}

// out[m][c] = Σ_s P[s][m][c] + s_a·Σ_j T[m][j]·F_a(j, c), four columns per
// thread, F_a(j, c) = B_a[c][j] (ALONG: the rank contiguous) or A_a[j][c].
template <bool ALONG>
__global__ __launch_bounds__(256) void adapters_up_kernel(const float* __restrict__ P, int splits, int64_t M, int64_t C,
                                                          const uint16_t* __restrict__ F, AdapterView ad, PlanView pl,
                                                          const float* __restrict__ T, void* __restrict__ out,
                                                          int out16) {
  const int64_t m = blockIdx.y, c = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (c >= C) return;
  f32x4_t y = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(P + ((int64_t)s * M + m) * C + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] += v[i];
  }
  const int a = pl.owner[m];
  if (a >= 0 && a < ad.count) {
    const uint16_t* f = F + (int64_t)a * C * ad.r;
    float dot[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < ad.r; ++j) {
      const float t = T[m * ad.r + j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dot[i] = __builtin_fmaf(t, bf16_to_f32(ALONG ? f[(c + i) * ad.r + j] : f[j * C + c + i]), dot[i]);
    }
    const float s = ad.s[a];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(s, dot[i], y[i]);
  }
  if (out16) {
    u32x2_t o;
    o[0] = pack_bf16x2(y[0], y[1]);
    o[1] = pack_bf16x2(y[2], y[3]);
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(out) + m * C + c) = o;
  } else {
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + m * C + c) = y;
  }
}

// One adapter's gradient: out[j][c] (or out[c][j], ALONG) = s_a·Σ_m S[m][j]·L[m][c]
// over its tokens in order; workgroup (256 columns, 8 ranks, adapter).
template <bool ALONG>
__global__ __launch_bounds__(256) void adapters_gradient_kernel(const uint16_t* __restrict__ L, int64_t M, int64_t C,
                                                                AdapterView ad, PlanView pl,
                                                                const float* __restrict__ S, float* __restrict__ out) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int j0 = 8 * (int)blockIdx.y, a = (int)blockIdx.z;
  const int g = pl.slot[a];
  float acc[8] = {};
  if (g >= 0 && g < ad.count) {
    const int64_t p1 = std::min<int64_t>(pl.start[g + 1], M);
    for (int64_t p = std::max(pl.start[g], 0); p < p1; ++p) {
      const int64_t m = pl.perm[p];
      if ((uint64_t)m >= (uint64_t)M) continue;
      const float x = c < C ? bf16_to_f32(L[m * C + c]) : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = __builtin_fmaf(S[m * ad.r + j0 + j], x, acc[j]);
    }
  }
  if (c >= C) return;
  const float s = g >= 0 ? ad.s[a] : 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    out[(int64_t)a * ad.r * C + (ALONG ? c * ad.r + j0 + j : (j0 + j) * C + c)] = s * acc[j];
}

}  // namespace

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

namespace {
constexpr int64_t kPlanHead = 16;  // words
int64_t plan_pad(int64_t n) { return round_up(n, 16); }
}  // namespace

size_t plan_bytes(int64_t M, int count) {
  return (size_t)(kPlanHead + 3 * plan_pad(M) + 3 * plan_pad(count + 1)) * 4;
}
PlanView plan_view(void* plan, int64_t M, int count) {
  PlanView v;
  v.head = static_cast<int32_t*>(plan);
  v.owner = v.head + kPlanHead;
  v.perm = v.owner + plan_pad(M);
  v.group = v.perm + plan_pad(M);
  v.id = v.group + plan_pad(M);
  v.start = v.id + plan_pad(count + 1);
  v.slot = v.start + plan_pad(count + 1);
  return v;
}
hipError_t launch_adapters_plan(const int32_t* index, int64_t M, int count, const PlanView& pl, hipStream_t st) {
  adapters_plan_kernel<<<1, 64 * kPlanWaves, (size_t)kPlanWaves * (count + 1) * 4, st>>>(index, M, count, pl);
  return hipGetLastError();
}

AdaptersFwdLayout adapters_fwd_layout(int64_t M, int64_t N, int64_t K, int r, int count) {
  AdaptersFwdLayout L{};
  L.splits = M > 0 ? fwd_gemm_splits(M, N, K, SIZE_MAX) : 1;
  L.off_T = 0;
  L.off_P = round_up(M * r * 4, 256);
  L.total = L.off_P + round_up((int64_t)L.splits * M * N * 4, 256);
  return L;
}
AdaptersBwdLayout adapters_bwd_layout(int64_t M, int64_t N, int64_t K, int r, int count) {
  AdaptersBwdLayout L{};
  L.splits = M > 0 ? dx_gemm_splits(M, N, K, SIZE_MAX) : 1;
  L.off_T = 0;
  L.off_U = round_up(M * r * 4, 256);
  L.off_P = 2 * L.off_U;
  L.total = L.off_P + round_up((int64_t)L.splits * M * K * 4, 256);
  return L;
}
// The split count depends on M through the number of 256-row tiles alone and
// the bytes grow with M within such a band: each band's largest M is taken.
size_t adapters_fwd_ws_max(int64_t M_max, int64_t N, int64_t K, int r, int count) {
  size_t most = 0;
  for (int64_t top = 256;; top += 256) {
    most = std::max(most, adapters_fwd_layout(std::min(top, M_max), N, K, r, count).total);
    if (top >= M_max) return most;
  }
}
size_t adapters_bwd_ws_max(int64_t M_max, int64_t N, int64_t K, int r, int count) {
  size_t most = 0;
  for (int64_t top = 256;; top += 256) {
    most = std::max(most, adapters_bwd_layout(std::min(top, M_max), N, K, r, count).total);
    if (top >= M_max) return most;
  }
}

hipError_t launch_adapters_fwd(const Nf4View& W, const uint16_t* X, int64_t M, const AdapterView& ad,
                               const PlanView& pl, void* Y, bool y16, float* T_save, char* ws,
                               const AdaptersFwdLayout& L, hipStream_t st) {
  if (M == 0) return hipSuccess;
  float* T = T_save ? T_save : reinterpret_cast<float*>(ws + L.off_T);
  float* P = reinterpret_cast<float*>(ws + L.off_P);
  adapters_down_kernel<<<dim3((unsigned)M, cdiv(ad.r, 16)), 256, 0, st>>>(X, W.K, ad, pl, T);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = launch_fwd_gemm(W, X, M, nullptr, nullptr, 0, P, false, L.splits, P, false, st);
  if (e != hipSuccess) return e;
  adapters_up_kernel<true><<<dim3(cdiv(W.N, 1024), (unsigned)M), 256, 0, st>>>(P, L.splits, M, W.N, ad.B, ad, pl, T, Y,
                                                                               y16 ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_adapters_bwd(const Nf4View& W, const uint16_t* X, const uint16_t* dY, int64_t M,
                               const AdapterView& ad, const PlanView& pl, const float* T_saved, void* dX, bool dx16,
                               float* dA, float* dB, char* ws, const AdaptersBwdLayout& L, hipStream_t st) {
  const int64_t N = W.N, K = W.K;
  hipError_t e;
  if (M == 0) {
    e = launch_zero(dA, (int64_t)ad.count * ad.r * K, st);
    return e != hipSuccess ? e : launch_zero(dB, (int64_t)ad.count * ad.r * N, st);
  }
  float* T = reinterpret_cast<float*>(ws + L.off_T);
  float* U = reinterpret_cast<float*>(ws + L.off_U);
  float* P = reinterpret_cast<float*>(ws + L.off_P);
  const unsigned m = (unsigned)M, r16 = cdiv(ad.r, 16), r8 = (unsigned)(ad.r / 8), count = (unsigned)ad.count;
  if (!T_saved) {
    adapters_down_kernel<<<dim3(m, r16), 256, 0, st>>>(X, K, ad, pl, T);
    T_saved = T;
  }
  adapters_gradient_down_kernel<<<dim3(m, r16), 256, 0, st>>>(dY, N, ad, pl, U);
  e = hipGetLastError();
  if (e == hipSuccess) e = launch_dx_gemm(W, dY, M, nullptr, nullptr, 0, P, false, L.splits, P, false, st);
  if (e != hipSuccess) return e;
  adapters_up_kernel<false><<<dim3(cdiv(K, 1024), m), 256, 0, st>>>(P, L.splits, M, K, ad.A, ad, pl, U, dX,
                                                                    dx16 ? 1 : 0);
  adapters_gradient_kernel<false><<<dim3(cdiv(K, 256), r8, count), 256, 0, st>>>(X, M, K, ad, pl, U, dA);
  adapters_gradient_kernel<true><<<dim3(cdiv(N, 256), r8, count), 256, 0, st>>>(dY, M, N, ad, pl, T_saved, dB);
  return hipGetLastError();
}

}  // namespace qnf4
