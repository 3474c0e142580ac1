// Adapters with dropout on one quantized layer, and the gated feed-forward block
// of two such layers that share their input, gfx950.  With D the dropout of the
// adapters' input (dropout.h: one mask of X for both layers) and layer l's
//   Y_l = X·Ŵ_lᵀ + s·T_l·B_lᵀ,  T_l = D(X)·A_lᵀ,
// the gated block is H = act(Y_0)*Y_1 (G = Y_0, U = Y_1), and with dY_l what
// reaches Y_l and V_l = dY_l·B_l
//   dX = Σ_l dY_l·Ŵ_l + s·keep*(Σ_l V_l·A_l)   (keep: D's mask times its scale)
//   dA_l = s·V_lᵀ·D(X),  dB_l = s·dY_lᵀ·T_l.
// The base products run in the dequant-in-tile GEMMs (fwd.hip, dx.hip; up to 16
// tokens forward: gemv.hip), whose reductions go on over the low-rank factors;
// the kernels here make those, the gradients, and what is element by element.
#include <algorithm>

#include "dropout.h"
#include "gate.h"
#include "host.h"
#include "lowrank.h"
#include "splitk.h"
#include "tiling.h"

namespace qnf4 {

hipError_t launch_fwd_gemm_block(const Nf4View& W, const uint16_t* X, int64_t M, const BlockGemmArgs& ma, bool pair,
                                 void* Y, bool y16, int splits, float* P, hipStream_t st);
hipError_t launch_dx_gemm_block(const Nf4View& W, const uint16_t* dY, int64_t M, const BlockGemmArgs& ma, bool pair,
                                void* dX, bool dx16, int splits, float* P, hipStream_t st);
hipError_t launch_splitk_reduce(const float* P, int splits, int64_t n, void* out, bool out16, bool f16,
                                hipStream_t st);
hipError_t launch_gemv_sums(const Nf4View& W, const uint16_t* X, int64_t M, const float* P, int S, int JT,
                            const uint16_t* B, int32_t r, float scale, void* Y, bool y16, float* T, bool f16,
                            hipStream_t st);
hipError_t launch_gated_gemv(const BlockView& b, const uint16_t* X, int64_t M, const uint16_t* S, const GatedOut& out,
                             hipStream_t st);
int block_fwd_splits(int64_t M, int64_t N, int64_t K, int layers);
int block_dx_splits(int64_t M, int64_t N, int64_t K, int layers);

namespace {

unsigned cdiv(int64_t a, int64_t b) { return (unsigned)((a + b - 1) / b); }

// ---------------------------------------------------------------------------
// Low-rank factors: D[m][j] = Σ_k L[m][k]·R[j][k] for 64 tokens, 16·NJ ranks and
// one slice of the reduction, as fp32 partial sums P[slice][m][j].  R is A [r,
// Kred] (T, whose L = X has the dropped elements of each LDS stage cleared by the
// wave that copied them, before the stage is opened) or, NATURAL, B [Kred, r] (V,
// whose operand fragments are transposing reads).  Bound by reading L; both
// operands are copied straight into a ring of LDS stages of 64 reduction
// elements, all but one in flight.  4 waves: NJ across the ranks, 4/NJ across the
// rows.  (4096 tokens, K = 4096, r = 64, T with dropout 15.1 us, 34 MB of X at 2.2 TB/s, the
// generator's calls beside the products; V of two layers of 11008 rows 45 us, 180 MB of dG
// and dU at 4.0.  V in the kernel that finds dG and dU, from its registers through LDS: 124 us
// for both, against 75 + 44: half the waves, and a barrier between what they load and
// what they multiply.)
// ---------------------------------------------------------------------------
constexpr int kDownRing = 4;
struct DownJob {
  const uint16_t* L[2];
  const uint16_t* R[2];
  int64_t Kred;
  float* P;  // [layers][slices][M][r]
  int slices;
};

template <int NJ, bool NATURAL>
__device__ __forceinline__ void down_tile(const DownJob& J, int layer, int tile, int slice, int j0, int64_t M, int r,
                                          const DropView& drop, char* sl, char* sr) {
  constexpr int RI = NJ == 4 ? 2 : 1;               // R copies per wave and stage
  constexpr int LB = 64 * 128, RB = 4 * RI * 1024;  // stage bytes
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, kq = lane >> 4;
  const int64_t Kred = J.Kred, m0 = 64 * (int64_t)tile;
  const int all = (int)((Kred + 63) / 64);
  const int s0 = split_first(slice, J.slices, all), s1 = split_first(slice + 1, J.slices, all);
  const i32x4_t rl = rsrc_words(J.L[layer] + m0 * Kred, (M - m0) * Kred * 2);
  const i32x4_t rr = rsrc_words(J.R[layer], (int64_t)r * Kred * 2);
  const bool dropping = !NATURAL && drop.out > 0;
  // L: wave w copies rows 16w + 8c + (lane >> 3), lane i physical chunk i & 7
  const int lch = (lane & 7) ^ (lane >> 3);
  const int lrow = 16 * wave + (lane >> 3);
  const uint32_t chunk0 = (uint32_t)((m0 + lrow) * (Kred / 8)) + lch;
  auto issue = [&](int b, int s) __attribute__((always_inline)) {
    const int64_t k0 = 64 * (int64_t)s;
    const bool in = s < s1 && k0 + 8 * lch < Kred;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      dma_lds16(rl, sl + b * LB + (16 * wave + 8 * c) * 128,
                in ? (uint32_t)(((lrow + 8 * c) * Kred + k0 + 8 * lch) * 2) : 0x7fffffffu, 0u);
#pragma unroll
    for (int c = 0; c < RI; ++c) {
      uint32_t o = 0x7fffffffu;
      if constexpr (NATURAL) {
        // rows of the reduction, 2·NJ chunks of 8 ranks each
        const int idx = 64 * (RI * wave + c) + lane, row = idx / (2 * NJ);
        const int j = j0 + 8 * ((idx % (2 * NJ)) ^ rank_swz<NJ>(row));
        if (row < 64 && s < s1 && k0 + row < Kred && j < r) o = (uint32_t)(((k0 + row) * r + j) * 2);
      } else {
        const int row = 8 * (RI * wave + c) + (lane >> 3), j = j0 + row;
        const int64_t k = k0 + 8 * ((lane & 7) ^ (row & 7));
        if (row < 16 * NJ && j < r && s < s1 && k < Kred) o = (uint32_t)((j * Kred + k) * 2);
      }
      dma_lds16(rr, sr + b * RB + (RI * wave + c) * 1024, o, 0u);
    }
  };
  const int wj = wave % NJ, wr = wave / NJ;  // this wave's rank block, and its NJ row blocks
  f32x4_t acc[NJ];
#pragma unroll
  for (int i = 0; i < NJ; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i + 1 < kDownRing; ++i) issue(i, s0 + i);
  // the generator's bits for a stage are found beside the products of the one before
  u32x4_t bits[2];
  auto draw = [&](int s) __attribute__((always_inline)) {
    if (!dropping) return;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      bits[c] = philox(drop, chunk0 + (uint32_t)(8 * c * (Kred / 8)) + 8u * (uint32_t)s);
  };
  draw(s0);
  for (int s = s0; s < s1; ++s) {
    const int b = (s - s0) % kDownRing;
    if (dropping) {
      // this wave's own copies of the stage
      wait_vmem_le<(kDownRing - 2) * (2 + RI)>();
      asm volatile("" ::: "memory");
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        u32x4_t* const at = reinterpret_cast<u32x4_t*>(sl + b * LB + (16 * wave + 8 * c) * 128 + 16 * lane);
        *at = drop8(drop, bits[c], *at);
      }
    }
    open_stage<(kDownRing - 2) * (2 + RI)>();
    issue((s - s0 + kDownRing - 1) % kDownRing, s + kDownRing - 1);
    draw(s + 1);
    const char* const lt = sl + b * LB;
    const char* const rt = sr + b * RB;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4_t w;
      if constexpr (NATURAL) {
        u32x2_t h[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int row = 32 * ks + 8 * kq + 4 * q + (lr >> 2), col = 16 * wj + 4 * (lr & 3);
          h[q] = lds_read_tr(rt + row * 32 * NJ + (((col >> 3) ^ rank_swz<NJ>(row)) << 4) + 2 * (col & 7));
        }
        w = u32x4_t{h[0][0], h[0][1], h[1][0], h[1][1]};
      } else {
        w = *reinterpret_cast<const u32x4_t*>(rt + dswz(16 * wj + lr, 4 * ks + kq));
      }
#pragma unroll
      for (int i = 0; i < NJ; ++i) {
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(lt + dswz(16 * (NJ * wr + i) + lr, 4 * ks + kq));
        acc[i] = mfma_16x16x32(x, w, acc[i]);
      }
    }
  }
  wait_vmem();  // no copy may land in LDS after the workgroup ends
  const int j = j0 + 16 * wj + lr;
  if (j >= r) return;
  float* const P = J.P + ((int64_t)layer * J.slices + slice) * M * r;
#pragma unroll
  for (int i = 0; i < NJ; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t m = m0 + 16 * (NJ * wr + i) + 4 * kq + v;
      if (m < M) P[m * r + j] = acc[i][v];
    }
}

// Job t (T; no slices: not asked for) and job u (V) in one launch: blockIdx.x =
// tile of 64 tokens, y = slice of t, then of u, z = block of 16·NJ ranks of each
// layer in turn.
template <int NJ>
__global__ __launch_bounds__(256) void block_down_kernel(DownJob t, DownJob u, int64_t M, int r, DropView drop) {
  __shared__ __attribute__((aligned(1024))) char sl[kDownRing * 64 * 128];
  __shared__ __attribute__((aligned(1024))) char sr[kDownRing * 4 * (NJ == 4 ? 2 : 1) * 1024];
  const int tile = (int)blockIdx.x, y = (int)blockIdx.y, blocks = (r + 16 * NJ - 1) / (16 * NJ);
  const int layer = (int)blockIdx.z / blocks, j0 = 16 * NJ * ((int)blockIdx.z - layer * blocks);
  drop = drawn(drop);
  if (y < t.slices)
    down_tile<NJ, false>(t, layer, tile, y, j0, M, r, drop, sl, sr);
  else
    down_tile<NJ, true>(u, layer, tile, y - t.slices, j0, M, r, drop, sl, sr);
}

// T for up to 16 tokens, in one launch: a workgroup per (token, 4 ranks, layer),
// its 4 waves sharing the reduction, 8 elements per lane and step (one token, r = 16,
// two layers 3.7 us, 13 of r = 64 4.5: a launch and the latency of memory).  What is given
// of: T [layers][M][r]; Tt, the single layer's in the dequant-GEMV's tile layout; S
// [layers][M][C], the three-part splits of scale·T.
constexpr int kFewRanks = 4;
// The sums of each wave's v[j] added in wave order, for thread j < R.
template <int R>
__device__ __forceinline__ float few_sum(float (&v)[R]) {
  __shared__ float s_part[4][R];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    v[j] = wave_sum(v[j]);
    if (lane == 0) s_part[wave][j] = v[j];
  }
  __syncthreads();
  const int j = tid < R ? tid : 0;
  return ((s_part[0][j] + s_part[1][j]) + s_part[2][j]) + s_part[3][j];
}
__device__ __forceinline__ void few_split(float v, uint16_t* S, int r) {
  uint16_t o[3];
  split3(v, o);
#pragma unroll
  for (int i = 0; i < 3; ++i) S[i * r] = o[i];
}
// Thread j < kFewRanks: T[m][j0 + j] of the layer with A.
__device__ __forceinline__ float few_down(const uint16_t* __restrict__ X, int64_t m, int64_t K,
                                          const uint16_t* __restrict__ A, int j0, const DropView& drop) {
  constexpr int UN = 2;
  const int tid = threadIdx.x;
  const rsrc_t rl = make_rsrc(X + m * K, K * 2);
  const rsrc_t rr = make_rsrc(A + j0 * K, (int64_t)kFewRanks * K * 2);
  float acc[kFewRanks] = {};
  for (int64_t k0 = 8 * tid; k0 < K; k0 += 2048 * UN) {
    u32x4_t x[UN], w[UN][kFewRanks];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int64_t k = k0 + 2048 * u;
      const bool in = k < K;
      x[u] = buf_load16(rl, in ? (uint32_t)(k * 2) : 0x7fffffffu, 0u);
#pragma unroll
      for (int j = 0; j < kFewRanks; ++j)
        w[u][j] = buf_load16(rr, in ? (uint32_t)((j * K + k) * 2) : 0x7fffffffu, 0u);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (drop.out > 0) x[u] = drop8(drop, philox(drop, (uint32_t)((m * K + k0 + 2048 * u) / 8)), x[u]);
#pragma unroll
      for (int j = 0; j < kFewRanks; ++j) acc[j] = dot8(x[u], w[u][j], acc[j]);
    }
  }
  return __fmul_rn(few_sum(acc), drop.scale);
}
__global__ __launch_bounds__(256) void block_few_down_kernel(const uint16_t* __restrict__ X, int64_t M, int64_t K,
                                                             const uint16_t* __restrict__ A0,
                                                             const uint16_t* __restrict__ A1, int r, DropView drop,
                                                             float scale, float* __restrict__ T,
                                                             float* __restrict__ Tt, uint16_t* __restrict__ S) {
  const int m = (int)blockIdx.x, j0 = kFewRanks * (int)blockIdx.y, layer = (int)blockIdx.z;
  const float t = few_down(X, m, K, layer ? A1 : A0, j0, drawn(drop));
  if (threadIdx.x >= kFewRanks) return;
  const int j = j0 + (int)threadIdx.x;
  if (T) T[(layer * M + m) * r + j] = t;
  if (Tt) Tt[(j >> 4) * 256 + 16 * m + (j & 15)] = t;
  if (S) few_split(__fmul_rn(scale, t), S + (layer * M + m) * adapter_cols(r) + j, r);
}

// The splits of s·T (ST; from T_in where it was saved) and of s·V (SV) of few tokens
// in one launch, in place of block_down_kernel and block_factor_kernel: a workgroup
// per (token, 4 ranks of T) and, blockIdx.z >= layers, one per (token, 8 ranks of V),
// whose threads take two rows of B a step, 16 bytes of each.
__global__ __launch_bounds__(256) void block_few_factors_kernel(DownJob t, DownJob u, const float* __restrict__ T_in,
                                                                int64_t M, int r, int layers, DropView drop, float scale,
                                                                uint16_t* __restrict__ ST, uint16_t* __restrict__ SV) {
  const int tid = threadIdx.x, m = (int)blockIdx.x, z = (int)blockIdx.z, layer = z % layers;
  const int64_t at = layer * M + m;
  if (z < layers) {
    const int j0 = kFewRanks * (int)blockIdx.y;
    float v = 0.f;
    if (!T_in)
      v = few_down(t.L[layer], m, t.Kred, t.R[layer], j0, drawn(drop));
    else if (tid < kFewRanks)
      v = T_in[at * r + j0 + tid];
    if (tid < kFewRanks) few_split(__fmul_rn(scale, v), ST + at * adapter_cols(r) + j0 + tid, r);
    return;
  }
  const int j0 = 8 * (int)blockIdx.y;
  if (j0 >= r) return;
  constexpr int UN = 4;
  const int64_t N = u.Kred;
  const rsrc_t ry = make_rsrc(u.L[layer] + m * N, N * 2), rb = make_rsrc(u.R[layer], N * r * 2);
  float acc[8] = {};
  for (int64_t n0 = 2 * tid; n0 < N; n0 += 512 * UN) {
    uint32_t y[UN];
    u32x4_t b[UN][2];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int64_t n = n0 + 512 * i;
      const bool in = n < N;
      y[i] = buf_load4(ry, in ? (uint32_t)(n * 2) : 0x7fffffffu, 0u);
#pragma unroll
      for (int h = 0; h < 2; ++h) b[i][h] = buf_load16(rb, in ? (uint32_t)(((n + h) * r + j0) * 2) : 0x7fffffffu, 0u);
    }
#pragma unroll
    for (int i = 0; i < UN; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float d = h ? bf16hi(y[i]) : bf16lo(y[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[j] = __builtin_fmaf(d, j & 1 ? bf16hi(b[i][h][j >> 1]) : bf16lo(b[i][h][j >> 1]), acc[j]);
      }
  }
  const float v = __fmul_rn(few_sum(acc), drop.scale);  // (the mask's scale, for dX and dA)
  if (tid < 8) few_split(__fmul_rn(scale, v), SV + at * adapter_cols(r) + j0 + tid, r);
}

// The slices added in order, 16 tokens x 16 ranks per workgroup: v = mult·Σ, as
// fp32 into T_out and as the three-part split of scale·v into S [M, C].  A job
// without slices splits the T it is given.  blockIdx.z: job 0's layers, then job 1's.
struct FactorJob {
  const float* P;
  int slices;
  const float* T_in;
  float* T_out;
  uint16_t* S;
  float mult, scale;
};
__global__ __launch_bounds__(256) void block_factor_kernel(FactorJob t, FactorJob u, int64_t M, int r, int layers) {
  const FactorJob J = (int)blockIdx.z < layers ? t : u;
  const int layer = (int)blockIdx.z % layers;
  const int64_t m = 16 * (int64_t)blockIdx.x + (threadIdx.x >> 4);
  const int j = 16 * (int)blockIdx.y + (threadIdx.x & 15);
  if (m >= M || j >= r) return;
  float v = 0.f;
  if (J.slices == 0) {
    v = J.T_in[(layer * M + m) * r + j];
  } else {
    const float* const p = J.P + ((int64_t)layer * J.slices * M + m) * r + j;
    // (the loads of eight slices, of existing ones whatever their number, before their adds)
    for (int s = 0; s < J.slices; s += 8) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p[(int64_t)std::min(s + i, J.slices - 1) * M * r];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (s + i < J.slices) v += x[i];
    }
    v = __fmul_rn(v, J.mult);
  }
  if (J.T_out) J.T_out[(layer * M + m) * r + j] = v;
  if (!J.S) return;
  uint16_t o[3];
  split3(__fmul_rn(J.scale, v), o);
  uint16_t* const S = J.S + (layer * M + m) * adapter_cols(r) + j;
#pragma unroll
  for (int i = 0; i < 3; ++i) S[i * r] = o[i];
}

// ---------------------------------------------------------------------------
// Gradients: for one unit of tokens, 128 columns of L (X for dA, dY for dB) and
// up to 16·NJ ranks of one layer,
//   D[c][j] = Σ_m L[m][c]·(S[m][j] + S[m][r + j] + S[m][2r + j]).
// Stages of 32 tokens, both operands copied straight into a ring of LDS stages in
// their own layouts (X with its dropped elements cleared by the wave that copied
// them); the MFMA operands, 8 consecutive tokens of one column, are transposing
// reads.  One unit writes the gradient itself, several partial sums that are added
// in unit order.  (4096 tokens, r = 64: one layer of 4096 x 11008 53 us, both of a pair
// of 11008 x 4096 82, 246 MB of X, dG and dU at 3.0 TB/s, the units' sum in a launch after
// it 5 and 6 more; LDS reads of three parts of S
// for each column block, the generator for X of either layer, 10 us of it, and memory
// share the time.  256 columns a workgroup gained nothing.)
// ---------------------------------------------------------------------------
constexpr int kGradRing = 3;
struct GradientJob {
  const uint16_t* L[2];
  const uint16_t* S;  // [layers][M][C]
  int64_t cols;
  float* out[2];
  int64_t part_off;  // of this job within a layer's partial
};

// ALONG: out [cols][r] (dB), else [r][cols] (dA).
template <int NJ, bool ALONG>
__device__ __forceinline__ void gradient_unit(const GradientJob& J, int layer, int64_t c0, int j0, int64_t p0, int64_t p1,
                                              int64_t M, int r, const DropView& drop, float* __restrict__ out, char* sl,
                                              char* ss) {
  constexpr int SI = NJ == 4 ? 3 : NJ == 2 ? 2 : 1;  // S copies per wave and stage
  constexpr int LB = 32 * 256, SB = 4 * SI * 1024, SROW = 96 * NJ;
  // a wave's column and rank blocks: 32 columns of all ranks, of 64 ranks 64 of half of
  // them (20 reads of LDS a stage in place of 28)
  constexpr int PF = NJ == 4 ? 4 : 2, WC = 8 / PF, JF = NJ * WC / 4;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, kq = lane >> 4, C = (int)adapter_cols(r);
  const int stages = (int)((p1 - p0 + 31) / 32);
  const i32x4_t rl = rsrc_words(J.L[layer], p1 * J.cols * 2);
  const i32x4_t rs = rsrc_words(J.S + (int64_t)layer * M * C, p1 * C * 2);
  const bool dropping = !ALONG && drop.out > 0;
  auto issue = [&](int b, int s) __attribute__((always_inline)) {
    // L: wave w copies rows 8w + 4c + (lane >> 4), lane i physical chunk i & 15
    // (tokens past the unit lie past the resources: zeros)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = 8 * wave + 4 * c + (lane >> 4);
      const int64_t col = c0 + 8 * ((lane & 15) ^ ((row & 3) << 1));
      const int64_t m = p0 + 32 * (int64_t)s + row;
      dma_lds16(rl, sl + b * LB + (8 * wave + 4 * c) * 256,
                m < p1 && col < J.cols ? (uint32_t)((m * J.cols + col) * 2) : 0x7fffffffu, 0u);
    }
#pragma unroll
    for (int c = 0; c < SI; ++c) {
      const int idx = 64 * (SI * wave + c) + lane, row = idx / (6 * NJ);
      const int ch = (idx % (6 * NJ)) ^ rank_swz<NJ>(row), part = ch / (2 * NJ), j = j0 + 8 * (ch % (2 * NJ));
      const int64_t m = p0 + 32 * (int64_t)s + row;
      dma_lds16(rs, ss + b * SB + (SI * wave + c) * 1024,
                row < 32 && m < p1 && j < r ? (uint32_t)((m * C + part * r + j) * 2) : 0x7fffffffu, 0u);
    }
  };
  const int wc = 16 * PF * (wave % WC), wj = JF * (wave / WC);
  f32x4_t acc[PF][JF];
#pragma unroll
  for (int i = 0; i < PF; ++i)
#pragma unroll
    for (int j = 0; j < JF; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i + 1 < kGradRing; ++i) issue(i, i);
  // the generator's bits for a stage are found beside the products of the one before
  u32x4_t bits[2];
  auto draw = [&](int s) __attribute__((always_inline)) {
    if (!dropping) return;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = 8 * wave + 4 * c + (lane >> 4);
      const int64_t chunk = (p0 + 32 * (int64_t)s + row) * (J.cols / 8) + c0 / 8 + ((lane & 15) ^ ((row & 3) << 1));
      bits[c] = philox(drop, (uint32_t)chunk);
    }
  };
  draw(0);
  for (int s = 0; s < stages; ++s) {
    if (dropping) {
      // this wave's own copies of the stage
      wait_vmem_le<(kGradRing - 2) * (2 + SI)>();
      asm volatile("" ::: "memory");
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        u32x4_t* const at =
            reinterpret_cast<u32x4_t*>(sl + (s % kGradRing) * LB + (8 * wave + 4 * c) * 256 + 16 * lane);
        *at = drop8(drop, bits[c], *at);
      }
    }
    open_stage<(kGradRing - 2) * (2 + SI)>();
    issue((s + kGradRing - 1) % kGradRing, s + kGradRing - 1);
    draw(s + 1);
    const char* const lt = sl + (s % kGradRing) * LB;
    const char* const st = ss + (s % kGradRing) * SB;
    const int trow = 8 * kq + (lr >> 2), tcol = 4 * (lr & 3);  // this lane's part of a transposing read
    u32x4_t a[PF];
#pragma unroll
    for (int pf = 0; pf < PF; ++pf) {
      const u32x2_t h0 = lds_read_tr(lt + gswz(trow, wc + 16 * pf + tcol));
      const u32x2_t h1 = lds_read_tr(lt + gswz(trow + 4, wc + 16 * pf + tcol));
      a[pf] = u32x4_t{h0[0], h0[1], h1[0], h1[1]};
    }
#pragma unroll
    for (int part = 0; part < 3; ++part)
#pragma unroll
      for (int jf = 0; jf < JF; ++jf) {
        const int col = 16 * (NJ * part + wj + jf) + tcol;
        u32x2_t h[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int row = trow + 4 * q;
          h[q] = lds_read_tr(st + row * SROW + (((col >> 3) ^ rank_swz<NJ>(row)) << 4) + 2 * (col & 7));
        }
        const u32x4_t f = {h[0][0], h[0][1], h[1][0], h[1][1]};
#pragma unroll
        for (int pf = 0; pf < PF; ++pf)
          acc[pf][jf] = ALONG ? mfma_16x16x32(a[pf], f, acc[pf][jf]) : mfma_16x16x32(f, a[pf], acc[pf][jf]);
      }
  }
  wait_vmem();  // no copy may land in LDS after the workgroup ends
#pragma unroll
  for (int pf = 0; pf < PF; ++pf)
#pragma unroll
    for (int jf = 0; jf < JF; ++jf)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t cb = c0 + wc + 16 * pf;
        const int jbase = j0 + 16 * (wj + jf);
        const int64_t c = ALONG ? cb + 4 * kq + v : cb + lr;
        const int j = ALONG ? jbase + lr : jbase + 4 * kq + v;
        if (c < J.cols && j < r) out[ALONG ? c * r + j : j * J.cols + c] = acc[pf][jf][v];
      }
}

// The sum of dX's split partials (n4 = 0: none), for the workgroups past the units'.
struct SplitSum {
  const f32x4_t* P;
  int splits;
  int64_t n4;
  void* out;
  int out16;
};
// blockIdx.x: 128 columns of dA, then of dB; y: the unit; z: block of 16·NJ ranks
// of each layer in turn.  P [units][layers][r·(K + N)], or null with one unit.
template <int NJ>
__global__ __launch_bounds__(256) void block_gradient_kernel(GradientJob ja, GradientJob jb, unsigned tiles_a, int64_t M,
                                                             int r, int64_t unit, int units, int layers, DropView drop,
                                                             float* __restrict__ P, SplitSum sum) {
  __shared__ __attribute__((aligned(1024))) char sl[kGradRing * 32 * 256];
  __shared__ __attribute__((aligned(1024))) char ss[kGradRing * 4 * (NJ == 4 ? 3 : NJ == 2 ? 2 : 1) * 1024];
  const int blocks = (r + 16 * NJ - 1) / (16 * NJ);
  const int layer = (int)blockIdx.z / blocks, j0 = 16 * NJ * ((int)blockIdx.z - layer * blocks);
  if ((int)blockIdx.y >= units) {
    const int64_t block = ((int64_t)(blockIdx.y - units) * gridDim.z + blockIdx.z) * gridDim.x + blockIdx.x;
    const int64_t i = 256 * block + threadIdx.x;
    if (i < sum.n4) splitk_sum4<false>(sum.P, sum.splits, sum.n4, i, sum.out, sum.out16);
    return;
  }
  const int64_t p0 = unit * blockIdx.y, p1 = std::min<int64_t>(p0 + unit, M);
  const int64_t part = ((int64_t)blockIdx.y * layers + layer) * r * (ja.cols + jb.cols);
  drop = drawn(drop);
  // (dA's tiles, whose masks cost vector time, spread evenly between dB's)
  const unsigned tile_a = (unsigned)((uint64_t)blockIdx.x * tiles_a / gridDim.x);
  const bool is_a = (uint64_t)(blockIdx.x + 1) * tiles_a / gridDim.x > tile_a;
  if (is_a)
    gradient_unit<NJ, false>(ja, layer, 128 * (int64_t)tile_a, j0, p0, p1, M, r, drop,
                             P ? P + part + ja.part_off : ja.out[layer], sl, ss);
  else
    gradient_unit<NJ, true>(jb, layer, 128 * (int64_t)(blockIdx.x - tile_a), j0, p0, p1, M, r, drop,
                            P ? P + part + jb.part_off : jb.out[layer], sl, ss);
}

// The units' partial sums added in order, four values per thread; blockIdx.y: the layer.
__global__ __launch_bounds__(256) void block_gradient_finish_kernel(float* dA0, float* dB0, float* dA1, float* dB1,
                                                                    int64_t na, int64_t nb, int layers,
                                                                    const float* __restrict__ P, int units) {
  const int layer = (int)blockIdx.y;
  float* const dA = layer ? dA1 : dA0;
  float* const dB = layer ? dB1 : dB0;
  const float* const p = P + layer * (na + nb);
  for (int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x); i < na + nb; i += 1024 * (int64_t)gridDim.x) {
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int q = 0; q < units; ++q) {
      const f32x4_t x = *reinterpret_cast<const f32x4_t*>(p + (int64_t)q * layers * (na + nb) + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += x[e];
    }
    *reinterpret_cast<f32x4_t*>(i < na ? dA + i : dB + (i - na)) = v;
  }
}

// ---------------------------------------------------------------------------
// Element by element
// ---------------------------------------------------------------------------

// The gated block's split partials added in order, and its outputs; four columns a
// thread.  rows: [splits][M][2N], each row the gate's N columns, then the other
// layer's; else [2][splits][M][N].
__global__ __launch_bounds__(256) void gated_reduce_kernel(const f32x4_t* __restrict__ P, int splits, int64_t M, int64_t N,
                                                           bool rows, GatedOut out) {
  const int64_t n4 = N / 4, total = M * n4;
  const int64_t up = rows ? n4 : splits * total, split = rows ? 2 * total : total;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += 256 * (int64_t)gridDim.x) {
    const f32x4_t* const p = P + (rows ? i + i / n4 * n4 : i);
    f32x4_t g = p[0], u = p[up];
    for (int s = 1; s < splits; ++s) {
      const f32x4_t a = p[s * split], b = p[s * split + up];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] += a[e];
        u[e] += b[e];
      }
    }
    float h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = gate_act(out.act, g[e]) * u[e];
    reinterpret_cast<u32x2_t*>(out.H)[i] = u32x2_t{pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
    if (out.G) {
      reinterpret_cast<u32x2_t*>(out.G)[i] = u32x2_t{pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3])};
      reinterpret_cast<u32x2_t*>(out.U)[i] = u32x2_t{pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3])};
    }
  }
}

// dG = dH·U·act'(G) and dU = dH·act(G), eight elements a thread.  The products
// after it take them in 16 bits, so those are the definition's to the bit: RNE_bf16
// of the fp32 value nearest to the exact one.  fp32 arithmetic gives that unless
// the value lies within its error of a border between two bf16 numbers, and there
// (about one element in 1,000) 64 bits decide.  Bound by memory: 4096 x 11008 75 us,
// 472 MB at 6.3 TB/s, part of it the last-level cache's (95 with an exact division and
// a separate test of each rounding, 87 vector instructions an element).
// act' = σ·(1 + g·(1 − σ)·h'), with 1 − σ = σ(−h) from the same exponential.
struct GateGradient {
  float dg, du;
};
// In 64 bits: off by less than 2^-45 of the terms' size.
__device__ __noinline__ GateGradient gate_gradient_exact(int act, float g, float u, float dh) {
  const double x = g;
  double h = x, slope = 1.0;
  if (act == kActGeluTanh) {
    h = kGeluSlope * (x + kGeluCube * x * x * x);
    slope = kGeluSlope * (1.0 + 3.0 * kGeluCube * x * x);
  }
  const double s = 1.0 / (1.0 + exp(-h)), r = 1.0 / (1.0 + exp(h));
  const double t = r > 0.0 ? x * r * slope : 0.0;  // (0 in the limit of an infinite g)
  return {(float)((double)dh * u * (s * (1.0 + t))), (float)((double)dh * (x * s))};
}
// In 32 bits, and whether both round as the exact values do.  With u = 2^-24 and an
// exponential and a reciprocal of 1 ulp, σ(−|h|) is off by (6 + 2|h|)u of itself and
// σ(|h|) by 5u (GELU, whose h is off by 5u of itself: 6 + 7|h| and 6); dU adds two
// roundings, dG three and those of t = g·σ(−h)·h', and the test's own is one more.
__device__ __forceinline__ bool gate_gradient(int act, float g, float u, float dh, GateGradient& d) {
  float h = g, slope = 1.f, per_h = 2.f * 0x1p-24f, more = 8.f * 0x1p-24f;
  if (act == kActGeluTanh) {
    const float g2 = g * g;
    h = (float)kGeluSlope * __builtin_fmaf((float)kGeluCube * g2, g, g);
    slope = (float)kGeluSlope * __builtin_fmaf(3.f * (float)kGeluCube, g2, 1.f);
    per_h = 8.f * 0x1p-24f;
    more = 12.f * 0x1p-24f;
  }
  const float e = __builtin_amdgcn_exp2f(fabsf(h) * -1.44269502f), near = __builtin_amdgcn_rcpf(1.f + e), far = e * near;
  const float s = h < 0.f ? far : near, r = h < 0.f ? near : far;
  const float y = dh * s, t = g * r * slope, yu = y * u;
  d = {yu * (1.f + t), y * g};
  const float unit = __builtin_fmaf(per_h, fabsf(h), 10.f * 0x1p-24f);
  // (2^-140: what underflows behind y, 2^-150 times 1 + |t|, below 200 where h is above −80)
  const float off_u = __builtin_fmaf(unit, fabsf(d.du), 0x1p-140f);
  const float off_g = __builtin_fmaf((unit + more) * (1.f + fabsf(t)), fabsf(yu), 0x1p-140f);
  const uint32_t differ = pack_bf16x2(d.du - off_u, d.dg - off_g) ^ pack_bf16x2(d.du + off_u, d.dg + off_g);
  // (what dh·σ loses below fp32's normal numbers, U and G may bring back up; σ itself is
  // one above h = −80, and a dH of 0 loses nothing)
  const bool whole = fabsf(y) >= 0x1p-126f || dh == 0.f;
  // (zeros of either sign are alike; below −80 the exponential nears fp32's end and
  // loses bits; NaN may be an infinity times what is 0 in fp32 alone)
  return whole && h > -80.f && (differ & 0x7fff7fffu) == 0u && !__builtin_isunordered(d.du, d.dg);
}
__global__ __launch_bounds__(256) void gate_gradient_kernel(const uint16_t* __restrict__ dH, const uint16_t* __restrict__ G,
                                                            const uint16_t* __restrict__ U, int64_t n8, int act,
                                                            uint16_t* __restrict__ dG, uint16_t* __restrict__ dU) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += 256 * (int64_t)gridDim.x) {
    const u32x4_t h = reinterpret_cast<const u32x4_t*>(dH)[i], g = reinterpret_cast<const u32x4_t*>(G)[i],
                  u = reinterpret_cast<const u32x4_t*>(U)[i];
    u32x4_t og, ou;
    uint32_t unsure = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      GateGradient a, b;
      if (!gate_gradient(act, bf16lo(g[q]), bf16lo(u[q]), bf16lo(h[q]), a)) unsure |= 1u << (2 * q);
      if (!gate_gradient(act, bf16hi(g[q]), bf16hi(u[q]), bf16hi(h[q]), b)) unsure |= 2u << (2 * q);
      og[q] = pack_bf16x2(a.dg, b.dg);
      ou[q] = pack_bf16x2(a.du, b.du);
    }
    reinterpret_cast<u32x4_t*>(dG)[i] = og;
    reinterpret_cast<u32x4_t*>(dU)[i] = ou;
    asm volatile("" ::: "memory");  // (the stores below come after those above)
    for (; unsure != 0u; unsure &= unsure - 1u) {
      const int64_t at = 8 * i + __builtin_ctz(unsure);
      const GateGradient d = gate_gradient_exact(act, bf16lo(G[at]), bf16lo(U[at]), bf16lo(dH[at]));
      dG[at] = (uint16_t)(pack_bf16x2(d.dg, 0.f) & 0xffffu);
      dU[at] = (uint16_t)(pack_bf16x2(d.du, 0.f) & 0xffffu);
    }
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

// NJ blocks of 16 ranks per workgroup
int rank_blocks(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }

// Slices of a low-rank factor's reduction: about 512 workgroups, of 4 stages each
// or more, 16 at most.
int down_slices(int64_t M, int64_t Kred, int r, int layers) {
  const int64_t work = (int64_t)cdiv(M, 64) * cdiv(r, 16 * rank_blocks(r)) * layers;
  return (int)std::max<int64_t>(1, std::min<int64_t>({512 / work, (int64_t)cdiv(Kred, 256), 16}));
}

hipError_t launch_down(const DownJob& t, const DownJob& u, int64_t M, int r, int layers, const DropView& drop,
                       hipStream_t st) {
  const int nj = rank_blocks(r);
  const dim3 grid(cdiv(M, 64), (unsigned)(t.slices + u.slices), (unsigned)layers * cdiv(r, 16 * nj));
  if (nj == 1)
    block_down_kernel<1><<<grid, 256, 0, st>>>(t, u, M, r, drop);
  else if (nj == 2)
    block_down_kernel<2><<<grid, 256, 0, st>>>(t, u, M, r, drop);
  else
    block_down_kernel<4><<<grid, 256, 0, st>>>(t, u, M, r, drop);
  return hipGetLastError();
}

// Whether a backward pass takes its factors from block_few_factors_kernel: one launch
// for two, but each token reads its 16 bytes of every row of B, lines of which hold
// other ranks'.  (A whole pass of 61 tokens, N x K, replayed, us against the two:
// 4096 x 4096 r = 8 28.0 and 32.1, r = 32 30.3 and 33.2, r = 64 38.0 and 35.1; 4096 x
// 11008 r = 16 39.7 and 46.3, r = 32 43.0 and 47.1, r = 64 51.6 and 49.3; 11008 x 4096
// r = 16 38.7 and 39.0, r = 32 43.0 and 40.2.  4 tokens: 21.4 and 24.3, 32.7 and 39.2,
// 33.5 and 32.8 at r = 8, 16 and 16.)
bool few_factors(int64_t M, int64_t N, int64_t K, int r) {
  return M <= kMidTokens && (r <= 16 || (r <= 32 && N <= K));
}

// Units of tokens of the gradients' reduction: as many as fill the chip about
// twice over, of 64 tokens or more.
int64_t gradient_unit(int64_t M, int64_t N, int64_t K, int r, int layers) {
  const int64_t work = (int64_t)(cdiv(K, 128) + cdiv(N, 128)) * cdiv(r, 16 * rank_blocks(r)) * layers;
  const int64_t parts = std::max<int64_t>(1, (512 + work / 2) / work);
  return round_up((std::max<int64_t>(M, 1) + parts - 1) / parts, 64);
}

}  // namespace

BlockFwdLayout block_fwd_layout(int64_t M, int64_t N, int64_t K, int r, int layers) {
  BlockFwdLayout L{};
  L.splits = 1;
  if (M == 0) return L;
  if (M <= 16) {
    L.total = layers == 1 ? (int64_t)cdiv(r, 16) * 1024 : 2 * M * adapter_cols(r) * 2;  // T's tiles; S
    return L;
  }
  if (M <= kMidTokens) {
    L.splits = mid_fwd_plan(M, N, K, layers).splits;
  } else {
    L.splits = block_fwd_splits(M, N, K, layers);
    L.slices = down_slices(M, K, r, layers);
  }
  L.off_P = round_up(layers * M * adapter_cols(r) * 2, 256);
  // (two layers of few tokens leave fp32 sums whatever their splits)
  const bool sums = L.splits > 1 || (layers == 2 && M <= kMidTokens);
  const int64_t gemm = sums ? (int64_t)L.splits * M * N * layers * 4 : 0;
  L.total = L.off_P + round_up(std::max(gemm, (int64_t)L.slices * layers * M * r * 4), 256);
  return L;
}

BlockBwdLayout block_bwd_layout(int64_t M, int64_t N, int64_t K, int r, int layers) {
  BlockBwdLayout L{};
  if (M == 0) return L;
  L.splits = M <= kMidTokens ? layers * mid_dx_splits(M, N, K, layers) : block_dx_splits(M, N, K, layers);
  L.slices_T = down_slices(M, K, r, layers);
  L.slices_V = down_slices(M, N, r, layers);
  L.unit = gradient_unit(M, N, K, r, layers);
  L.units = (int)((M + L.unit - 1) / L.unit);
  size_t off = 0;
  L.off_dY = off;
  off += layers == 2 ? round_up(2 * M * N * 2, 256) : 0;
  L.off_V = off;
  off += round_up(layers * M * adapter_cols(r) * 2, 256);
  L.off_T = off;
  off += round_up(layers * M * adapter_cols(r) * 2, 256);
  L.off_P = off;
  const int64_t gemm = L.splits > 1 ? (int64_t)L.splits * M * K * 4 : 0;
  const int64_t factors = (int64_t)(L.slices_V + L.slices_T) * layers * M * r * 4;
  L.off_Q = off + round_up(gemm, 256);  // (read while the gradients' are written)
  const int64_t gradients = L.units > 1 ? round_up(gemm, 256) + (int64_t)L.units * layers * r * (K + N) * 4 : 0;
  L.total = off + round_up(std::max({gemm, factors, gradients}), 256);
  return L;
}

// The largest totals over M in [0, M_max].  Up to kMidTokens tokens each is taken.
// Above, split and slice counts are constant between multiples of 64 tokens, and
// what they count grows with M: the last of every 64 and the first of the next are
// taken.
namespace {
template <typename F>
size_t most_of(int64_t M_max, F&& total) {
  size_t most = 0;
  for (int64_t M = 1; M <= std::min(M_max, kMidTokens); ++M) most = std::max(most, total(M));
  if (M_max > kMidTokens) most = std::max(most, total(kMidTokens + 1));
  for (int64_t top = kMidTokens + 64; M_max > kMidTokens; top += 64) {
    most = std::max(most, total(std::min(top, M_max)));
    if (top >= M_max) break;
    most = std::max(most, total(top + 1));
  }
  return most;
}
}  // namespace
size_t block_fwd_ws_max(int64_t M_max, int64_t N, int64_t K, int r, int layers) {
  return most_of(M_max, [&](int64_t M) { return block_fwd_layout(M, N, K, r, layers).total; });
}
size_t block_bwd_ws_max(int64_t M_max, int64_t N, int64_t K, int r, int layers) {
  return most_of(M_max, [&](int64_t M) { return block_bwd_layout(M, N, K, r, layers).total; });
}

hipError_t launch_block_fwd(const BlockView& b, const uint16_t* X, int64_t M, void* Y, bool y16, float* T,
                            const GatedOut& out, char* ws, const BlockFwdLayout& L, hipStream_t st) {
  if (M == 0) return hipSuccess;
  const int64_t N = b.W[0].N, K = b.W[0].K;
  const bool pair = b.layers == 2;
  float* P = reinterpret_cast<float*>(ws + L.off_P);
  if (M <= 16) {
    uint16_t* const S = pair ? reinterpret_cast<uint16_t*>(ws) : nullptr;
    block_few_down_kernel<<<dim3((unsigned)M, (unsigned)(b.r / kFewRanks), (unsigned)b.layers), 256, 0, st>>>(
        X, M, K, b.A[0], b.A[1], b.r, b.drop, b.scale, T, pair ? nullptr : P, S);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    float* const kept = nullptr;  // (T is written)
    return pair ? launch_gated_gemv(b, X, M, S, out, st)
                : launch_gemv_sums(b.W[0], X, M, P, 1, (int)cdiv(b.r, 16), b.B[0], b.r, b.scale, Y, y16, kept, false, st);
  }
  uint16_t* S = reinterpret_cast<uint16_t*>(ws);
  const int C = (int)adapter_cols(b.r), cols = (pair || y16 ? 2 : 3) * b.r;
  auto reduce = [&](bool rows) {
    gated_reduce_kernel<<<std::min(cdiv(M * N / 4, 256), 2048u), 256, 0, st>>>(reinterpret_cast<const f32x4_t*>(P),
                                                                               L.splits, M, N, rows, out);
    return hipGetLastError();
  };
  if (M <= kMidTokens) {
    // (at every rank; launch_down's tiles were not measured here)
    float* const none = nullptr;
    block_few_down_kernel<<<dim3((unsigned)M, (unsigned)(b.r / kFewRanks), (unsigned)b.layers), 256, 0, st>>>(
        X, M, K, b.A[0], b.A[1], b.r, b.drop, b.scale, T, none, S);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const DenseGemmArgs ma{S, b.B[0], b.r, C, 1, cols, (int)M, b.drop, b.W[pair ? 1 : 0], X, b.B[pair ? 1 : 0],
                           M * C, (int64_t)L.splits * M * N};
    e = launch_mid_fwd_block(b.W[0], X, M, ma, pair ? (void*)P : Y, !pair && y16, mid_fwd_plan(M, N, K, b.layers), P,
                             b.layers, st);
    if (e != hipSuccess) return e;
    if (pair) return reduce(false);
    return L.splits > 1 ? launch_splitk_reduce(P, L.splits, M * N, Y, y16, false, st) : hipSuccess;
  }
  const DownJob t{{X, X}, {b.A[0], b.A[1]}, K, P, L.slices};
  hipError_t e = launch_down(t, DownJob{}, M, b.r, b.layers, b.drop, st);
  if (e != hipSuccess) return e;
  const FactorJob f{P, L.slices, nullptr, T, S, b.drop.scale, b.scale};
  block_factor_kernel<<<dim3(cdiv(M, 16), cdiv(b.r, 16), (unsigned)b.layers), 256, 0, st>>>(f, f, M, b.r, b.layers);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  // (the partial sums of T have been consumed: P now takes the split partials.  16-bit outputs take
  // 16 bits of s·T, as AdapterGemmArgs says)
  const BlockGemmArgs ma{S, {b.B[0], b.B[1]}, b.r, C, cols, b.W[pair ? 1 : 0], out.G, out.U, out.act, nullptr, b.drop};
  e = launch_fwd_gemm_block(b.W[0], X, M, ma, pair, pair ? (void*)out.H : Y, y16, L.splits, P, st);
  if (e != hipSuccess || L.splits == 1) return e;
  return pair ? reduce(true) : launch_splitk_reduce(P, L.splits, M * N, Y, y16, false, st);
}

hipError_t launch_block_bwd(const BlockView& b, const uint16_t* X, int64_t M, const uint16_t* dY, const GatedIn& in,
                            const float* T_saved, void* dX, bool dx16, float* const dA[2], float* const dB[2], char* ws,
                            const BlockBwdLayout& L, hipStream_t st) {
  const int64_t N = b.W[0].N, K = b.W[0].K, r = b.r;
  const int layers = b.layers;
  const bool pair = layers == 2;
  hipError_t e;
  if (M == 0) {  // no tokens: the adapter gradients are zero
    for (int l = 0; l < layers; ++l) {
      if ((e = launch_zero(dA[l], r * K, st)) != hipSuccess) return e;
      if ((e = launch_zero(dB[l], N * r, st)) != hipSuccess) return e;
    }
    return hipSuccess;
  }
  uint16_t* SV = reinterpret_cast<uint16_t*>(ws + L.off_V);
  uint16_t* ST = reinterpret_cast<uint16_t*>(ws + L.off_T);
  float* P = reinterpret_cast<float*>(ws + L.off_P);
  const uint16_t* d[2] = {dY, nullptr};
  if (pair) {
    uint16_t* dG = reinterpret_cast<uint16_t*>(ws + L.off_dY);
    uint16_t* dU = dG + M * N;
    gate_gradient_kernel<<<std::min(cdiv(M * N / 8, 256), 8192u), 256, 0, st>>>(
        in.dH, in.G, in.U, M * N / 8, in.act, dG, dU);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    d[0] = dG;
    d[1] = dU;
  }
  // V, and T unless it was saved
  const int slices_T = T_saved ? 0 : L.slices_T;
  float* const PV = P + (int64_t)slices_T * layers * M * r;
  const DownJob t{{X, X}, {b.A[0], b.A[1]}, K, P, slices_T}, v{{d[0], d[1]}, {b.B[0], b.B[1]}, N, PV, L.slices_V};
  if (few_factors(M, N, K, r)) {
    block_few_factors_kernel<<<dim3((unsigned)M, (unsigned)(r / kFewRanks), 2u * layers), 256, 0, st>>>(
        t, v, T_saved, M, r, layers, b.drop, b.scale, ST, SV);
  } else {
    if ((e = launch_down(t, v, M, r, layers, b.drop, st)) != hipSuccess) return e;
    const FactorJob ft{P, slices_T, T_saved, nullptr, ST, b.drop.scale, b.scale};
    const FactorJob fv{PV, L.slices_V, nullptr, nullptr, SV, b.drop.scale, b.scale};
    block_factor_kernel<<<dim3(cdiv(M, 16), cdiv(r, 16), 2u * layers), 256, 0, st>>>(ft, fv, M, r, layers);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int C = (int)adapter_cols(r), cols = (dx16 ? 2 : 3) * b.r;
  if (M <= kMidTokens) {
    // (each layer's splits into their own partials, added together)
    const int splits = L.splits / layers;
    const DenseGemmArgs ma{SV, b.A[0], b.r, C, 1, cols, (int)M, b.drop, b.W[pair ? 1 : 0], d[1], b.A[pair ? 1 : 0],
                           M * C, (int64_t)splits * M * K};
    e = launch_mid_dx_block(b.W[0], d[0], M, ma, L.splits > 1 ? (void*)P : dX, L.splits == 1 && dx16, splits, P, layers,
                            st);
  } else {
    const BlockGemmArgs ma{SV, {b.A[0], b.A[1]}, b.r, C, cols, b.W[pair ? 1 : 0], nullptr, nullptr, in.act, d[1], b.drop};
    e = launch_dx_gemm_block(b.W[0], d[0], M, ma, pair, dX, dx16, L.splits, P, st);
  }
  if (e != hipSuccess) return e;
  // the gradients; with them the sum of dX's splits
  const GradientJob ja{{X, X}, SV, K, {dA[0], dA[1]}, 0}, jb{{d[0], d[1]}, ST, N, {dB[0], dB[1]}, r * K};
  const int nj = rank_blocks(b.r);
  const unsigned ta = cdiv(K, 128);
  const unsigned gx = ta + cdiv(N, 128), gz = (unsigned)layers * cdiv(r, 16 * nj);
  const SplitSum sum{reinterpret_cast<const f32x4_t*>(P), L.splits, L.splits > 1 ? M * K / 4 : 0, dX, dx16 ? 1 : 0};
  const dim3 grid(gx, (unsigned)L.units + cdiv(sum.n4, (int64_t)256 * gx * gz), gz);
  float* const parts = L.units > 1 ? reinterpret_cast<float*>(ws + L.off_Q) : nullptr;
  if (nj == 1)
    block_gradient_kernel<1><<<grid, 256, 0, st>>>(ja, jb, ta, M, b.r, L.unit, L.units, layers, b.drop, parts, sum);
  else if (nj == 2)
    block_gradient_kernel<2><<<grid, 256, 0, st>>>(ja, jb, ta, M, b.r, L.unit, L.units, layers, b.drop, parts, sum);
  else
    block_gradient_kernel<4><<<grid, 256, 0, st>>>(ja, jb, ta, M, b.r, L.unit, L.units, layers, b.drop, parts, sum);
  e = hipGetLastError();
  if (e != hipSuccess || L.units == 1) return e;
  block_gradient_finish_kernel<<<dim3(std::min(cdiv(r * (K + N), 1024), 1024u), (unsigned)layers), 256, 0, st>>>(
      dA[0], dB[0], dA[1], dB[1], r * K, r * N, layers, parts, L.units);
  return hipGetLastError();
}

}  // namespace qnf4
