// Low-rank adapters of many requests beside one quantized weight, gfx950:
//   Y[m] = X[m]·Ŵᵀ + s_a·(X[m]·A_aᵀ)·B_aᵀ,  a = a(m) the adapter of token m,
// and its gradients, with T = X[m]·A_aᵀ and U = dY[m]·B_a:
//   dX[m] = dY[m]·Ŵ + s_a·U[m]·A_a,
//   dA_a = s_a·Σ_{m: a(m) = a} U[m]ᵀ·X[m],  dB_a = s_a·Σ_{m: a(m) = a} dY[m]ᵀ·T[m].
// A plan sorts the batch's tokens by adapter.  The low-rank factors T and U are
// small products over tiles of 16 sorted positions; the base products run in
// the dequant-in-tile GEMMs over the sorted positions, whose reductions go on
// over the low-rank factors (fwd.hip, dx.hip; up to 16 tokens: gemv.hip), so
// that Y and dX are written once; the adapters' gradients are reductions over
// runs of positions.
#include <algorithm>

#include "host.h"
#include "splitk.h"
#include "tiling.h"

namespace qnf4 {

hipError_t launch_dx_gemm_adapters(const Nf4View& W, const uint16_t* dY, int64_t M, const AdapterGemmArgs& ma, void* dX,
                                   bool dx16, int splits, float* P, hipStream_t st);
hipError_t launch_fwd_gemm_adapters(const Nf4View& W, const uint16_t* X, int64_t M, const AdapterGemmArgs& ma, void* Y,
                                    bool y16, int splits, float* P, hipStream_t st);
hipError_t launch_gemv_adapters(const Nf4View& W, const uint16_t* X, int64_t M, const AdapterView& ad,
                                const int32_t* owner, void* Y, bool y16, const float* T, hipStream_t st);
hipError_t launch_splitk_reduce(const float* P, int splits, int64_t n, void* out, bool out16, bool f16,
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
// adapter's number.  Bound by latency: 5.6 us for 64 tokens or fewer, 8.5 for
// 2,045 of 40 adapters, 12 to 15 for 4,096, once for every layer and both passes.
// ---------------------------------------------------------------------------
constexpr int kPlanWaves = 16;
static_assert(kMaxAdapters <= 64 * kPlanWaves, "a thread per adapter");
__global__ __launch_bounds__(64 * kPlanWaves) void adapters_plan_kernel(const int32_t* __restrict__ index, int64_t M,
                                                                        int count, PlanView pl) {
  extern __shared__ int32_t hist[];  // [16][count + 1]; column `count`: no adapter
  __shared__ int32_t s_wave[3][kPlanWaves];
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
  // the tokens, of "carries any token" and of the 64-position tiles
  int total = 0;
  if (tid < count)
    for (int w = 0; w < kPlanWaves; ++w) total += hist[w * cols + tid];
  const int used = total > 0 ? 1 : 0;
  const int tiles = (total + 63) / 64;
  int st = total, su = used, sx = tiles;
  for (int o = 1; o < 64; o <<= 1) {
    const int a = __shfl_up(st, o, 64), b = __shfl_up(su, o, 64), c = __shfl_up(sx, o, 64);
    if (lane >= o) {
      st += a;
      su += b;
      sx += c;
    }
  }
  if (lane == 63) {
    s_wave[0][wave] = st;
    s_wave[1][wave] = su;
    s_wave[2][wave] = sx;
  }
  __syncthreads();
  int all = 0, nact = 0, all_tiles = 0;
  st -= total;
  su -= used;
  sx -= tiles;
  for (int w = 0; w < kPlanWaves; ++w) {
    if (w < wave) {
      st += s_wave[0][w];
      su += s_wave[1][w];
      sx += s_wave[2][w];
    }
    all += s_wave[0][w];
    nact += s_wave[1][w];
    all_tiles += s_wave[2][w];
  }
  __syncthreads();
  if (tid < count) {
    pl.slot[tid] = used ? su : -1;
    if (used) {
      pl.id[su] = tid;
      pl.start[su] = st;
      for (int i = 0; i < tiles; ++i) pl.tile[sx + i] = int2{su, st + 64 * i};
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
    pl.head[2] = all_tiles;
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
// Low-rank factors, three-part: v = s_a·D as hi + mid + lo in bf16 (24 bits:
// products with it are as exact as fp32 ones).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void split3(float v, uint16_t* o) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t h = pack_bf16x2(v, 0.0f) & 0xffffu;
    o[i] = (uint16_t)h;
    v = __fsub_rn(v, __uint_as_float(h << 16));
  }
}

// D[p][j] = Σ_k L[token(p)][k]·R_a(j, k) for the positions of one plan tile (up
// to 64 of one adapter), 16·NJ ranks and one slice of the reduction, as fp32
// partial sums P[slice][p][j].  R_a is A_a [r, Kred] (T = X·A_aᵀ) or, NATURAL,
// B_a [Kred, r] (U = dY·B_a), whose operand fragments are transposing reads.
// Bound by reading L once: both operands are copied straight into a ring of
// LDS stages (64 reduction elements; L rows gathered through the plan), all
// but one in flight, and the slices give every compute unit a part of the
// ring's traffic (64 positions per tile read R a quarter as often as 16).  4
// waves: NJ across the ranks, 4/NJ across the rows.  (4096 x 4096, r = 64, 8
// adapters: 16.8 us, 68 MB at 4.1 TB/s; tiles of 16 positions with operands
// straight from memory took 43.  U of 4096 x 4096, r = 16: 10.0 us, 4.1 TB/s.)
constexpr int kDownRing = 4;
struct DownJob {
  const uint16_t* L;
  int64_t Kred;
  const uint16_t* R;
  float* P;
  int slices;
};
// NATURAL: the 16-byte chunks of a reduction row (2·NJ of them) XORed by bits
// of the row, so that the 4 rows of a transposing read lie on different banks.
template <int NJ>
__device__ __forceinline__ int rank_swz(int row) {
  return NJ == 4 ? (row & 3) << 1 : NJ == 2 ? row & 2 : 0;
}
__device__ __forceinline__ int dswz(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

template <int NJ, bool NATURAL>
__device__ __forceinline__ void down_tile(const DownJob& J, int tile, int slice, int j0, int64_t M,
                                          const AdapterView& ad, const PlanView& pl, char* sl, char* sr) {
  constexpr int RI = NJ == 4 ? 2 : 1;                  // R copies per wave and stage
  constexpr int LB = 64 * 128, RB = 4 * RI * 1024;     // stage bytes
  const int2 tl = pl.tile[tile];
  const int g = std::min(std::max(tl.x, 0), ad.count - 1), r = ad.r;
  const int p0 = std::max(tl.y, 0), p1 = (int)std::min<int64_t>(std::min(p0 + 64, pl.start[g + 1]), M);
  const int id = pl.id[g];
  if ((unsigned)id >= (unsigned)ad.count || p0 >= p1) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, kq = lane >> 4;
  const int64_t Kred = J.Kred;
  const int all = (int)((Kred + 63) / 64);
  const int s0 = split_first(slice, J.slices, all), s1 = split_first(slice + 1, J.slices, all);
  const i32x4_t rl = rsrc_words(J.L, M * Kred * 2);
  const i32x4_t rr = rsrc_words(J.R + (int64_t)id * r * Kred, (int64_t)r * Kred * 2);
  // L: wave w copies rows 16w + 8c + (lane >> 3), lane i physical chunk i & 7
  const int lch = (lane & 7) ^ (lane >> 3);
  uint32_t vl[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int pos = p0 + 16 * wave + 8 * c + (lane >> 3);
    const int tok = pl.perm[std::min(pos, p1 - 1)];
    vl[c] = pos < p1 && (uint32_t)tok < (uint32_t)M ? (uint32_t)tok * (uint32_t)Kred * 2u + 16u * lch : 0x7fffffffu;
  }
  auto issue = [&](int b, int s) __attribute__((always_inline)) {
    const int64_t k0 = 64 * (int64_t)s;
    const bool in = s < s1 && k0 + 8 * lch < Kred;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      dma_lds16(rl, sl + b * LB + (16 * wave + 8 * c) * 128, in ? vl[c] + (uint32_t)(k0 * 2) : 0x7fffffffu, 0u);
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
  for (int s = s0; s < s1; ++s) {
    const int b = (s - s0) % kDownRing;
    open_stage<(kDownRing - 2) * (2 + RI)>();
    issue((s - s0 + kDownRing - 1) % kDownRing, s + kDownRing - 1);
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
#pragma unroll
  for (int i = 0; i < NJ; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int pos = p0 + 16 * (NJ * wr + i) + 4 * kq + v;
      if (pos < p1) J.P[((int64_t)slice * M + pos) * r + j] = acc[i][v];
    }
}

// Job t (T = X·A_aᵀ; no slices: not asked for) and job u (U = dY·B_a) in one
// launch: blockIdx.x = tile, y = slice of t, then of u, z = block of 16·NJ ranks.
template <int NJ>
__global__ __launch_bounds__(256) void adapters_down_kernel(DownJob t, DownJob u, int64_t M, AdapterView ad,
                                                            PlanView pl) {
  __shared__ __attribute__((aligned(1024))) char sl[kDownRing * 64 * 128];
  __shared__ __attribute__((aligned(1024))) char sr[kDownRing * 4 * (NJ == 4 ? 2 : 1) * 1024];
  const int tile = (int)blockIdx.x, y = (int)blockIdx.y, j0 = 16 * NJ * (int)blockIdx.z;
  if (tile >= pl.head[2]) return;
  if (y < t.slices)
    down_tile<NJ, false>(t, tile, y, j0, M, ad, pl, sl, sr);
  else
    down_tile<NJ, true>(u, tile, y - t.slices, j0, M, ad, pl, sl, sr);
}

// The slices added in order, for 16 positions x 16 ranks per workgroup (one
// value a thread): S [M, C] by position, and T [M, r] fp32 by token (zeros for
// a token without an adapter).  A job without slices splits the T it is given.
// One workgroup more (blockIdx.x == 0, if the table is asked for) cuts every
// used adapter's positions into units of at most `unit`, the gradients' work
// items.  (4096 x 64 from 4 slices: 5.2 us, mostly latency; its sums inside the
// down-projection would need the slices' workgroups to wait for each other.)
struct FactorJob {
  const float* P;
  int slices;
  const float* T_in;
  float* T_out;
  uint16_t* S;
};
// {used adapter, first position, end, partial slot or -1: written directly}
struct UnitTable {
  int32_t* head;   // [0] units
  int4* unit;      // [units]
  int4* of_group;  // [count] {first slot or -1, units, 0, 0}
};
__device__ __forceinline__ int block_scan256(int v, int* s, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) s[wave] = x;
  __syncthreads();
  total = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) x += s[w];
    total += s[w];
  }
  return x - v;
}
__device__ __forceinline__ void cut_units(const AdapterView& ad, const PlanView& pl, const UnitTable& ut, int64_t M,
                                          int unit, int max_units, int max_slots) {
  __shared__ int s_scan[4];
  const int used = std::min(std::max(pl.head[0], 0), ad.count);
  const int64_t held = std::min<int64_t>(pl.head[1], M);
  int u0 = 0, s0 = 0;
  for (int b = 0; b < used; b += 256) {
    const int g = b + (int)threadIdx.x;
    int p0 = 0, p1 = 0;
    if (g < used) {
      p0 = std::max(pl.start[g], 0);
      p1 = (int)std::min<int64_t>(pl.start[g + 1], held);
    }
    const int n = p1 > p0 ? (p1 - p0 + unit - 1) / unit : 0;
    int tu, ts;
    const int u = u0 + block_scan256(n, s_scan, tu), s = s0 + block_scan256(n > 1 ? n : 0, s_scan, ts);
    if (g < used) ut.of_group[g] = int4{n > 1 ? s : -1, n, 0, 0};
    for (int i = 0; i < n; ++i)
      if (u + i < max_units && (n == 1 || s + i < max_slots))
        ut.unit[u + i] = int4{g, p0 + i * unit, std::min(p0 + (i + 1) * unit, p1), n > 1 ? s + i : -1};
    u0 += tu;
    s0 += ts;
  }
  if (threadIdx.x == 0) ut.head[0] = std::min(u0, max_units);
}

__global__ __launch_bounds__(256) void adapters_factor_kernel(FactorJob t, FactorJob u, int64_t M, AdapterView ad,
                                                              PlanView pl, unsigned first, UnitTable ut, int unit,
                                                              int max_units, int max_slots) {
  if (blockIdx.x < first) {
    if (blockIdx.y == 0 && blockIdx.z == 0) cut_units(ad, pl, ut, M, unit, max_units, max_slots);
    return;
  }
  const FactorJob J = blockIdx.z ? u : t;
  const int64_t pos = 16 * (int64_t)(blockIdx.x - first) + (threadIdx.x >> 4);
  const int r = ad.r, j = 16 * (int)blockIdx.y + (threadIdx.x & 15);
  if (pos >= M || j >= r) return;
  const int tok = pl.perm[pos];
  if ((uint32_t)tok >= (uint32_t)M) return;
  const bool has = pos < std::min<int64_t>(pl.head[1], M);
  float v = 0.f;
  if (has) {
    if (J.slices == 0) {
      v = J.T_in[(int64_t)tok * r + j];
    } else {
      const float* const p = J.P + pos * r + j;
      // (the loads of eight slices, of existing ones whatever their number, before their adds)
      for (int s = 0; s < J.slices; s += 8) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = p[(int64_t)std::min(s + i, J.slices - 1) * M * r];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (s + i < J.slices) v += x[i];
      }
    }
  }
  if (J.T_out) J.T_out[(int64_t)tok * r + j] = v;
  if (!has || !J.S) return;
  const int id = pl.owner[tok];
  if ((unsigned)id >= (unsigned)ad.count) return;
  uint16_t o[3];
  split3(__fmul_rn(ad.s[id], v), o);
#pragma unroll
  for (int i = 0; i < 3; ++i) J.S[pos * adapter_cols(r) + i * r + j] = o[i];
}

// T for few tokens, in one launch: a workgroup per (position, kFewRanks ranks), its 4
// waves sharing the reduction, 8 elements per lane and step; each token reads
// its own adapter (tokens of one adapter share it in L2).  Fewer dependent
// loads before the data than with tiles, and the adapters' rows spread over
// many workgroups.  Up to 16 tokens positions are tokens (the plan's order
// does not matter to the dequant-GEMV).  (16 tokens and adapters, K = 4096, r =
// 64: 4.4 us, 2.0 TB/s of 8.5 MB; 53 tokens of 24 adapters, K = 11008, r = 32:
// 9.2 us, 41 MB at 4.5 TB/s, each adapter read once per token that carries it,
// mostly from L2.)  At 17 to 64 tokens against the tiles of adapters_down_kernel,
// whole forwards: r = 64, 4096 x 4096, 53 tokens of 8 adapters 26.9 us against 29.4,
// of as many adapters 40.4 against 47.2; r = 8 23.3 against 26.8; r = 256, of as
// many adapters 96 against 112.  Where long adapters are shared the tiles are
// faster (r = 256, 53 tokens of 8 adapters, 44.8 against 35.2; r = 128, K = 11008,
// 58.4 against 44.5), but how many tokens share one is known on the device alone.
constexpr int kFewTokens = 64, kFewRanks = 4;
__device__ __forceinline__ float dot8(const u32x4_t a, const u32x4_t b, float acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = __builtin_fmaf(bf16lo(a[i]), bf16lo(b[i]), acc);
    acc = __builtin_fmaf(bf16hi(a[i]), bf16hi(b[i]), acc);
  }
  return acc;
}
// This thread's part of kFewRanks ranks of one token: x·R[j], rows of Kred.
__device__ __forceinline__ void few_rows(const uint16_t* x_row, const uint16_t* R, int64_t Kred, int tid, float* acc) {
  constexpr int UN = 3;
  const rsrc_t rl = make_rsrc(x_row, Kred * 2), rr = make_rsrc(R, (int64_t)kFewRanks * Kred * 2);
  for (int64_t k0 = 8 * tid; k0 < Kred; k0 += 2048 * UN) {
    u32x4_t x[UN], w[UN][kFewRanks];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int64_t k = k0 + 2048 * u;
      const bool in = k < Kred;
      x[u] = buf_load16(rl, in ? (uint32_t)(k * 2) : 0x7fffffffu, 0u);
#pragma unroll
      for (int j = 0; j < kFewRanks; ++j)
        w[u][j] = buf_load16(rr, in ? (uint32_t)((j * Kred + k) * 2) : 0x7fffffffu, 0u);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int j = 0; j < kFewRanks; ++j) acc[j] = dot8(x[u], w[u][j], acc[j]);
  }
}
template <bool TOKENS>
__global__ __launch_bounds__(256) void adapters_few_down_kernel(const uint16_t* __restrict__ L, int64_t M, int64_t Kred,
                                                                AdapterView ad, PlanView pl, float* __restrict__ T,
                                                                float* __restrict__ Tt, uint16_t* __restrict__ S) {
  __shared__ float s_part[4][kFewRanks];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t pos = blockIdx.x;
  const int j0 = kFewRanks * (int)blockIdx.y, r = ad.r;
  const int tok = TOKENS ? (int)pos : pl.perm[pos];
  if ((uint32_t)tok >= (uint32_t)M) return;
  const int id = pl.owner[tok];
  const bool has = (unsigned)id < (unsigned)ad.count;
  float acc[kFewRanks] = {};
  if (has) few_rows(L + (int64_t)tok * Kred, ad.A + ((int64_t)id * r + j0) * Kred, Kred, tid, acc);
#pragma unroll
  for (int j = 0; j < kFewRanks; ++j) {
    acc[j] = wave_sum(acc[j]);
    if (lane == 0) s_part[wave][j] = acc[j];
  }
  __syncthreads();
  if (tid >= kFewRanks) return;
  const int j = j0 + tid;
  const float t = ((s_part[0][tid] + s_part[1][tid]) + s_part[2][tid]) + s_part[3][tid];
  if (T) T[(int64_t)tok * r + j] = t;
  if (Tt) Tt[(j >> 4) * 256 + 16 * tok + (j & 15)] = t;
  if (has && S) {
    uint16_t v[3];
    split3(__fmul_rn(ad.s[id], t), v);
#pragma unroll
    for (int i = 0; i < 3; ++i) S[pos * adapter_cols(r) + i * r + j] = v[i];
  }
}

// Both factors of a backward pass over few tokens, and its unit table, in one
// launch in place of adapters_down_kernel and adapters_factor_kernel: a workgroup
// per (position, 8 ranks of U), one per (position, kFewRanks of T; blockIdx.z
// = 1) and one for the table (blockIdx.x == 0).  U[m][j] = Σ_n dY[m][n]·B_a[n][j]:
// a thread takes two rows of B_a a step, 16 bytes of each.  (61 tokens of 4 adapters,
// r = 8, 4096 x 4096: 6.0 us, latency, against 5.2 + 4.0 for the two.)
__global__ __launch_bounds__(256) void adapters_few_factors_kernel(const uint16_t* __restrict__ X,
                                                                   const uint16_t* __restrict__ dY, int64_t M,
                                                                   int64_t N, int64_t K, AdapterView ad, PlanView pl,
                                                                   const float* __restrict__ T_in,
                                                                   uint16_t* __restrict__ ST, uint16_t* __restrict__ SU,
                                                                   UnitTable ut, int unit, int max_units,
                                                                   int max_slots) {
  if (blockIdx.x == 0) {
    if (blockIdx.y == 0 && blockIdx.z == 0) cut_units(ad, pl, ut, M, unit, max_units, max_slots);
    return;
  }
  __shared__ float s_part[4][8];
  const bool is_u = blockIdx.z == 0;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = ad.r;
  const int ranks = is_u ? 8 : kFewRanks, j0 = ranks * (int)blockIdx.y;
  const int64_t pos = blockIdx.x - 1;
  if (j0 >= r) return;
  const int tok = pl.perm[pos];
  if ((uint32_t)tok >= (uint32_t)M) return;
  const int id = pl.owner[tok];
  if ((unsigned)id >= (unsigned)ad.count) return;
  float acc[8] = {};
  if (is_u) {
    constexpr int UN = 4;
    const rsrc_t rl = make_rsrc(dY + (int64_t)tok * N, N * 2), rr = make_rsrc(ad.B + (int64_t)id * N * r, N * r * 2);
    for (int64_t n0 = 2 * tid; n0 < N; n0 += 512 * UN) {
      uint32_t y[UN];
      u32x4_t w[UN][2];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int64_t n = n0 + 512 * u;  // (N is even)
        const bool in = n < N;
        y[u] = buf_load4(rl, in ? (uint32_t)(n * 2) : 0x7fffffffu, 0u);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w[u][i] = buf_load16(rr, in ? (uint32_t)(((n + i) * r + j0) * 2) : 0x7fffffffu, 0u);
      }
#pragma unroll
      for (int u = 0; u < UN; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float v = i ? bf16hi(y[u]) : bf16lo(y[u]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[2 * q] = __builtin_fmaf(v, bf16lo(w[u][i][q]), acc[2 * q]);
            acc[2 * q + 1] = __builtin_fmaf(v, bf16hi(w[u][i][q]), acc[2 * q + 1]);
          }
        }
    }
  } else if (!T_in) {
    few_rows(X + (int64_t)tok * K, ad.A + ((int64_t)id * r + j0) * K, K, tid, acc);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    acc[j] = wave_sum(acc[j]);
    if (lane == 0) s_part[wave][j] = acc[j];
  }
  __syncthreads();
  if (tid >= ranks) return;
  const int j = j0 + tid;
  const float t = !is_u && T_in ? T_in[(int64_t)tok * r + j]
                                : ((s_part[0][tid] + s_part[1][tid]) + s_part[2][tid]) + s_part[3][tid];
  uint16_t* const S = is_u ? SU : ST;
  uint16_t v[3];
  split3(__fmul_rn(ad.s[id], t), v);
#pragma unroll
  for (int i = 0; i < 3; ++i) S[pos * adapter_cols(r) + i * r + j] = v[i];
}

// ---------------------------------------------------------------------------
// The adapters' gradients: for one unit (positions [p0, p1) of one used
// adapter), 128 columns of L (X for dA, dY for dB) and up to 16·NJ ranks,
//   D[c][j] = Σ_p L[token(p)][c]·(S[p][j] + S[p][r + j] + S[p][2r + j]).
// Stages of 32 positions, both operands copied straight into a ring of LDS
// stages in their own layouts (L rows gathered through the plan); the MFMA
// operands, 8 consecutive positions of one column, are transposing reads.
// Positions outside the unit read as zero on both sides.  A unit that is its
// adapter's only one writes the gradient itself, the others partial sums,
// added in unit order by the finishing kernel.  Bound by reading X and dY and
// by writing dA and dB: 4096 tokens of 6 adapters, r = 16, 4096 x 11008, 24.6 us,
// 140 MB at 5.7 TB/s (in part from the last-level cache); 2045 tokens of 40
// adapters, r = 64, 8192 x 8192, 63 us, 168 MB written of 244 in all, 3.9 TB/s.
// ---------------------------------------------------------------------------
constexpr int kMaxUnit = 1024, kGradRing = 3;
struct GradientJob {
  const uint16_t* L;
  int64_t cols;
  const uint16_t* S;
  float* out;        // [count][r·cols]
  int64_t part_off;  // of this job within a partial slot
};
// 16-byte chunk c of L row p at c ^ ((p & 3) << 1): the 4 rows of a transposing
// read on different banks
__device__ __forceinline__ int lswz(int row, int col) {
  return row * 256 + (((col >> 3) ^ ((row & 3) << 1)) << 4) + 2 * (col & 7);
}
// The same for S rows of 6·NJ chunks (three parts of 2·NJ).
template <int NJ>
__device__ __forceinline__ int factor_swz(int row) {
  return NJ == 4 ? (row & 3) << 1 : NJ == 2 ? row & 2 : 0;
}

// ALONG: out [cols][r] (dB), else [r][cols] (dA).
template <int NJ, bool ALONG>
__device__ __forceinline__ void gradient_unit(const GradientJob& J, int64_t c0, int j0, const int4 u, int64_t M,
                                              const AdapterView& ad, const PlanView& pl, float* __restrict__ P,
                                              int64_t slot_floats, char* sl, char* ss, int* s_tok) {
  constexpr int SI = NJ == 4 ? 3 : NJ == 2 ? 2 : 1;  // S copies per wave and stage
  constexpr int LB = 32 * 256, SB = 4 * SI * 1024, SROW = 96 * NJ;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, kq = lane >> 4, r = ad.r, C = (int)adapter_cols(r);
  const int p0 = u.y, p1 = std::min(u.z, u.y + kMaxUnit);
  const int stages = (p1 - p0 + 31) / 32;
  for (int i = tid; i < 32 * stages; i += 256) s_tok[i] = p0 + i < p1 ? pl.perm[p0 + i] : -1;
  __syncthreads();
  const i32x4_t rl = rsrc_words(J.L, M * J.cols * 2), rs = rsrc_words(J.S, M * C * 2);
  auto issue = [&](int b, int s) __attribute__((always_inline)) {
    // L: wave w copies rows 8w + 4c + (lane >> 4), lane i physical chunk i & 15
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = 8 * wave + 4 * c + (lane >> 4);
      const int64_t col = c0 + 8 * ((lane & 15) ^ ((row & 3) << 1));
      const int tok = s < stages ? s_tok[32 * s + row] : -1;
      const bool in = (uint32_t)tok < (uint32_t)M && col < J.cols;
      dma_lds16(rl, sl + b * LB + (8 * wave + 4 * c) * 256,
                in ? ((uint32_t)tok * (uint32_t)J.cols + (uint32_t)col) * 2u : 0x7fffffffu, 0u);
    }
#pragma unroll
    for (int c = 0; c < SI; ++c) {
      const int idx = 64 * (SI * wave + c) + lane, row = idx / (6 * NJ);
      const int ch = (idx % (6 * NJ)) ^ factor_swz<NJ>(row), part = ch / (2 * NJ), j = j0 + 8 * (ch % (2 * NJ));
      const int pos = p0 + 32 * s + row;
      const bool in = row < 32 && pos < p1 && j < r;
      dma_lds16(rs, ss + b * SB + (SI * wave + c) * 1024,
                in ? ((uint32_t)pos * (uint32_t)C + (uint32_t)(part * r + j)) * 2u : 0x7fffffffu, 0u);
    }
  };
  f32x4_t acc[2][NJ];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i + 1 < kGradRing; ++i) issue(i, i);
  for (int s = 0; s < stages; ++s) {
    open_stage<(kGradRing - 2) * (2 + SI)>();
    issue((s + kGradRing - 1) % kGradRing, s + kGradRing - 1);
    const char* const lt = sl + (s % kGradRing) * LB;
    const char* const st = ss + (s % kGradRing) * SB;
    const int trow = 8 * kq + (lr >> 2), tcol = 4 * (lr & 3);  // this lane's part of a transposing read
    u32x4_t a[2];
#pragma unroll
    for (int pf = 0; pf < 2; ++pf) {
      const u32x2_t h0 = lds_read_tr(lt + lswz(trow, 32 * wave + 16 * pf + tcol));
      const u32x2_t h1 = lds_read_tr(lt + lswz(trow + 4, 32 * wave + 16 * pf + tcol));
      a[pf] = u32x4_t{h0[0], h0[1], h1[0], h1[1]};
    }
#pragma unroll
    for (int part = 0; part < 3; ++part)
#pragma unroll
      for (int jf = 0; jf < NJ; ++jf) {
        const int col = 16 * (NJ * part + jf) + tcol;
        u32x2_t h[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int row = trow + 4 * q;
          h[q] = lds_read_tr(st + row * SROW + (((col >> 3) ^ factor_swz<NJ>(row)) << 4) + 2 * (col & 7));
        }
        const u32x4_t f = {h[0][0], h[0][1], h[1][0], h[1][1]};
#pragma unroll
        for (int pf = 0; pf < 2; ++pf)
          acc[pf][jf] = ALONG ? mfma_16x16x32(a[pf], f, acc[pf][jf]) : mfma_16x16x32(f, a[pf], acc[pf][jf]);
      }
  }
  wait_vmem();  // no copy may land in LDS after the workgroup ends
  const int id = pl.id[u.x];
  if ((unsigned)id >= (unsigned)ad.count) return;
  float* const o = u.w < 0 ? J.out + (int64_t)id * r * J.cols : P + (int64_t)u.w * slot_floats + J.part_off;
#pragma unroll
  for (int pf = 0; pf < 2; ++pf)
#pragma unroll
    for (int jf = 0; jf < NJ; ++jf)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t cb = c0 + 32 * wave + 16 * pf;
        const int jbase = j0 + 16 * jf;
        const int64_t c = ALONG ? cb + 4 * kq + v : cb + lr;
        const int j = ALONG ? jbase + lr : jbase + 4 * kq + v;
        if (c < J.cols && j < r) o[ALONG ? c * r + j : j * J.cols + c] = acc[pf][jf][v];
      }
}

// Zeros in the same part of an adapter without tokens.
template <int NJ>
__device__ __forceinline__ void zero_part(float* out, int64_t cols, int r, int64_t c0, int j0, bool along) {
  // along: 128 rows c of 4·NJ chunks of 4 ranks; else 16·NJ rows j of 32 chunks of 4 columns
  const int per = along ? 4 * NJ : 32;
  for (int i = threadIdx.x; i < 512 * NJ; i += 256) {
    const int64_t c = c0 + (along ? i / per : 4 * (i % per));
    const int j = j0 + (along ? 4 * (i % per) : i / per);
    if (c < cols && j < r)
      *reinterpret_cast<f32x4_t*>(out + (along ? c * r + j : j * cols + c)) = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
}
// blockIdx.y: a unit, or from max_units on an adapter, for its zeros, and then a
// part of the sum of dX's split partials (launched so where every adapter is one
// unit: no partial sums of gradients take the partials' place, and nothing is
// left to finish).
struct TailJobs {
  int adapters;      // whose zeros are looked after: all of them or none
  const f32x4_t* P;  // dX's partials; n4 = 0: none
  int splits;
  int64_t n4;
  void* out;
  int out16;
};
template <int NJ>
__global__ __launch_bounds__(256) void adapters_gradient_kernel(GradientJob ja, GradientJob jb, unsigned tiles_a,
                                                                int64_t M, AdapterView ad, PlanView pl, UnitTable ut,
                                                                int max_units, float* __restrict__ P,
                                                                int64_t slot_floats, TailJobs tail) {
  __shared__ __attribute__((aligned(1024))) char sl[kGradRing * 32 * 256];
  __shared__ __attribute__((aligned(1024))) char ss[kGradRing * 4 * (NJ == 4 ? 3 : NJ == 2 ? 2 : 1) * 1024];
  __shared__ int s_tok[kMaxUnit];
  const int j0 = 16 * NJ * (int)blockIdx.z;
  if ((int)blockIdx.y >= max_units) {
    const int64_t a = blockIdx.y - max_units;
    if (a >= tail.adapters) {
      const int64_t block = ((a - tail.adapters) * gridDim.z + blockIdx.z) * gridDim.x + blockIdx.x;
      const int64_t i = 256 * block + threadIdx.x;
      if (i < tail.n4) splitk_sum4<false>(tail.P, tail.splits, tail.n4, i, tail.out, tail.out16);
      return;
    }
    const int g = pl.slot[a];
    if (g >= 0 && g < ad.count) return;
    const bool along = blockIdx.x >= tiles_a;
    const GradientJob& J = along ? jb : ja;
    zero_part<NJ>(J.out + a * ad.r * J.cols, J.cols, ad.r, 128 * (int64_t)(blockIdx.x - (along ? tiles_a : 0u)), j0, along);
    return;
  }
  if ((int)blockIdx.y >= ut.head[0]) return;
  const int4 u = ut.unit[blockIdx.y];
  if (blockIdx.x < tiles_a)
    gradient_unit<NJ, false>(ja, 128 * (int64_t)blockIdx.x, j0, u, M, ad, pl, P, slot_floats, sl, ss, s_tok);
  else
    gradient_unit<NJ, true>(jb, 128 * (int64_t)(blockIdx.x - tiles_a), j0, u, M, ad, pl, P, slot_floats, sl, ss, s_tok);
}

// Partial sums added in unit order; zeros for an adapter without tokens.
__global__ __launch_bounds__(256) void adapters_gradient_finish_kernel(float* __restrict__ dA, float* __restrict__ dB,
                                                                       int64_t na, int64_t nb, int count, PlanView pl,
                                                                       UnitTable ut, const float* __restrict__ P,
                                                                       int max_slots) {
  const int a = (int)blockIdx.y, g = pl.slot[a];
  int first = -1, n = 0;
  if (g >= 0 && g < count) {
    const int4 t = ut.of_group[g];
    first = t.x;
    n = t.y;
    if (n == 1 || (n > 0 && (first < 0 || first + n > max_slots))) return;
  }
  for (int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x); i < na + nb; i += 1024 * (int64_t)gridDim.x) {
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int q = 0; q < n; ++q) {
      const f32x4_t x = *reinterpret_cast<const f32x4_t*>(P + (int64_t)(first + q) * (na + nb) + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += x[e];
    }
    float* const o = i < na ? dA + a * na + i : dB + a * nb + (i - na);
    *reinterpret_cast<f32x4_t*>(o) = v;
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

size_t plan_bytes(int64_t M, int count) {
  return (size_t)(kPlanHead + 3 * plan_pad(M) + 3 * plan_pad(count + 1) + plan_pad(2 * plan_tiles(M, count))) * 4;
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
  v.tile = reinterpret_cast<int2*>(v.slot + plan_pad(count + 1));
  return v;
}
hipError_t launch_adapters_plan(const int32_t* index, int64_t M, int count, const PlanView& pl, hipStream_t st) {
  adapters_plan_kernel<<<1, 64 * kPlanWaves, (size_t)kPlanWaves * (count + 1) * 4, st>>>(index, M, count, pl);
  return hipGetLastError();
}

namespace {

// NJ blocks of 16 ranks per workgroup
int rank_blocks(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }

// Slices of a low-rank factor's reduction: about 512 workgroups over the
// tiles that M tokens make at least, of 4 stages each or more, 16 at most.
int down_slices(int64_t M, int64_t Kred, int r) {
  const int64_t work = std::max<int64_t>(1, M / 64) * cdiv(r, 16 * rank_blocks(r));
  return (int)std::max<int64_t>(1, std::min<int64_t>({512 / work, (int64_t)cdiv(Kred, 256), 16}));
}

hipError_t launch_down(const DownJob& t, const DownJob& u, int64_t M, const AdapterView& ad, const PlanView& pl,
                       hipStream_t st) {
  const int nj = rank_blocks(ad.r);
  const dim3 grid((unsigned)plan_tiles(M, ad.count), (unsigned)(t.slices + u.slices), cdiv(ad.r, 16 * nj));
  if (nj == 1)
    adapters_down_kernel<1><<<grid, 256, 0, st>>>(t, u, M, ad, pl);
  else if (nj == 2)
    adapters_down_kernel<2><<<grid, 256, 0, st>>>(t, u, M, ad, pl);
  else
    adapters_down_kernel<4><<<grid, 256, 0, st>>>(t, u, M, ad, pl);
  return hipGetLastError();
}

}  // namespace

AdaptersFwdLayout adapters_fwd_layout(int64_t M, int64_t N, int64_t K, int r, int count) {
  AdaptersFwdLayout L{};
  L.splits = M > kMidTokens ? fwd_gemm_splits(M, N, K, SIZE_MAX) : M > 16 ? mid_fwd_plan(M, N, K).splits : 1;
  L.slices = M > kFewTokens ? down_slices(M, K, r) : 0;
  L.off_S = 0;
  L.off_P = M > 16 ? round_up(M * adapter_cols(r) * 2, 256) : M > 0 ? round_up((int64_t)cdiv(r, 16) * 1024, 256) : 0;
  const int64_t gemm = L.splits > 1 ? (int64_t)L.splits * M * N * 4 : 0;
  L.total = L.off_P + round_up(std::max(gemm, (int64_t)L.slices * M * r * 4), 256);
  return L;
}
namespace {
// Column tiles times rank blocks of the gradients, and the units they need to
// fill the chip about twice over.
int64_t gradient_parts(int64_t N, int64_t K, int r) {
  const int64_t work = (int64_t)(cdiv(K, 128) + cdiv(N, 128)) * cdiv(r, 16 * rank_blocks(r));
  return std::max<int64_t>(1, (512 + work - 1) / work);
}
int64_t unit_table_bytes(int64_t units, int count) { return round_up(256 + (units + count) * 16, 256); }
}  // namespace
// Whether a backward pass takes its factors from adapters_few_factors_kernel: one
// launch for two, but a token's 16 bytes of every row of B_a waste more of the
// lines they come in, and are read by more tokens, the longer the rows are.  (A
// whole pass, replayed: 61 tokens, r = 8, 4096 x 4096, 31.8 us against 34.7; 64
// tokens, 11008 x 4096, r = 16, 52.5 against 52.4; r = 32, 70.9 against 55.4.)
bool few_factors(int64_t M, int r) { return M <= kFewTokens && r <= 16; }
AdaptersBwdLayout adapters_bwd_layout(int64_t M, int64_t N, int64_t K, int r, int count) {
  AdaptersBwdLayout L{};
  L.splits = M > kMidTokens ? dx_gemm_splits(M, N, K, SIZE_MAX) : M > 0 ? mid_dx_splits(M, N, K) : 1;
  if (M == 0) return L;
  const bool few = few_factors(M, r);
  L.slices_U = few ? 0 : down_slices(M, N, r);
  L.slices_T = few ? 0 : down_slices(M, K, r);
  const int64_t parts = gradient_parts(N, K, r);
  L.unit = (int)std::min<int64_t>(kMaxUnit, round_up((M + parts - 1) / parts, 64));
  L.units = (int)(M / L.unit + std::min<int64_t>(count, M));
  L.slots = (int)(2 * M / L.unit);  // (an adapter of n > 1 units has more than (n - 1)·unit tokens)
  size_t off = 0;
  L.off_U = off;
  off += round_up(M * adapter_cols(r) * 2, 256);
  L.off_T = off;
  off += round_up(M * adapter_cols(r) * 2, 256);
  L.off_units = off;
  off += unit_table_bytes(L.units, count);
  L.off_P = off;
  const int64_t gemm = L.splits > 1 ? (int64_t)L.splits * M * K * 4 : 0;
  const int64_t factors = (int64_t)(L.slices_U + L.slices_T) * M * r * 4;
  off += round_up(std::max({gemm, factors, (int64_t)L.slots * r * (K + N) * 4}), 256);
  L.total = off;
  return L;
}

// Up to kMidTokens tokens the split count may change at any of them, so each is
// taken; above, it is constant within a band of 256 tokens (the GEMMs' tiles)
// and the partials grow with M, and so are a factor's slices between multiples
// of 64: the last of every 64 and the first of the next are taken.
namespace {
template <typename F>
void each_worst(int64_t M_max, F&& take) {
  for (int64_t M = 1; M <= std::min(M_max, kMidTokens); ++M) take(M);
  for (int64_t top = kMidTokens + 63; M_max > kMidTokens; top += 64) {
    take(std::min(top, M_max));
    if (top >= M_max) break;
    take(top + 1);
  }
}
}  // namespace
size_t adapters_fwd_ws_max(int64_t M_max, int64_t N, int64_t K, int r, int count) {
  size_t most = 0;
  each_worst(M_max, [&](int64_t M) { most = std::max(most, adapters_fwd_layout(M, N, K, r, count).total); });
  return most;
}
size_t adapters_bwd_ws_max(int64_t M_max, int64_t N, int64_t K, int r, int count) {
  // the factors grow with M; the shared area is bounded by the products' and
  // the factors' partials as above, and for the gradients' by 2M/unit slots:
  // units of at least M/parts give 2·parts, units of 1,024 2M/1,024
  const AdaptersBwdLayout L = adapters_bwd_layout(M_max, N, K, r, count);
  if (M_max == 0) return L.total;
  int64_t area = 0;
  each_worst(M_max, [&](int64_t M) {
    const AdaptersBwdLayout l = adapters_bwd_layout(M, N, K, r, count);
    if (l.splits > 1) area = std::max(area, l.splits * M * K * 4);
    area = std::max(area, (int64_t)(l.slices_U + l.slices_T) * M * r * 4);
  });
  const int64_t parts = gradient_parts(N, K, r);
  const int64_t slots = std::min(std::max<int64_t>(2 * parts, 2 * M_max / kMaxUnit), 2 * M_max / 64);
  area = std::max(area, slots * r * (K + N) * 4);
  const int64_t units = std::max(parts, M_max / kMaxUnit) + std::min<int64_t>(count, M_max);
  return L.off_units + unit_table_bytes(units, count) + round_up(area, 256);
}

hipError_t launch_adapters_fwd(const Nf4View& W, const uint16_t* X, int64_t M, const AdapterView& ad,
                               const PlanView& pl, void* Y, bool y16, float* T_save, char* ws,
                               const AdaptersFwdLayout& L, hipStream_t st) {
  if (M == 0) return hipSuccess;
  const dim3 few((unsigned)M, (unsigned)(ad.r / kFewRanks));
  uint16_t* const none = nullptr;
  if (M <= 16) {
    float* Tt = reinterpret_cast<float*>(ws + L.off_S);
    adapters_few_down_kernel<true><<<few, 256, 0, st>>>(X, M, W.K, ad, pl, T_save, Tt, none);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_gemv_adapters(W, X, M, ad, pl.owner, Y, y16, Tt, st);
  }
  uint16_t* S = reinterpret_cast<uint16_t*>(ws + L.off_S);
  float* P = reinterpret_cast<float*>(ws + L.off_P);
  hipError_t e;
  if (M <= kFewTokens) {
    adapters_few_down_kernel<false><<<few, 256, 0, st>>>(X, M, W.K, ad, pl, T_save, (float*)nullptr, S);
    e = hipGetLastError();
  } else {
    e = launch_down(DownJob{X, W.K, ad.A, P, L.slices}, DownJob{}, M, ad, pl, st);
    if (e != hipSuccess) return e;
    const FactorJob t{P, L.slices, nullptr, T_save, S};
    adapters_factor_kernel<<<dim3(cdiv(M, 16), cdiv(ad.r, 16)), 256, 0, st>>>(t, t, M, ad, pl, 0u, UnitTable{}, 1, 0, 0);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  // (the partial sums of T have been consumed: P now takes the split partials)
  const AdapterGemmArgs ma{pl.head, (int)plan_pad(M), (int)plan_pad(ad.count + 1), S, ad.B, ad.r,
                           (int)adapter_cols(ad.r), ad.count, (y16 ? 2 : 3) * ad.r};
  e = M <= kMidTokens ? launch_mid_fwd(W, X, M, ma, Y, y16, mid_fwd_plan(M, W.N, W.K), P, st)
                      : launch_fwd_gemm_adapters(W, X, M, ma, Y, y16, L.splits, P, st);
  if (e != hipSuccess || L.splits == 1) return e;
  return launch_splitk_reduce(P, L.splits, M * W.N, Y, y16, false, st);
}

hipError_t launch_adapters_bwd(const Nf4View& W, const uint16_t* X, const uint16_t* dY, int64_t M,
                               const AdapterView& ad, const PlanView& pl, const float* T_saved, void* dX, bool dx16,
                               float* dA, float* dB, char* ws, const AdaptersBwdLayout& L, hipStream_t st) {
  const int64_t N = W.N, K = W.K, r = ad.r;
  hipError_t e;
  if (M == 0) {
    e = launch_zero(dA, ad.count * r * K, st);
    return e != hipSuccess ? e : launch_zero(dB, ad.count * r * N, st);
  }
  uint16_t* U = reinterpret_cast<uint16_t*>(ws + L.off_U);
  uint16_t* T = reinterpret_cast<uint16_t*>(ws + L.off_T);
  float* P = reinterpret_cast<float*>(ws + L.off_P);
  UnitTable ut;
  ut.head = reinterpret_cast<int32_t*>(ws + L.off_units);
  ut.unit = reinterpret_cast<int4*>(ws + L.off_units + 256);
  ut.of_group = ut.unit + L.units;
  // U, and T unless it was saved
  if (L.slices_U == 0) {
    adapters_few_factors_kernel<<<dim3((unsigned)(M + 1), (unsigned)(r / kFewRanks), 2), 256, 0, st>>>(
        X, dY, M, N, K, ad, pl, T_saved, T, U, ut, L.unit, L.units, L.slots);
    e = hipGetLastError();
  } else {
    float* const PU = P + (T_saved ? 0 : (int64_t)L.slices_T * M * r);
    const DownJob dt{X, K, ad.A, P, T_saved ? 0 : L.slices_T}, du{dY, N, ad.B, PU, L.slices_U};
    e = launch_down(dt, du, M, ad, pl, st);
    if (e != hipSuccess) return e;
    const FactorJob ft{P, dt.slices, T_saved, nullptr, T}, fu{PU, L.slices_U, nullptr, nullptr, U};
    adapters_factor_kernel<<<dim3(1 + cdiv(M, 16), cdiv(r, 16), 2), 256, 0, st>>>(ft, fu, M, ad, pl, 1u, ut, L.unit,
                                                                                 L.units, L.slots);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  const AdapterGemmArgs ma{pl.head, (int)plan_pad(M), (int)plan_pad(ad.count + 1), U, ad.A, ad.r,
                           (int)adapter_cols(r), ad.count, (dx16 ? 2 : 3) * ad.r};
  e = M <= kMidTokens ? launch_mid_dx(W, dY, M, ma, dX, dx16, L.splits, P, st)
                      : launch_dx_gemm_adapters(W, dY, M, ma, dX, dx16, L.splits, P, st);
  // up to one unit of tokens no adapter has partial sums to add: the zeros of
  // those without tokens, and the sum of dX's splits, come with the gradients
  // (61 tokens, 4096 x 4096, r = 8: 25.9 us
  // the whole pass, 31 with launches of their own)
  const bool finish = M > L.unit, sum = L.splits > 1;
  if (e == hipSuccess && sum && finish) e = launch_splitk_reduce(P, L.splits, M * K, dX, dx16, false, st);
  if (e != hipSuccess) return e;
  const int64_t slot = r * (K + N);
  const GradientJob ja{X, K, U, dA, 0}, jo{dY, N, T, dB, r * K};
  const int nj = rank_blocks(ad.r);
  const unsigned ta = cdiv(K, 128);
  const unsigned gx = ta + cdiv(N, 128), gz = cdiv(r, 16 * nj);
  const TailJobs tail{finish ? 0 : ad.count, reinterpret_cast<const f32x4_t*>(P), L.splits,
                      sum && !finish ? M * K / 4 : 0, dX, dx16 ? 1 : 0};
  const dim3 grid(gx, (unsigned)L.units + tail.adapters + cdiv(tail.n4, (int64_t)256 * gx * gz), gz);
  if (nj == 1)
    adapters_gradient_kernel<1><<<grid, 256, 0, st>>>(ja, jo, ta, M, ad, pl, ut, L.units, P, slot, tail);
  else if (nj == 2)
    adapters_gradient_kernel<2><<<grid, 256, 0, st>>>(ja, jo, ta, M, ad, pl, ut, L.units, P, slot, tail);
  else
    adapters_gradient_kernel<4><<<grid, 256, 0, st>>>(ja, jo, ta, M, ad, pl, ut, L.units, P, slot, tail);
  e = hipGetLastError();
  if (e != hipSuccess || !finish) return e;
  adapters_gradient_finish_kernel<<<dim3(std::min(cdiv(slot, 1024), 256u), (unsigned)ad.count), 256, 0, st>>>(
      dA, dB, r * K, r * N, ad.count, pl, ut, P, L.slots);
  return hipGetLastError();
}

}  // namespace qnf4
