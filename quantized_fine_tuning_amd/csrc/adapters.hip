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
#include <type_traits>

#include "host.h"

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
// Low-rank factors.  For the 16 sorted positions of a tile and one of the used
// adapters among them (blockIdx.y, its stride gridDim.y): D[p][j] =
// Σ_k L[token(p)][k]·R_a[j][k] over NJ blocks of 16 ranks, 16 waves taking
// 64-element runs of the reduction in turn, each lane whole 32-byte pieces of
// its row (L read straight from memory: every byte is used once), the waves'
// sums added in wave order.  Only the positions of that adapter are written:
//   T   [M, r] fp32 by token (zeros for a token without an adapter), or
//   Tt  the same in the dequant-GEMV's tiles (M <= 16),
//   S   [M, C] by position, v = s_a·D as hi + mid + lo in bf16 (24 bits: the
//       products with it are as exact as fp32 ones),
//   ST  its transpose [3r, Mp].
// ---------------------------------------------------------------------------
constexpr int kDownWaves = 16;
struct DownOut {
  float* T;
  float* Tt;
  uint16_t* S;
  uint16_t* ST;
  int64_t Mp;
};

__device__ __forceinline__ void split3(float v, uint16_t* o) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t h = pack_bf16x2(v, 0.0f) & 0xffffu;
    o[i] = (uint16_t)h;
    v = __fsub_rn(v, __uint_as_float(h << 16));
  }
}

template <int NJ>
__global__ __launch_bounds__(64 * kDownWaves) void adapters_down_kernel(const uint16_t* __restrict__ L, int64_t M,
                                                                        int64_t Kred, const uint16_t* __restrict__ R,
                                                                        int by_id, AdapterView ad, PlanView pl,
                                                                        DownOut out) {
  __shared__ f32x4_t s_acc[kDownWaves][NJ][64];
  constexpr int UN = NJ == 1 ? 4 : NJ == 2 ? 3 : 2;  // runs in flight per wave
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, kq = lane >> 4;
  const int64_t pos0 = 16 * (int64_t)blockIdx.x;
  const int jb0 = NJ * (int)blockIdx.z, r = ad.r, C = (int)adapter_cols(r);
  const int64_t held = std::min<int64_t>(pl.head[1], M);
  // (the row loaded by lanes lr, and the output row of thread tid / 16 % 16)
  const int64_t lpos = pos0 + lr, opos = pos0 + ((tid >> 4) & 15);
  const int64_t ltok = lpos < held ? pl.perm[lpos] : -1;
  const int64_t otok = opos < M ? pl.perm[opos] : -1;
  const bool otok_ok = (uint64_t)otok < (uint64_t)M;
  if (blockIdx.y == 0 && opos >= held && otok_ok) {
    for (int o = tid; o < 256 * NJ; o += 64 * kDownWaves) {
      const int j = 16 * (jb0 + (o >> 8)) + (o & 15);
      if (j < r && out.T) out.T[otok * r + j] = 0.f;
      if (j < r && out.Tt) out.Tt[(j >> 4) * 256 + 16 * otok + (j & 15)] = 0.f;
    }
  }
  if (pos0 >= held) return;
  const int g0 = std::max(pl.group[pos0], 0);
  const int g1 = std::min(pl.group[std::min(pos0 + 16, held) - 1], ad.count - 1);
  const int ogroup = opos < held ? pl.group[opos] : -1;
  const rsrc_t rl = make_rsrc(L, M * Kred * 2);
  const bool lok = (uint64_t)ltok < (uint64_t)M;
  const uint32_t loff = lok ? (uint32_t)(ltok * Kred * 2) : 0u;
  const int runs = (int)((Kred + 63) / 64);
  for (int g = g0 + (int)blockIdx.y; g <= g1; g += (int)gridDim.y) {
    const int id = pl.id[g];
    if ((unsigned)id >= (unsigned)ad.count) break;
    const rsrc_t rr = make_rsrc(R + (int64_t)(by_id ? id : g) * r * Kred, (int64_t)r * Kred * 2);
    f32x4_t acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int run = wave; run < runs; run += UN * kDownWaves) {
      u32x4_t x[UN][2], w[UN][NJ][2];
#pragma unroll
      for (int u = 0; u < UN; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t k = 64 * (int64_t)(run + u * kDownWaves) + 16 * kq + 8 * h;
          const bool in = k < Kred;
          x[u][h] = buf_load16(rl, in && lok ? loff + (uint32_t)(k * 2) : 0x7fffffffu, 0u);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int row = 16 * (jb0 + j) + lr;
            w[u][j][h] = buf_load16(rr, in && row < r ? (uint32_t)((row * Kred + k) * 2) : 0x7fffffffu, 0u);
          }
        }
#pragma unroll
      for (int u = 0; u < UN; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NJ; ++j) acc[j] = mfma_16x16x32(x[u][h], w[u][j][h], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) s_acc[wave][j][lane] = acc[j];
    __syncthreads();
    if (ogroup == g && otok_ok) {
      const float s = ad.s[id];
      for (int o = tid; o < 256 * NJ; o += 64 * kDownWaves) {
        const int jb = o >> 8, row = (o >> 4) & 15, jj = o & 15, j = 16 * (jb0 + jb) + jj;
        if (j >= r) continue;
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) t += s_acc[w][jb][16 * (row >> 2) + jj][row & 3];
        if (out.T) out.T[otok * r + j] = t;
        if (out.Tt) out.Tt[(j >> 4) * 256 + 16 * otok + (j & 15)] = t;
        if (out.S || out.ST) {
          uint16_t v[3];
          split3(__fmul_rn(s, t), v);
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            if (out.S) out.S[opos * C + i * r + j] = v[i];
            if (out.ST) out.ST[(int64_t)(i * r + j) * out.Mp + opos] = v[i];
          }
        }
      }
    }
    __syncthreads();
  }
}

// The same for few tokens: a workgroup per (position, kFewRanks ranks), its 4
// waves sharing the reduction, 8 elements per lane and step; each token reads
// its own adapter (tokens of one adapter share it in L2).  Fewer dependent
// loads before the data than with tiles, and the adapters' rows spread over
// many workgroups.  Up to 16 tokens positions are tokens (the plan's order
// does not matter to the dequant-GEMV).
constexpr int kFewTokens = 64, kFewRanks = 4;
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
template <bool TOKENS>
__global__ __launch_bounds__(256) void adapters_few_down_kernel(const uint16_t* __restrict__ L, int64_t M, int64_t Kred,
                                                                const uint16_t* __restrict__ R, int by_id,
                                                                AdapterView ad, PlanView pl, DownOut out) {
  constexpr int UN = 3;
  __shared__ float s_part[4][kFewRanks];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t pos = blockIdx.x;
  const int j0 = kFewRanks * (int)blockIdx.y, r = ad.r;
  const int tok = TOKENS ? (int)pos : pl.perm[pos];
  if ((uint32_t)tok >= (uint32_t)M) return;
  const int id = pl.owner[tok];
  const bool has = (unsigned)id < (unsigned)ad.count;
  float acc[kFewRanks] = {};
  if (has) {
    const int g = by_id ? id : std::max(pl.slot[id], 0);
    const rsrc_t rl = make_rsrc(L + (int64_t)tok * Kred, Kred * 2);
    const rsrc_t rr = make_rsrc(R + ((int64_t)g * r + j0) * Kred, (int64_t)kFewRanks * Kred * 2);
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
#pragma unroll
  for (int j = 0; j < kFewRanks; ++j) {
    acc[j] = wave_sum(acc[j]);
    if (lane == 0) s_part[wave][j] = acc[j];
  }
  __syncthreads();
  if (tid >= kFewRanks) return;
  const int j = j0 + tid;
  const float t = ((s_part[0][tid] + s_part[1][tid]) + s_part[2][tid]) + s_part[3][tid];
  if (out.T) out.T[(int64_t)tok * r + j] = t;
  if (out.Tt) out.Tt[(j >> 4) * 256 + 16 * tok + (j & 15)] = t;
  if (has && (out.S || out.ST)) {
    uint16_t v[3];
    split3(__fmul_rn(ad.s[id], t), v);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (out.S) out.S[pos * adapter_cols(r) + i * r + j] = v[i];
      if (out.ST) out.ST[(int64_t)(i * r + j) * out.Mp + pos] = v[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Operand copies of the backward pass, one launch: block 0 cuts every used
// adapter's positions into units of at most `unit` (the gradients' work
// items); the next bt blocks split a saved T into ST [3r, Mp]; the rest
// transpose the used adapters: BT [used, r, N], AT [used, K, r], in 64 x 64
// tiles through LDS.
// ---------------------------------------------------------------------------
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
__global__ __launch_bounds__(256) void adapters_prep_kernel(const float* __restrict__ T, int64_t M, int64_t Mp,
                                                            uint16_t* __restrict__ ST, uint16_t* __restrict__ BT,
                                                            int64_t N, uint16_t* __restrict__ AT, int64_t K,
                                                            AdapterView ad, PlanView pl, UnitTable ut, int unit,
                                                            int max_units, int max_slots, unsigned bt, unsigned nb,
                                                            unsigned na, unsigned jb) {
  __shared__ uint16_t sh[3][64][66];
  __shared__ int s_scan[4];
  const int col = threadIdx.x & 63, row = threadIdx.x >> 6, r = ad.r;
  const int used = std::min(std::max(pl.head[0], 0), ad.count);
  const int64_t held = std::min<int64_t>(pl.head[1], M);
  if (blockIdx.x == 0) {
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
    return;
  }
  unsigned b = blockIdx.x - 1;
  if (b < bt) {
    // positions p, ranks j of s·T
    const int64_t q0 = (int64_t)(b / jb) * 64;
    const int j0 = (int)(b % jb) * 64, j = j0 + col;
    // (unconditional loads of clamped addresses: each step's 16 go out together)
    int tok[16], id[16];
    float sv[16], tv[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) tok[i] = pl.perm[std::min<int64_t>(q0 + 4 * i + row, M - 1)];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (q0 + 4 * i + row >= held || j >= r || (uint32_t)tok[i] >= (uint32_t)M) tok[i] = -1;
      id[i] = pl.owner[std::max(tok[i], 0)];
      tv[i] = T[(int64_t)std::max(tok[i], 0) * r + std::min(j, r - 1)];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if ((unsigned)id[i] >= (unsigned)ad.count) tok[i] = -1;
      sv[i] = ad.s[tok[i] < 0 ? 0 : id[i]];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint16_t v[3];
      split3(tok[i] < 0 ? 0.f : __fmul_rn(sv[i], tv[i]), v);
#pragma unroll
      for (int t = 0; t < 3; ++t) sh[t][col][4 * i + row] = v[t];
    }
    __syncthreads();
    for (int i = 0; i < 16; ++i) {
      const int jj = 4 * i + row;
      const int64_t pos = q0 + col;
      if (j0 + jj < r && pos < Mp)
#pragma unroll
        for (int t = 0; t < 3; ++t) ST[(int64_t)(t * r + j0 + jj) * Mp + pos] = sh[t][jj][col];
    }
    return;
  }
  b -= bt;
  const int g = (int)(b / (nb + na));
  if (g >= used) return;
  const int id = pl.id[g];
  if ((unsigned)id >= (unsigned)ad.count) return;
  unsigned t = b % (nb + na);
  // in [rows, cols] -> out [cols, rows]
  const bool isb = t < nb;
  if (!isb) t -= nb;
  const int64_t rows = isb ? N : r, cols = isb ? r : K;
  const uint16_t* in = isb ? ad.B + (int64_t)id * N * r : ad.A + (int64_t)id * r * K;
  uint16_t* o = isb ? BT + (int64_t)g * N * r : AT + (int64_t)g * K * r;
  const int64_t r0 = 64 * (int64_t)(isb ? t / jb : t % jb), c0 = 64 * (int64_t)(isb ? t % jb : t / jb);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t rr = r0 + 4 * i + row, cc = c0 + col;
    const bool ok = rr < rows && cc < cols;
    const uint16_t v = in[ok ? rr * cols + cc : 0];
    sh[0][col][4 * i + row] = ok ? v : 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t cc = c0 + 4 * i + row, rr = r0 + col;
    if (cc < cols && rr < rows) o[cc * rows + rr] = sh[0][4 * i + row][col];
  }
}

// ---------------------------------------------------------------------------
// The adapters' gradients: for one unit (positions [p0, p1) of one used
// adapter), 128 columns of L (X for dA, dY for dB) and up to 16·NJ ranks,
//   D[c][j] = Σ_p L[token(p)][c]·(ST[j][p] + ST[r + j][p] + ST[2r + j][p]).
// Stages of 64 positions, both operands copied straight into LDS, one stage
// ahead; L rows are gathered through the plan and kept in their natural
// layout, an MFMA operand (8 consecutive positions of one column) gathered
// with 2-byte reads.  Positions outside the unit read as zero on both sides.
// A unit that is its adapter's only one writes the gradient itself, the
// others partial sums, added in unit order by the finishing kernel.
// ---------------------------------------------------------------------------
constexpr int kMaxUnit = 1024;
struct GradientJob {
  const uint16_t* L;
  int64_t cols;
  const uint16_t* ST;
  float* out;       // [count][r·cols]
  int64_t part_off; // of this job within a partial slot
  int along;        // out [cols][r] (dB), else [r][cols] (dA)
};
__device__ __forceinline__ int lswz(int row, int chunk) {
  return row * 256 + ((chunk ^ (((row >> 3) & 7) << 1)) << 4);
}
__device__ __forceinline__ int sswz(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

template <int NJ>
__global__ __launch_bounds__(256) void adapters_gradient_kernel(GradientJob ja, GradientJob jb, unsigned tiles_a,
                                                                int64_t M, int64_t Mp, AdapterView ad, PlanView pl,
                                                                UnitTable ut, float* __restrict__ P,
                                                                int64_t slot_floats) {
  constexpr int SI = NJ == 1 ? 2 : NJ == 2 ? 3 : 6;  // S copies per wave and stage (8 rows each)
  __shared__ __attribute__((aligned(1024))) char sl[2][64 * 256];
  __shared__ __attribute__((aligned(1024))) char ss[2][4 * SI * 8 * 128];
  __shared__ int s_tok[kMaxUnit + 128];
  if ((int)blockIdx.y >= ut.head[0]) return;
  const bool second = blockIdx.x >= tiles_a;
  const GradientJob J = second ? jb : ja;
  const int4 u = ut.unit[blockIdx.y];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, kq = lane >> 4, r = ad.r;
  const int64_t c0 = 128 * (int64_t)(second ? blockIdx.x - tiles_a : blockIdx.x);
  const int j0 = 16 * NJ * (int)blockIdx.z;
  const int p0 = u.y, p1 = std::min(u.z, u.y + kMaxUnit), base = p0 & ~7;
  const int stages = (p1 - base + 63) / 64;
  for (int i = tid; i < 64 * stages; i += 256) {
    const int pos = base + i;
    s_tok[i] = pos >= p0 && pos < p1 ? pl.perm[pos] : -1;
  }
  __syncthreads();

  const i32x4_t rl = rsrc_words(J.L, M * J.cols * 2), rs = rsrc_words(J.ST, (int64_t)3 * r * Mp * 2);
  auto issue = [&](int b, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = 16 * wave + 4 * c + (lane >> 4);
      const int64_t col = c0 + 8 * ((lane & 15) ^ (((row >> 3) & 7) << 1));
      const int tok = s_tok[64 * s + row];
      const bool in = (uint64_t)(int64_t)tok < (uint64_t)M && col < J.cols;
      dma_lds16(rl, sl[b] + (16 * wave + 4 * c) * 256, in ? (uint32_t)((tok * J.cols + col) * 2) : 0x7fffffffu, 0u);
    }
#pragma unroll
    for (int c = 0; c < SI; ++c) {
      const int row = 8 * (SI * wave + c) + (lane >> 3);
      const int part = row / (16 * NJ), j = j0 + row % (16 * NJ);
      const int64_t pos = base + 64 * s + 8 * ((lane & 7) ^ (row & 7));
      const bool in = part < 3 && j < r && pos < Mp;
      dma_lds16(rs, ss[b] + 8 * (SI * wave + c) * 128, in ? (uint32_t)(((part * r + j) * Mp + pos) * 2) : 0x7fffffffu,
                0u);
    }
  };
  f32x4_t acc[2][NJ];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](auto along, int b, int s) __attribute__((always_inline)) {
    const char* const lt = sl[b];
    const char* const st = ss[b];
    const bool inside = base + 64 * s >= p0 && base + 64 * s + 64 <= p1;
#pragma unroll
    for (int mh = 0; mh < 2; ++mh) {
      u32x4_t a[2];
#pragma unroll
      for (int pf = 0; pf < 2; ++pf) {
        const int c = 32 * wave + 16 * pf + lr;
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          h[i] = *reinterpret_cast<const uint16_t*>(lt + lswz(32 * mh + 8 * kq + i, c >> 3) + 2 * (c & 7));
#pragma unroll
        for (int t = 0; t < 4; ++t) a[pf][t] = h[2 * t] | (h[2 * t + 1] << 16);
      }
      u32x4_t mask = {~0u, ~0u, ~0u, ~0u};
      if (!inside) {
        const int q = base + 64 * s + 32 * mh + 8 * kq;
#pragma unroll
        for (int t = 0; t < 4; ++t)
          mask[t] = (q + 2 * t >= p0 && q + 2 * t < p1 ? 0xffffu : 0u) |
                    (q + 2 * t + 1 >= p0 && q + 2 * t + 1 < p1 ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int part = 0; part < 3; ++part)
#pragma unroll
        for (int jf = 0; jf < NJ; ++jf) {
          u32x4_t f = *reinterpret_cast<const u32x4_t*>(st + sswz(16 * NJ * part + 16 * jf + lr, 4 * mh + kq));
          if (!inside)
#pragma unroll
            for (int t = 0; t < 4; ++t) f[t] &= mask[t];
#pragma unroll
          for (int pf = 0; pf < 2; ++pf)
            acc[pf][jf] = decltype(along)::value ? mfma_16x16x32(a[pf], f, acc[pf][jf])
                                                 : mfma_16x16x32(f, a[pf], acc[pf][jf]);
        }
    }
  };
  issue(0, 0);
  for (int s = 0; s < stages; ++s) {
    if (s + 1 < stages) {
      issue((s + 1) & 1, s + 1);
      wait_vmem_le<4 + SI>();
    } else {
      wait_vmem();
    }
    asm volatile("" ::: "memory");
    __syncthreads();
    if (J.along)
      compute(std::true_type(), s & 1, s);
    else
      compute(std::false_type(), s & 1, s);
    __syncthreads();
  }
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
        const int64_t c = J.along ? cb + 4 * kq + v : cb + lr;
        const int j = J.along ? jbase + lr : jbase + 4 * kq + v;
        if (c < J.cols && j < r) o[J.along ? c * r + j : j * J.cols + c] = acc[pf][jf][v];
      }
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
    if (n == 1 || first + n > max_slots) return;
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

namespace {

int64_t position_stride(int64_t M) { return round_up(std::max<int64_t>(M, 1), 64); }

// NJ blocks of 16 ranks per workgroup
int rank_blocks(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }

hipError_t launch_down(const uint16_t* L, int64_t M, int64_t Kred, const uint16_t* R, int by_id, const AdapterView& ad,
                       const PlanView& pl, const DownOut& out, hipStream_t st) {
  if (M <= kFewTokens) {
    const dim3 grid((unsigned)M, (unsigned)(ad.r / kFewRanks));
    if (M <= 16 && out.S == nullptr && out.ST == nullptr)
      adapters_few_down_kernel<true><<<grid, 256, 0, st>>>(L, M, Kred, R, by_id, ad, pl, out);
    else
      adapters_few_down_kernel<false><<<grid, 256, 0, st>>>(L, M, Kred, R, by_id, ad, pl, out);
    return hipGetLastError();
  }
  const unsigned tiles = cdiv(M, 16);
  // few tokens: one workgroup per 16 ranks, so that each reads less of the
  // adapter; then as many workgroups per tile as fill the chip once
  const int nj = tiles < 64 ? 1 : rank_blocks(ad.r);
  const unsigned z = cdiv(ad.r, 16 * nj);
  const unsigned want = 512 / (tiles * z) + 1;
  const unsigned y = std::min<unsigned>({want, 16u, (unsigned)ad.count});
  const dim3 grid(tiles, y, z), block(64 * kDownWaves);
  if (nj == 1)
    adapters_down_kernel<1><<<grid, block, 0, st>>>(L, M, Kred, R, by_id, ad, pl, out);
  else if (nj == 2)
    adapters_down_kernel<2><<<grid, block, 0, st>>>(L, M, Kred, R, by_id, ad, pl, out);
  else
    adapters_down_kernel<4><<<grid, block, 0, st>>>(L, M, Kred, R, by_id, ad, pl, out);
  return hipGetLastError();
}

}  // namespace

AdaptersFwdLayout adapters_fwd_layout(int64_t M, int64_t N, int64_t K, int r, int count) {
  AdaptersFwdLayout L{};
  L.splits = M > 16 ? fwd_gemm_splits(M, N, K, SIZE_MAX) : 1;
  L.off_S = 0;
  L.off_P = M > 16 ? round_up(M * adapter_cols(r) * 2, 256) : M > 0 ? round_up((int64_t)cdiv(r, 16) * 1024, 256) : 0;
  L.total = L.off_P + (L.splits > 1 ? round_up((int64_t)L.splits * M * N * 4, 256) : 0);
  return L;
}
AdaptersBwdLayout adapters_bwd_layout(int64_t M, int64_t N, int64_t K, int r, int count) {
  AdaptersBwdLayout L{};
  L.splits = M > 0 ? dx_gemm_splits(M, N, K, SIZE_MAX) : 1;
  if (M == 0) return L;
  const int64_t Mp = position_stride(M), used = std::min<int64_t>(count, M);
  // about 512 workgroups or more: units of 64 to 1,024 positions
  const int64_t work = (int64_t)(cdiv(K, 128) + cdiv(N, 128)) * cdiv(r, 16 * rank_blocks(r));
  const int64_t parts = std::max<int64_t>(1, (512 + work - 1) / work);
  L.unit = (int)std::min<int64_t>(kMaxUnit, round_up((M + parts - 1) / parts, 64));
  L.units = (int)(M / L.unit + used);
  L.slots = (int)(2 * M / L.unit);  // (an adapter of n > 1 units has more than (n - 1)·unit tokens)
  size_t off = 0;
  L.off_U = off;
  off += round_up(M * adapter_cols(r) * 2, 256);
  L.off_UT = off;
  off += round_up(3 * r * Mp * 2, 256);
  L.off_TT = off;
  off += round_up(3 * r * Mp * 2, 256);
  L.off_AT = off;
  off += round_up(used * K * r * 2, 256);
  L.off_BT = off;
  off += round_up(used * N * r * 2, 256);
  L.off_units = off;
  off += round_up(256 + (int64_t)(L.units + count) * 16, 256);
  L.off_P = off;
  const int64_t gemm = L.splits > 1 ? (int64_t)L.splits * M * K * 4 : 0;
  off += round_up(std::max<int64_t>(gemm, (int64_t)L.slots * r * (K + N) * 4), 256);
  L.total = off;
  return L;
}

size_t adapters_fwd_ws_max(int64_t M_max, int64_t N, int64_t K, int r, int count) {
  size_t most = adapters_fwd_layout(std::min<int64_t>(M_max, 16), N, K, r, count).total;
  // the split count depends on M through the number of 256-row tiles alone
  // and the bytes grow with M within such a band: each band's largest M
  for (int64_t top = 256; M_max > 16; top += 256) {
    most = std::max(most, adapters_fwd_layout(std::min(top, M_max), N, K, r, count).total);
    if (top >= M_max) break;
  }
  return most;
}
size_t adapters_bwd_ws_max(int64_t M_max, int64_t N, int64_t K, int r, int count) {
  // every part but the shared area grows with M; that one is bounded band by
  // band for the GEMM's partials, and for the gradients by 2M/unit slots:
  // units of at least M/parts give 2·parts, units of 1,024 at most 2M/1,024
  const AdaptersBwdLayout L = adapters_bwd_layout(M_max, N, K, r, count);
  if (M_max == 0) return L.total;
  int64_t area = 0;
  for (int64_t top = 256;; top += 256) {
    const int64_t M = std::min(top, M_max);
    const int splits = dx_gemm_splits(M, N, K, SIZE_MAX);
    if (splits > 1) area = std::max(area, splits * M * K * 4);
    if (top >= M_max) break;
  }
  const int64_t work = (int64_t)(cdiv(K, 128) + cdiv(N, 128)) * cdiv(r, 16 * rank_blocks(r));
  const int64_t parts = std::max<int64_t>(1, (512 + work - 1) / work);
  const int64_t slots = std::min(std::max<int64_t>(2 * parts, 2 * M_max / kMaxUnit), 2 * M_max / 64);
  area = std::max(area, slots * r * (K + N) * 4);
  // the units' table: M / unit is at most parts or M / 1,024
  const int64_t units = std::max(parts, M_max / kMaxUnit) + std::min<int64_t>(count, M_max);
  return L.off_units + round_up(256 + (units + count) * 16, 256) + round_up(area, 256);
}

hipError_t launch_adapters_fwd(const Nf4View& W, const uint16_t* X, int64_t M, const AdapterView& ad,
                               const PlanView& pl, void* Y, bool y16, float* T_save, char* ws,
                               const AdaptersFwdLayout& L, hipStream_t st) {
  if (M == 0) return hipSuccess;
  if (M <= 16) {
    float* Tt = reinterpret_cast<float*>(ws + L.off_S);
    const hipError_t e = launch_down(X, M, W.K, ad.A, 1, ad, pl, DownOut{T_save, Tt, nullptr, nullptr, 0}, st);
    return e != hipSuccess ? e : launch_gemv_adapters(W, X, M, ad, pl.owner, Y, y16, Tt, st);
  }
  uint16_t* S = reinterpret_cast<uint16_t*>(ws + L.off_S);
  float* P = reinterpret_cast<float*>(ws + L.off_P);
  hipError_t e = launch_down(X, M, W.K, ad.A, 1, ad, pl, DownOut{T_save, nullptr, S, nullptr, 0}, st);
  if (e != hipSuccess) return e;
  const AdapterGemmArgs ma{pl.head, (int)plan_pad(M), (int)plan_pad(ad.count + 1), S, ad.B, ad.r,
                           (int)adapter_cols(ad.r), ad.count, 1};
  e = launch_fwd_gemm_adapters(W, X, M, ma, Y, y16, L.splits, P, st);
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
  const int64_t Mp = position_stride(M);
  uint16_t* U = reinterpret_cast<uint16_t*>(ws + L.off_U);
  uint16_t* UT = reinterpret_cast<uint16_t*>(ws + L.off_UT);
  uint16_t* TT = reinterpret_cast<uint16_t*>(ws + L.off_TT);
  uint16_t* AT = reinterpret_cast<uint16_t*>(ws + L.off_AT);
  uint16_t* BT = reinterpret_cast<uint16_t*>(ws + L.off_BT);
  float* P = reinterpret_cast<float*>(ws + L.off_P);
  UnitTable ut;
  ut.head = reinterpret_cast<int32_t*>(ws + L.off_units);
  ut.unit = reinterpret_cast<int4*>(ws + L.off_units + 256);
  ut.of_group = ut.unit + L.units;
  const unsigned jb = cdiv(r, 64), bt = T_saved ? cdiv(Mp, 64) * jb : 0u;
  const unsigned nb = cdiv(N, 64) * jb, na = cdiv(K, 64) * jb;
  const unsigned used = (unsigned)std::min<int64_t>(ad.count, M);
  adapters_prep_kernel<<<1 + bt + used * (nb + na), 256, 0, st>>>(T_saved, M, Mp, TT, BT, N, AT, K, ad, pl, ut, L.unit,
                                                                  L.units, L.slots, bt, nb, na, jb);
  e = hipGetLastError();
  if (e == hipSuccess && !T_saved)
    e = launch_down(X, M, K, ad.A, 1, ad, pl, DownOut{nullptr, nullptr, nullptr, TT, Mp}, st);
  if (e == hipSuccess) e = launch_down(dY, M, N, BT, 0, ad, pl, DownOut{nullptr, nullptr, U, UT, Mp}, st);
  if (e != hipSuccess) return e;
  const AdapterGemmArgs ma{pl.head, (int)plan_pad(M), (int)plan_pad(ad.count + 1), U, AT, ad.r,
                           (int)adapter_cols(r), ad.count, 0};
  e = launch_dx_gemm_adapters(W, dY, M, ma, dX, dx16, L.splits, P, st);
  if (e == hipSuccess && L.splits > 1) e = launch_splitk_reduce(P, L.splits, M * K, dX, dx16, false, st);
  if (e != hipSuccess) return e;
  const int64_t slot = r * (K + N);
  const GradientJob ja{X, K, UT, dA, 0, 0}, jo{dY, N, TT, dB, r * K, 1};
  const int nj = rank_blocks(ad.r);
  const unsigned ta = cdiv(K, 128);
  const dim3 grid(ta + cdiv(N, 128), (unsigned)L.units, cdiv(r, 16 * nj));
  if (nj == 1)
    adapters_gradient_kernel<1><<<grid, 256, 0, st>>>(ja, jo, ta, M, Mp, ad, pl, ut, P, slot);
  else if (nj == 2)
    adapters_gradient_kernel<2><<<grid, 256, 0, st>>>(ja, jo, ta, M, Mp, ad, pl, ut, P, slot);
  else
    adapters_gradient_kernel<4><<<grid, 256, 0, st>>>(ja, jo, ta, M, Mp, ad, pl, ut, P, slot);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  adapters_gradient_finish_kernel<<<dim3(std::min(cdiv(slot, 1024), 256u), (unsigned)ad.count), 256, 0, st>>>(
      dA, dB, r * K, r * N, ad.count, pl, ut, P, L.slots);
  return hipGetLastError();
}

}  // namespace qnf4
