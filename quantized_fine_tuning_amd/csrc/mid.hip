// Base products of a batch of few tokens that carry different adapters (17 to
// kMidTokens), gfx950.  The dequant-in-tile GEMMs (fwd.hip, dx.hip) decode
// 256 weight rows for 256 tokens and are bound by that decode long before the
// tokens are many; here a weight fragment goes from its codes to the MFMA
// operand with as little between as its layout allows, and every tile of 16
// tokens uses it (forward of 32 tokens, 4096 x 4096, 18.8 us against 28.9 with
// the GEMM; 11008 x 4096, 34.1 against 40.7 and at 64 tokens 41.4 against 43.4;
// at 128 the GEMM is faster, 50 against 58).  A stage takes about 2.3 us of
// decode (lookups and operand reads share the LDS), with 7.7 us around all of
// them.  Tokens are taken in plan order (AdapterGemmArgs), the
// reduction is split over workgroups, fp32 partial sums are added in split
// order by splitk_reduce_kernel.
#include <algorithm>

#include "host.h"
#include "tiling.h"

namespace qnf4 {
namespace {

constexpr int kMidThreads = 512, kMidWaves = kMidThreads / 64;

// Waits for this wave's copies but the newest N and for its LDS reads, then
// for the workgroup.
template <int N>
__device__ __forceinline__ void open_stage() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));  // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Output rows of an accumulator tile back to their tokens: lane holds rows
// 4kq + v of each 16-position tile, one column; the tokens of its rows are
// loaded at the kernel's start.
template <int NT>
struct RowTokens {
  int t[NT][4];
  __device__ __forceinline__ RowTokens(const AdapterGemmArgs& ma, int p0, int64_t M, int kq) {
    int4 v[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
      v[i] = *reinterpret_cast<const int4*>(ma.perm() + std::min(p0 + 16 * i + 4 * kq, ((int)M - 1) & ~3));
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) t[i][q] = p0 + 16 * i + 4 * kq + q < (int)M && (uint32_t)w[q] < (uint32_t)M ? w[q] : -1;
    }
  }
  template <typename Put>
  __device__ __forceinline__ void scatter(const f32x4_t* acc, Put&& put) const {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (t[i][q] >= 0) put(t[i][q], acc[i][q]);
  }
};

// The adapters' share as more reduction stages of 256 columns: the `cols` split
// ranks of each used adapter among positions [p0, p0 + rows), one adapter after
// another (column c belongs to used adapter gfirst + c / cols); `all` columns,
// this split's stages [first, last).
struct LoraShare {
  int gfirst, all, first, last;
};
__device__ __forceinline__ LoraShare lora_share(const AdapterGemmArgs& ma, int p0, int rows, int64_t M, int sp,
                                                int splits) {
  LoraShare s{0, 0, 0, 0};
  const int held = std::min(ma.held(), (int)M);
  if (p0 < held) {
    s.gfirst = ma.group(p0);
    const int glast = std::min(ma.group(std::min(p0 + rows, held) - 1), ma.count - 1);
    s.all = s.gfirst >= 0 && glast >= s.gfirst ? std::min(glast - s.gfirst + 1, rows) * ma.cols : 0;
    const int stages = (s.all + 255) / 256;
    s.first = split_first(sp, splits, stages);
    s.last = split_first(sp + 1, splits, stages);
  }
  return s;
}

// ---------------------------------------------------------------------------
// Y = X·Ŵᵀ + S·Bᵀ for 16·NT positions and 128 weight rows, 16 per wave.  A
// stage is 256 reduction elements: four NF4 blocks of each row, lane (row l % 16,
// q = l / 16) owning block q with its one constant.  The lane decodes 8 codes
// at a time straight into an MFMA operand (levels from a 16-entry LDS table;
// its 8 reduction slots are elements 8t .. 8t + 7 of its block) and multiplies
// it with NT operands of X, which is copied into LDS a stage ahead (row p's
// 16-byte chunk c at c ^ (p & 15), so that the 16 rows of one read differ in
// bank: 256 bytes a clock).  The adapters come first, as stages of the same
// shape (LoraShare): S rows into a free stage of the ring, every 8-rank piece of
// B_a[n] straight into its operand register.
// ---------------------------------------------------------------------------
template <int NT>
__global__ __launch_bounds__(kMidThreads) void mid_fwd_kernel(Nf4View W, const uint16_t* __restrict__ X, int64_t M,
                                                              void* __restrict__ Y, int y_bf16, int tiles_n, int splits,
                                                              float* __restrict__ P, Codebook cb, AdapterGemmArgs ma) {
  constexpr int TM = 16 * NT, ROW = 512, XB = TM * ROW, WB = 2560;  // bytes: X of a stage, one wave's codes and constants
  constexpr int D = NT == 2 ? 4 : 3;                                // ring depth
  __shared__ __attribute__((aligned(1024))) char sx[D][XB];
  __shared__ __attribute__((aligned(1024))) char sc[D][kMidWaves * WB];
  __shared__ __attribute__((aligned(256))) float sq[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, kq = lane >> 4;
  const int64_t K = W.K, N = W.N;
  const int tn = (int)blockIdx.x % tiles_n, tm = (int)blockIdx.x / tiles_n, sp = (int)blockIdx.y;
  const int p0 = TM * tm;
  const int64_t n0 = 128 * (int64_t)tn + 16 * wave;  // this wave's rows
  const uint32_t kpr = (uint32_t)(K / kBlock);
  const int all = (int)((K + 255) / 256);
  const int s0 = split_first(sp, splits, all), s1 = split_first(sp + 1, splits, all);
  const float mu = *W.mu;
  const i32x4_t rc = rsrc_words(W.codes + n0 * (K / 2), (N - n0) * (K / 2));
  const i32x4_t re = rsrc_words(W.e, N * kpr);
  const i32x4_t rs = rsrc_words(W.s, ((N * kpr + kDqBlock - 1) / kDqBlock) * 4);
  const i32x4_t rx = rsrc_words(X, M * K * 2);

  // X: wave w copies rows 2(NT·w + c), +1; lane l physical chunk l % 32
  uint32_t vx[NT];
  int ch[NT];
  {
    int tok[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) tok[c] = ma.perm()[std::min(p0 + 2 * (NT * wave + c) + (lane >> 5), (int)M - 1)];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      const int row = 2 * (NT * wave + c) + (lane >> 5);
      ch[c] = (lane & 31) ^ (row & 15);
      vx[c] = p0 + row < (int)M && (uint32_t)tok[c] < (uint32_t)M ? (uint32_t)tok[c] * (uint32_t)K * 2u + 16u * ch[c]
                                                                  : 0x7fffffffu;
    }
  }
  // The codes, their e4m3 bytes' dwords and their scales go through LDS too:
  // with every load a copy that the compiler does not track, the waits are
  // the explicit ones alone and a stage has D - 1 stages of time to arrive.
  const uint32_t vcode = (uint32_t)(lr * (K / 2)) + 32u * kq, blk0 = (uint32_t)(n0 + lr) * kpr + kq;
  const bool row_ok = n0 + lr < N;
  auto issue = [&](int b, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < NT; ++c)
      dma_lds16(rx, sx[b] + (NT * wave + c) * 1024,
                s < s1 && 256 * (int64_t)s + 8 * ch[c] < K ? vx[c] : 0x7fffffffu, (uint32_t)s * 512u);
    const bool ok = s < s1 && row_ok && 4 * (uint32_t)s + kq < kpr;
    char* const w = sc[b] + wave * WB;
    const uint32_t blk = blk0 + 4 * (uint32_t)s;
    dma_lds16(rc, w, ok ? vcode + 128u * s : 0x7fffffffu, 0u);
    dma_lds16(rc, w + 1024, ok ? vcode + 128u * s + 16u : 0x7fffffffu, 0u);
    dma_lds4(re, w + 2048, ok ? blk & ~3u : 0x7fffffffu, 0u);
    dma_lds4(rs, w + 2304, ok ? (blk / kDqBlock) * 4u : 0x7fffffffu, 0u);
  };
  f32x4_t acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint32_t sqb = lds_offset(sq);
  auto consume = [&](const char* xt, const char* w, int s) __attribute__((always_inline)) {
    u32x4_t c[2];
    c[0] = *reinterpret_cast<const u32x4_t*>(w + 16 * lane);
    c[1] = *reinterpret_cast<const u32x4_t*>(w + 1024 + 16 * lane);
    const uint32_t e4 = *reinterpret_cast<const uint32_t*>(w + 2048 + 4 * lane);
    const float sg = *reinterpret_cast<const float*>(w + 2304 + 4 * lane);
    const float cp = decode_constant((e4 >> (8 * ((blk0 + 4 * (uint32_t)s) & 3u))) & 0xffu, sg, mu);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t cw = c[t >> 2][t & 3];  // codes 8t .. 8t+7
      const uint32_t we = (cw << 2) & 0x3C3C3C3Cu, wo = (cw >> 2) & 0x3C3C3C3Cu;
      u32x4_t bf;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float qe = *(const __attribute__((address_space(3))) float*)(uintptr_t)__builtin_amdgcn_perm(
            sqb, we, 0x07060500u | (uint32_t)p);
        const float qo = *(const __attribute__((address_space(3))) float*)(uintptr_t)__builtin_amdgcn_perm(
            sqb, wo, 0x07060500u | (uint32_t)p);
        bf[p] = pack_bf16x2(__fmul_rn(qe, cp), __fmul_rn(qo, cp));
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const u32x4_t a =
            *reinterpret_cast<const u32x4_t*>(xt + (16 * i + lr) * ROW + (((8 * kq + t) ^ lr) << 4));
        acc[i] = mfma_16x16x32(a, bf, acc[i]);
      }
    }
  };
  const RowTokens<NT> rows(ma, p0, M, kq);
  const float cbq = cb.q[tid & 15];
#pragma unroll
  for (int i = 0; i + 1 < D; ++i) issue(i, s0 + i);
  if (tid < 16) sq[tid] = cbq;

  // the adapters, while the first stages are on their way, through the ring's
  // free stage
  const LoraShare L = lora_share(ma, p0, TM, M, sp, splits);
  if (L.first < L.last) {
    const i32x4_t rS = rsrc_words(ma.S, M * ma.C * 2);
    const float inv_cols = 1.0f / (float)ma.cols;
    // (c + 0.5) / cols is never nearer than 0.5 / cols to a whole number
    auto adapter_of = [&](int c) __attribute__((always_inline)) { return (int)(((float)c + 0.5f) * inv_cols); };
    for (int ls = L.first; ls < L.last; ++ls) {
      int id[8], at[8], lo[NT], hi[NT], col[NT];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int c = 256 * ls + 64 * kq + 8 * t, cc = std::min(c, L.all - 8), g = adapter_of(cc);
        at[t] = c < L.all && row_ok ? (cc - g * ma.cols) % ma.r : -1;
        id[t] = ma.id(L.gfirst + g);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int c = 256 * ls + 8 * ch[i], cc = std::min(c, L.all - 8), g = adapter_of(cc);
        col[i] = c < L.all ? cc - g * ma.cols : -1;
        lo[i] = ma.start(L.gfirst + g) - p0;
        hi[i] = std::min(ma.start(L.gfirst + g + 1), (int)M) - p0;
      }
      if (ls > L.first) open_stage<0>();  // (the free stage is read)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int row = 2 * (NT * wave + i) + (lane >> 5);
        const bool in = col[i] >= 0 && row >= lo[i] && row < hi[i];
        dma_lds16(rS, sx[D - 1] + (NT * wave + i) * 1024,
                  in ? (uint32_t)(((p0 + row) * ma.C + col[i]) * 2) : 0x7fffffffu, 0u);
      }
      u32x4_t bf[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const bool ok = at[t] >= 0 && (unsigned)id[t] < (unsigned)ma.count;
        bf[t] = *reinterpret_cast<const u32x4_t*>(
            ma.F + (ok ? ((int64_t)id[t] * N + n0 + lr) * ma.r + at[t] : 0));
        if (!ok) bf[t] = u32x4_t{0u, 0u, 0u, 0u};
      }
      open_stage<0>();
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const u32x4_t a = *reinterpret_cast<const u32x4_t*>(sx[D - 1] + (16 * i + lr) * ROW +
                                                              (((8 * kq + t) ^ lr) << 4));
          acc[i] = mfma_16x16x32(a, bf[t], acc[i]);
        }
    }
  }

  int b = 0;
  for (int s = s0; s < s1; ++s) {
    open_stage<(D - 2) * (NT + 4)>();
    issue(b == 0 ? D - 1 : b - 1, s + D - 1);
    consume(sx[b], sc[b] + wave * WB, s);
    b = b + 1 == D ? 0 : b + 1;
  }
  wait_vmem();  // no copy may land in LDS after the workgroup ends

  const int64_t n = n0 + lr;
  if (n >= N) return;
  if (splits > 1) {
    float* const D0 = P + (int64_t)sp * M * N + n;
    rows.scatter(acc, [&](int tok, float v) { D0[(int64_t)tok * N] = v; });
  } else if (y_bf16) {
    uint16_t* const D0 = static_cast<uint16_t*>(Y) + n;
    rows.scatter(acc, [&](int tok, float v) { D0[(int64_t)tok * N] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu); });
  } else {
    float* const D0 = static_cast<float*>(Y) + n;
    rows.scatter(acc, [&](int tok, float v) { D0[(int64_t)tok * N] = v; });
  }
}

// Positions per workgroup, in tiles of 16.
int mid_tiles(int64_t M) { return M <= 32 ? 2 : 4; }

}  // namespace

// The split count with the least estimated time, in microseconds: rounds of
// workgroups over the 256 compute units at 2.3 us a stage and 7.7 around them,
// and the fp32 partials written and read at 4 TB/s.
int mid_splits(int64_t tiles, int64_t stages, int64_t elements) {
  int best = 1;
  double least = 0;
  for (int64_t s = 1; s <= 16 && 2 * s <= std::max<int64_t>(stages, 2); ++s) {
    const double t = (double)((tiles * s + 255) / 256) * ((double)((stages + s - 1) / s) * 2.3 + 7.7) +
                     (s > 1 ? (double)s * (double)elements * 8 / 4e6 : 0.0);
    if (s == 1 || t < least) {
      least = t;
      best = (int)s;
    }
  }
  return best;
}
int mid_fwd_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t tm = 16 * mid_tiles(M);
  return mid_splits(((M + tm - 1) / tm) * ((N + 127) / 128), (K + 255) / 256, M * N);
}

hipError_t launch_mid_fwd(const Nf4View& W, const uint16_t* X, int64_t M, const AdapterGemmArgs& ma, void* Y, bool y16,
                          int splits, float* P, hipStream_t st) {
  const int nt = mid_tiles(M), tm = 16 * nt, tiles_n = (int)((W.N + 127) / 128);
  const dim3 grid((unsigned)(tiles_n * ((M + tm - 1) / tm)), (unsigned)splits);
#define QNF4_MID(NT) \
  mid_fwd_kernel<NT><<<grid, kMidThreads, 0, st>>>(W, X, M, Y, y16 ? 1 : 0, tiles_n, splits, P, codebook(), ma)
  if (nt == 2)
    QNF4_MID(2);
  else
    QNF4_MID(4);
#undef QNF4_MID
  return hipGetLastError();
}

}  // namespace qnf4
