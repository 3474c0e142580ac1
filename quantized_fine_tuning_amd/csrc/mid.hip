// Base products of a batch of few tokens (17 to kMidTokens) that carry different
// adapters (AdapterGemmArgs), or one that may have dropout (DenseGemmArgs: in dX the
// adapter's share is summed and masked before the base product; 61 tokens, 4096 x
// 4096, 17.6 us of 26.1 for the pass), gfx950.  The dequant-in-tile GEMMs (fwd.hip,
// dx.hip) decode 256 weight rows for 256 tokens and are bound by that decode long
// before the tokens are many; here a weight fragment goes from its codes to the MFMA
// operand with as little between as its layout allows, and every tile of 16
// tokens uses it (forward of 32 tokens, 4096 x 4096, 18.8 us against 28.9 with
// the GEMM; 11008 x 4096, 34.1 against 40.7 and at 64 tokens 41.4 against 43.4;
// at 128 the GEMM is faster, 50 against 58).  A stage takes about 2.3 us of
// decode (lookups and operand reads share the LDS), with 7.7 us around all of
// them.  Tokens are taken in plan order (AdapterGemmArgs), the
// reduction is split over workgroups, fp32 partial sums are added in split
// order by splitk_reduce_kernel.
#include <algorithm>
#include <type_traits>

#include "dropout.h"
#include "host.h"
#include "tiling.h"

namespace qnf4 {
namespace {

// blockIdx.z = 1: the second layer of a pair, which has fp32 outputs.
__device__ __forceinline__ void other_layer(Nf4View& W, const uint16_t* __restrict__& L, void* __restrict__& out,
                                            float* __restrict__& P, DenseGemmArgs& ma) {
  if (blockIdx.z == 0) return;
  W = ma.W1;
  L = ma.L1;
  ma.F = ma.F1;
  ma.S += ma.next_S;
  out = static_cast<float*>(out) + ma.next_P;
  P += ma.next_P;
}

// Output rows of an accumulator tile back to their tokens: lane holds rows
// 4kq + v of each 16-position tile, one column; the tokens of its rows are
// loaded at the kernel's start.
template <int NT>
struct RowTokens {
  int t[NT][4];
  template <typename Args>
  __device__ __forceinline__ RowTokens(const Args& ma, int p0, int64_t M, int kq) {
    int4 v[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) v[i] = ma.tokens4(std::min(p0 + 16 * i + 4 * kq, ((int)M - 1) & ~3));
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

// The adapters' share as more reduction stages of `width` columns: the split
// ranks of each used adapter among positions [p0, p0 + rows), one adapter after
// another, `each` columns (`cols` and zeros up to a multiple of 32, so that the
// 32 columns of one matrix instruction are one adapter's and its result can be
// kept to that adapter's rows where the adapter holds an infinity or NaN, which
// times another row's zeros is NaN); `all` columns, this split's stages [first, last).
struct LoraShare {
  int gfirst, each, all, first, last;
  float inv_each;
  // ((c + 0.5) / each is never nearer than 0.5 / each to a whole number)
  __device__ __forceinline__ int adapter_of(int c) const { return (int)(((float)c + 0.5f) * inv_each); }
  // the rows, from p0 on, of the adapter that columns [c, c + 32) belong to
  template <typename Args>
  __device__ __forceinline__ void rows(const Args& ma, int c, int p0, int64_t M, int& lo, int& hi) const {
    const int g = adapter_of(std::min(c, all - 32));
    lo = c < all ? ma.start(gfirst + g) - p0 : 0;
    hi = c < all ? std::min(ma.start(gfirst + g + 1), (int)M) - p0 : 0;
  }
};
template <typename Args>
__device__ __forceinline__ LoraShare lora_share(const Args& ma, int p0, int rows, int64_t M, int sp,
                                                int splits, int width) {
  const int each = (ma.cols + 31) & ~31;
  LoraShare s{0, each, 0, 0, 0, 1.0f / (float)each};
  const int held = std::min(ma.held(), (int)M);
  if (p0 < held) {
    s.gfirst = ma.group(p0);
    const int glast = std::min(ma.group(std::min(p0 + rows, held) - 1), ma.count - 1);
    s.all = s.gfirst >= 0 && glast >= s.gfirst ? std::min(glast - s.gfirst + 1, rows) * each : 0;
    const int stages = (s.all + width - 1) / width;
    s.first = split_first(sp, splits, stages);
    s.last = split_first(sp + 1, splits, stages);
  }
  return s;
}

// ---------------------------------------------------------------------------
// Y = X·Ŵᵀ + S·Bᵀ for 16·NT positions and 16 weight rows per wave.  A
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
// WV waves: 8, or 16 with twice the weight rows (four waves on a SIMD cover each
// other's lookups better, 2.9 us for a stage of twice the weights, but the
// tiles are fewer: mid_fwd_plan).
template <int NT, int WV, typename Args>
__global__ __launch_bounds__(64 * WV) void mid_fwd_kernel(Nf4View W, const uint16_t* __restrict__ X, int64_t M,
                                                              void* __restrict__ Y, int y_bf16, int tiles_n, int splits,
                                                              float* __restrict__ P, Codebook cb, Args ma) {
  constexpr int TM = 16 * NT, ROW = 512, XB = TM * ROW, WB = 2560;  // bytes: X of a stage, one wave's codes and constants
  if constexpr (Args::kPair) other_layer(W, X, Y, P, ma);
  constexpr int D = WV == 16 ? 2 : NT == 2 ? 4 : 3, XI = 8 * NT / WV;                                // ring depth
  __shared__ __attribute__((aligned(1024))) char sx[D][XB];
  __shared__ __attribute__((aligned(1024))) char sc[D][WV * WB];
  __shared__ __attribute__((aligned(256))) float sq[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, kq = lane >> 4;
  const int64_t K = W.K, N = W.N;
  const int tn = (int)blockIdx.x % tiles_n, tm = (int)blockIdx.x / tiles_n, sp = (int)blockIdx.y;
  const int p0 = TM * tm;
  const int64_t n0 = 16 * WV * (int64_t)tn + 16 * wave;  // this wave's rows
  const uint32_t kpr = (uint32_t)(K / kBlock);
  const int all = (int)((K + 255) / 256);
  const int s0 = split_first(sp, splits, all), s1 = split_first(sp + 1, splits, all);
  const float mu = *W.mu;
  const i32x4_t rc = rsrc_words(W.codes + n0 * (K / 2), (N - n0) * (K / 2));
  const i32x4_t re = rsrc_words(W.e, N * kpr);
  const i32x4_t rs = rsrc_words(W.s, ((N * kpr + kDqBlock - 1) / kDqBlock) * 4);
  const i32x4_t rx = rsrc_words(X, M * K * 2);

  // X: wave w copies rows 2(XI·w + c), +1; lane l physical chunk l % 32
  uint32_t vx[XI];
  int ch[XI];
  {
    int tok[XI];
#pragma unroll
    for (int c = 0; c < XI; ++c) tok[c] = ma.token(std::min(p0 + 2 * (XI * wave + c) + (lane >> 5), (int)M - 1));
#pragma unroll
    for (int c = 0; c < XI; ++c) {
      const int row = 2 * (XI * wave + c) + (lane >> 5);
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
    for (int c = 0; c < XI; ++c)
      dma_lds16(rx, sx[b] + (XI * wave + c) * 1024,
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
  const LoraShare L = lora_share(ma, p0, TM, M, sp, splits, 256);
  if (L.first < L.last) {
    const i32x4_t rS = rsrc_words(ma.S, M * ma.C * 2);
    for (int ls = L.first; ls < L.last; ++ls) {
      // matrix instruction t: columns [32t, +32) of the stage, 8 per lane
      int id[8], at[8], lo[XI], hi[XI], col[XI];
      auto piece = [&](int t, int& a, int& rank) __attribute__((always_inline)) {
        const int c = 256 * ls + 32 * t, cc = std::min(c, L.all - 32), g = L.adapter_of(cc), j = cc - g * L.each + 8 * kq;
        rank = c < L.all && j < ma.cols && row_ok ? j % ma.r : -1;
        a = ma.id(L.gfirst + g);
      };
      auto load_piece = [&](int a, int rank) __attribute__((always_inline)) {
        const bool ok = rank >= 0 && (unsigned)a < (unsigned)ma.count;
        const u32x4_t v =
            *reinterpret_cast<const u32x4_t*>(ma.F + (ok ? ((int64_t)a * N + n0 + lr) * ma.r + rank : 0));
        return ok ? v : u32x4_t{0u, 0u, 0u, 0u};
      };
#pragma unroll
      for (int t = 0; t < 8; ++t) piece(t, id[t], at[t]);
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int c = 256 * ls + 8 * ch[i], cc = std::min(c, L.all - 8), g = L.adapter_of(cc);
        col[i] = c < L.all && cc - g * L.each < ma.cols ? cc - g * L.each : -1;
        lo[i] = ma.start(L.gfirst + g) - p0;
        hi[i] = std::min(ma.start(L.gfirst + g + 1), (int)M) - p0;
      }
      if (ls > L.first) open_stage<0>();  // (the free stage is read)
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int row = 2 * (XI * wave + i) + (lane >> 5);
        const bool in = col[i] >= 0 && row >= lo[i] && row < hi[i];
        dma_lds16(rS, sx[D - 1] + (XI * wave + i) * 1024,
                  in ? (uint32_t)(((p0 + row) * ma.C + col[i]) * 2) : 0x7fffffffu, 0u);
      }
      u32x4_t bf[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) bf[t] = load_piece(id[t], at[t]);
      open_stage<0>();
      const bool apart = any_not_finite<false>(bf, 8);
      auto operand = [&](int i, int t) __attribute__((always_inline)) {
        return *reinterpret_cast<const u32x4_t*>(sx[D - 1] + (16 * i + lr) * ROW + (((4 * t + kq) ^ lr) << 4));
      };
      if (!apart) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
#pragma unroll
          for (int i = 0; i < NT; ++i) acc[i] = mfma_16x16x32(operand(i, t), bf[t], acc[i]);
          if (t % 2) __builtin_amdgcn_sched_barrier(0);  // (not every operand's registers at once)
        }
      }
      asm volatile("" ::: "memory");
      if (apart) {
#pragma unroll 1
        for (int t = 0; t < 8; ++t) {
          int first, end, a, rank;
          L.rows(ma, 256 * ls + 32 * t, p0, M, first, end);
          piece(t, a, rank);
          const u32x4_t f = load_piece(a, rank);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            bool in[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) in[v] = 16 * i + 4 * kq + v >= first && 16 * i + 4 * kq + v < end;
            mfma_rows<false, false>(operand(i, t), f, acc[i], in);
          }
        }
      }
    }
  }

  int b = 0;
  for (int s = s0; s < s1; ++s) {
    open_stage<(D - 2) * (XI + 4)>();
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

// ---------------------------------------------------------------------------
// dX = dY·Ŵ + S·A for 16·NT positions and 128 columns k, 32 per wave.  The
// reduction runs over weight rows while a row's codes run along k, so a stage
// of 64 rows is decoded into a bf16 tile [row][k] (thread: 32 codes of a row)
// and the MFMA operands, 8 rows of one column, are transposing reads of it.
// dY rows, codes and constants are copied into LDS two stages ahead; within a
// stage the products come first and the next stage's decode after them.  The
// adapters come first of all, as stages of 64 split ranks (LoraShare): rows of
// A_a in the tile's place.  Two workgroups share a compute unit.  (61 tokens,
// 4096 x 4096: 17.7 us against 25.3 with the GEMM.)
// ---------------------------------------------------------------------------
constexpr int kDxThreads = 256;
// byte of column `col` (a multiple of 4) of tile row `row`: 16-byte chunk c at
// c ^ ((row & 3) << 1), the 4 rows of a transposing read on different banks
__device__ __forceinline__ int tswz(int row, int col) {
  return row * 256 + (((col >> 3) ^ ((row & 3) << 1)) << 4) + 2 * (col & 7);
}
// (DenseGemmArgs with dropout: between the adapters and the weight the sums are the
// low-rank product alone, and those of dropped elements become zero.)
template <int NT, typename Args>
__global__ __launch_bounds__(kDxThreads) void mid_dx_kernel(Nf4View W, const uint16_t* __restrict__ dY, int64_t M,
                                                            void* __restrict__ dX, int dx_bf16, int tiles_k, int splits,
                                                            float* __restrict__ P, Codebook cb, Args ma) {
  if constexpr (Args::kPair) other_layer(W, dY, dX, P, ma);
  constexpr int TM = 16 * NT, D = 3, YI = NT / 2;  // dY copies per wave and stage (8 rows each)
  __shared__ __attribute__((aligned(1024))) char sy[D][TM * 128];
  __shared__ __attribute__((aligned(1024))) char sc[D][4 * 1536];  // per wave: codes 1 KB, e4m3 dwords, scales
  __shared__ __attribute__((aligned(1024))) char sw[2][64 * 256];
  __shared__ __attribute__((aligned(256))) float sq[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, kq = lane >> 4;
  const int64_t K = W.K, N = W.N;
  const int tk = (int)blockIdx.x % tiles_k, tm = (int)blockIdx.x / tiles_k, sp = (int)blockIdx.y;
  const int p0 = TM * tm;
  const int64_t k0 = 128 * (int64_t)tk;
  const uint32_t kpr = (uint32_t)(K / kBlock);
  const int all = (int)((N + 63) / 64);
  const int s0 = split_first(sp, splits, all), s1 = split_first(sp + 1, splits, all);
  const float mu = *W.mu;
  const i32x4_t ry = rsrc_words(dY, M * N * 2), rc = rsrc_words(W.codes, N * (K / 2)), re = rsrc_words(W.e, N * kpr);
  const i32x4_t rs = rsrc_words(W.s, ((N * kpr + kDqBlock - 1) / kDqBlock) * 4);
  const RowTokens<NT> rows(ma, p0, M, kq);

  // dY: wave w copies rows 8(YI·w + c) + (lane >> 3), lane l physical chunk l % 8
  const int ych = (lane & 7) ^ (lane >> 3);
  uint32_t vy[YI];
  {
    int tok[YI];
#pragma unroll
    for (int c = 0; c < YI; ++c) tok[c] = ma.token(std::min(p0 + 8 * (YI * wave + c) + (lane >> 3), (int)M - 1));
#pragma unroll
    for (int c = 0; c < YI; ++c)
      vy[c] = p0 + 8 * (YI * wave + c) + (lane >> 3) < (int)M && (uint32_t)tok[c] < (uint32_t)M
                  ? (uint32_t)tok[c] * (uint32_t)N * 2u + 16u * ych
                  : 0x7fffffffu;
  }
  // this thread's codes: row drow of a stage, columns [32·dq, +32) of the tile
  const int drow = tid >> 2, dq = tid & 3;
  const bool dcol = k0 + 32 * dq < K;
  const uint32_t vcode = (uint32_t)(drow * (K / 2)) + (uint32_t)(k0 / 2) + 16u * dq;
  const uint32_t blk0 = (uint32_t)drow * kpr + (uint32_t)(k0 / kBlock) + (dq >> 1);
  auto issue = [&](int b, int s) __attribute__((always_inline)) {
    const bool in = s < s1 && 64 * (int64_t)s + 8 * ych < N;
#pragma unroll
    for (int c = 0; c < YI; ++c)
      dma_lds16(ry, sy[b] + (YI * wave + c) * 1024, in ? vy[c] : 0x7fffffffu, (uint32_t)s * 128u);
    const bool ok = s < s1 && dcol && 64 * (int64_t)s + drow < N;
    char* const w = sc[b] + wave * 1536;
    const uint32_t blk = blk0 + 64 * (uint32_t)s * kpr;
    dma_lds16(rc, w, ok ? vcode + (uint32_t)(32 * (int64_t)s * K) : 0x7fffffffu, 0u);
    dma_lds4(re, w + 1024, ok ? blk & ~3u : 0x7fffffffu, 0u);
    dma_lds4(rs, w + 1280, ok ? (blk / kDqBlock) * 4u : 0x7fffffffu, 0u);
  };
  const uint32_t sqb = lds_offset(sq);
  // this thread's 32 values of stage s into the tile (zeros past N: with no
  // scale and no code they would be level 0 times the mean)
  auto decode = [&](const char* w, char* t, int s) __attribute__((always_inline)) {
    const u32x4_t c = *reinterpret_cast<const u32x4_t*>(w + 16 * lane);
    const uint32_t e4 = *reinterpret_cast<const uint32_t*>(w + 1024 + 4 * lane);
    const float sg = *reinterpret_cast<const float*>(w + 1280 + 4 * lane);
    const uint32_t blk = blk0 + 64 * (uint32_t)s * kpr;
    const bool ok = dcol && 64 * (int64_t)s + drow < N;
    const float cp = ok ? decode_constant((e4 >> (8 * (blk & 3u))) & 0xffu, sg, mu) : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t we = (c[i] << 2) & 0x3C3C3C3Cu, wo = (c[i] >> 2) & 0x3C3C3C3Cu;
      u32x4_t o;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float qe = *(const __attribute__((address_space(3))) float*)(uintptr_t)__builtin_amdgcn_perm(
            sqb, we, 0x07060500u | (uint32_t)p);
        const float qo = *(const __attribute__((address_space(3))) float*)(uintptr_t)__builtin_amdgcn_perm(
            sqb, wo, 0x07060500u | (uint32_t)p);
        o[p] = pack_bf16x2(__fmul_rn(qe, cp), __fmul_rn(qo, cp));
      }
      *reinterpret_cast<u32x4_t*>(t + tswz(drow, 32 * dq + 8 * i)) = o;
    }
  };
  f32x4_t acc[2][NT];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[f][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const char* y, const char* t, auto&& add) __attribute__((always_inline)) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4_t b[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int row = 32 * ks + 8 * kq + (lr >> 2), col = 32 * wave + 16 * f + 4 * (lr & 3);
        const u32x2_t h0 = lds_read_tr(t + tswz(row, col)), h1 = lds_read_tr(t + tswz(row + 4, col));
        b[f] = u32x4_t{h0[0], h0[1], h1[0], h1[1]};
      }
      add(ks, b, [&](int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const u32x4_t*>(y + (16 * i + lr) * 128 + (((4 * ks + kq) ^ (lr & 7)) << 4));
      });
    }
  };
  auto all_rows = [&](int, const u32x4_t* w, auto&& y) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const u32x4_t a = y(i);
#pragma unroll
      for (int f = 0; f < 2; ++f) acc[f][i] = mfma_16x16x32(a, w[f], acc[f][i]);
    }
  };
  constexpr int PER = YI + 3;  // copies per wave and stage
  const float cbq = cb.q[tid & 15];
  issue(0, s0);
  issue(1, s0 + 1);
  if (tid < 16) sq[tid] = cbq;

  // the adapters, through the ring's free stage and the second tile
  const LoraShare L = lora_share(ma, p0, TM, M, sp, splits, 64);
  if (L.first < L.last) {
    const i32x4_t rS = rsrc_words(ma.S, M * ma.C * 2);
    for (int ls = L.first; ls < L.last; ++ls) {
      if (ls > L.first) open_stage<0>();  // (stage and tile are read)
      const int c = 64 * ls + 8 * ych, cc = std::min(c, L.all - 8), g = L.adapter_of(cc);
      const int lo = ma.start(L.gfirst + g) - p0, hi = std::min(ma.start(L.gfirst + g + 1), (int)M) - p0;
#pragma unroll
      for (int i = 0; i < YI; ++i) {
        const int row = 8 * (YI * wave + i) + (lane >> 3);
        const bool in = c < L.all && cc - g * L.each < ma.cols && row >= lo && row < hi;
        dma_lds16(rS, sy[2] + (YI * wave + i) * 1024,
                  in ? (uint32_t)(((p0 + row) * ma.C + cc - g * L.each) * 2) : 0x7fffffffu, 0u);
      }
      // tile rows 16w + 4i + (lane >> 4), physical chunk lane % 16
      int id[4], at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 64 * ls + 16 * wave + 4 * i + (lane >> 4), tc = std::min(t, L.all - 1), ga = L.adapter_of(tc);
        at[i] = t < L.all && tc - ga * L.each < ma.cols ? (tc - ga * L.each) % ma.r : -1;
        id[i] = ma.id(L.gfirst + ga);
      }
      u32x4_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * wave + 4 * i + (lane >> 4);
        const int64_t k = k0 + 8 * ((lane & 15) ^ ((row & 3) << 1));
        const bool ok = at[i] >= 0 && (unsigned)id[i] < (unsigned)ma.count && k < K;
        v[i] = *reinterpret_cast<const u32x4_t*>(ma.F + (ok ? ((int64_t)id[i] * ma.r + at[i]) * K + k : 0));
        if (!ok) v[i] = u32x4_t{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x4_t*>(sw[1] + (16 * wave + 4 * i) * 256 + 16 * lane) = v[i];
      open_stage<0>();
      multiply(sy[2], sw[1], [&](int ks, const u32x4_t* w, auto&& y) __attribute__((always_inline)) {
        const bool apart = any_not_finite<false>(w, 2);
        if (!apart) all_rows(ks, w, y);
        asm volatile("" ::: "memory");
        if (apart) {
          int lo, hi;
          L.rows(ma, 64 * ls + 32 * ks, p0, M, lo, hi);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            bool in[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) in[v] = 16 * i + 4 * kq + v >= lo && 16 * i + 4 * kq + v < hi;
#pragma unroll
            for (int f = 0; f < 2; ++f) mfma_rows<false, false>(y(i), w[f], acc[f][i], in);
          }
        }
      });
    }
  }

  if constexpr (std::is_same_v<Args, DenseGemmArgs>) {
    if (L.first < L.last && ma.drop.out > 0) {
      // lane l finds the masks of rows 16i + l/4, chunk l%4 of the wave's four; the
      // lane of row 16i + 4kq + v, column 16f + lr takes them from lane
      // 4·(4kq + v) + 2f + lr/8
      const DropView drop = drawn(ma.drop);
      const uint32_t c0 = (uint32_t)((p0 + (lane >> 2)) * (K / 8) + (k0 + 32 * wave) / 8 + (lane & 3));
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int keep = (int)keep8(drop, c0 + (uint32_t)(16 * i * (K / 8)));
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int m = __builtin_amdgcn_ds_bpermute(4 * (4 * (4 * kq + v) + 2 * f + (lr >> 3)), keep) >> (lr & 7);
            acc[f][i][v] = m & 1 ? acc[f][i][v] : 0.f;
          }
      }
    }
  }

  // stage s0 decoded; then per stage: its products, the next one's decode
  open_stage<PER>();  // (the levels are in LDS, and this wave's copies of stage s0)
  if (s0 < s1) decode(sc[0] + wave * 1536, sw[0], s0);
  int b = 0;
  for (int s = s0; s < s1; ++s) {
    const int b1 = b + 1 == D ? 0 : b + 1, b2 = b1 + 1 == D ? 0 : b1 + 1;
    // tile s is written, and every wave has waited for its copies of stage s
    open_stage<PER>();
    issue(b2, s + 2);
    multiply(sy[b], sw[(s - s0) & 1], all_rows);
    wait_vmem_le<PER>();  // this wave's copies of stage s + 1
    asm volatile("" ::: "memory");
    if (s + 1 < s1) decode(sc[b1] + wave * 1536, sw[(s + 1 - s0) & 1], s + 1);
    b = b1;
  }
  wait_vmem();  // no copy may land in LDS after the workgroup ends

#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const int64_t k = k0 + 32 * wave + 16 * f + lr;
    if (k >= K) continue;
    if (splits > 1) {
      float* const D0 = P + (int64_t)sp * M * K + k;
      rows.scatter(acc[f], [&](int tok, float v) { D0[(int64_t)tok * K] = v; });
    } else if (dx_bf16) {
      uint16_t* const D0 = static_cast<uint16_t*>(dX) + k;
      rows.scatter(acc[f], [&](int tok, float v) { D0[(int64_t)tok * K] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu); });
    } else {
      float* const D0 = static_cast<float*>(dX) + k;
      rows.scatter(acc[f], [&](int tok, float v) { D0[(int64_t)tok * K] = v; });
    }
  }
}

// Positions per workgroup, in tiles of 16.
int mid_tiles(int64_t M) { return M <= 32 ? 2 : 4; }

}  // namespace

// The split count with the least estimated time, in microseconds: rounds of
// `slots` workgroups at `stage` us a stage and `around` all of them, and the
// fp32 partials written and read at 4 TB/s.
MidPlan mid_splits(int64_t tiles, int64_t stages, int64_t elements, int64_t slots, double stage, double around) {
  MidPlan best{1, 8, 0.0};
  for (int64_t s = 1; s <= 16 && 2 * s <= std::max<int64_t>(stages, 2); ++s) {
    const double t = (double)((tiles * s + slots - 1) / slots) * ((double)((stages + s - 1) / s) * stage + around) +
                     (s > 1 ? (double)s * (double)elements * 8 / 4e6 : 0.0);
    if (s == 1 || t < best.us) best = MidPlan{(int)s, 8, t};
  }
  return best;
}
// One workgroup per compute unit (its LDS), 2.3 us a stage with 8 waves and 2.9
// with 16: 64 tokens, 4096 x 4096, 24 us in all with 8 and 27 with 16; 11008 x
// 4096, 41 and 36.
MidPlan mid_fwd_plan(int64_t M, int64_t N, int64_t K, int layers) {
  const int64_t tm = 16 * mid_tiles(M), mt = layers * ((M + tm - 1) / tm), stages = (K + 255) / 256;
  const MidPlan narrow = mid_splits(mt * ((N + 127) / 128), stages, layers * M * N, 256, 2.3, 7.7);
  MidPlan wide = mid_splits(mt * ((N + 255) / 256), stages, layers * M * N, 256, 2.9, 7.5);
  wide.waves = 16;
  return wide.us < narrow.us ? wide : narrow;
}
// Two workgroups per compute unit.
int mid_dx_splits(int64_t M, int64_t N, int64_t K, int layers) {
  const int64_t tm = 16 * mid_tiles(M), tiles = layers * ((M + tm - 1) / tm) * ((K + 127) / 128);
  return mid_splits(tiles, (N + 63) / 64, layers * M * K, 512, 1.0, 6.0).splits;
}

namespace {

template <typename Args>
hipError_t launch_fwd(const Nf4View& W, const uint16_t* X, int64_t M, const Args& ma, void* Y, bool y16,
                      const MidPlan& plan, float* P, int layers, hipStream_t st) {
  const int nt = mid_tiles(M), tm = 16 * nt, rows = 16 * plan.waves, tiles_n = (int)((W.N + rows - 1) / rows);
  const dim3 grid((unsigned)(tiles_n * ((M + tm - 1) / tm)), (unsigned)plan.splits, (unsigned)layers);
#define QNF4_MID(NT, WV)                                                                                              \
  mid_fwd_kernel<NT, WV, Args><<<grid, 64 * WV, 0, st>>>(W, X, M, Y, y16 ? 1 : 0, tiles_n, plan.splits, P, codebook(), \
                                                         ma)
  if (plan.waves == 16) {
    if (nt == 2)
      QNF4_MID(2, 16);
    else
      QNF4_MID(4, 16);
  } else {
    if (nt == 2)
      QNF4_MID(2, 8);
    else
      QNF4_MID(4, 8);
  }
#undef QNF4_MID
  return hipGetLastError();
}

template <typename Args>
hipError_t launch_dx(const Nf4View& W, const uint16_t* dY, int64_t M, const Args& ma, void* dX, bool dx16, int splits,
                     float* P, int layers, hipStream_t st) {
  const int nt = mid_tiles(M), tm = 16 * nt, tiles_k = (int)((W.K + 127) / 128);
  const dim3 grid((unsigned)(tiles_k * ((M + tm - 1) / tm)), (unsigned)splits, (unsigned)layers);
#define QNF4_MID(NT)                                                                                              \
  mid_dx_kernel<NT, Args><<<grid, kDxThreads, 0, st>>>(W, dY, M, dX, dx16 ? 1 : 0, tiles_k, splits, P, codebook(), ma)
  if (nt == 2)
    QNF4_MID(2);
  else
    QNF4_MID(4);
#undef QNF4_MID
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mid_fwd(const Nf4View& W, const uint16_t* X, int64_t M, const AdapterGemmArgs& ma, void* Y, bool y16,
                          const MidPlan& plan, float* P, hipStream_t st) {
  return launch_fwd(W, X, M, ma, Y, y16, plan, P, 1, st);
}
hipError_t launch_mid_fwd_block(const Nf4View& W, const uint16_t* X, int64_t M, const DenseGemmArgs& ma, void* Y, bool y16,
                                const MidPlan& plan, float* P, int layers, hipStream_t st) {
  return launch_fwd(W, X, M, ma, Y, y16, plan, P, layers, st);
}
hipError_t launch_mid_dx(const Nf4View& W, const uint16_t* dY, int64_t M, const AdapterGemmArgs& ma, void* dX, bool dx16,
                         int splits, float* P, hipStream_t st) {
  return launch_dx(W, dY, M, ma, dX, dx16, splits, P, 1, st);
}
hipError_t launch_mid_dx_block(const Nf4View& W, const uint16_t* dY, int64_t M, const DenseGemmArgs& ma, void* dX,
                               bool dx16, int splits, float* P, int layers, hipStream_t st) {
  return launch_dx(W, dY, M, ma, dX, dx16, splits, P, layers, st);
}

}  // namespace qnf4
