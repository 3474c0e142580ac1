// Forward product of the QLoRA linear layer for M > 16 tokens, gfx950:
//   Y[M, N] = X·Ŵᵀ + s·T·Bᵀ  =  [X | sT_hi | sT_lo] · [Ŵ | B | B]ᵀ
// (P1 §七 dataflow figure: the 4-bit base is dequantized to BF16 for the
// matmul and the LoRA path is added to the output.)
//
// Design
//   * One output tile per workgroup of 12 waves, three per SIMD, in two
//     roles; the tile is 256x256, or 512x128 from 2048 tokens on and from
//     512 on where it adds no padding rows (one kernel template, TMV = 256 or
//     512 token rows).  Waves 0..7 only
//     multiply: wave (wm, wn) owns token rows [128wm, +128) and weight rows
//     [64wn, +64) of the tile (2 x 4 waves, or 4 x 2), 64
//     v_mfma_f32_16x16x32_bf16 per 64-wide reduction step, operands read
//     from LDS one MFMA group ahead.  Waves 8..11 (one per SIMD) produce the
//     operands of the next step: each copies a quarter of the X tile
//     straight into LDS and dequantizes a quarter of the tile's weight rows
//     into the shared bf16 tile Ŵ[n][k].  Their arithmetic and copies
//     overlap the MFMAs of the other two waves of their SIMD.
//   * The 512x128 tile decodes each weight row of a step once for 512
//     tokens: half the producers' decode per MFMA for twice their X copy
//     (64 KB of X and 16 KB of Ŵ per step, 160 KB of LDS with both
//     buffers).  On the 7B MLP shapes it takes the forward GEMM from ≈322 to
//     ≈310 µs (bit-identical output), at 1,024–1,536 tokens by 4-6 % (with
//     or without a split reduction).
//   * Dequantization in registers: producer p owns tile rows
//     [WR p, +WR) (WR = 64 or 32): lane l takes row WR p + l % WR and, when
//     two lanes share a row, half l / WR of its 64 codes.  Per step a lane
//     builds its row's table of the 16 values RNE_bf16(fl32(q_j * c')) of
//     the step's block (bit-identical to multiplying per element, since the
//     value depends only on code and row), held as four byte planes (low
//     bytes of values 0-3, 4-7, 8-11, 12-15, likewise the high bytes), and
//     decodes its codes with byte permutes: four codes per permute pair,
//     the code's low three bits selecting within 8 bytes and its top bit
//     between the two halves; the low and high bytes are then interleaved
//     into bf16 pairs and the row's 16-byte chunks stored.  No LDS lookups,
//     no tables in LDS.
//   * Each producer step first waits for the codes and constants it loaded a
//     step earlier, then issues the X copy of the next step, then the loads
//     of the step after (into the other of two register sets, so that no
//     register a load in flight writes is copied), then decodes; at its end
//     only the X copy must be complete.  (The X copy is the long-latency
//     transfer; issued first it has the whole step to land.)
//   * Tiles are stored with 16-byte chunks XOR-swizzled by row (xswz) so that
//     MFMA operand reads of 8 rows cover the 32 LDS banks once.
//   * One barrier per step: after it the MFMA waves use X(s) and Ŵ(s) while
//     the producers fill the other buffers with X(s+1) and Ŵ(s+1).
//   * All operand reads are buffer loads whose resources end at the tensor's
//     last row, so ragged tiles read zeros without per-lane branches.
//   * The LoRA up-projection is 2*Rp/64 extra reduction steps whose A operand
//     is the bf16 hi/lo split of s·T and whose B operand is the padded copy
//     B2 = [B | 0 | B | 0] ([N, 2Rp] bf16), both copied straight into LDS.
//   * Workgroups are mapped to tiles so that each XCD (workgroup id mod 8)
//     walks a contiguous run of a grouped tile order (4 M-tiles per group):
//     the ~32 workgroups resident on one XCD share X and code rows in its L2.
//   * With few tokens the tiles alone leave most compute units idle; then
//     the K steps are split over `splits` workgroups per tile (the last
//     split also takes the LoRA steps), each writing its fp32 partial tile
//     to P[split][M][N], summed in split order by splitk_reduce_kernel.
#include <algorithm>
#include <type_traits>

#include "gate.h"
#include "host.h"
#include "modes.h"
#include "tiling.h"

namespace qnf4 {
namespace {

constexpr int TM = 256, TN = 256, KSTEP = 64;  // the square tile (split plans)
constexpr int kMfmaWaves = 8, kProdWaves = 4, kWaves = kMfmaWaves + kProdWaves;
constexpr int kThreads = 64 * kWaves;
// 512 x 128 tiles from 2048 tokens on, and from 512 tokens on where they
// add no padding rows over 256-row tiles
constexpr int64_t kTallMinTokens = 512, kTallAlwaysTokens = 2048;
inline bool fwd_tall(int64_t M) {
  return M >= kTallAlwaysTokens || (M >= kTallMinTokens && ((M + 255) / 256) % 2 == 0);
}

// A tile row = 64 bf16 = eight 16-byte chunks; chunk c of row r is stored at
// physical chunk c ^ sw(r & 7), where sw swaps bits 0 and 1 of its argument.
// An MFMA operand read gives the 64 lanes 16 consecutive rows at 4 chunks;
// with this permutation the gfx950 LDS serves it at its full 16-byte read
// rate (measured: 4 clocks per wave instruction), where the plain c ^ (r & 7)
// takes twice as long.  The write paths are indifferent to the choice.
__device__ __forceinline__ int rsw(int row) { return ((row >> 1) & 1) | ((row & 1) << 1) | (row & 4); }
__device__ __forceinline__ int xswz(int row, int chunk) {
  return row * 128 + ((chunk ^ rsw(row & 7)) << 4);
}

// TMV x (65536 / TMV) output tiles: 256 x 256, or 512 x 128 (the weight
// rows of a step decoded once for twice the tokens: half the producers'
// decode per MFMA, twice their X copy).
// MULTI: the tokens carry different adapters (AdapterGemmArgs): tile rows are
// sorted positions, X rows are gathered and output rows scattered through
// the plan, and the LoRA steps run over the used adapters whose tokens the
// tile holds, cols/64 steps each, rounded up (rows of other adapters read as
// zero; the split reductions share these steps out as they do the K steps).
// BLOCK: one layer (kBlock1) or the two of a gated block (kBlock2) whose low-rank
// factors come as three-part splits (BlockGemmArgs).  Of two layers a tile holds
// as many weight rows of each, the gate's first: an MFMA wave's 64 columns are 32
// of each layer's, the same ones, so that a lane holds both factors of the outputs
// it writes; a LoRA step belongs to one layer and adds to its half.
// (4096 tokens, two of 11008 x 4096, r = 64: 662 us with H alone, 683 with G and U
// too, 1.1 PFLOP/s, where two plain layers take 645; with dropout 694 in all.)
template <int LSTEPS, bool F16, int TMV, int MODE = kPlain>
__global__ __launch_bounds__(kThreads, 1) void fwd_gemm_kernel(Nf4View W, const uint16_t* __restrict__ X,
                                                               int64_t M, const uint16_t* __restrict__ sT,
                                                               const uint16_t* __restrict__ B2,
                                                               int64_t Rp, void* __restrict__ Y,
                                                               int y_bf16, int tiles_m, int tiles_n,
                                                               int splits, float* __restrict__ P,
                                                               Codebook cb,
                                                               ModeArgs<MODE> ma) {
  constexpr bool MULTI = MODE == kMulti, BLOCK = MODE >= kBlock1, PAIR = MODE == kBlock2;
  constexpr int TM = TMV, TN = 65536 / TMV;
  constexpr int LAYERS = PAIR ? 2 : 1;
  constexpr int WGN = TN / 64;           // MFMA waves along N (4 or 2), each 128 x 64
  constexpr int XR = TM / kProdWaves;    // X rows copied per producer and step (64 or 128)
  constexpr int WR = TN / kProdWaves;    // weight rows decoded per producer (64 or 32)
  constexpr int HALVES = 64 / WR;        // lanes per weight row (1 or 2)
  constexpr int NLOADS = 2 / HALVES + 2;  // vector loads per producer step (codes, e byte, scale)
  __shared__ __attribute__((aligned(16))) char sx0[TM * 128], sx1[TM * 128];  // A tiles: X, then sT
  __shared__ __attribute__((aligned(16))) char sw[2][TN * 128];  // B tiles: Ŵ, then B2
  int tmi, tni, sp;
  if (!tile_of<TMV == 512 ? 2 : kGroupM>(blockIdx.x, tiles_m, tiles_n, splits, tmi, tni, sp)) return;

  // (the wave index in a scalar register: the LDS addresses and offsets of
  // the copies derived from it are then formed by scalar instructions)
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t K = W.K, N = W.N;
  const int64_t m0 = (int64_t)tmi * TM, n0 = (int64_t)tni * (TN / LAYERS);
  // this workgroup's K steps [kfirst, kfirst + ksteps) (step indices below
  // are relative to kfirst) and its LoRA steps
  const int kall = (int)(K / KSTEP);
  const int kfirst = split_first(sp, splits, kall);
  const int ksteps = split_first(sp + 1, splits, kall) - kfirst;
  int lsteps = sp == splits - 1 ? LSTEPS : 0;
  // MULTI: this workgroup's LoRA steps [lfirst, lfirst + lsteps) of the
  // tile's; step i belongs to used adapter gfirst + i / lper, chunk i % lper
  int lfirst = 0, gfirst = 0, lper = 1;
  if constexpr (MULTI) {
    const int held = std::min(ma.held(), (int)M);
    lper = (ma.cols + 63) / 64;
    if ((int)m0 < held) {
      gfirst = ma.group((int)m0);
      const int glast = std::min(ma.group(std::min((int)m0 + TM, held) - 1), ma.count - 1);
      const int all = gfirst >= 0 && glast >= gfirst ? std::min(glast - gfirst + 1, TM) * lper : 0;
      lfirst = split_first(sp, splits, all);
      lsteps = split_first(sp + 1, splits, all) - lfirst;
    }
  }
  // BLOCK: this workgroup's LoRA steps of the layers', lper each
  if constexpr (BLOCK) {
    lper = (ma.cols + 63) / 64;
    lfirst = split_first(sp, splits, LAYERS * lper);
    lsteps = split_first(sp + 1, splits, LAYERS * lper) - lfirst;
  }
  // the sorted positions [p0, p1) of LoRA step l's adapter, relative to m0
  auto rows_of = [&](int l, int& p0, int& p1) __attribute__((always_inline)) {
    if constexpr (MULTI) {
      const int g = gfirst + (lfirst + l) / lper;
      p0 = ma.start(g) - (int)m0;
      p1 = std::min(ma.start(g + 1), (int)M) - (int)m0;
    }
  };
  auto sxb = [&](int i) { return i ? sx1 : sx0; };

  // Resources start at this tile's first row and end at the tensor's last
  // row: rows past M or N read as zero.  (Rows past M only feed output rows
  // past M, rows past N only output columns past N; neither is stored.)
  // Reads of weight data one or two steps past the last step stay inside
  // these buffers or return zeros; their results are never used.
  // (PAIR: producers 2 and 3 decode the second layer's rows)
  const bool second = PAIR && wave >= kMfmaWaves + 2;
  const rsrc_t rc = make_rsrc(layer(W, ma, second).codes + n0 * (K / 2), (N - n0) * (K / 2));

  auto no_issue = [](int) {};

  if (wave < kMfmaWaves) {
    // ---------------------------------------------------------------- MFMA
    const int lr = lane & 15, kq = lane >> 4;
    const int wm = wave / WGN, wn = wave % WGN;
    f32x4_t acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // MFMA group g (0..15) of a step: k-half ks = g / 8, token block i = g % 8.
    // A fragments are read one group ahead: group g first reads the A
    // fragment of group g + 1, so the read's latency overlaps this group's
    // MFMAs.  At a step's start the A fragment of group 0 is requested before
    // the four B fragments, so that its first MFMA waits for two reads, not
    // five (LDS reads return in order; about 1% on the step).  The B
    // fragments of the second k-half are read right after the MFMAs of
    // group 7.
    const int arow = 128 * wm + lr, brow = 64 / LAYERS * wn + lr;
    // tile row of column block j (PAIR: blocks 0, 1 are the gate's, 2, 3 the other layer's)
    auto block_row = [&](int j) __attribute__((always_inline)) {
      return PAIR ? brow + 16 * (j & 1) + TN / 2 * (j >> 1) : brow + 16 * j;
    };
    u32x4_t bfr[4], anext;
    auto read_b = [&](const char* wb, int ks, u32x4_t* b) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[j] = *reinterpret_cast<const u32x4_t*>(wb + xswz(block_row(j), 2 * kq + ks));
    };
    auto read_a = [&](const char* xa, int g) __attribute__((always_inline)) {
      return *reinterpret_cast<const u32x4_t*>(xa + xswz(arow + 16 * (g & 7), 2 * kq + (g >> 3)));
    };
    auto mfma_step = [&](const char* xa, const char* wb) __attribute__((always_inline)) {
      anext = read_a(xa, 0);
      read_b(wb, 0, bfr);
#pragma unroll
      for (int g = 0; g < 16; ++g) {
        const int i = g & 7;
        const u32x4_t a = anext;
        if (g < 15) anext = read_a(xa, g + 1);
        // keep the reads ahead of the MFMAs (the scheduler would sink them
        // below to reuse the fragment's registers)
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma16<F16>(a, bfr[j], acc[i][j]);
        if (g == 7) read_b(wb, 1, bfr);
      }
    };
    // MULTI, a LoRA step of an adapter that has some of the wave's rows: those of
    // other adapters read as zero, but zero times an infinity or NaN is NaN.  A
    // B tile that holds one goes through lora_step_rows, where rows [lo, hi)
    // alone take the sums (8 matrix instructions against 64 to find out: 362 us
    // for 4096 tokens of 8 requests, r = 64, 11008 x 4096, against 382 always
    // adding by rows and 357 with neither).
    using LdsTile = const __attribute__((address_space(3))) char*;
    auto read_tile = [&](LdsTile t, int row, int ks) __attribute__((always_inline)) {
      return *(const __attribute__((address_space(3))) u32x4_t*)(t + xswz(row, 2 * kq + ks));
    };
    auto not_finite = [&](LdsTile wb) __attribute__((always_inline)) {
      bool bad = false;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int j = 0; j < 4; ++j) bfr[j] = read_tile(wb, brow + 16 * j, ks);
        bad |= any_not_finite<F16>(bfr, 4);
      }
      return bad;
    };
    auto lora_step_rows = [&](LdsTile xa, LdsTile wb, int lo, int hi) __attribute__((always_inline)) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int j = 0; j < 4; ++j) bfr[j] = read_tile(wb, brow + 16 * j, ks);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          bool in[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) in[v] = 16 * i + 4 * kq + v >= lo && 16 * i + 4 * kq + v < hi;
          const u32x4_t a = read_tile(xa, arow + 16 * i, ks);
#pragma unroll
          for (int j = 0; j < 4; ++j) mfma_rows<F16, true>(a, bfr[j], acc[i][j], in);
        }
      }
    };

    // PAIR, a LoRA step of layer q: its two column blocks alone
    auto lora_step_half = [&](auto q, const char* xa, const char* wb) __attribute__((always_inline)) {
      constexpr int J0 = 2 * decltype(q)::value;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4_t b[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          b[j] = *reinterpret_cast<const u32x4_t*>(wb + xswz(block_row(J0 + j), 2 * kq + ks));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const u32x4_t a = read_a(xa, 8 * ks + i);
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][J0 + j] = mfma16<F16>(a, b[j], acc[i][J0 + j]);
        }
      }
    };

    __syncthreads();  // (the producers' prologue)
    __syncthreads();  // step 0 in place
#pragma unroll 1
    for (int s = 0; s + 1 < ksteps; ++s) {
      mfma_step(sxb(s & 1), sw[s & 1]);
      __syncthreads();
    }
    if constexpr (PAIR) {
      mfma_step(sxb((ksteps - 1) & 1), sw[(ksteps - 1) & 1]);
      __syncthreads();
#pragma unroll 1
      for (int l = 0; l < lsteps; ++l) {
        const int s = ksteps + l;
        const bool up = lfirst + l >= lper;
        if (!up) lora_step_half(std::integral_constant<int, 0>(), sxb(s & 1), sw[s & 1]);
        asm volatile("" ::: "memory");  // (two branches, not one of two arms, whose sums would not stay in place)
        if (up) lora_step_half(std::integral_constant<int, 1>(), sxb(s & 1), sw[s & 1]);
        __syncthreads();
      }
    } else if constexpr (!MULTI) {
#pragma unroll 1
      for (int s = ksteps - 1; s < ksteps + lsteps; ++s) {
        mfma_step(sxb(s & 1), sw[s & 1]);
        __syncthreads();
      }
    } else {
      mfma_step(sxb((ksteps - 1) & 1), sw[(ksteps - 1) & 1]);
      __syncthreads();
#pragma unroll 1
      for (int l = 0; l < lsteps; ++l) {
        const int s = ksteps + l;
        int p0, p1;
        rows_of(l, p0, p1);  // (waves whose rows hold none of the adapter's tokens skip its steps)
        p0 = __builtin_amdgcn_readfirstlane(p0);
        p1 = __builtin_amdgcn_readfirstlane(p1);
        const bool some = p0 < 128 * wm + 128 && p1 > 128 * wm, whole = p0 <= 128 * wm && p1 >= 128 * wm + 128;
        const bool apart = some && !whole && not_finite((LdsTile)sw[0] + (s & 1) * sizeof(sw[0]));
        if (some && !apart) mfma_step(sxb(s & 1), sw[s & 1]);
        asm volatile("" ::: "memory");  // (two branches, not one of two arms, whose sums would not stay in place)
        if (apart) {
          const LdsTile xa = s & 1 ? (LdsTile)sx1 : (LdsTile)sx0;
          lora_step_rows(xa, (LdsTile)sw[0] + (s & 1) * sizeof(sw[0]), p0 - 128 * wm, p1 - 128 * wm);
        }
        __syncthreads();
      }
    }

    // epilogue: lane holds rows 128wm + 16i + 4kq + v of column 64wn + 16j + lr.
    // The row/column bases go through an empty asm so that their address
    // arithmetic is not hoisted above the main loop (it would stay live there).
    int row0 = 128 * wm + 4 * kq, col0 = 64 / LAYERS * wn + lr;
    asm volatile("" : "+v"(row0), "+v"(col0));
    const bool full = (m0 + TM <= M) && (n0 + TN / LAYERS <= N);
    if constexpr (PAIR) {
      if (splits > 1) {
        // rows of a split's partials: the gate's N columns, then the other layer's
        float* Pp = P + ((int64_t)sp * M + m0 + row0) * 2 * N + n0 + col0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int64_t m = m0 + row0 + 16 * i + v, n = n0 + col0 + 16 * (j & 1);
              if (full || (m < M && n < N)) Pp[(16 * i + v) * 2 * N + (j >> 1) * N + 16 * (j & 1)] = acc[i][j][v];
            }
      } else {
        uint16_t* const H = static_cast<uint16_t*>(Y);
        const int64_t at0 = (m0 + row0) * N + n0 + col0;
        const bool save = ma.G != nullptr;
        // the wave's gate that is furthest below zero, as a number whose order is that of
        // negative floats' sizes
        uint32_t most = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int64_t m = m0 + row0 + 16 * i + v, n = n0 + col0 + 16 * j;
              if (!full && (m >= M || n >= N)) continue;
              const int64_t at = at0 + (int64_t)(16 * i + v) * N + 16 * j;
              const float g = acc[i][j][v], u = acc[i][j + 2][v];
              most = std::max(most, __float_as_uint(g));
              H[at] = (uint16_t)(pack16<F16>(gate_act<false>(ma.act, g) * u, 0.0f) & 0xffffu);
              if (save) {
                const uint32_t gu = pack16<F16>(g, u);
                ma.G[at] = (uint16_t)(gu & 0xffffu);
                ma.U[at] = (uint16_t)(gu >> 16);
              }
            }
        // (once more where it has to be, not a branch for each output: 700 us for 4096
        // tokens of 11008 x 4096, not 689)
        if (__builtin_amdgcn_ballot_w64(most > __float_as_uint(far_gate(ma.act))) != 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int64_t m = m0 + row0 + 16 * i + v, n = n0 + col0 + 16 * j;
                const float g = acc[i][j][v], u = acc[i][j + 2][v];
                if (m < M && n < N && g < far_gate(ma.act))
                  H[at0 + (int64_t)(16 * i + v) * N + 16 * j] =
                      (uint16_t)(pack16<F16>(gate_act(ma.act, g) * u, 0.0f) & 0xffffu);
              }
        }
      }
    } else if constexpr (MULTI) {
      // rows back to their tokens, as buffer stores: a row or column past the
      // output's end gets an offset past the buffer's (no branches; the 16-bit
      // output and the partials of a split are below 2^31 bytes)
      auto scatter = [&](auto size, auto&& put) __attribute__((always_inline)) {
        constexpr uint32_t SZ = decltype(size)::value;
        const bool whole = n0 + TN <= N;
        const uint32_t colb = ((uint32_t)n0 + (uint32_t)col0) * SZ;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int pos = (int)m0 + row0 + 16 * i;
          const int4 tok = *reinterpret_cast<const int4*>(ma.perm() + std::min(pos, ((int)M - 1) & ~3));
          const int t4[4] = {tok.x, tok.y, tok.z, tok.w};
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const bool row_ok = pos + v < (int)M && (uint32_t)t4[v] < (uint32_t)M;
            const uint32_t o = row_ok ? (uint32_t)t4[v] * (uint32_t)N * SZ : 0x80000000u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t at = o + colb + 16 * SZ * j;
              if (!whole) at = n0 + col0 + 16 * j < N ? at : 0xffffffffu;
              put(at, acc[i][j][v]);
            }
          }
        }
      };
      if (splits > 1) {
        const rsrc_t rp = make_rsrc(P + (int64_t)sp * M * N, M * N * 4);
        scatter(std::integral_constant<uint32_t, 4>(),
                [&](uint32_t at, float v) { __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rp, at, 0, 0); });
      } else if (y_bf16) {
        const rsrc_t ry = make_rsrc(Y, M * N * 2);
        scatter(std::integral_constant<uint32_t, 2>(), [&](uint32_t at, float v) {
          __builtin_amdgcn_raw_buffer_store_b16((short)(pack16<F16>(v, 0.0f) & 0xffffu), ry, at, 0, 0);
        });
      } else {
        // (64-bit addresses: an fp32 output goes past the 2^31 bytes that a buffer's
        // offsets reach.  One load of the plan a row, in a rolled loop.  4096 tokens without adapters, 11008 x 4096: 334 us
        // against 308 for a bf16 output; the one-adapter path's fp32 output costs
        // 4 us more than its bf16 one)
        float* const D = static_cast<float*>(Y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int pos = (int)m0 + row0 + 16 * i;
#pragma unroll 1
          for (int v = 0; v < 4; ++v) {
            const int tok = pos + v < (int)M ? ma.perm()[pos + v] : -1;
            if ((uint32_t)tok >= (uint32_t)M) continue;
            float* const Dr = D + (int64_t)tok * N + n0 + col0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (n0 + col0 + 16 * j < N) Dr[16 * j] = v == 0 ? acc[i][j][0] : v == 1 ? acc[i][j][1] : v == 2 ? acc[i][j][2] : acc[i][j][3];
          }
        }
      }
    } else if (splits > 1) {
      float* Pp = P + ((int64_t)sp * M + m0 + row0) * N + n0 + col0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + row0 + 16 * i + v, n = n0 + col0 + 16 * j;
            if (full || (m < M && n < N)) Pp[(16 * i + v) * N + 16 * j] = acc[i][j][v];
          }
    } else if (y_bf16) {
      uint16_t* Yb = static_cast<uint16_t*>(Y) + (m0 + row0) * N + n0 + col0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + row0 + 16 * i + v, n = n0 + col0 + 16 * j;
            if (full || (m < M && n < N))
              Yb[(16 * i + v) * N + 16 * j] = (uint16_t)(pack16<F16>(acc[i][j][v], 0.0f) & 0xffffu);
          }
    } else {
      float* Yf = static_cast<float*>(Y) + (m0 + row0) * N + n0 + col0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + row0 + 16 * i + v, n = n0 + col0 + 16 * j;
            if (full || (m < M && n < N)) Yf[(16 * i + v) * N + 16 * j] = acc[i][j][v];
          }
    }
    return;
  }

  // ------------------------------------------------------------ producers
  // Producer p dequantizes weight rows [WR p, +WR) and copies X rows
  // [XR p, +XR) of every step (WR = XR = 64 on the square tile; WR = 32,
  // XR = 128 on the tall one).
  const int p = wave - kMfmaWaves;
  const uint32_t kpr = (uint32_t)(K / kBlock);  // blocks per weight row
  const float mu = *layer(W, ma, second).mu;
  const rsrc_t rt = make_rsrc(sT + m0 * 2 * Rp, (M - m0) * 2 * Rp * 2);
  const rsrc_t re = make_rsrc(layer(W, ma, second).e + n0 * kpr, (N - n0) * kpr);
  const rsrc_t rs = make_rsrc(layer(W, ma, second).s, ((N * kpr + kDqBlock - 1) / kDqBlock) * 4);
  const rsrc_t rb = make_rsrc(B2 + n0 * 2 * Rp, (N - n0) * 2 * Rp * 2);

  // X rows [XR p, +XR) of a step, copied straight into LDS: part c
  // moves rows XR p + 8c + (l >> 3), lane l into physical chunk l & 7, so it
  // fetches logical chunk (l & 7) ^ sw(l >> 3) (row & 7 = l >> 3).  Each
  // instruction fills 1 KB of LDS contiguously.  (Written as assembly: the
  // compiler then inserts no wait for these copies in front of the
  // producer's own LDS reads; the wait before the step's closing barrier is
  // explicit.)
  const int xlch = (lane & 7) ^ rsw(lane >> 3);
  const uint32_t vx = (uint32_t)(((XR * p + (lane >> 3)) * K + 8 * xlch) * 2);
  const uint32_t x_gstride = (uint32_t)(8 * K * 2);
  const i32x4_t rxw = MULTI ? rsrc_words(X, M * K * 2) : rsrc_words(X + m0 * K, (M - m0) * K * 2);
  // MULTI: the byte offset of each row's token (past every buffer for none)
  uint32_t vtok[MULTI ? XR / 8 : 1];
  if constexpr (MULTI) {
    // (unconditional loads, all in flight together)
    int tok[XR / 8];
#pragma unroll
    for (int c = 0; c < XR / 8; ++c)
      tok[c] = ma.perm()[std::min((int)m0 + XR * p + 8 * c + (lane >> 3), (int)M - 1)];
#pragma unroll
    for (int c = 0; c < XR / 8; ++c) {
      const bool ok = (int)m0 + XR * p + 8 * c + (lane >> 3) < (int)M && (uint32_t)tok[c] < (uint32_t)M;
      vtok[c] = ok ? ((uint32_t)tok[c] * (uint32_t)K + 8 * xlch) * 2u : 0x7fffffffu;
    }
  }
  auto copy_x_part = [&](char* t, int s, int c) __attribute__((always_inline)) {
    dma_lds16(rxw, t + (XR * p + 8 * c) * 128, MULTI ? vtok[c] : vx + c * x_gstride, (uint32_t)(kfirst + s) * 128u);
  };
  auto copy_x = [&](char* t, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < XR / 8; ++c) copy_x_part(t, s, c);
  };
  // LoRA tiles (sT rows, B2 rows), the same pattern over rows of 2Rp bf16.
  const uint32_t l_gstride = (uint32_t)(8 * 2 * Rp * 2);
  auto copy_lora = [&](rsrc_t r, char* t, int l, auto rows) __attribute__((always_inline)) {
    constexpr int RR = decltype(rows)::value;  // rows per producer
    const uint32_t vl = (uint32_t)(((RR * p + (lane >> 3)) * 2 * Rp + 8 * xlch) * 2);
#pragma unroll
    for (int c = 0; c < RR / 8; ++c)
      buf_load_lds16(r, t + (RR * p + 8 * c) * 128, vl, c * l_gstride + (uint32_t)l * 128u);
  };
  // MULTI: the LoRA step's tiles straight from S and the adapter's factor, each
  // 16-byte chunk from column (64l + 8 chunk) mod r of its part; rows of other
  // adapters, columns past `cols` and rows past N read as zero
  auto copy_multi = [&](char* ts, char* tf, int l) __attribute__((always_inline)) {
    if constexpr (MULTI) {
      const int i = lfirst + l, g = gfirst + i / lper, col = 64 * (i % lper) + 8 * xlch;
      const bool in = col < ma.cols;
      int p0, p1;
      rows_of(l, p0, p1);
      const rsrc_t rt3 = make_rsrc(ma.S, M * ma.C * 2);
#pragma unroll
      for (int c = 0; c < XR / 8; ++c) {
        const int row = XR * p + 8 * c + (lane >> 3);
        const uint32_t o = (uint32_t)(((m0 + row) * ma.C + col) * 2);
        buf_load_lds16(rt3, ts + (XR * p + 8 * c) * 128, in && row >= p0 && row < p1 ? o : 0x7fffffffu, 0u);
      }
      const int a = ma.id(g);
      const bool ok = (unsigned)a < (unsigned)ma.count;
      const rsrc_t rf = make_rsrc(ma.F + (int64_t)(ok ? a : 0) * N * ma.r, ok ? N * ma.r * 2 : 0);
#pragma unroll
      for (int c = 0; c < WR / 8; ++c) {
        const int row = WR * p + 8 * c + (lane >> 3);
        buf_load_lds16(rf, tf + (WR * p + 8 * c) * 128,
                       in ? (uint32_t)(((n0 + row) * ma.r + col % ma.r) * 2) : 0x7fffffffu, 0u);
      }
    }
  };
  // BLOCK: the same for one layer's S and factor; of two layers the producers of
  // the other one's rows copy S alone
  auto copy_block = [&](char* ts, char* tf, int l) __attribute__((always_inline)) {
    if constexpr (BLOCK) {
      const int i = lfirst + l, q = PAIR && i >= lper ? 1 : 0, col = 64 * (i - q * lper) + 8 * xlch;
      const bool in = col < ma.cols;
      const rsrc_t rS = make_rsrc(ma.S + (int64_t)q * M * ma.C, M * ma.C * 2);
#pragma unroll
      for (int c = 0; c < XR / 8; ++c) {
        const int row = XR * p + 8 * c + (lane >> 3);
        buf_load_lds16(rS, ts + (XR * p + 8 * c) * 128, in ? (uint32_t)(((m0 + row) * ma.C + col) * 2) : 0x7fffffffu, 0u);
      }
      if (PAIR && q != (p >> 1)) return;
      const rsrc_t rf = make_rsrc(ma.F[q], N * ma.r * 2);
#pragma unroll
      for (int c = 0; c < WR / 8; ++c) {
        const int row = (PAIR ? WR * (p & 1) : WR * p) + 8 * c + (lane >> 3);
        buf_load_lds16(rf, tf + (WR * p + 8 * c) * 128,
                       in ? (uint32_t)(((n0 + row) * ma.r + col % ma.r) * 2) : 0x7fffffffu, 0u);
      }
    }
  };
  using XRows = std::integral_constant<int, XR>;
  using WRows = std::integral_constant<int, WR>;

  // Row trow = WR p + lane % WR of the tile is this lane's: the dword
  // holding its e4m3 byte and its group scale, and per step its 32 bytes of
  // codes (the 16 of half lane / WR when two lanes share the row).
  const int trow = WR * p + lane % WR, half = lane / WR;
  const int nrow = PAIR ? WR * (p & 1) + lane % WR : trow;  // from the layer's row n0 on
  const uint32_t ve_me = (uint32_t)nrow * kpr;
  const uint32_t blk_me = (uint32_t)(n0 + nrow) * kpr;
  struct Consts {
    uint32_t e, s;
  };
  auto load_consts = [&](Consts& r, int t) __attribute__((always_inline)) {
    r.e = buf_load4(re, (ve_me + (uint32_t)(kfirst + t)) & ~3u, 0u);
    r.s = buf_load4(rs, ((blk_me + (uint32_t)(kfirst + t)) / kDqBlock) * 4u, 0u);
  };
  const uint32_t vrow = (uint32_t)nrow * (uint32_t)(K / 2);
  auto load_row = [&](u32x4_t* c, int t) __attribute__((always_inline)) {
    if constexpr (HALVES == 1) {
      c[0] = buf_load16(rc, vrow, (uint32_t)(kfirst + t) * 32u);
      c[1] = buf_load16(rc, vrow, (uint32_t)(kfirst + t) * 32u + 16u);
    } else {
      c[0] = buf_load16(rc, vrow + 16u * (uint32_t)half, (uint32_t)(kfirst + t) * 32u);
    }
  };
  auto row_table = [&](int t, const Consts& r, uint32_t* L, uint32_t* H) __attribute__((always_inline)) {
    const uint32_t e = (r.e >> (8 * ((ve_me + (uint32_t)(kfirst + t)) & 3u))) & 0xffu;
    const float cp = decode_constant(e, __uint_as_float(r.s), mu);
    uint32_t d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = pack16<F16>(__fmul_rn(cb.q[2 * j], cp), __fmul_rn(cb.q[2 * j + 1], cp));
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      L[g] = __builtin_amdgcn_perm(d[2 * g + 1], d[2 * g], 0x06040200u);
      H[g] = __builtin_amdgcn_perm(d[2 * g + 1], d[2 * g], 0x07050301u);
    }
  };
  // T: a byte plane; the bytes of c are four codes (0..15)
  auto look = [&](uint32_t c, const uint32_t* T) __attribute__((always_inline)) {
    const uint32_t s7 = c & 0x07070707u;
    const uint32_t sel = ((c >> 1) & 0x04040404u) | 0x03020100u;
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(T[3], T[2], s7), __builtin_amdgcn_perm(T[1], T[0], s7), sel);
  };
  // eight codes (one dword: element 2b in the low nibble of byte b, 2b+1 in
  // its high nibble) into four bf16 pairs in element order
  auto decode8 = [&](uint32_t w, const uint32_t* L, const uint32_t* H, u32x4_t& o) __attribute__((always_inline)) {
    const uint32_t ev = w & 0x0F0F0F0Fu, od = (w >> 4) & 0x0F0F0F0Fu;
    const uint32_t le = look(ev, L), he = look(ev, H), lo = look(od, L), ho = look(od, H);
    const uint32_t E01 = __builtin_amdgcn_perm(he, le, 0x05010400u), E23 = __builtin_amdgcn_perm(he, le, 0x07030602u);
    const uint32_t O01 = __builtin_amdgcn_perm(ho, lo, 0x05010400u), O23 = __builtin_amdgcn_perm(ho, lo, 0x07030602u);
    o[0] = __builtin_amdgcn_perm(O01, E01, 0x05040100u);
    o[1] = __builtin_amdgcn_perm(O01, E01, 0x07060302u);
    o[2] = __builtin_amdgcn_perm(O23, E23, 0x05040100u);
    o[3] = __builtin_amdgcn_perm(O23, E23, 0x07060302u);
  };
  auto decode_row = [&](const u32x4_t* c, const uint32_t* L, const uint32_t* H, char* dst, auto&& issue)
      __attribute__((always_inline)) {
#pragma unroll
    for (int jj = 0; jj < 8 / HALVES; ++jj) {
      const int j = HALVES == 1 ? jj : 4 * half + jj;  // chunk of the row
      u32x4_t o;
      decode8(c[jj >> 2][jj & 3], L, H, o);
      *reinterpret_cast<u32x4_t*>(dst + xswz(trow, j)) = o;
      issue(jj);
    }
  };

  u32x4_t cw[2], cwn[2];
  Consts cc, cn;
  // prologue: X of step 0, codes and constants of steps 0 and 1, step 0 decoded
  {
    Consts c0;
    u32x4_t k0[2];
    copy_x(sx0, 0);
    load_consts(c0, 0);
    load_consts(cc, 1);
    load_row(k0, 0);
    load_row(cw, 1);
    uint32_t L[4], H[4];
    row_table(0, c0, L, H);
    decode_row(k0, L, H, sw[0], no_issue);
  }
  __syncthreads();
  wait_vmem();
  __syncthreads();  // step 0 in place

  // Weight steps 0 .. ksteps-2, one step: the table of step s+1 from constants loaded a step earlier
  // (their first use, where the compiler waits for them), then the X copy of
  // step s+1 and the loads of step s+2 (into the other register set: no
  // copies of registers that loads in flight are writing), then the decode;
  // at the end the X copy must be done while the 4 loads of step s+2 may
  // still be in flight.
  auto pstep = [&](int s, const u32x4_t* cur, u32x4_t* nxt, const Consts& ccur, Consts& cnxt)
      __attribute__((always_inline)) {
    uint32_t L[4], H[4];
    row_table(s + 1, ccur, L, H);
    // the table and this step's codes exist before the copies are issued
    // (the compiler's waits for them would otherwise also wait for copies
    // issued before them, which it does not track)
    asm volatile("" : "+v"(L[0]), "+v"(L[1]), "+v"(L[2]), "+v"(L[3]), "+v"(H[0]), "+v"(H[1]), "+v"(H[2]),
                 "+v"(H[3]) : "v"(cur[0]), "v"(cur[HALVES == 1 ? 1 : 0]));
    copy_x(sxb((s + 1) & 1), s + 1);
    load_row(nxt, s + 2);
    load_consts(cnxt, s + 2);
    decode_row(cur, L, H, sw[(s + 1) & 1], no_issue);
    wait_vmem_le<NLOADS>();
    __syncthreads();
  };
#pragma unroll 1
  for (int s = 0; s + 1 < ksteps; s += 2) {
    pstep(s, cw, cwn, cc, cn);
    if (s + 2 < ksteps) pstep(s + 1, cwn, cw, cn, cc);
  }
  // last weight step: copy LoRA step 0 (sT and B2 tiles) into the other
  // buffers; then the LoRA steps
  if (lsteps > 0) {
    if constexpr (MULTI) {
      copy_multi(sxb(ksteps & 1), sw[ksteps & 1], 0);
    } else if constexpr (BLOCK) {
      copy_block(sxb(ksteps & 1), sw[ksteps & 1], 0);
    } else {
      copy_lora(rt, sxb(ksteps & 1), 0, XRows{});
      copy_lora(rb, sw[ksteps & 1], 0, WRows{});
    }
  }
  wait_vmem();
  __syncthreads();
#pragma unroll 1
  for (int l = 0; l < lsteps; ++l) {
    const int s = ksteps + l;
    if (l + 1 < lsteps) {
      if constexpr (MULTI) {
        copy_multi(sxb((s + 1) & 1), sw[(s + 1) & 1], l + 1);
      } else if constexpr (BLOCK) {
        copy_block(sxb((s + 1) & 1), sw[(s + 1) & 1], l + 1);
      } else {
        copy_lora(rt, sxb((s + 1) & 1), l + 1, XRows{});
        copy_lora(rb, sw[(s + 1) & 1], l + 1, WRows{});
      }
    }
    wait_vmem();
    __syncthreads();
  }
}

}  // namespace

int fwd_gemm_splits(int64_t M, int64_t N, int64_t K, size_t cap) {
  const int64_t tiles = ((M + TM - 1) / TM) * ((N + TN - 1) / TN);
  return gemm_splits(tiles, K / KSTEP, M, N, cap);
}

hipError_t launch_fwd_gemm(const Nf4View& W, const uint16_t* X, int64_t M, const uint16_t* sT,
                           const uint16_t* B2, int64_t Rp, void* Y, bool y16, int splits, float* P, bool f16,
                           hipStream_t st) {
  // 512 x 128 tiles (also with a split reduction: the split ranges, and so
  // every output's order of additions, are those of the square tile)
  const bool tall = fwd_tall(M);
  const int tmv = tall ? 512 : 256;
  const int tm = (int)((M + tmv - 1) / tmv), tn = (int)((W.N + 65536 / tmv - 1) / (65536 / tmv));
  const unsigned grid = tile_grid(tm, tn, splits);
  const int yb = y16 ? 1 : 0;
#define QNF4_FWD_LAUNCH(LS, F16V, TMV)                                                                        \
  timed_launch(kKernFwdGemm, fwd_gemm_kernel<LS, F16V, TMV>, dim3(grid), dim3(kThreads), st, W, X, M,        \
               (const uint16_t*)sT, (const uint16_t*)B2, Rp, Y, yb, tm, tn, splits, P, codebook(), NoAdapters{})
#define QNF4_FWD_CASE(LS)                                                                                    \
  case LS:                                                                                                   \
    if (tall) return f16 ? QNF4_FWD_LAUNCH(LS, true, 512) : QNF4_FWD_LAUNCH(LS, false, 512);                 \
    return f16 ? QNF4_FWD_LAUNCH(LS, true, 256) : QNF4_FWD_LAUNCH(LS, false, 256);
  switch (2 * Rp / KSTEP) {
    QNF4_FWD_CASE(1)
    QNF4_FWD_CASE(2)
    QNF4_FWD_CASE(3)
    QNF4_FWD_CASE(4)
    QNF4_FWD_CASE(5)
    QNF4_FWD_CASE(6)
    QNF4_FWD_CASE(7)
    QNF4_FWD_CASE(8)
    default:
      return hipErrorInvalidValue;
  }
#undef QNF4_FWD_CASE
#undef QNF4_FWD_LAUNCH
}

hipError_t launch_fwd_gemm_adapters(const Nf4View& W, const uint16_t* X, int64_t M, const AdapterGemmArgs& ma, void* Y,
                                    bool y16, int splits, float* P, hipStream_t st) {
  const bool tall = fwd_tall(M);
  const int tmv = tall ? 512 : 256;
  const int tm = (int)((M + tmv - 1) / tmv), tn = (int)((W.N + 65536 / tmv - 1) / (65536 / tmv));
  const unsigned grid = tile_grid(tm, tn, splits);
  const uint16_t* none = nullptr;
  if (tall)
    hipLaunchKernelGGL((fwd_gemm_kernel<0, false, 512, kMulti>), dim3(grid), dim3(kThreads), 0, st, W, X, M, none, none,
                       (int64_t)0, Y, y16 ? 1 : 0, tm, tn, splits, P, codebook(), ma);
  else
    hipLaunchKernelGGL((fwd_gemm_kernel<0, false, 256, kMulti>), dim3(grid), dim3(kThreads), 0, st, W, X, M, none, none,
                       (int64_t)0, Y, y16 ? 1 : 0, tm, tn, splits, P, codebook(), ma);
  return hipGetLastError();
}

// Tiles of the gated block's forward, whose N is that of one layer: half a tile's
// weight rows are the gate's.
// Short reductions are split down to four steps where the sum of the partials, a
// launch of its own, is small (us with eight and with four, one layer and two: 153
// tokens, 2536 x 768, r = 112, 38.7 and 30.3, 41.6 and 34.4; 300, 1024 x 1024, 31.9 and
// 27.9, 33.8 and 30.8; larger, 1000, 2048 x 512, 29.1 and 35.8, 31.2 and 39.5; longer,
// 200, 2048 x 2048, 32.5 and 33.0).
int block_fwd_splits(int64_t M, int64_t N, int64_t K, int layers) {
  const int64_t tiles = ((M + TM - 1) / TM) * ((layers * N + TN - 1) / TN), steps = K / KSTEP;
  const bool small = round_up(M, 64) * layers * N <= (int64_t)1 << 20;
  return gemm_splits(tiles, steps, M, layers * N, SIZE_MAX, small && steps < 24 ? 4 : 8);
}

hipError_t launch_fwd_gemm_block(const Nf4View& W, const uint16_t* X, int64_t M, const BlockGemmArgs& ma, bool pair,
                                 void* Y, bool y16, int splits, float* P, hipStream_t st) {
  const bool tall = fwd_tall(M);
  const int tmv = tall ? 512 : 256, tnv = 65536 / tmv / (pair ? 2 : 1);
  const int tm = (int)((M + tmv - 1) / tmv), tn = (int)((W.N + tnv - 1) / tnv);
  const unsigned grid = tile_grid(tm, tn, splits);
  const uint16_t* none = nullptr;
#define QNF4_FWD_BLOCK(TMV, MODE)                                                                                  \
  hipLaunchKernelGGL((fwd_gemm_kernel<0, false, TMV, MODE>), dim3(grid), dim3(kThreads), 0, st, W, X, M, none, none, \
                     (int64_t)0, Y, y16 ? 1 : 0, tm, tn, splits, P, codebook(), ma)
  if (pair) {
    if (tall)
      QNF4_FWD_BLOCK(512, kBlock2);
    else
      QNF4_FWD_BLOCK(256, kBlock2);
  } else {
    if (tall)
      QNF4_FWD_BLOCK(512, kBlock1);
    else
      QNF4_FWD_BLOCK(256, kBlock1);
  }
#undef QNF4_FWD_BLOCK
  return hipGetLastError();
}

}  // namespace qnf4
