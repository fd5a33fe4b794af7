// Training pass of the experts' gated feed-forward block, as grouped GEMMs on tcgen05 (bf16).
//
// Forward (per expert e and row r): g = x Wg^T + bg, u = x Wu^T + bu, h = f(g') u',
// y = h Wd^T + bd, with f(a) = a s(alpha a), s the sigmoid, and g' = clip(g, gate_lo, L),
// u' = clip(u, -L, L) (SiLU: no clips, alpha = 1):
//   GATEUP  gu [R, 2, F] = (g, u) and h [R, F];   DOWN  y.
// Backward, given dy:
//   DH  dh = dy Wd;  dg = dh u' f'(g') [gate_lo <= g <= L],  du = dh f(g') [|u| <= L],
//       f'(a) = s + alpha a s (1 - s)                                  -> dgu [R, 2, F]
//   DX  dx = dg Wg + du Wu
//   DW  dWd = dy^T h, dWg = dg^T x, dWu = du^T x over each expert's rows (zero where it has
//       none), and the bias gradients, the column sums of dy, dg, du over the same rows.
//
// Operand orders: the weights are stored [N, K] for the forward pass, so here the reduction
// runs along their slow dimension: "MN-major" operands (output index contiguous), which the
// tensor core reads directly (instruction descriptor transpose bits, 128-byte swizzle: 64
// elements x 8 K-rows per 1024-byte atom) at the rate of K-major ones.  DW has both operands
// MN-major, its K running over rows.  TMA brings [64 K-rows x 64 elements] boxes; nothing is
// transposed in memory.  All but DW put the weights in M (their output transposed, 256
// output columns a tile) and the expert's rows in N, split evenly into tiles of at most 256
// in steps of 16: a ragged expert wastes at most 15 rows of MMA work a tile, where rows in M
// would round every expert up to 128 or 256.  GATEUP has two accumulators (gate and up of
// the same 256 features) and tiles of at most 128 rows.

// DW's K range is an expert's row range, of any length.  Its last block may reach into
// rows of the next expert: whole 16-row MMA steps past the end are not issued, and the
// rows past the end of the last step are overwritten with zeros in shared memory, in both
// operands, before the MMA reads them (zeroing one would let an infinity or a NaN of a
// neighbouring expert through as 0 * inf).
//
// Bias gradients.  db_down = column sums of dy: for the tiles of the first column block,
// which that gradient keeps 128 columns wide, the issuer adds one N = 16 MMA a step whose B
// operand is a tile of ones, into TMEM columns that the tile leaves free: no further pass
// over dy.  db_gate and db_up are sums of dg and du before their rounding to bf16: DH's
// epilogue lanes, each one column, add up their rows and leave the sums of a tile in the
// workspace; DW adds an expert's tiles in order.  (Sums of the rounded values, by the same
// ones, were off by up to twice as much where a sum cancels.)
//
// Dependent launches.  A call's kernels but its last let their dependents go once their own
// wait is over, so that everything before the call is complete when the second and third
// start: their schedulers read the offsets and decode the first tiles at once, and the rest
// waits for the kernel before.  DW needs nothing of DX, whose last wave of tiles leaves CTA
// pairs idle: it starts on those (what DH wrote is complete when DX's wait is over) and waits
// for DX at its end instead, so that the call's last kernel ends last.  Its pairs then start
// at different times, so after their first tile they take tiles from a counter that DH has
// zeroed, one ahead of their producers (a tile's result does not depend on who computes it).
//
// Roundings to bf16: g and u as kept for the backward pass (bf16_keep_side); h, an output and the
// down product's operand; dg and du between DH and the two products that read them.  The last
// two are tensor-core operands, at the rate that the whole pass is about, and the layer's own
// forward pass rounds h alike.  Against the formulas in 64 bits they put the relative error of
// y, of dx and of the gate and up gradients at 2.3e-3 where one rounding of the result has
// 1.7e-3; two bf16 halves of each would double the products that read them.  All sums are fp32.
//
// CTA pairs (cta_group::2): a tile of M = 256 x N <= 256 a pair, every CTA staging its own 128
// rows of A and half of B, 32 KB a 64-deep stage where a CTA alone takes 48 KB for the same
// MMA time.  N is a multiple of 16 from 16 on: each CTA then holds whole groups of eight rows of B,
// and an expert of a few rows pays for no more than 16 (every width is compared in the tests).
// DW's columns are split into blocks of 256 and 128 (narrow ones first), so that
// every box row is one 128-byte line.
//
// Roles (384 threads a CTA): warp 0 TMA producer; warp 1 TMEM and, in the leader, the MMA
// issuer; warps 2..9 epilogue of the CTA's own 128 accumulator rows; warp 10 the tile scheduler, which
// decodes tiles ahead of everyone into a ring (decoding costs some 500 cycles of division,
// a DW tile of a few hundred rows only some thousands); warp 11 blanks tails (DW) or
// prefetches g and u (DH).  Producer and issuer walk the stages as whole warps with uniform
// values, one elected lane issuing (a lone lane moves every descriptor into uniform registers
// first: 830 cycles a stage against 460).  Waits bounded as in grouped_gemm.cuh, two
// accumulator buffers, and the closing cluster barrier of grouped_gemm_pair.cuh.
//
// Measured, 32 experts, D = F = 2880, 16384 rows, passes one after another: GATEUP 537 us
// (1.01 PFLOP/s), DOWN 276 (0.99), DH 323 to 385 (0.71 to 0.84), DX 547 (0.99), DW 962 with bf16
// gradients (0.85).  Such runs sit at the power limit (990 W, 1.1 to 1.3 GHz of 1.965), where a
// library product of the same sizes in even groups runs at 0.95 to 1.09.  Power is not all of it:
// one launch alone at 1.6 GHz (8 experts, 4096 rows) has the tensor pipe busy 67 / 58 / 39 / 64 /
// 62 % of the time.  GATEUP's two accumulators of N <= 128 stage 40 KB for the MMA time of DOWN's 32.
// DH, with DOWN's operations, takes 47 to 109 us longer: its epilogue also reads g and u and
// writes dg and du, 378 MB in four-byte accesses.  Of 323 us, 253 are left without the loads of
// g and u, 271 without the stores, 286 without the activation's instructions (each taken out
// alone): the loads cost the most.  The epilogue takes 12 to 15 us for 256 rows where DOWN's takes
// 2 (tiles of 48 rows, one a launch: 6.2 us, 4.2 with the pairs of act_grad and the lane selectors,
// 2.9 with its instructions fetched before); a 256-row tile's MMAs take 19 us.
// Seven experts of 143 rows, D = 1440, F = 720 (43 us a backward pass): DH takes 2.5 us from
// the end of its wait to its first copy, DX 0.4 (see above); then 1.5 to the copy's arrival and
// 0.35 a stage, six stages deep; DW's tiles there are bound by their epilogue, 2 us for
// 128 x 256 a CTA (4 TB/s of stores).
// Single CTAs of 128 x 256 with the rows in M: DX 529 to 545 us, DH 296 to 305 and DW 947 to
// 967 against 524 / 327 / 849 for the pairs of their time; halving DX's row tiles past one wave
// of CTA pairs, an L2 prefetch of the weights, and staggered K orders in DW gained 1 % or lost.
#pragma once

#include "grouped_gemm_mx4.cuh"

namespace moe {

enum TrainKind : int { TR_GATEUP = 0, TR_DOWN = 1, TR_DH = 2, TR_DX = 3, TR_DW = 4 };

constexpr int kTrBM = 256;           // M of a pair's tile
constexpr int kTrBK = 64;           // K per stage
constexpr int kTrBox = 64 * 128;    // bytes of a [64 K-rows x 64 elements] box
constexpr int kTrOnesCol = 128;     // TMEM column of the bias sums inside an accumulator buffer
constexpr int kTrUpCol = 128;        // GATEUP: TMEM column of the up accumulator
constexpr int kTrThreads = 384;
constexpr int kTrEpiWarps = 8;
constexpr int kTrSched = 4;         // tiles the scheduler is ahead

template <int KIND>
struct TrainLayout {
  static constexpr int ROWS = KIND == TR_GATEUP ? 128 : 256;    // most rows in a tile's N (not DW)
  static constexpr int NA = KIND == TR_GATEUP ? 2 : 1;          // A operands (and accumulators)
  static constexpr bool A_KMAJOR = KIND == TR_GATEUP || KIND == TR_DOWN;
  static constexpr int STAGES = KIND == TR_GATEUP ? 5 : 6;
  static constexpr int A_BYTES = NA * 2 * kTrBox;
  static constexpr int B_BYTES = ROWS / 2 * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int ONES = KIND == TR_DW ? 1024 : 0;   // 8 rows x 128 B of bf16 ones: half of N = 16
  static constexpr int STAGING_WARP = KIND == TR_DW ? 32 * 80 : 0;   // epilogue: 32 rows of 64 B + 16 B
  static constexpr int STAGING = kTrEpiWarps * STAGING_WARP;
  static constexpr int EXTRA = 4096;   // alignment to 1024, barriers and tables
  static constexpr int SMEM = STAGES * STAGE_BYTES + ONES + STAGING + EXTRA;
  static_assert(SMEM <= 232448, "shared memory budget");
};

// Column blocks of N columns: 1 or 2 units of 128 each (1 for the first one if `spare`), the
// narrower ones first.
__host__ __device__ constexpr int train_col_blocks(int N, bool spare) {
  return ((N + 127) / 128 + (spare ? 1 : 0) + 1) / 2;
}
struct TrainCols {
  int first, units;   // first column, number of 128-column units
};
__host__ __device__ inline TrainCols train_cols(int N, int blocks, int j) {
  const int n = (N + 127) / 128;
  const int q = n / blocks, narrow = blocks - n % blocks;
  return TrainCols{128 * (j * q + (j > narrow ? j - narrow : 0)), q + (j >= narrow ? 1 : 0)};
}

// One product of a launch.  DW: a, bw = the two row-major operands whose rows are summed
// over.  Else a (and a2) = the weights, b = the rows: GATEUP Wg, Wu and x;  DOWN Wd and h;
// DH Wd and dy;  DX Wg, Wu and dgu.  K-major operands have boxes of 64 K elements x 128
// weight rows (a.single) or 32 (q + 1) rows (b[q]).
// Two boxes of a K-rows x elements operand come in one copy: the matrix seen as {64 columns,
// K rows, N / 64} (and groups), a box of 64 x 64 x 2 landing as consecutive [64 x 64] boxes.
// Where the partial box of an N that is no multiple of 64 is met, and for one box alone, the
// copies are single boxes.  (One TMA instruction costs the producer thread some 100 cycles.)
struct TrainMaps {
  CUtensorMap two, single;
};
struct TrainJob {
  TrainMaps a, a2;
  union {
    TrainMaps bw;         // DW
    CUtensorMap b[4];   // the others
  };
  void* out;
  void* bias_out;     // DW: [G, m] bias gradient, or null
  const float* part;  // DW: its sums by row tile and epilogue half, part_ld apart; null: column sums of A
  const __nv_bfloat16 *bias0, *bias1;   // GATEUP (gate, up), DOWN: [G, m], or null
  int m, n;         // DW: rows and columns of the gradient;  else m = columns of the output
  int nt;           // DW: column blocks
};

template <int KIND>
struct TrainArgs {
  TrainJob job[KIND == TR_DW ? 3 : 1];
  int num_jobs;
  const int32_t* group_off;   // [G+1]
  int num_groups;
  int m_total;                // R
  int early;                  // DW: behind a DX launch, starts beside it
  int* counter;               // DH (zeroes it), DW if early: tiles taken beyond the pairs' first ones
  int tile_rows;              // most rows in a tile's N: TrainLayout::ROWS, or a half or quarter (DW: DH's)
  int k_dim;                  // K (DX: of one half)
  __nv_bfloat16* gu;          // GATEUP (written), DH: [R, 2, F]
  float* part;                // DH: [part_tiles][2 halves][2][F] sums of dg and du
  int part_tiles;             // DH, DW (clamp for offsets that are not ascending)
  int part_ld;                // 2 F
  float limit, alpha, gate_lo;
  unsigned long long wait_limit_ns;
};

__device__ __forceinline__ void tma_load_4d_pair(void* dst, const void* tmap, uint32_t bar_cluster, int c0, int c1,
                                                 int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// K-rows x elements operand ("MN-major"), 128-byte swizzle: 64-element blocks kTrBox bytes
// apart (leading offset), 8-row groups 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kTrBox >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// A lane's values of one column in rows j (a) and j + 1 (b), rounded to bf16 and traded with
// the neighbouring lane: the even lane gets both columns of row j, the odd one of row j + 1.
// `sel` is the lane's byte selector, trade_sel.
__device__ __forceinline__ uint32_t trade_sel() { return (threadIdx.x & 1) ? 0x3276u : 0x5410u; }
__device__ __forceinline__ uint32_t trade_pair(float a, float b, uint32_t sel) {
  const __nv_bfloat162 mine = __floats2bfloat162_rn(a, b);
  const uint32_t x = *reinterpret_cast<const uint32_t*>(&mine);
  return __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 1), sel);
}
// The way back: both columns of the lane's row to its own column in rows j and j + 1.
__device__ __forceinline__ float2 untrade_pair(uint32_t x, uint32_t sel) {
  const uint32_t z = __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 1), sel);
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&z));
}

// v rounded to bf16, kept on its side of the bounds +-lim: the backward pass decides from the
// stored value whether the clip let the gradient through, so rounding must not move it across.
// The gate's lower bound is lo = 0 (-inf: none): a negative value too small for bf16 stays at
// the smallest negative one instead of becoming -0, which lies inside the clip.
__device__ __forceinline__ float bf16_keep_side(float v, float lim, float lo = -INFINITY) {
  const float a = fabsf(v);
  uint16_t b = __bfloat16_as_ushort(__float2bfloat16_rn(a));
  const bool over = a > lim;
  if ((__bfloat162float(__ushort_as_bfloat16(b)) > lim) != over) b += over ? 1 : -1;
  if (v < lo && b == 0) b = 1;
  return copysignf(__bfloat162float(__ushort_as_bfloat16(b)), v);
}

// Derivatives of h = f(clip(g)) clip(u) times dh, for two rows.  The clips pass the gradient
// at their ends, and that of a NaN.
__device__ __forceinline__ void act_grad(float2 dh, float2 g, float2 u, float limit, float alpha, float gate_lo,
                                         float2& dg, float2& du) {
  const float2 gc = make_float2(clip_nan(g.x, gate_lo, limit), clip_nan(g.y, gate_lo, limit));
  const float2 uc = make_float2(clip_nan(u.x, limit), clip_nan(u.y, limit));
  const float2 a2 = make_float2(alpha, alpha);
  const float zl = -alpha * 1.44269504f;   // log2(e)
  const float2 s = sigmoid2_neg_log2(__fmul2_rn(gc, make_float2(zl, zl)));
  const float2 f = __fmul2_rn(gc, s);
  const float2 rest = __ffma2_rn(s, make_float2(-1.0f, -1.0f), make_float2(1.0f, 1.0f));
  const float2 slope = __ffma2_rn(__fmul2_rn(a2, f), rest, s);
  const float2 vg = __fmul2_rn(__fmul2_rn(dh, uc), slope), vu = __fmul2_rn(dh, f);
  dg = make_float2((g.x < gate_lo || g.x > limit) ? 0.0f : vg.x, (g.y < gate_lo || g.y > limit) ? 0.0f : vg.y);
  du = make_float2(fabsf(u.x) > limit ? 0.0f : vu.x, fabsf(u.y) > limit ? 0.0f : vu.y);
}

struct TrainTile {
  int job, g;           // job -1: no more tiles
  int m0;               // first row of the gradient (DW), first column of the output (others)
  int n0, units;        // DW: first column, 128-column units
  int n;                // MMA N
  int kb;               // 64-deep K blocks
  int r0, rows;         // DW: the expert's rows;  others: the tile's
  int sums;             // DW: bias gradient wanted of this tile: 1 by the ones, 2 from the row tiles' sums
  int rt;               // DH: row tile, counted over the experts
};

// DW: the last K block of the tile ends inside a 16-row MMA step.
__device__ __forceinline__ bool train_ragged(const TrainTile& t) { return (t.rows & 15) != 0; }

template <int KIND>
__device__ __forceinline__ TrainTile train_tile(int i, const int* tile_off, const int* goff, const TrainArgs<KIND>& a) {
  TrainTile t{};
  if constexpr (KIND == TR_DW) {
    int mt, nt;
    for (;; ++t.job) {
      nt = a.job[t.job].nt;
      mt = (a.job[t.job].m + kTrBM - 1) / kTrBM;
      const int n = a.num_groups * mt * nt;
      if (i < n || t.job + 1 == a.num_jobs) break;
      i -= n;
    }
    t.g = i / (mt * nt);
    i -= t.g * mt * nt;
    // bands of row blocks, the row block fastest: neighbours share operand rows in L2
    constexpr int kBand = 8;
    const int band = i / (kBand * nt);
    const int rem = i - band * kBand * nt;
    const int rows = min(kBand, mt - band * kBand);
    const int nb = rem / rows;
    t.m0 = (band * kBand + rem - nb * rows) * kTrBM;
    const TrainCols c = train_cols(a.job[t.job].n, nt, nb);
    t.n0 = c.first;
    t.units = c.units;
    t.n = 128 * c.units;
    t.r0 = goff[t.g];
    t.rows = max(0, goff[t.g + 1] - t.r0);
    t.kb = (t.rows + kTrBK - 1) / kTrBK;
    t.sums = t.n0 != 0 || a.job[t.job].bias_out == nullptr ? 0 : a.job[t.job].part == nullptr ? 1 : 2;
  } else {
    // tiles of an expert: its row tiles fastest (they share the weight columns)
    const int mt = (a.job[0].m + kTrBM - 1) / kTrBM;
    int lo = 0, hi = a.num_groups;            // tile_off[lo] * mt <= i < tile_off[hi] * mt
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_off[mid] * mt <= i) lo = mid; else hi = mid;
    }
    t.g = lo;
    const int rt = tile_off[lo + 1] - tile_off[lo], rows = goff[lo + 1] - goff[lo];
    i -= tile_off[lo] * mt;
    const int mb = i / rt, r = i - mb * rt;
    const int per = ((rows + rt - 1) / rt + 15) / 16 * 16;
    t.m0 = mb * kTrBM;
    t.rt = tile_off[lo] + r;
    t.r0 = goff[lo] + r * per;
    t.rows = min(per, rows - r * per);
    t.n = (t.rows + 15) / 16 * 16;
    const int kb = (a.k_dim + kTrBK - 1) / kTrBK;
    t.kb = KIND == TR_DX ? 2 * kb : kb;
  }
  return t;
}

// 32 rows x 64 bytes that the warp's lanes hold (lane = row, v its columns) to global rows
// through the warp's staging area: a store instruction covers eight 64-byte runs of rows.
template <typename T>
__device__ __forceinline__ void store_rows64(uint8_t* stage, T* out, size_t ldo, int rows, int cols, const float* v) {
  constexpr int PER = 16 / static_cast<int>(sizeof(T));   // columns per 16-byte piece
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint4 u;
    if constexpr (sizeof(T) == 2) {
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(v[p * PER + 2 * j], v[p * PER + 2 * j + 1]);
    } else {
      u = make_uint4(__float_as_uint(v[p * PER]), __float_as_uint(v[p * PER + 1]), __float_as_uint(v[p * PER + 2]),
                     __float_as_uint(v[p * PER + 3]));
    }
    *reinterpret_cast<uint4*>(stage + lane * 80 + p * 16) = u;
  }
  __syncwarp();
  const int piece = lane & 3;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int r = it * 8 + (lane >> 2);
    if (r < rows && piece * PER < cols)
      *reinterpret_cast<uint4*>(out + r * ldo + piece * PER) = *reinterpret_cast<const uint4*>(stage + r * 80 + piece * 16);
  }
}

template <int KIND, typename OutT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTrThreads, 1)
    ffn_train_kernel(const __grid_constant__ TrainArgs<KIND> args) {
  if constexpr (KIND == TR_DOWN || KIND == TR_DW) pdl_launch_dependents();
  using LY = TrainLayout<KIND>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ones = smem + LY::STAGES * LY::STAGE_BYTES;
  uint8_t* staging = ones + LY::ONES;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + LY::STAGING);   // leader's: both CTAs' stage is in place
  uint64_t* landed = full + LY::STAGES;         // DW: a ragged tail's loads have landed in this CTA
  uint64_t* empty = landed + LY::STAGES;
  uint64_t* tfull = empty + LY::STAGES;
  uint64_t* tempty = tfull + 2;                 // leader's
  uint64_t* sfull = tempty + 2;                 // scheduler ring
  uint64_t* sempty = sfull + kTrSched;
  uint64_t* drain = sempty + kTrSched;
  uint64_t* taken = drain + 1;                  // DW: the leader's producer has the tile
  uint64_t* boxed = taken + 1;                  // DW: the leader's choices for the other CTA
  TrainTile* ring = reinterpret_cast<TrainTile*>(boxed + 2 * kTrSched);
  int* box = reinterpret_cast<int*>(ring + kTrSched);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(box + 2 * kTrSched);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* never_flag = abort_flag + 1;
  int* tile_off = never_flag + 1;              // [G+1]
  int* goff = tile_off + (kMaxGroups + 1);     // [G+1]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());   // 0 = leader (issues the MMAs)
  const int G = args.num_groups;
  const uint64_t lim = args.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < LY::STAGES; ++s) {
      mbar_init(&full[s], 2);      // one arrival a CTA: its producer's, or its blanker's
      mbar_init(&landed[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kTrEpiWarps);
    }
    for (int q = 0; q < kTrSched; ++q) {
      mbar_init(&sfull[q], 1);
      mbar_init(&sempty[q], 1 + (rank == 0 ? 1 : 0) + kTrEpiWarps + (KIND == TR_DH || KIND == TR_DW ? 1 : 0));   // who reads a tile
    }
    mbar_init(drain, 1);
    mbar_init(taken, 1);
    for (int q = 0; q < 2 * kTrSched; ++q) mbar_init(&boxed[q], 1);
    *abort_flag = 0;
    *never_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    if (lane < args.num_jobs) {
      tma_prefetch_desc(&args.job[lane].a.single);
      tma_prefetch_desc(KIND == TR_DW ? &args.job[lane].bw.single : &args.job[lane].b[0]);
    }
  } else if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  } else if (KIND == TR_DW && warp < 6) {
    for (int i = threadIdx.x - 64; i < LY::ONES / 4; i += 128) reinterpret_cast<uint32_t*>(ones)[i] = 0x3F803F80u;
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // both CTAs' barriers are initialised before any signal between them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (KIND == TR_GATEUP || KIND == TR_DH || (KIND == TR_DW && !args.early)) pdl_wait();
  else if (KIND != TR_DW && warp != 2 + kTrEpiWarps) pdl_wait();
  if ((KIND == TR_DX && warp != 2 + kTrEpiWarps) || KIND == TR_GATEUP || KIND == TR_DH) pdl_launch_dependents();
  const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
  const int KB1 = (args.k_dim + kTrBK - 1) / kTrBK;   // DX: K blocks of one half

  // The next tile from the scheduler's ring; false when a wait gave up.  For a whole
  // warp, which agrees on the answer.
  auto next_tile = [&](int n, TrainTile& t) {
    const int q = n % kTrSched;
    if (!__all_sync(0xffffffffu, mbar_wait(&sfull[q], (n / kTrSched) & 1, abort_flag, lim))) return false;
    t = ring[q];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sempty[q]);
    return true;
  };
  // A tile that the whole warp has read, as values the compiler knows to be the same in every lane.
  auto uniform = [](TrainTile& t) {
    int* f = reinterpret_cast<int*>(&t);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(TrainTile) / sizeof(int)); ++i) f[i] = __shfl_sync(0xffffffffu, f[i], 0);
  };
  bool ok = true;

  if (warp == 2 + kTrEpiWarps) {
    // ------------------------------------------------------------ scheduler
    group_table(args.group_off, G, args.m_total, args.tile_rows, goff, tile_off);
    __syncwarp();   // the ring's barrier passes the table on with the first tile
    if (lane == 0) {
      int total = 0;
      if constexpr (KIND == TR_DW) {
        for (int j = 0; j < args.num_jobs; ++j) total += G * ((args.job[j].m + kTrBM - 1) / kTrBM) * args.job[j].nt;
      } else {
        total = tile_off[G] * ((args.job[0].m + kTrBM - 1) / kTrBM);
      }
      if (KIND == TR_DH && blockIdx.x == 0) *args.counter = 0;
      const int pairs = gridDim.x >> 1;
      int n = 0;
      for (int i = blockIdx.x >> 1;; ++n) {
        TrainTile t;
        t.job = -1;
        if (i < total) t = train_tile<KIND>(i, tile_off, goff, args);
        const int q = n % kTrSched;
        if (!mbar_wait(&sempty[q], ((n / kTrSched) & 1) ^ 1, abort_flag, lim)) { ok = false; break; }
        ring[q] = t;
        mbar_arrive(&sfull[q]);
        if (i >= total) break;
        if (KIND == TR_DW && args.early) {
          // A box is written again eight tiles on: by then the other CTA's epilogue, which the
          // accumulators' barriers keep within three tiles of the issuer, has long read it.
          const int b = n % (2 * kTrSched);
          if (rank == 0) {
            if (!mbar_wait(taken, n & 1, abort_flag, lim)) { ok = false; break; }
            i = pairs + atomicAdd(args.counter, 1);
            st_async(mapa_shared(smem_u32(&box[b]), 1), i, mapa_shared(smem_u32(&boxed[b]), 1));
          } else {
            mbar_arrive_expect_tx(&boxed[b], 4);
            if (!mbar_wait_cluster(&boxed[b], (n / (2 * kTrSched)) & 1, abort_flag, lim)) { ok = false; break; }
            i = box[b];
          }
        } else {
          i += pairs;
        }
      }
      if (!ok) {
        *abort_flag = 1;
        flag_error(DEVERR_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    // As in the issuer, the whole warp walks the stages with uniform values and one elected
    // lane issues the copies.
    {
      const bool leader = elect_one();
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;         // stages counted on the leader's full
      uint32_t tails = 0, tail_par = 0, tail_uses = 0;     // stages counted on this CTA's landed
      TrainTile ti;
      for (int n = 0;; ++n) {
        if (!next_tile(n, ti)) { ok = false; break; }
        uniform(ti);
        if (ti.job < 0) break;
        if (KIND == TR_DW && leader) mbar_arrive(taken);
        const TrainJob& jb = args.job[ti.job];
        const int a_row = ti.m0 + rank * 128;
        const bool a_two = a_row + 128 <= (jb.m & ~63) || (jb.m & 63) == 0;
        const int b_col = ti.n0 + rank * 64 * ti.units;                       // DW
        const bool b_two = ti.units == 2 && b_col + 128 <= (jb.n & ~63);
        const int b_row = ti.r0 + rank * (ti.n / 2), q32 = (ti.n + 63) / 64;   // others: boxes of 32 rows
        const uint32_t tx = LY::A_BYTES + (KIND == TR_DW ? ti.units * kTrBox : q32 * (kTrBox / 2));
        for (int kb = 0; kb < ti.kb; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, abort_flag, lim))) { ok = false; break; }
          uint8_t* sa = smem + s * LY::STAGE_BYTES;
          uint8_t* sb = sa + LY::A_BYTES;
          const uint32_t fb = full_leader + static_cast<uint32_t>(s) * 8u;
          if (KIND == TR_DW && kb == ti.kb - 1 && train_ragged(ti)) {
            // the blanker is told here, and passes the stage on to the leader
            const int r = ti.r0 + kb * kTrBK;
            if (leader) {
              mbar_arrive_expect_tx(&landed[s], tx);
              if (b_two) tma_load_3d(sb, &jb.bw.two, &landed[s], 0, r, b_col / 64);
              else
                for (int q = 0; q < ti.units; ++q) tma_load_2d(sb + q * kTrBox, &jb.bw.single, &landed[s], b_col + 64 * q, r);
              if (a_two) tma_load_3d(sa, &jb.a.two, &landed[s], 0, r, a_row / 64);
              else
                for (int q = 0; q < 2; ++q) tma_load_2d(sa + q * kTrBox, &jb.a.single, &landed[s], a_row + 64 * q, r);
            }
            issued &= ~(1u << s);   // its earlier loads have landed, or the slot were not free
            tails |= 1u << s;
            tail_par = (tail_par & ~(1u << s)) | (tail_uses & (1u << s));
            tail_uses ^= 1u << s;
          } else {
            if (leader) {
              if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * tx);
              else mbar_arrive_cluster(fb);
              if constexpr (KIND == TR_DW) {
                const int r = ti.r0 + kb * kTrBK;
                if (b_two) tma_load_3d_pair(sb, &jb.bw.two, fb, 0, r, b_col / 64);
                else
                  for (int q = 0; q < ti.units; ++q) tma_load_2d_pair(sb + q * kTrBox, &jb.bw.single, fb, b_col + 64 * q, r);
                if (a_two) tma_load_3d_pair(sa, &jb.a.two, fb, 0, r, a_row / 64);
                else
                  for (int q = 0; q < 2; ++q) tma_load_2d_pair(sa + q * kTrBox, &jb.a.single, fb, a_row + 64 * q, r);
              } else {
                if constexpr (LY::A_KMAJOR) {
                  tma_load_3d_pair(sa, &jb.a.single, fb, kb * kTrBK, a_row, ti.g);
                  if (LY::NA == 2) tma_load_3d_pair(sa + 2 * kTrBox, &jb.a2.single, fb, kb * kTrBK, a_row, ti.g);
                  tma_load_2d_pair(sb, &jb.b[q32 - 1], fb, kb * kTrBK, b_row);
                } else {
                  const int half = (KIND == TR_DX && kb >= KB1) ? 1 : 0;
                  const int k0 = (kb - half * KB1) * kTrBK;
                  const TrainMaps& ma = half ? jb.a2 : jb.a;
                  if (a_two) tma_load_4d_pair(sa, &ma.two, fb, 0, k0, a_row / 64, ti.g);
                  else
                    for (int q = 0; q < 2; ++q) tma_load_3d_pair(sa + q * kTrBox, &ma.single, fb, a_row + 64 * q, k0, ti.g);
                  if (KIND == TR_DX) tma_load_3d_pair(sb, &jb.b[q32 - 1], fb, k0, half, b_row);
                  else tma_load_2d_pair(sb, &jb.b[q32 - 1], fb, k0, b_row);
                }
              }
            }
            issued |= 1u << s;
            issued_par = (issued_par & ~(1u << s)) | (ph << s);
          }
          __syncwarp();
          if (++s == LY::STAGES) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
      }
      // every copy has landed before the CTA may leave (those counted on the peer's barriers: see the end)
      if (leader) {
        const uint64_t t0 = global_timer_ns();
        if (rank == 0 && !wait_landed(full, LY::STAGES, issued, issued_par, never_flag, t0)) ok = false;
        if (!wait_landed(landed, LY::STAGES, tails, tail_par, never_flag, t0)) ok = false;
      }
      if (!ok) {
        *abort_flag = 1;
        flag_error(DEVERR_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    // The whole warp walks the stages, so that addresses and descriptors (made once, stepped
    // by additions) are uniform values the tensor instructions take as they are; one elected
    // lane issues them.
    if (rank == 0) {
      const bool leader = elect_one();
      const uint32_t s_addr = smem_u32(smem);
      const uint64_t a_desc = LY::A_KMAJOR ? sw128_kmajor_desc(s_addr) : sw128_mnmajor_desc(s_addr);
      const uint64_t b_desc = KIND == TR_DW ? sw128_mnmajor_desc(s_addr + LY::A_BYTES) : sw128_kmajor_desc(s_addr + LY::A_BYTES);
      const uint64_t ones_desc = sw128_kmajor_desc(smem_u32(ones));
      constexpr int kAStep = LY::A_KMAJOR ? 32 / 16 : 2048 / 16, kBStep = KIND == TR_DW ? 2048 / 16 : 32 / 16;   // of 16 K
      const uint32_t idesc_ones = make_idesc(kTrBM, 16, 1u) | (1u << 15);
      int s = 0;
      uint32_t ph = 0;
      bool issued_any = false;
      TrainTile ti;
      for (int n = 0;; ++n) {
        if (!next_tile(n, ti)) { ok = false; break; }
        uniform(ti);
        if (ti.job < 0) break;
        const uint32_t idesc = make_idesc(kTrBM, ti.n, 1u) | (LY::A_KMAJOR ? 0u : 1u << 15) | (KIND == TR_DW ? 1u << 16 : 0u);
        const bool sums = KIND == TR_DW && ti.sums == 1;
        const int acc = n & 1;
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kAccStride);
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(&tempty[acc], ((n >> 1) & 1) ^ 1u, abort_flag, lim))) { ok = false; break; }
        tc_fence_after();
        for (int kb = 0; kb < ti.kb; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&full[s], ph, abort_flag, lim))) { ok = false; break; }
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>(s * (LY::STAGE_BYTES >> 4));
          const uint64_t ad = a_desc + so, bd = b_desc + so;
          const int steps = KIND == TR_DW ? min(kTrBK / 16, (ti.rows - kb * kTrBK + 15) / 16) : kTrBK / 16;
          if (leader) {
            if (steps == kTrBK / 16 && !sums) {
#pragma unroll
              for (int kk = 0; kk < kTrBK / 16; ++kk) {
                tc_mma_pair(d_tmem, ad + kk * kAStep, bd + kk * kBStep, idesc, (kb | kk) != 0 ? 1u : 0u);
                if (LY::NA == 2)
                  tc_mma_pair(d_tmem + kTrUpCol, ad + (2 * kTrBox >> 4) + kk * kAStep, bd + kk * kBStep, idesc,
                              (kb | kk) != 0 ? 1u : 0u);
              }
            } else {
              for (int kk = 0; kk < steps; ++kk) {
                const uint32_t accumulate = (kb | kk) != 0 ? 1u : 0u;
                tc_mma_pair(d_tmem, ad + kk * kAStep, bd + kk * kBStep, idesc, accumulate);
                if (sums) tc_mma_pair(d_tmem + kTrOnesCol, ad + kk * kAStep, ones_desc, idesc_ones, accumulate);
              }
            }
            tc_commit_pair_mc(&empty[s], 0x3);
          }
          __syncwarp();
          issued_any = true;
          if (++s == LY::STAGES) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        if (leader) tc_commit_pair_mc(&tfull[acc], 0x3);
        __syncwarp();
      }
      if (leader) {
        if (!ok) {
          *abort_flag = 1;
          flag_error(DEVERR_TIMEOUT);
        }
        if (issued_any) {
          tc_commit_pair(drain);
          if (!mbar_wait(drain, 0, never_flag, kDrainLimitNs)) flag_error(DEVERR_TIMEOUT);
        }
      }
    }
    __syncwarp();
  } else if (warp < 2 + kTrEpiWarps) {
    // ------------------------------------------------------------ epilogue (warps 2..9)
    // Two warps share a TMEM lane quarter and take its column chunks in turn.
    const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    // DH's epilogue begins with a tile that has no rows of its own: a first pass over its 900
    // instructions fetches them while the first operands are on their way (ragged SiLU backward
    // 44.6 -> 42.9 us; GATEUP gains nothing by it).  Its loads from the second accumulator are in no
    // order with the second tile's MMAs, which may be writing there: what they bring is dropped.
    TrainTile ti{};
    ti.rows = 32;
    for (int n = KIND == TR_DH ? -1 : 0;; ++n) {
      const bool dry = n < 0;
      if (!dry && !next_tile(n, ti)) { ok = false; break; }
      if (ti.job < 0) break;
      const TrainJob& jb = args.job[ti.job];
      const int acc = n & 1;
      const int row0 = ti.m0 + rank * 128 + quarter * 32;   // of the warp's accumulator rows
      const uint32_t tbase =
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * kAccStride);
      if constexpr (KIND == TR_DW) {
        constexpr int COLS = 64 / static_cast<int>(sizeof(OutT));
        uint8_t* stage = staging + (warp - 2) * LY::STAGING_WARP;
        const int rows = jb.m - row0, width = min(ti.n, jb.n - ti.n0);
        if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], (n >> 1) & 1, abort_flag, lim))) { ok = false; break; }
        tc_fence_after();
        const bool none = ti.rows == 0;   // the gradient is zero
        const size_t row_base = static_cast<size_t>(ti.g) * jb.m;
        OutT* out = static_cast<OutT*>(jb.out) + (row_base + row0) * jb.n + ti.n0;
#pragma unroll 1
        for (int c = COLS * half; c < width; c += 2 * COLS) {
          float v[COLS];
#pragma unroll
          for (int j = 0; j < COLS; j += 8) tmem_ld8(tbase + c + j, *reinterpret_cast<float(*)[8]>(v + j));
          tmem_ld_wait();
          if (none) {
#pragma unroll
            for (int j = 0; j < COLS; ++j) v[j] = 0.0f;
          }
          store_rows64<OutT>(stage, out + c, jb.n, rows, width - c, v);
        }
        if (half == 0 && ti.sums) {
          float sum = 0.0f;
          if (ti.sums == 1) {
            float b[8];
            tmem_ld8(tbase + kTrOnesCol, b);
            tmem_ld_wait();
            sum = none ? 0.0f : b[0];
          } else if (lane < rows) {
            const int last = min(tile_off[ti.g + 1], args.part_tiles);
            for (int t = 2 * tile_off[ti.g]; t < 2 * last; ++t) sum += __ldcg(jb.part + static_cast<size_t>(t) * args.part_ld + row0 + lane);
          }
          if (lane < rows) {
            OutT* bo = static_cast<OutT*>(jb.bias_out) + row_base + row0 + lane;
            if constexpr (sizeof(OutT) == 2) *bo = __float2bfloat16_rn(sum);
            else *bo = sum;
          }
        }
      } else {
        // Lane = output column, accumulator column = row, 16 rows at a time.  Neighbouring
        // lanes trade halves (trade_pair), so that the even one holds both columns of a row
        // and the odd one both of the next: every access is four bytes a lane, 64-byte runs
        // of two rows.  DH's g and u of the next 16 rows are on their way while these are
        // computed, the first before the accumulator is complete.
        const int col = row0 + lane, M = jb.m;
        const bool cvalid = col < M && !dry;                  // M is a multiple of 16: of both lanes
        constexpr int kRowElems = KIND == TR_DH ? 2 : 1;      // DH: [R, 2, F]
        const size_t ld = static_cast<size_t>(kRowElems) * M;
        const int odd = lane & 1;
        const int rows = (cvalid ? ti.rows : 0) - odd;        // this lane's rows are j + odd
        const size_t at = static_cast<size_t>(ti.r0) * ld + col + odd * (ld - 1);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(jb.out) + at;
        const size_t gu_at = static_cast<size_t>(ti.r0) * 2 * M + col + odd * (2 * static_cast<size_t>(M) - 1);
        __nv_bfloat16* gu = args.gu + gu_at;
        float bias0 = 0.0f, bias1 = 0.0f;
        if constexpr (LY::A_KMAJOR) {
          const size_t bi = static_cast<size_t>(ti.g) * M + col;
          if (cvalid && jb.bias0 != nullptr) bias0 = __bfloat162float(jb.bias0[bi]);
          if (KIND == TR_GATEUP && cvalid && jb.bias1 != nullptr) bias1 = __bfloat162float(jb.bias1[bi]);
        }
        const uint32_t sel = trade_sel();
        float2 sum_g = {}, sum_u = {};      // DH: of this lane's column, even and odd rows
        uint32_t pg[8], pu[8];
        auto fetch = [&](int c) {
          if constexpr (KIND == TR_DH) {
            const __nv_bfloat16* p = gu + c * ld;
#pragma unroll
            for (int j = 0; j < 8; ++j, p += 2 * ld)
              if (c + 2 * j < rows) {
                pg[j] = *reinterpret_cast<const uint32_t*>(p);
                pu[j] = *reinterpret_cast<const uint32_t*>(p + M);
              } else {
                pg[j] = pu[j] = 0;
              }
          }
        };
        fetch(16 * half);
        if (!dry && !__all_sync(0xffffffffu, mbar_wait(&tfull[acc], (n >> 1) & 1, abort_flag, lim))) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int c = 16 * half; c < ti.rows; c += 32) {
          float v[16];
          tmem_ld8(tbase + c, *reinterpret_cast<float(*)[8]>(v));
          tmem_ld8(tbase + c + 8, *reinterpret_cast<float(*)[8]>(v + 8));
          if constexpr (KIND == TR_GATEUP) {
            float u[16];
            tmem_ld8(tbase + kTrUpCol + c, *reinterpret_cast<float(*)[8]>(u));
            tmem_ld8(tbase + kTrUpCol + c + 8, *reinterpret_cast<float(*)[8]>(u + 8));
            tmem_ld_wait();
            __nv_bfloat16* o = out + c * ld;
            __nv_bfloat16* p = gu + c * 2 * ld;
#pragma unroll
            for (int j = 0; j < 16; j += 2, o += 2 * ld, p += 4 * ld) {
              float h[2], g[2], w[2];
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const float gv = v[j + q] + bias0, uv = u[j + q] + bias1;
                const float gc = clip_nan(gv, args.gate_lo, args.limit);
                const float uc = clip_nan(uv, args.limit);
                h[q] = __fdividef(gc, 1.0f + __expf(-args.alpha * gc)) * uc;
                g[q] = bf16_keep_side(gv, args.limit, args.gate_lo);
                w[q] = bf16_keep_side(uv, args.limit);
              }
              const uint32_t ph = trade_pair(h[0], h[1], sel), pgv = trade_pair(g[0], g[1], sel), puv = trade_pair(w[0], w[1], sel);
              if (c + j < rows) {
                *reinterpret_cast<uint32_t*>(o) = ph;
                *reinterpret_cast<uint32_t*>(p) = pgv;
                *reinterpret_cast<uint32_t*>(p + M) = puv;
              }
            }
          } else if constexpr (KIND == TR_DH) {
            tmem_ld_wait();
            uint32_t dgs[8], dus[8];
            if (c + 16 > ti.rows) {   // columns past the tile's rows hold other rows' products
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = c + j < ti.rows ? v[j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float2 dg, du;
              act_grad(make_float2(v[2 * j], v[2 * j + 1]), untrade_pair(pg[j], sel), untrade_pair(pu[j], sel),
                       args.limit, args.alpha, args.gate_lo, dg, du);
              sum_g = __fadd2_rn(sum_g, dg);
              sum_u = __fadd2_rn(sum_u, du);
              dgs[j] = trade_pair(dg.x, dg.y, sel);
              dus[j] = trade_pair(du.x, du.y, sel);
            }
            fetch(c + 32);
            __nv_bfloat16* o = out + c * ld;
#pragma unroll
            for (int j = 0; j < 8; ++j, o += 2 * ld)
              if (c + 2 * j < rows) {
                *reinterpret_cast<uint32_t*>(o) = dgs[j];
                *reinterpret_cast<uint32_t*>(o + M) = dus[j];
              }
          } else {
            tmem_ld_wait();
            __nv_bfloat16* o = out + c * ld;
#pragma unroll
            for (int j = 0; j < 16; j += 2, o += 2 * ld) {
              const uint32_t both = trade_pair(v[j] + bias0, v[j + 1] + bias0, sel);
              if (c + j < rows) *reinterpret_cast<uint32_t*>(o) = both;
            }
          }
        }
        if (KIND == TR_DH && args.part != nullptr && cvalid && ti.rt < args.part_tiles) {
          float* p = args.part + static_cast<size_t>(2 * ti.rt + half) * args.part_ld + col;
          p[0] = sum_g.x + sum_g.y;
          p[M] = sum_u.x + sum_u.y;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && !dry) mbar_arrive_cluster(tempty_leader + static_cast<uint32_t>(acc) * 8u);
    }
    if (!ok) {
      *abort_flag = 1;
      flag_error(DEVERR_TIMEOUT);
    }
  } else if (KIND == TR_DH) {
    // ------------------------------------------------------------ prefetcher
    // g and u of coming tiles into the L2: the epilogue's loads look only 16 rows ahead.
    TrainTile ti;
    for (int n = 0;; ++n) {
      if (!next_tile(n, ti)) { ok = false; break; }
      if (ti.job < 0) break;
      const int F = args.job[0].m;
      const int col = ti.m0 + rank * 128 + (lane & 1) * 64;
      if (col < F)
        for (int r = lane >> 1; r < 2 * ti.rows; r += 16)   // g and u of a row: two runs of F elements
          asm volatile("prefetch.global.L2 [%0];" ::"l"(args.gu + (static_cast<size_t>(ti.r0) * 2 + r) * F + col));
    }
    if (!ok) {
      *abort_flag = 1;
      flag_error(DEVERR_TIMEOUT);
    }
  } else if (KIND == TR_DW) {
    // ------------------------------------------------------------ blanker (both CTAs)
    // Blanks the rows between the end of an expert and the end of its last 16-row step in
    // this CTA's operands, then makes the CTA's arrival on the leader's full barrier (the
    // proxy fence publishes the writes to the tensor core, as in grouped_gemm_pair_mx.cuh).
    int s = 0;
    uint32_t uses = 0;
    TrainTile ti;
    for (int n = 0;; ++n) {
      if (!next_tile(n, ti)) { ok = false; break; }
      if (ti.job < 0) break;
      if (ti.kb > 0 && train_ragged(ti)) {
        const int q = (s + ti.kb - 1) % LY::STAGES;
        if (!__all_sync(0xffffffffu, mbar_wait(&landed[q], (uses >> q) & 1u, abort_flag, lim))) { ok = false; break; }
        uses ^= 1u << q;
        const int valid = ti.rows - (ti.kb - 1) * kTrBK;
        uint8_t* st = smem + q * LY::STAGE_BYTES + valid * 128;
        const int pieces = (16 - (valid & 15)) * 8;
        for (int box = 0; box < 2 + ti.units; ++box)
          for (int p = lane; p < pieces; p += 32)
            *reinterpret_cast<uint4*>(st + box * kTrBox + p * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();   // read by the tensor core (async proxy)
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(full_leader + static_cast<uint32_t>(q) * 8u);
      }
      s = (s + ti.kb) % LY::STAGES;
    }
    if (!ok) {
      *abort_flag = 1;
      flag_error(DEVERR_TIMEOUT);
    }
  }

  tc_fence_before();
  __syncthreads();
  // A role that gave up may leave copies in flight that count on the peer's barriers, which cannot
  // be polled from here, or on a stage that does not complete: both CTAs give them 2 ms to land
  // (the peer waits for this one at the cluster barrier).
  if (threadIdx.x == 0 && *abort_flag)
    for (int q = 0; q < 2000; ++q) __nanosleep(1000);
  if (KIND == TR_DW && args.early) pdl_wait();
  cluster_sync_all();   // no CTA leaves while its peer may still signal it or read its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

}  // namespace moe
