// Backward pass of the experts' gated feed-forward block, as grouped GEMMs on tcgen05.
//
// Forward (per expert e and row r): g = x Wg^T + bg, u = x Wu^T + bu, h = f(g') u',
// y = h Wd^T + bd, with f(a) = a s(alpha a), s the sigmoid, and g' = clip(g, gate_lo, L),
// u' = clip(u, -L, L) (SiLU: no clips, alpha = 1).  Given dy:
//   DH  dh = dy Wd;  dg = dh u' f'(g') [gate_lo <= g <= L],  du = dh f(g') [|u| <= L],
//       f'(a) = s + alpha a s (1 - s)                                  -> dgu [R, 2, F]
//   DX  dx = dg Wg + du Wu
//   DW  dWd = dy^T h, dWg = dg^T x, dWu = du^T x over each expert's rows (zero where it has
//       none), and the bias gradients, the column sums of dy, dg, du over the same rows.
//
// Operand orders: the weights are stored [N, K] for the forward pass, so here the reduction
// runs along their slow dimension: B is "MN-major" (N contiguous), which the tensor core
// reads directly (instruction descriptor transpose bits, 128-byte swizzle: 64 N-elements x
// 8 K-rows per 1024-byte atom).  DW has both operands MN-major, its K running over rows.
// TMA brings [64 K-rows x 64 elements] boxes; no operand is transposed in memory.
//
// DW's K range is an expert's row range, of any length.  Its last block may reach into
// rows of the next expert: whole 16-row MMA steps past the end are not issued, and the
// rows past the end of the last step are overwritten with zeros in shared memory, in both
// operands, before the MMA reads them (zeroing one would let an infinity or a NaN of a
// neighbouring expert through as 0 * inf).
//
// Bias gradients: for the tiles of the first column block, which DW keeps at most 192
// columns wide, the issuer adds one N = 16 MMA a step whose B operand is a tile of ones, into
// TMEM columns that the tile leaves free: the sums cost no further pass over dy and dgu.
//
// dg and du are rounded to bf16 between DH and the two products that read them (they are
// tensor-core operands); all sums are fp32.
//
// Tile 128 x (64 to 256 columns): the columns are split into blocks of 1 to 4 boxes of 64,
// as even as that allows (2880 = 3 x 192 + 9 x 256), so that every box row is one 128-byte
// line of L2 -- evener blocks of 240 columns start between lines, and each box row then
// takes two L2 requests.  Four 64-deep stages, two accumulator buffers; roles as in
// grouped_gemm.cuh.  DH and DX walk (expert, row block, column block) tiles of the ragged
// rows, DW walks (matrix, expert, 128-row block, column block) tiles of the gradients.
#pragma once

#include "grouped_gemm_mx4.cuh"

namespace moe {

enum BwdKind : int { BWD_DH = 0, BWD_DX = 1, BWD_DW = 2 };

constexpr int kBwdBK = 64;           // K per stage
constexpr int kBwdStages = 4;
constexpr int kBwdBox = 64 * 128;    // bytes of a [64 K-rows x 64 elements] box
constexpr int kBwdOnesCol = 192;     // TMEM column of the bias sums inside an accumulator buffer

constexpr int kBwdThreads = 384;
constexpr int kBwdEpiWarps = 8;
constexpr int kBwdSched = 4;         // tiles the scheduler is ahead

template <int KIND>
struct BwdLayout {
  static constexpr int A_BYTES = 2 * kBwdBox;
  static constexpr int B_BYTES = 4 * kBwdBox;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int ONES = KIND == BWD_DW ? 2048 : 0;                     // 16 rows x 128 B of bf16 ones
  // epilogue staging of a warp: 32 rows of 64 B + 16 B;  DH: of g and u, 32 B + 16 B each
  static constexpr int STAGING_WARP = KIND == BWD_DH ? 2 * 32 * 48 : 32 * 80;
  static constexpr int STAGING = kBwdEpiWarps * STAGING_WARP;
  static constexpr int EXTRA = 1024 + 3072;
  static constexpr int SMEM = kBwdStages * STAGE_BYTES + ONES + STAGING + EXTRA;
  static_assert(SMEM <= 232448, "shared memory budget");
};

// Column blocks of N columns: 1 to 4 boxes of 64 each (3 at most for the first one if
// `spare`), differing by at most one box, the narrower ones first.
__host__ __device__ constexpr int bwd_col_blocks(int N, bool spare) {
  return ((N + 63) / 64 + (spare ? 1 : 0) + 3) / 4;
}
struct BwdCols {
  int first, boxes;   // first column, number of 64-column boxes
};
__host__ __device__ inline BwdCols bwd_cols(int N, int blocks, int j) {
  const int n64 = (N + 63) / 64;
  const int q = n64 / blocks, narrow = blocks - n64 % blocks;
  return BwdCols{64 * (j * q + (j > narrow ? j - narrow : 0)), q + (j >= narrow ? 1 : 0)};
}

// One product of a launch.  DH: A = dy, B0 = Wd.  DX: A = dgu (halves), B0 = Wg, B1 = Wu.
// DW: A, B0 = the two row-major operands whose rows are summed over.
struct BwdJob {
  CUtensorMap a, b0, b1;
  void* out;
  void* bias_out;   // DW: [G, m] column sums of A, or null
  int m, n;         // DW: rows and columns of the gradient;  DH, DX: n = columns of the output
  int nt;           // column blocks
};

template <int KIND>
struct BwdArgs {
  BwdJob job[KIND == BWD_DW ? 3 : 1];
  int num_jobs;
  const int32_t* group_off;   // [G+1]
  int num_groups;
  int m_total;                // R
  int k_dim;                  // DH: D;  DX: F
  const __nv_bfloat16* gu;    // DH: [R, 2, F]
  float limit, alpha, gate_lo;
  unsigned long long wait_limit_ns;
};

// K-rows x elements operand ("MN-major"), 128-byte swizzle: 64-element blocks kBwdBox bytes
// apart (leading offset), 8-row groups 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kBwdBox >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Derivatives of h = f(clip(g)) clip(u) times dh.  The clips pass the gradient at their ends.
__device__ __forceinline__ void act_grad(float dh, float g, float u, float limit, float alpha, float gate_lo,
                                         float& dg, float& du) {
  const float gc = fminf(fmaxf(g, gate_lo), limit), uc = fminf(fmaxf(u, -limit), limit);
  const float s = __fdividef(1.0f, 1.0f + __expf(-alpha * gc));
  const float f = gc * s;
  dg = (g >= gate_lo && g <= limit) ? dh * uc * (s + alpha * f * (1.0f - s)) : 0.0f;
  du = (u >= -limit && u <= limit) ? dh * f : 0.0f;
}

struct BwdTile {
  int job, g;           // job -1: no more tiles
  int m0, m_end;        // DW: rows of the gradient;  DH, DX: rows of A
  int n0, boxes;        // first column, 64-column boxes
  int kb;               // 64-deep K blocks
  int r0, rows;         // DW: the expert's rows
};

template <int KIND>
__device__ __forceinline__ BwdTile bwd_tile(int i, const int* tile_off, const int* goff, const BwdArgs<KIND>& a) {
  BwdTile t;
  t.job = 0;
  int nb;
  if constexpr (KIND == BWD_DW) {
    int mt = 0;
    for (;; ++t.job) {
      mt = (a.job[t.job].m + kBM - 1) / kBM;
      const int n = a.num_groups * mt * a.job[t.job].nt;
      if (i < n || t.job + 1 == a.num_jobs) break;
      i -= n;
    }
    const int nt = a.job[t.job].nt;
    t.g = i / (mt * nt);
    i -= t.g * mt * nt;
    // bands of kGroupBand row blocks, the row block fastest: neighbours share operand rows in L2
    const int band = i / (kGroupBand * nt);
    const int rem = i - band * kGroupBand * nt;
    const int rows = min(kGroupBand, mt - band * kGroupBand);
    nb = rem / rows;
    t.m0 = (band * kGroupBand + rem - nb * rows) * kBM;
    t.m_end = a.job[t.job].m;
  } else {
    const TileInfo ti = decode_tile(i, tile_off, goff, a.num_groups, a.job[0].nt, 1);
    t.g = ti.g;
    t.m0 = ti.m0;
    t.m_end = ti.m_end;
    nb = ti.n0;
  }
  const BwdCols c = bwd_cols(a.job[t.job].n, a.job[t.job].nt, nb);
  t.n0 = c.first;
  t.boxes = c.boxes;
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
__global__ void __launch_bounds__(kBwdThreads, 1) ffn_backward_kernel(const __grid_constant__ BwdArgs<KIND> args) {
  pdl_enter();
  using LY = BwdLayout<KIND>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ones = smem + kBwdStages * LY::STAGE_BYTES;
  uint8_t* staging = ones + LY::ONES;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + LY::STAGING);
  uint64_t* ready = full + kBwdStages;          // DW: the blanker has seen the stage
  uint64_t* empty = ready + kBwdStages;
  uint64_t* tfull = empty + kBwdStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* sfull = tempty + 2;                 // scheduler ring
  uint64_t* sempty = sfull + kBwdSched;
  uint64_t* drain = sempty + kBwdSched;
  BwdTile* ring = reinterpret_cast<BwdTile*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring + kBwdSched);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* never_flag = abort_flag + 1;
  int* tile_off = never_flag + 1;              // [G+1]
  int* goff = tile_off + (kMaxGroups + 1);     // [G+1]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = args.num_groups;
  const uint64_t lim = args.wait_limit_ns;
  constexpr int kConsumers = 2 + kBwdEpiWarps + (KIND == BWD_DW ? 1 : 0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kBwdStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&ready[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 32 * kBwdEpiWarps);
    }
    for (int q = 0; q < kBwdSched; ++q) {
      mbar_init(&sfull[q], 1);
      mbar_init(&sempty[q], kConsumers);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    mx4_group_table(args.group_off, G, args.m_total, goff, tile_off);
    if (lane < args.num_jobs) {
      tma_prefetch_desc(&args.job[lane].a);
      tma_prefetch_desc(&args.job[lane].b0);
      if (KIND == BWD_DX) tma_prefetch_desc(&args.job[lane].b1);
    }
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  } else if (KIND == BWD_DW && warp < 6) {
    for (int i = threadIdx.x - 64; i < LY::ONES / 4; i += 128) reinterpret_cast<uint32_t*>(ones)[i] = 0x3F803F80u;
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int KB1 = (args.k_dim + kBwdBK - 1) / kBwdBK;   // DH, DX: K blocks (of one half)

  // The next tile from the scheduler's ring; false when a wait gave up.  One thread, or a
  // whole warp (which then agrees on the answer).
  auto next_tile = [&](int n, BwdTile& t, bool whole_warp) {
    const int q = n % kBwdSched;
    bool got = mbar_wait(&sfull[q], (n / kBwdSched) & 1, abort_flag, lim);
    if (whole_warp) got = __all_sync(0xffffffffu, got);
    if (!got) return false;
    t = ring[q];
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(&sempty[q]);
    return true;
  };
  bool ok = true;

  if (warp == 2 + kBwdEpiWarps) {
    // ------------------------------------------------------------ scheduler
    if (lane == 0) {
      int total = 0;
      if constexpr (KIND == BWD_DW) {
        for (int j = 0; j < args.num_jobs; ++j) total += G * ((args.job[j].m + kBM - 1) / kBM) * args.job[j].nt;
      } else {
        total = tile_off[G] * args.job[0].nt;
      }
      int n = 0;
      for (int i = blockIdx.x;; i += gridDim.x, ++n) {
        BwdTile t;
        t.job = -1;
        if (i < total) {
          t = bwd_tile<KIND>(i, tile_off, goff, args);
          t.r0 = goff[t.g];
          t.rows = max(0, goff[t.g + 1] - t.r0);
          t.kb = KIND == BWD_DW ? (t.rows + kBwdBK - 1) / kBwdBK : KIND == BWD_DX ? 2 * KB1 : KB1;
        }
        const int q = n % kBwdSched;
        if (!mbar_wait(&sempty[q], ((n / kBwdSched) & 1) ^ 1, abort_flag, lim)) { ok = false; break; }
        ring[q] = t;
        mbar_arrive(&sfull[q]);
        if (i >= total) break;
      }
      if (!ok) {
        *abort_flag = 1;
        flag_error(DEVERR_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      BwdTile ti;
      for (int n = 0;; ++n) {
        if (!next_tile(n, ti, false)) { ok = false; break; }
        if (ti.job < 0) break;
        const BwdJob& jb = args.job[ti.job];
        for (int kb = 0; kb < ti.kb; ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, lim)) { ok = false; break; }
          mbar_arrive_expect_tx(&full[s], LY::A_BYTES + ti.boxes * kBwdBox);
          uint8_t* sa = smem + s * LY::STAGE_BYTES;
          uint8_t* sb = sa + LY::A_BYTES;
          if constexpr (KIND == BWD_DW) {
            const int r = ti.r0 + kb * kBwdBK;
            for (int q = 0; q < ti.boxes; ++q) tma_load_2d(sb + q * kBwdBox, &jb.b0, &full[s], ti.n0 + 64 * q, r);
            for (int q = 0; q < 2; ++q) tma_load_2d(sa + q * kBwdBox, &jb.a, &full[s], ti.m0 + 64 * q, r);
          } else {
            const int half = (KIND == BWD_DX && kb >= KB1) ? 1 : 0;
            const int k0 = (kb - half * KB1) * kBwdBK;
            const CUtensorMap* tb = half ? &jb.b1 : &jb.b0;
            for (int q = 0; q < ti.boxes; ++q) tma_load_3d(sb + q * kBwdBox, tb, &full[s], ti.n0 + 64 * q, k0, ti.g);
            if (KIND == BWD_DX) tma_load_3d(sa, &jb.a, &full[s], k0, half, ti.m0);
            else tma_load_2d(sa, &jb.a, &full[s], k0, ti.m0);
          }
          issued |= 1u << s;
          issued_par = (issued_par & ~(1u << s)) | (ph << s);
          if (++s == kBwdStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
      }
      if (!ok) {
        *abort_flag = 1;
        flag_error(DEVERR_TIMEOUT);
      }
      for (int q = 0; q < kBwdStages; ++q)
        if ((issued >> q) & 1u)
          if (!mbar_wait(&full[q], (issued_par >> q) & 1u, never_flag, kDrainLimitNs)) flag_error(DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // One thread issues every MMA (128 cycles each at 256 columns): descriptors are made
    // once and stepped by additions (built per MMA they took 264 cycles an MMA).
    if (lane == 0) {
      const uint32_t s_addr = smem_u32(smem);
      const uint64_t a_desc = KIND == BWD_DW ? sw128_mnmajor_desc(s_addr) : sw128_kmajor_desc(s_addr);
      const uint64_t b_desc = sw128_mnmajor_desc(s_addr + LY::A_BYTES);
      const uint64_t ones_desc = sw128_kmajor_desc(smem_u32(ones));
      constexpr int kAStep = KIND == BWD_DW ? 2048 / 16 : 32 / 16;   // of 16 K elements
      const uint32_t idesc_ones = make_idesc(kBM, 16, 1u) | (1u << 15);
      uint64_t* loaded = KIND == BWD_DW ? ready : full;
      int s = 0;
      uint32_t ph = 0;
      BwdTile ti;
      for (int n = 0;; ++n) {
        if (!next_tile(n, ti, false)) { ok = false; break; }
        if (ti.job < 0) break;
        const uint32_t idesc = make_idesc(kBM, 64 * ti.boxes, 1u) | (1u << 16) | (KIND == BWD_DW ? 1u << 15 : 0u);
        const bool sums = KIND == BWD_DW && ti.n0 == 0 && args.job[ti.job].bias_out != nullptr;
        const int acc = n & 1;
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kAccStride);
        if (!mbar_wait(&tempty[acc], ((n >> 1) & 1) ^ 1u, abort_flag, lim)) { ok = false; break; }
        tc_fence_after();
        for (int kb = 0; kb < ti.kb; ++kb) {
          if (!mbar_wait(&loaded[s], ph, abort_flag, lim)) { ok = false; break; }
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>(s * (LY::STAGE_BYTES >> 4));
          const uint64_t ad = a_desc + so, bd = b_desc + so;
          const int steps = KIND == BWD_DW ? min(kBwdBK / 16, (ti.rows - kb * kBwdBK + 15) / 16) : kBwdBK / 16;
          if (steps == kBwdBK / 16 && !sums) {
#pragma unroll
            for (int kk = 0; kk < kBwdBK / 16; ++kk)
              tc_mma<false>(d_tmem, ad + kk * kAStep, bd + kk * 128, idesc, (kb | kk) != 0 ? 1u : 0u);
          } else {
            for (int kk = 0; kk < steps; ++kk) {
              const uint32_t accumulate = (kb | kk) != 0 ? 1u : 0u;
              tc_mma<false>(d_tmem, ad + kk * kAStep, bd + kk * 128, idesc, accumulate);
              if (sums) tc_mma<false>(d_tmem + kBwdOnesCol, ad + kk * kAStep, ones_desc, idesc_ones, accumulate);
            }
          }
          tc_commit(&empty[s]);
          if (++s == kBwdStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        tc_commit(&tfull[acc]);
      }
      if (!ok) {
        *abort_flag = 1;
        flag_error(DEVERR_TIMEOUT);
      }
      tc_commit(drain);
      if (!mbar_wait(drain, 0, never_flag, kDrainLimitNs)) flag_error(DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp < 2 + kBwdEpiWarps) {
    // ------------------------------------------------------------ epilogue (warps 2..9)
    // Two warps share a TMEM lane quarter and take its column chunks in turn.
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stage = staging + (warp - 2) * LY::STAGING_WARP;
    BwdTile ti;
    for (int n = 0;; ++n) {
      if (!next_tile(n, ti, true)) { ok = false; break; }
      if (ti.job < 0) break;
      const BwdJob& jb = args.job[ti.job];
      const int acc = n & 1;
      const int row0 = ti.m0 + quarter * 32;
      const int rows = ti.m_end - row0;
      const int width = min(64 * ti.boxes, jb.n - ti.n0);
      const uint32_t tbase =
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * kAccStride);
      if constexpr (KIND == BWD_DH) {
        // 16 columns at a time: g and u come in 32-byte runs of rows (the next chunk's while
        // this one is computed, the first before the accumulator is complete), turn into row
        // order through the staging area, and dg and du leave the same way
        const int F = jb.n;
        const int r2 = lane >> 1, piece = lane & 1;
        const __nv_bfloat16* gu = args.gu + static_cast<size_t>(row0) * 2 * F + ti.n0 + piece * 8;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(jb.out) + static_cast<size_t>(row0) * 2 * F + ti.n0 + piece * 8;
        uint8_t* su = stage + 32 * 48;         // u's half of the warp's staging
        uint4 pre[4];
        auto fetch = [&](int c) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int r = p * 16 + r2;
            pre[p] = pre[2 + p] = make_uint4(0, 0, 0, 0);
            if (c < width && r < rows) {
              pre[p] = *reinterpret_cast<const uint4*>(gu + static_cast<size_t>(r) * 2 * F + c);
              pre[2 + p] = *reinterpret_cast<const uint4*>(gu + static_cast<size_t>(r) * 2 * F + F + c);
            }
          }
        };
        fetch(16 * half);
        if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], (n >> 1) & 1, abort_flag, lim))) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int c = 16 * half; c < width; c += 32) {
          __syncwarp();
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            *reinterpret_cast<uint4*>(stage + (p * 16 + r2) * 48 + piece * 16) = pre[p];
            *reinterpret_cast<uint4*>(su + (p * 16 + r2) * 48 + piece * 16) = pre[2 + p];
          }
          __syncwarp();
          fetch(c + 32);
          float v[16];
          tmem_ld8(tbase + c, *reinterpret_cast<float(*)[8]>(v));
          tmem_ld8(tbase + c + 8, *reinterpret_cast<float(*)[8]>(v + 8));
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            float gv[8], uv[8], dg[8], du[8];
            __nv_bfloat16* pg = reinterpret_cast<__nv_bfloat16*>(stage + lane * 48 + j * 2);
            __nv_bfloat16* pu = reinterpret_cast<__nv_bfloat16*>(su + lane * 48 + j * 2);
            load8<__nv_bfloat16>(pg, gv);
            load8<__nv_bfloat16>(pu, uv);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              act_grad(v[j + q], gv[q], uv[q], args.limit, args.alpha, args.gate_lo, dg[q], du[q]);
            store8<__nv_bfloat16>(pg, dg);
            store8<__nv_bfloat16>(pu, du);
          }
          __syncwarp();
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int r = p * 16 + r2;
            if (r < rows) {
              *reinterpret_cast<uint4*>(out + static_cast<size_t>(r) * 2 * F + c) =
                  *reinterpret_cast<const uint4*>(stage + r * 48 + piece * 16);
              *reinterpret_cast<uint4*>(out + static_cast<size_t>(r) * 2 * F + F + c) =
                  *reinterpret_cast<const uint4*>(su + r * 48 + piece * 16);
            }
          }
        }
      } else {
        constexpr int COLS = 64 / static_cast<int>(sizeof(OutT));
        if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], (n >> 1) & 1, abort_flag, lim))) { ok = false; break; }
        tc_fence_after();
        const bool none = KIND == BWD_DW && ti.rows == 0;   // the gradient is zero
        const size_t row_base = KIND == BWD_DW ? static_cast<size_t>(ti.g) * jb.m : 0;
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
        if (KIND == BWD_DW && half == 0 && ti.n0 == 0 && jb.bias_out != nullptr) {
          float b[8];
          tmem_ld8(tbase + kBwdOnesCol, b);
          tmem_ld_wait();
          if (lane < rows) {
            const float sum = none ? 0.0f : b[0];
            OutT* bo = static_cast<OutT*>(jb.bias_out) + row_base + row0 + lane;
            if constexpr (sizeof(OutT) == 2) *bo = __float2bfloat16_rn(sum);
            else *bo = sum;
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&tempty[acc]);
    }
    if (!ok) {
      *abort_flag = 1;
      flag_error(DEVERR_TIMEOUT);
    }
  } else if (KIND == BWD_DW) {
    // ------------------------------------------------------------ blanker
    // Passes every loaded stage on to the issuer, after blanking the rows between the end
    // of the expert and the end of the last 16-row step.
    int s = 0;
    uint32_t ph = 0;
    BwdTile ti;
    for (int n = 0; ok; ++n) {
      if (!next_tile(n, ti, true)) { ok = false; break; }
      if (ti.job < 0) break;
      for (int kb = 0; kb < ti.kb; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[s], ph, abort_flag, lim))) { ok = false; break; }
        const int valid = ti.rows - kb * kBwdBK;
        if (valid < kBwdBK && (valid & 15) != 0) {
          uint8_t* st = smem + s * LY::STAGE_BYTES + valid * 128;
          const int pieces = (16 - (valid & 15)) * 8;
          for (int box = 0; box < 2 + ti.boxes; ++box)
            for (int q = lane; q < pieces; q += 32)
              *reinterpret_cast<uint4*>(st + box * kBwdBox + q * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();   // read by the tensor core (async proxy)
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ready[s]);
        if (++s == kBwdStages) { s = 0; ph ^= 1u; }
      }
    }
    if (!ok) {
      *abort_flag = 1;
      flag_error(DEVERR_TIMEOUT);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// fp32 layers: the same three products in fp32 FMA (no TF32), 64 x 64 tiles
// ---------------------------------------------------------------------------
struct SimtBwdArgs {
  const int32_t* group_off;
  int num_groups, m_total;
  int m, n, k;                // DH, DX: n, k;  DW: gradient rows m, columns n
  const float *a, *b0, *b1;
  int lda, ldb;               // DW: row strides of A and B0
  const float* gu;            // DH: [R, 2, F]
  float limit, alpha, gate_lo;
  float *out, *bias_out;
};

template <int KIND>
__global__ void __launch_bounds__(256) simt_backward_kernel(const SimtBwdArgs p) {
  pdl_enter();
  __shared__ float sa[kSimtBK][kSimtBM + 4];
  __shared__ float sb[kSimtBK][kSimtBN + 4];
  __shared__ int goff[kMaxGroups + 2];
  __shared__ int toff[kMaxGroups + 2];
  const int G = p.num_groups;
  for (int g = threadIdx.x; g <= G; g += blockDim.x) {
    const int v = p.group_off[g];
    if (v < 0 || v > p.m_total) flag_error(DEVERR_BOUNDS);
    goff[g] = min(max(v, 0), p.m_total);
  }
  __syncthreads();
  const int n0 = blockIdx.x * kSimtBN;
  int g, m0, m_end, r0 = 0, K = p.k;
  if constexpr (KIND == BWD_DW) {
    g = blockIdx.z;
    m0 = blockIdx.y * kSimtBM;
    m_end = p.m;
    r0 = goff[g];
    K = max(0, goff[g + 1] - r0);
  } else {
    if (threadIdx.x == 0) {
      toff[0] = 0;
      for (int q = 0; q < G; ++q) toff[q + 1] = toff[q] + max(0, (goff[q + 1] - goff[q] + kSimtBM - 1) / kSimtBM);
    }
    __syncthreads();
    const int mt = blockIdx.y;
    if (mt >= toff[G]) return;
    g = 0;
    while (toff[g + 1] <= mt) ++g;
    m0 = goff[g] + (mt - toff[g]) * kSimtBM;
    m_end = goff[g + 1];
  }
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {}, sum[4] = {};
  const int KT = KIND == BWD_DX ? 2 * K : K;
  for (int k0 = 0; k0 < KT; k0 += kSimtBK) {
    for (int i = threadIdx.x; i < kSimtBM * kSimtBK; i += 256) {
      if constexpr (KIND == BWD_DW) {
        const int kk = i / kSimtBM, r = i % kSimtBM, col = k0 + kk;
        sa[kk][r] = (m0 + r < m_end && col < K) ? p.a[static_cast<size_t>(r0 + col) * p.lda + m0 + r] : 0.0f;
        sb[kk][r] = (n0 + r < p.n && col < K) ? p.b0[static_cast<size_t>(r0 + col) * p.ldb + n0 + r] : 0.0f;
      } else {
        {
          const int r = i / kSimtBK, kk = i % kSimtBK, row = m0 + r, col = k0 + kk;
          sa[kk][r] = (row < m_end && col < KT) ? p.a[static_cast<size_t>(row) * KT + col] : 0.0f;
        }
        const int kk = i / kSimtBN, c = i % kSimtBN, col = k0 + kk;
        const bool second = KIND == BWD_DX && col >= K;
        const float* b = second ? p.b1 : p.b0;
        const int kr = second ? col - K : col;
        sb[kk][c] = (n0 + c < p.n && col < KT) ? b[(static_cast<size_t>(g) * K + kr) * p.n + n0 + c] : 0.0f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kSimtBK; ++kk) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = sa[kk][ty * 4 + i];
        b[i] = sb[kk][tx * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (KIND == BWD_DW) sum[i] += a[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = m0 + ty * 4 + i;
    if (row >= m_end) continue;
    const size_t orow = KIND == BWD_DW ? static_cast<size_t>(g) * p.m + row : row;
    if (KIND == BWD_DW && p.bias_out != nullptr && n0 == 0 && tx == 0) p.bias_out[orow] = sum[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (n >= p.n) continue;
      if constexpr (KIND == BWD_DH) {
        const float gv = p.gu[orow * 2 * p.n + n], uv = p.gu[orow * 2 * p.n + p.n + n];
        const float gc = fminf(fmaxf(gv, p.gate_lo), p.limit), uc = fminf(fmaxf(uv, -p.limit), p.limit);
        const float s = 1.0f / (1.0f + expf(-p.alpha * gc)), f = gc * s, dh = acc[i][j];
        p.out[orow * 2 * p.n + n] =
            (gv >= p.gate_lo && gv <= p.limit) ? dh * uc * (s + p.alpha * f * (1.0f - s)) : 0.0f;
        p.out[orow * 2 * p.n + p.n + n] = (uv >= -p.limit && uv <= p.limit) ? dh * f : 0.0f;
      } else {
        p.out[orow * p.n + n] = acc[i][j];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// combine, backward: dy_perm[row(t, j)] = w[t, j] dy[t], dw[t, j] = dy[t] . y_perm[row(t, j)]
// ---------------------------------------------------------------------------
// One CTA a token: dy[t] is read once and meets its k rows.  Bound by memory: (1 + 2 k) D
// elements a token.  The dot products are summed per thread, then over the warp and the
// CTA's warps in a fixed order.
constexpr int kCombineBwdThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kCombineBwdThreads)
    combine_backward_kernel(const T* __restrict__ dy, const T* __restrict__ y_perm,
                            const int32_t* __restrict__ row_of_slot, const float* __restrict__ w, int Tn, int k, int D,
                            T* __restrict__ dy_perm, float* __restrict__ dw) {
  pdl_enter();
  __shared__ float part[kCombineBwdThreads / 32][8];
  const int t = blockIdx.x;
  const int R = Tn * k;
  int row[8];
  float wt[8], acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    row[j] = -1;
    acc[j] = wt[j] = 0.0f;
    if (j < k) {
      row[j] = row_of_slot[static_cast<size_t>(t) * k + j];
      wt[j] = w[static_cast<size_t>(t) * k + j];
      if (row[j] < 0 || row[j] >= R) {
        if (threadIdx.x == 0) flag_error(DEVERR_BOUNDS);
        row[j] = -1;
      }
    }
  }
  for (int c = threadIdx.x * 8; c < D; c += kCombineBwdThreads * 8) {
    float d[8];
    load8<T>(dy + static_cast<size_t>(t) * D + c, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (row[j] < 0) continue;
      float y[8], o[8];
      load8<T>(y_perm + static_cast<size_t>(row[j]) * D + c, y);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        acc[j] = fmaf(d[q], y[q], acc[j]);
        o[q] = wt[j] * d[q];
      }
      store8<T>(dy_perm + static_cast<size_t>(row[j]) * D + c, o);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= k) break;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][j] = acc[j];
  }
  __syncthreads();
  if (threadIdx.x < k) {
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < kCombineBwdThreads / 32; ++q) s += part[q][threadIdx.x];
    dw[static_cast<size_t>(t) * k + threadIdx.x] = s;
  }
}

}  // namespace moe
