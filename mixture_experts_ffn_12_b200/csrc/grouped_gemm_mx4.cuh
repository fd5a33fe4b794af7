// Grouped product of MXFP4 rows with MXFP4 weights on the block-scaled tensor cores:
//   out[r, n] = sum_k A[r, k] * W_g[n, k] + b_g[n]    for the rows r of group g
// with both operands E2M1 with one E8M0 scale per 32 elements along K
// (tcgen05.mma kind::mxf4, block scales applied by the tensor core, fp32 accumulators).
//
// At four times the bf16 rate the tensor core outruns what the L2 delivers to an SM, and for
// few rows the weights are a plain stream from HBM, so the tile is chosen for its bytes:
// CTA pairs (cta_group::2) with the weights in M (256 output columns a pair, 128 a CTA) and
// the group's rows in N, at most 192, half of them staged by each CTA: 31 KB a stage of 256 K
// where a CTA alone would take 43 KB for the same MMA time, and a group's last tile only as
// wide as its rows (a step of 16), so a decode batch pays for its weights only.  Why 192:
// two accumulator buffers (a tile's epilogue overlaps the next tile's MMAs) leave 2 x 64 of
// the 512 TMEM columns, and the scales of a stage take 24; 2 x 256 columns would leave none.
//
// Stage = 256 elements of K = one 128-byte swizzled row of packed codes (plain byte boxes:
// the mxf4 MMA reads 4-bit operands packed); the scales come as ready-made 512-byte chunks
// (mxfp4_quant.cuh) by TMA, tcgen05.cp brings them to TMEM, four MMAs of K = 64.
//
// Roles (384 threads a CTA): warp 0 producer of the weights, warp 11 of the rows (weights are
// on their way while the quantizer before this kernel still writes the rows: decode experts
// 30.5 -> 27.4 us); warp 1 TMEM and, in the leader, the MMA issuer; warps 2..9 epilogue;
// warp 10 the tile scheduler.  Waits bounded and the closing cluster barrier as in
// grouped_gemm_pair.cuh.
//
// Measured, 32 groups, N = K = 2880: 16384 rows 78 us (3.5 PFLOP/s, tensor pipe busy 50 % of
// the time, 237 MB from and to HBM), 128 rows 24 us (5.9 TB/s of weights: HBM).  At 16384 rows one
// launch alone, at 1.6 to 1.9 GHz, is not bound by power: at the tensor pipe's nominal rate a
// stage's 31 KB a CTA in 384 cycles would ask some 21 TB/s of the L2, more than it was seen to give
// (15.5), and a wider tile has no room in TMEM beside two scale sets.  Single CTAs with the rows
// in M took 125 and 41 us.
#pragma once

#include "mxfp4_quant.cuh"

namespace moe {

constexpr int kMx4BK = 256;       // K elements per stage
constexpr int kMx4Stages = 7;
constexpr int kMx4BM = 256;       // output columns of a pair's tile
constexpr int kMx4Threads = 384;
constexpr int kMx4EpiWarps = 8;
constexpr int kMx4Sched = 4;      // tiles the scheduler is ahead

struct Mx4Layout {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = kMx4Rows / 2 * 128;
  static constexpr int SFA_BYTES = 1024;          // 2 chunks of 128 K
  static constexpr int SFB_BYTES = 2048;          // 2 chunks of 128 K x 2 of 128 rows
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int EXTRA = 4096;   // alignment to 1024, barriers and tables
  static constexpr int SMEM = kMx4Stages * STAGE_BYTES + EXTRA;
  // TMEM: accumulators at columns 0 and 256; scales of even / odd stages behind them:
  // weights 2 chunks x 4 columns, then rows 2 chunks x 2 x 4 columns
  static constexpr int SF_COL = kMx4Rows;
  static constexpr int SFB_COL = 8;
  static_assert(STAGE_BYTES % 1024 == 0, "stages keep the swizzle alignment");
  static_assert(SF_COL + 24 <= kAccStride, "scales fit behind an accumulator");
  static_assert(SMEM <= 232448, "shared memory budget");
};

// Instruction descriptor of kind::mxf4.block_scale: A and B E2M1 (1), E8M0 scales, K-major,
// K = 64; the scale-factor ids (0 or 2) pick the byte pair of each TMEM scale column.
__host__ __device__ constexpr uint32_t make_idesc_mx4(int M, int N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((static_cast<uint32_t>(N) >> 3) << 17) | (1u << 23) |
         ((static_cast<uint32_t>(M) >> 4) << 24) | (sf_id << 29);
}

__device__ __forceinline__ void tc_mma_mx4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

// tc_cp_sf in both CTAs of the pair, each from its own shared memory to its own TMEM.
__device__ __forceinline__ void tc_cp_sf_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

struct Mx4Args {
  CUtensorMap w;              // weight codes [G][n_out][K/2] bytes, boxes of 128 rows
  CUtensorMap x[3];           // row codes [m_total][K/2] bytes, boxes of 32, 64, 96 rows
  const int32_t* group_off;   // [G+1]; null: one group of m_total rows
  int num_groups;
  int m_total;
  int n_out;
  int k_dim;
  CUtensorMap sw, sx;         // scale tiles of W, [G][ceil(n_out / 128)] row blocks, and of the row
                              //   tiles: runs of 1024 and 2048 bytes, seen as rows of 256 B
  int row_tiles;              // number of row tiles (clamp for offsets that are not ascending)
  const __nv_bfloat16* bias;  // [G, n_out] or null
  void* out;                  // [m_total, n_out]
  unsigned long long wait_limit_ns;
};

struct Mx4Tile {
  int g;                // -1: no more tiles
  int m0;               // first output column
  int r0, rows, n;      // first row, rows, MMA N
  int xt;               // row tile (of the scales)
};

// Waits for the copies counted on `stages` barriers (bit q of `issued`: some on barrier q, in the
// phase that bit q of `par` says), also after a wait that gave up: a copy must not land in
// shared memory that the CTA has left.  kDrainLimitNs from t0 on for all of them, since a
// stage whose other copies were never issued does not complete.
__device__ __forceinline__ bool wait_landed(uint64_t* bars, int stages, uint32_t issued, uint32_t par,
                                            volatile int* never, uint64_t t0) {
  bool all = true;
  for (int q = 0; q < stages; ++q) {
    if (!((issued >> q) & 1u)) continue;
    const uint64_t gone = global_timer_ns() - t0;
    all &= mbar_wait(&bars[q], (par >> q) & 1u, never, gone < kDrainLimitNs ? kDrainLimitNs - gone : 1);
  }
  return all;
}

template <typename OutT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMx4Threads, 1)
    grouped_gemm_mx4_kernel(const __grid_constant__ Mx4Args args) {
  pdl_launch_dependents();
  using LY = Mx4Layout;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kMx4Stages * LY::STAGE_BYTES);   // leader's: both CTAs' stage
  uint64_t* empty = full + kMx4Stages;
  uint64_t* tfull = empty + kMx4Stages;
  uint64_t* tempty = tfull + 2;                // leader's
  uint64_t* rfull = tempty + 2;                // scheduler ring
  uint64_t* rempty = rfull + kMx4Sched;
  uint64_t* drain = rempty + kMx4Sched;
  Mx4Tile* ring = reinterpret_cast<Mx4Tile*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring + kMx4Sched);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* never_flag = abort_flag + 1;
  int* tile_off = never_flag + 1;              // [G+1] row tiles before each group
  int* goff = tile_off + (kMaxGroups + 1);     // [G+1]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());   // 0 = leader (issues the MMAs)
  const int G = args.group_off == nullptr ? 1 : args.num_groups;
  const int MT = (args.n_out + kMx4BM - 1) / kMx4BM;
  const int KB = (args.k_dim + kMx4BK - 1) / kMx4BK;
  const uint64_t lim = args.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMx4Stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kMx4EpiWarps);
    }
    for (int q = 0; q < kMx4Sched; ++q) {
      mbar_init(&rfull[q], 1);
      mbar_init(&rempty[q], 2 + (rank == 0 ? 1 : 0) + kMx4EpiWarps);   // who reads a tile
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&args.w);
      tma_prefetch_desc(&args.x[0]);
      tma_prefetch_desc(&args.x[2]);
      tma_prefetch_desc(&args.sw);
      tma_prefetch_desc(&args.sx);
    }
  } else if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  // No wait for the quantizer here: it started after every earlier kernel was complete, so the
  // offsets and the weights are in place; only the producer of the rows waits for it.
  if (warp == 0) group_table(args.group_off, G, args.m_total, kMx4Rows, goff, tile_off);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // both CTAs' barriers are initialised before any signal between them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // The next tile from the scheduler's ring; false when a wait gave up.  For a whole
  // warp, which agrees on the answer.
  auto next_tile = [&](int n, Mx4Tile& t) {
    const int q = n % kMx4Sched;
    if (!__all_sync(0xffffffffu, mbar_wait(&rfull[q], (n / kMx4Sched) & 1, abort_flag, lim))) return false;
    t = ring[q];
    __syncwarp();
    if (lane == 0) mbar_arrive(&rempty[q]);
    return true;
  };
  // A tile that the whole warp has read, as values the compiler knows to be the same in every lane.
  auto uniform = [](Mx4Tile& t) {
    t.g = __shfl_sync(0xffffffffu, t.g, 0);
    t.m0 = __shfl_sync(0xffffffffu, t.m0, 0);
    t.r0 = __shfl_sync(0xffffffffu, t.r0, 0);
    t.rows = __shfl_sync(0xffffffffu, t.rows, 0);
    t.n = __shfl_sync(0xffffffffu, t.n, 0);
    t.xt = __shfl_sync(0xffffffffu, t.xt, 0);
  };
  bool ok = true;

  if (warp == 10) {
    // ------------------------------------------------------------ scheduler
    if (lane == 0) {
      const int total = tile_off[G] * MT;
      int n = 0;
      for (int i = blockIdx.x >> 1;; i += gridDim.x >> 1, ++n) {
        Mx4Tile t{};
        t.g = -1;
        if (i < total) {
          int lo = 0, hi = G;                  // tile_off[lo] * MT <= i < tile_off[hi] * MT
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tile_off[mid] * MT <= i) lo = mid; else hi = mid;
          }
          // a group's row tiles fastest: they share the weight columns
          const int rt = tile_off[lo + 1] - tile_off[lo], j = i - tile_off[lo] * MT;
          const int mb = j / rt, r = j - mb * rt;
          const int rows = goff[lo + 1] - goff[lo], per = mx4_rows_per_tile(rows, rt);
          t.g = lo;
          t.m0 = mb * kMx4BM;
          t.r0 = goff[lo] + r * per;
          t.rows = min(per, rows - r * per);
          t.n = (t.rows + 15) / 16 * 16;
          t.xt = min(tile_off[lo] + r, args.row_tiles - 1);
        }
        const int q = n % kMx4Sched;
        if (!mbar_wait(&rempty[q], ((n / kMx4Sched) & 1) ^ 1, abort_flag, lim)) { ok = false; break; }
        ring[q] = t;
        mbar_arrive(&rfull[q]);
        if (i >= total) break;
      }
      if (!ok) {
        *abort_flag = 1;
        flag_error(DEVERR_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer of the weights (both CTAs)
    {
      const bool leader = elect_one();
      const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
      const int NBW = (args.n_out + 127) / 128;
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      Mx4Tile ti;
      for (int n = 0;; ++n) {
        if (!next_tile(n, ti)) { ok = false; break; }
        uniform(ti);
        if (ti.g < 0) break;
        const int q32 = (ti.n + 63) / 64;                  // boxes of 32 rows in half of the rows
        const int col = ti.m0 + rank * 128;
        // the pair's second block may lie behind the last one: its columns are not stored
        const int wrow = (ti.g * NBW + min(ti.m0 / 128 + rank, NBW - 1)) * KB * (LY::SFA_BYTES / 256);
        const uint32_t bytes = 2u * (LY::A_BYTES + q32 * 32 * 128 + LY::SFA_BYTES + LY::SFB_BYTES);
        for (int kb = 0; kb < KB; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, abort_flag, lim))) { ok = false; break; }
          uint8_t* st = smem + s * LY::STAGE_BYTES;
          const uint32_t fb = full_leader + static_cast<uint32_t>(s) * 8u;
          if (leader) {
            if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
            tma_load_3d_pair(st, &args.w, fb, kb * 128, col, ti.g);
            tma_load_2d_pair(st + LY::A_BYTES + LY::B_BYTES, &args.sw, fb, 0, wrow + kb * (LY::SFA_BYTES / 256));
          }
          __syncwarp();
          issued |= 1u << s;
          issued_par = (issued_par & ~(1u << s)) | (ph << s);
          if (++s == kMx4Stages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
      }
      // every copy has landed before the CTA may leave (those counted on the peer's barriers: see the end)
      if (leader && rank == 0 && !wait_landed(full, kMx4Stages, issued, issued_par, never_flag, global_timer_ns())) ok = false;
      if (!ok) {
        *abort_flag = 1;
        flag_error(DEVERR_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // ------------------------------------------------------------ producer of the rows (both CTAs)
    {
      const bool leader = elect_one();
      const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      Mx4Tile ti;
      pdl_wait();   // the quantizer's codes and scales
      for (int n = 0;; ++n) {
        if (!next_tile(n, ti)) { ok = false; break; }
        uniform(ti);
        if (ti.g < 0) break;
        const CUtensorMap* tx = &args.x[(ti.n + 63) / 64 - 1];
        const int row = ti.r0 + rank * (ti.n / 2), xrow = ti.xt * KB * (LY::SFB_BYTES / 256);
        for (int kb = 0; kb < KB; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, abort_flag, lim))) { ok = false; break; }
          uint8_t* st = smem + s * LY::STAGE_BYTES + LY::A_BYTES;
          const uint32_t fb = full_leader + static_cast<uint32_t>(s) * 8u;
          if (leader) {
            tma_load_2d_pair(st, tx, fb, kb * 128, row);
            tma_load_2d_pair(st + LY::B_BYTES + LY::SFA_BYTES, &args.sx, fb, 0, xrow + kb * (LY::SFB_BYTES / 256));
          }
          __syncwarp();
          issued |= 1u << s;
          issued_par = (issued_par & ~(1u << s)) | (ph << s);
          if (++s == kMx4Stages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
      }
      if (leader && rank == 0 && !wait_landed(full, kMx4Stages, issued, issued_par, never_flag, global_timer_ns())) ok = false;
      if (!ok) {
        *abort_flag = 1;
        flag_error(DEVERR_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    // The whole warp walks the stages, so that addresses and descriptors are uniform values
    // the tensor instructions take as they are; one elected lane issues them.  (One lane
    // walking alone moves every operand over: 830 cycles a stage for 460 of instructions.)
    if (rank == 0) {
      const uint32_t s_addr = smem_u32(smem);
      const uint64_t a_desc = sw128_kmajor_desc(s_addr), b_desc = sw128_kmajor_desc(s_addr + LY::A_BYTES);
      const uint64_t sf_desc = sf_chunk_desc(s_addr + LY::A_BYTES + LY::B_BYTES);
      const bool leader = elect_one();
      int s = 0;
      uint32_t ph = 0, par = 0;
      bool issued_any = false;
      Mx4Tile ti;
      for (int n = 0;; ++n) {
        if (!next_tile(n, ti)) { ok = false; break; }
        uniform(ti);
        if (ti.g < 0) break;
        const int acc = n & 1;
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(&tempty[acc], ((n >> 1) & 1) ^ 1u, abort_flag, lim))) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kAccStride);
        const uint32_t idesc = make_idesc_mx4(kMx4BM, ti.n, 0);
        constexpr uint32_t kSfId2 = (2u << 4) | (2u << 29);
        const bool two = ti.n > 128;                       // the rows' scales take two chunks
        for (int kb = 0; kb < KB; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&full[s], ph, abort_flag, lim))) { ok = false; break; }
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>(s * (LY::STAGE_BYTES >> 4));
          const uint64_t ad = a_desc + so, bd = b_desc + so, fd = sf_desc + so;
          // scales of even and odd stages sit in different columns: a stage's copies need not
          // wait for the MMAs of the stage before it to have read theirs
          const uint32_t sf = tmem_base + static_cast<uint32_t>(LY::SF_COL) + par * kAccStride;
          if (leader) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              tc_cp_sf_pair(sf + 4 * c, fd + c * (512 >> 4));
              tc_cp_sf_pair(sf + LY::SFB_COL + 8 * c, fd + ((LY::SFA_BYTES + 1024 * c) >> 4));
              if (two) tc_cp_sf_pair(sf + LY::SFB_COL + 8 * c + 4, fd + ((LY::SFA_BYTES + 1024 * c + 512) >> 4));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {                  // K = 64 each: chunk q / 2, byte pair q % 2
              const uint32_t sel = static_cast<uint32_t>(2 * (q & 1)) << 30;
              tc_mma_mx4_pair(d_tmem, ad + q * 2, bd + q * 2, (q & 1) ? (idesc | kSfId2) : idesc,
                              (sf + 4 * (q >> 1)) | sel, (sf + LY::SFB_COL + 8 * (q >> 1)) | sel,
                              (kb | q) != 0 ? 1u : 0u);
            }
            tc_commit_pair_mc(&empty[s], 0x3);
          }
          __syncwarp();
          issued_any = true;
          par ^= 1u;
          if (++s == kMx4Stages) { s = 0; ph ^= 1u; }
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
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..9)
    // Lane = output column, accumulator column = row: each store of the warp is one run of a
    // row.  Two warps share a TMEM lane quarter and take 16 rows in turn.
    const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    Mx4Tile ti;
    for (int n = 0;; ++n) {
      if (!next_tile(n, ti)) { ok = false; break; }
      if (ti.g < 0) break;
      const int acc = n & 1;
      const int col = ti.m0 + rank * 128 + quarter * 32 + lane;
      const int rows = col < args.n_out ? ti.rows : 0;
      float bias = 0.0f;
      if (args.bias != nullptr && col < args.n_out)
        bias = __bfloat162float(args.bias[static_cast<size_t>(ti.g) * args.n_out + col]);
      const uint32_t tbase =
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * kAccStride);
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], (n >> 1) & 1, abort_flag, lim))) { ok = false; break; }
      tc_fence_after();
#pragma unroll 1
      for (int c = 16 * half; c < ti.rows; c += 32) {
        float v[16];
        tmem_ld8(tbase + c, *reinterpret_cast<float(*)[8]>(v));
        tmem_ld8(tbase + c + 8, *reinterpret_cast<float(*)[8]>(v + 8));
        tmem_ld_wait();
        OutT* o = static_cast<OutT*>(args.out) + static_cast<size_t>(ti.r0 + c) * args.n_out + col;
        if constexpr (sizeof(OutT) == 2) {
          // neighbouring lanes trade, so that one has both columns of row j, the other of row
          // j + 1: a store of four bytes a lane covers 64 bytes of two rows
          o += (lane & 1) * (args.n_out - 1);
#pragma unroll
          for (int j = 0; j < 16; j += 2, o += 2 * static_cast<size_t>(args.n_out)) {
            const __nv_bfloat162 mine = __floats2bfloat162_rn(v[j] + bias, v[j + 1] + bias);
            const uint32_t a = *reinterpret_cast<const uint32_t*>(&mine);
            const uint32_t b = __shfl_xor_sync(0xffffffffu, a, 1);
            const uint32_t both = (lane & 1) ? __byte_perm(b, a, 0x7632) : __byte_perm(a, b, 0x5410);
            if (c + j + (lane & 1) < rows) *reinterpret_cast<uint32_t*>(o) = both;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j, o += args.n_out)
            if (c + j < rows) *o = v[j] + bias;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty_leader + static_cast<uint32_t>(acc) * 8u);
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
  cluster_sync_all();   // no CTA leaves while its peer may still signal it or read its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

}  // namespace moe
