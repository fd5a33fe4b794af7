// Grouped product of MXFP4 rows with MXFP4 weights on the block-scaled tensor cores:
//   out[r, n] = sum_k A[r, k] * W_g[n, k] + b_g[n]    for the rows r of group g
// with both operands E2M1 with one E8M0 scale per 32 elements along K
// (tcgen05.mma kind::mxf4, block scales applied by the tensor core, fp32 accumulators).
//
// Stage = 256 elements of K = one 128-byte swizzled row of packed codes: A 128 rows and B
// 192 rows by TMA (plain byte boxes: the mxf4 MMA reads 4-bit operands packed), the scales
// as ready-made 512-byte chunks (mxfp4_quant.cuh) by bulk copies, four MMAs of K = 64.
// Why 192 columns: two accumulator buffers (so a tile's epilogue overlaps the next tile's
// loads and MMAs) leave 128 of the 512 TMEM columns, and the scales of a stage take 24 of
// them; 2 x 256 columns would leave none.  A tile starts at a multiple of 192, so every
// second one starts in the middle of a 128-row scale chunk: its MMAs read the scales two
// TMEM columns (64 rows) further on.
//
// Roles (one CTA per SM, 192 threads) and tile order as in grouped_gemm.cuh; waits bounded.
#pragma once

#include "mxfp4_quant.cuh"

namespace moe {

constexpr int kMx4BK = 256;       // K elements per stage
constexpr int kMx4TN = 192;       // output columns per tile
constexpr int kMx4Stages = 4;

struct Mx4Layout {
  static constexpr int A_BYTES = kBM * 128;
  static constexpr int B_BYTES = kMx4TN * 128;
  static constexpr int SFA_BYTES = 1024;          // 2 chunks of 128 K
  static constexpr int SFB_BYTES = 2048;          // 2 row blocks x 2 chunks
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int STAGING = 4 * 32 * 144;    // epilogue: 32 rows of 128 B (+ 16 B) a warp
  static constexpr int EXTRA = 1024 + 4096;
  static constexpr int SMEM = kMx4Stages * STAGE_BYTES + STAGING + EXTRA;
  // TMEM: accumulators at columns 0 and 256; scales of even / odd stages behind them:
  // A 2 chunks x 4 columns, then B 2 chunks x 2 row blocks x 4 columns
  static constexpr int SF_COL = kMx4TN;
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

__device__ __forceinline__ void tc_mma_mx4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

// Contiguous bytes (a multiple of 16, both addresses 16-byte aligned) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

struct Mx4Args {
  const int32_t* group_off;   // [G+1]; null: one group of m_total rows
  int num_groups;
  int m_total;
  int n_out;
  int k_dim;
  const uint8_t* tiles_a;     // scale tiles of A, row blocks counted group after group
  int row_blocks;             // their number (clamp for offsets that are not ascending)
  const uint8_t* tiles_w;     // scale tiles of W, [G][ceil(n_out / 128)] row blocks
  const __nv_bfloat16* bias;  // [G, n_out] or null
  void* out;                  // [m_total, n_out]
  unsigned long long wait_limit_ns;
};

// Writes 32 rows x (8 * PIECES) columns that the warp's lanes hold (lane = row) through its
// staging area, so that each store instruction covers whole 128-byte runs of rows.
// T = bf16: 64 columns a call; float: 32.
template <typename T>
__device__ __forceinline__ void store_rows_staged(uint8_t* stage, T* out, size_t ldo, int rows, int cols,
                                                  const float* v) {
  constexpr int COLS = 128 / static_cast<int>(sizeof(T));
  constexpr int PER = 16 / static_cast<int>(sizeof(T));   // columns per 16-byte piece
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    uint4 u;
    if constexpr (sizeof(T) == 2) {
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(v[p * PER + 2 * j], v[p * PER + 2 * j + 1]);
    } else {
      u = make_uint4(__float_as_uint(v[p * PER]), __float_as_uint(v[p * PER + 1]), __float_as_uint(v[p * PER + 2]),
                     __float_as_uint(v[p * PER + 3]));
    }
    *reinterpret_cast<uint4*>(stage + lane * 144 + p * 16) = u;
  }
  __syncwarp();
  const int piece = lane & 7;
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int r = it * 4 + (lane >> 3);
    if (r < rows && piece * PER < cols)
      *reinterpret_cast<uint4*>(out + r * ldo + piece * PER) =
          *reinterpret_cast<const uint4*>(stage + r * 144 + piece * 16);
  }
  (void)COLS;
}

template <typename OutT>
__global__ void __launch_bounds__(kGemmThreads, 1)
    grouped_gemm_mx4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                            const Mx4Args args) {
  pdl_enter();
  using LY = Mx4Layout;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + kMx4Stages * LY::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + LY::STAGING);
  uint64_t* empty = full + kMx4Stages;
  uint64_t* tfull = empty + kMx4Stages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* never_flag = abort_flag + 1;
  int* tile_off = never_flag + 2;              // [G+1]
  int* goff = tile_off + (kMaxGroups + 2);     // [G+1]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = args.group_off == nullptr ? 1 : args.num_groups;
  const int NT = (args.n_out + kMx4TN - 1) / kMx4TN;
  const int KB = (args.k_dim + kMx4BK - 1) / kMx4BK;
  const int NBW = (args.n_out + kBM - 1) / kBM;      // row blocks of W's scale tiles
  const uint64_t lim = args.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMx4Stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 128);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    mx4_group_table(args.group_off, G, args.m_total, goff, tile_off);
    if (lane == 0) {
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmB);
    }
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = tile_off[G] * NT;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const size_t row_block = static_cast<size_t>(KB) * 1024;   // bytes of one row block of scale tiles
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < total; i += gridDim.x) {
        const TileInfo ti = decode_tile(i, tile_off, goff, G, NT, kMx4TN);
        const int rba = min(tile_off[ti.g] + (ti.m0 - goff[ti.g]) / kBM, args.row_blocks - 1);
        const int rbw = ti.n0 / kBM;
        const int nrb = min(2, NBW - rbw);
        const uint8_t* sa = args.tiles_a + rba * row_block;
        const uint8_t* sw = args.tiles_w + (static_cast<size_t>(ti.g) * NBW + rbw) * row_block;
        const uint32_t tx = LY::A_BYTES + LY::B_BYTES + LY::SFA_BYTES + nrb * 1024u;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, lim)) { ok = false; break; }
          mbar_arrive_expect_tx(&full[s], tx);
          uint8_t* st = smem + s * LY::STAGE_BYTES;
          tma_load_3d(st + LY::A_BYTES, &tmB, &full[s], kb * 128, ti.n0, ti.g);
          tma_load_2d(st, &tmA, &full[s], kb * 128, ti.m0);
          uint8_t* sf = st + LY::A_BYTES + LY::B_BYTES;
          bulk_load(sf, sa + kb * 1024, 1024, &full[s]);
          for (int q = 0; q < nrb; ++q) bulk_load(sf + 1024 * (1 + q), sw + q * row_block + kb * 1024, 1024, &full[s]);
          issued |= 1u << s;
          issued_par = (issued_par & ~(1u << s)) | (ph << s);
          if (++s == kMx4Stages) { s = 0; ph ^= 1u; }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        flag_error(DEVERR_TIMEOUT);
      }
      for (int q = 0; q < kMx4Stages; ++q)
        if ((issued >> q) & 1u)
          if (!mbar_wait(&full[q], (issued_par >> q) & 1u, never_flag, kDrainLimitNs)) flag_error(DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int s = 0, it = 0;
      uint32_t ph = 0, par = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < total; i += gridDim.x, ++it) {
        const TileInfo ti = decode_tile(i, tile_off, goff, G, NT, kMx4TN);
        const int acc = it & 1;
        if (!mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, abort_flag, lim)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kAccStride);
        const uint32_t half = (ti.n0 & 127) != 0 ? 2u : 0u;   // the tile starts 64 rows into a chunk
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&full[s], ph, abort_flag, lim)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + s * LY::STAGE_BYTES);
          const uint32_t b_addr = a_addr + LY::A_BYTES;
          const uint32_t sf_addr = b_addr + LY::B_BYTES;
          // scales of even and odd stages sit in different columns: a stage's copy need not
          // wait for the MMAs of the stage before it to have read theirs
          const uint32_t sf = tmem_base + static_cast<uint32_t>(LY::SF_COL) + par * kAccStride;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tc_cp_sf(sf + 4 * c, sf_chunk_desc(sf_addr + 512 * c));
#pragma unroll
            for (int q = 0; q < 2; ++q)
              tc_cp_sf(sf + LY::SFB_COL + 8 * c + 4 * q, sf_chunk_desc(sf_addr + 1024 * (1 + q) + 512 * c));
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              const uint32_t sel = static_cast<uint32_t>(2 * kk) << 30;
              tc_mma_mx4(d_tmem, sw128_kmajor_desc(a_addr + c * 64 + kk * 32),
                         sw128_kmajor_desc(b_addr + c * 64 + kk * 32), make_idesc_mx4(kBM, kMx4TN, 2 * kk),
                         (sf + 4 * c) | sel, (sf + LY::SFB_COL + 8 * c + half) | sel, (kb | c | kk) != 0 ? 1u : 0u);
            }
          }
          tc_commit(&empty[s]);
          par ^= 1u;
          if (++s == kMx4Stages) { s = 0; ph ^= 1u; }
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
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..5)
    constexpr int COLS = 128 / static_cast<int>(sizeof(OutT));
    const int quarter = warp & 3;
    uint8_t* stage = staging + quarter * (32 * 144);
    int it = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < total; i += gridDim.x, ++it) {
      const TileInfo ti = decode_tile(i, tile_off, goff, G, NT, kMx4TN);
      const int acc = it & 1;
      const bool got = __all_sync(0xffffffffu, mbar_wait(&tfull[acc], (it >> 1) & 1, abort_flag, lim));
      if (!got) { ok = false; break; }
      tc_fence_after();
      const uint32_t tbase =
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * kAccStride);
      const int row0 = ti.m0 + quarter * 32;
      OutT* out = static_cast<OutT*>(args.out) + static_cast<size_t>(row0) * args.n_out + ti.n0;
      const __nv_bfloat16* bias =
          args.bias == nullptr ? nullptr : args.bias + static_cast<size_t>(ti.g) * args.n_out + ti.n0;
#pragma unroll 1
      for (int c = 0; c < kMx4TN; c += COLS) {
        const int left = args.n_out - ti.n0 - c;
        if (left <= 0) break;
        float v[COLS];
#pragma unroll
        for (int j = 0; j < COLS; j += 8) tmem_ld8(tbase + c + j, *reinterpret_cast<float(*)[8]>(v + j));
        tmem_ld_wait();
        if (bias != nullptr) {
#pragma unroll
          for (int j = 0; j < COLS; j += 8)
            if (j < left) {
              float b[8];
              load8<__nv_bfloat16>(bias + c + j, b);
#pragma unroll
              for (int q = 0; q < 8; ++q) v[j + q] += b[q];
            }
        }
        store_rows_staged<OutT>(stage, out + c, args.n_out, ti.m_end - row0, left, v);
      }
      tc_fence_before();
      mbar_arrive(&tempty[acc]);
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

}  // namespace moe
