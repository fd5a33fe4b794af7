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
// Bias gradients: for the tiles of the first column block the issuer adds one N = 16 MMA a
// step whose B operand is a tile of ones, into the 16 TMEM columns that the <= 240-column
// tile leaves free: the sums cost no further pass over dy and dgu.
//
// dg and du are rounded to bf16 between DH and the two products that read them (they are
// tensor-core operands); all sums are fp32.
//
// Tile 128 x tn, tn = the columns split evenly into blocks of at most 240 (a multiple of
// 16; 2880 = 12 x 240), four 64-deep stages, two accumulator buffers; roles as in
// grouped_gemm.cuh.  DH and DX walk (expert, row block, column block) tiles of the ragged
// rows, DW walks (matrix, expert, 128-row block, column block) tiles of the gradients.
#pragma once

#include "grouped_gemm_mx4.cuh"

namespace moe {

enum BwdKind : int { BWD_DH = 0, BWD_DX = 1, BWD_DW = 2 };

constexpr int kBwdTN = 240;          // most columns of a tile
constexpr int kBwdBK = 64;           // K per stage
constexpr int kBwdStages = 4;
constexpr int kBwdBox = 64 * 128;    // bytes of a [64 K-rows x 64 elements] box
constexpr int kBwdOnesCol = 240;     // TMEM column of the bias sums inside an accumulator buffer

struct BwdLayout {
  static constexpr int A_BYTES = 2 * kBwdBox;
  static constexpr int B_BYTES = 4 * kBwdBox;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int ONES = 2048;               // 16 rows x 128 B of bf16 ones
  static constexpr int STAGING = 4 * 32 * 144;
  static constexpr int EXTRA = 1024 + 4096;
  static constexpr int SMEM = kBwdStages * STAGE_BYTES + ONES + STAGING + EXTRA;
  static_assert(SMEM <= 232448, "shared memory budget");
};

// Columns per tile: N split evenly into blocks of at most 240, in steps of 16.
__host__ __device__ constexpr int bwd_tile_n(int N) {
  const int blocks = (N + kBwdTN - 1) / kBwdTN;
  return ((N + blocks - 1) / blocks + 15) / 16 * 16;
}

// One product of a launch.  DH: A = dy, B0 = Wd.  DX: A = dgu (halves), B0 = Wg, B1 = Wu.
// DW: A, B0 = the two row-major operands whose rows are summed over.
struct BwdJob {
  CUtensorMap a, b0, b1;
  void* out;
  void* bias_out;   // DW: [G, m] column sums of A, or null
  int m, n;         // DW: rows and columns of the gradient;  DH, DX: n = columns of the output
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
  int job, g, m0, m_end, n0;   // DW: m0 / n0 inside the gradient;  DH, DX: m0 a row of A
};

template <int KIND>
__device__ __forceinline__ BwdTile bwd_tile(int i, const int* tile_off, const int* goff, const BwdArgs<KIND>& a) {
  BwdTile t;
  if constexpr (KIND == BWD_DW) {
    t.job = 0;
    int mt = 0, nt = 0;
    for (;; ++t.job) {
      mt = (a.job[t.job].m + kBM - 1) / kBM;
      nt = (a.job[t.job].n + bwd_tile_n(a.job[t.job].n) - 1) / bwd_tile_n(a.job[t.job].n);
      const int n = a.num_groups * mt * nt;
      if (i < n || t.job + 1 == a.num_jobs) break;
      i -= n;
    }
    t.g = i / (mt * nt);
    i -= t.g * mt * nt;
    // bands of kGroupBand row blocks, the row block fastest: neighbours share operand rows in L2
    const int band = i / (kGroupBand * nt);
    const int rem = i - band * kGroupBand * nt;
    const int rows = min(kGroupBand, mt - band * kGroupBand);
    t.n0 = (rem / rows) * bwd_tile_n(a.job[t.job].n);
    t.m0 = (band * kGroupBand + rem % rows) * kBM;
    t.m_end = a.job[t.job].m;
  } else {
    const int tn = bwd_tile_n(a.job[0].n);
    const TileInfo ti = decode_tile(i, tile_off, goff, a.num_groups, (a.job[0].n + tn - 1) / tn, tn);
    t.job = 0;
    t.g = ti.g;
    t.m0 = ti.m0;
    t.m_end = ti.m_end;
    t.n0 = ti.n0;
  }
  return t;
}

template <int KIND, typename OutT>
__global__ void __launch_bounds__(kGemmThreads, 1) ffn_backward_kernel(const __grid_constant__ BwdArgs<KIND> args) {
  pdl_enter();
  using LY = BwdLayout;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ones = smem + kBwdStages * LY::STAGE_BYTES;
  uint8_t* staging = ones + LY::ONES;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + LY::STAGING);
  uint64_t* empty = full + kBwdStages;
  uint64_t* tfull = empty + kBwdStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* never_flag = abort_flag + 1;
  int* tile_off = never_flag + 2;              // [G+1]
  int* goff = tile_off + (kMaxGroups + 2);     // [G+1]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = args.num_groups;
  const uint64_t lim = args.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kBwdStages; ++s) {
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
    if (lane < args.num_jobs) {
      tma_prefetch_desc(&args.job[lane].a);
      tma_prefetch_desc(&args.job[lane].b0);
      if (KIND == BWD_DX) tma_prefetch_desc(&args.job[lane].b1);
    }
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  } else if (KIND == BWD_DW) {
    for (int i = threadIdx.x - 64; i < LY::ONES / 4; i += 128) reinterpret_cast<uint32_t*>(ones)[i] = 0x3F803F80u;
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  int total = 0;
  if constexpr (KIND == BWD_DW) {
    for (int j = 0; j < args.num_jobs; ++j) {
      const int tn = bwd_tile_n(args.job[j].n);
      total += G * ((args.job[j].m + kBM - 1) / kBM) * ((args.job[j].n + tn - 1) / tn);
    }
  } else {
    const int tn = bwd_tile_n(args.job[0].n);
    total = tile_off[G] * ((args.job[0].n + tn - 1) / tn);
  }
  // 64-deep K blocks of a tile (DW: of its expert's rows; DX: of both halves)
  const int KB1 = (args.k_dim + kBwdBK - 1) / kBwdBK;
  auto k_blocks = [&](const BwdTile& t) {
    if (KIND == BWD_DW) return max(0, goff[t.g + 1] - goff[t.g] + kBwdBK - 1) / kBwdBK;
    return KIND == BWD_DX ? 2 * KB1 : KB1;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < total; i += gridDim.x) {
        const BwdTile ti = bwd_tile<KIND>(i, tile_off, goff, args);
        const BwdJob& jb = args.job[ti.job];
        const int nbox = (bwd_tile_n(jb.n) + 63) / 64;
        const int KB = k_blocks(ti);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, lim)) { ok = false; break; }
          mbar_arrive_expect_tx(&full[s], LY::A_BYTES + nbox * kBwdBox);
          uint8_t* sa = smem + s * LY::STAGE_BYTES;
          uint8_t* sb = sa + LY::A_BYTES;
          if constexpr (KIND == BWD_DW) {
            const int r = goff[ti.g] + kb * kBwdBK;
            for (int q = 0; q < nbox; ++q) tma_load_2d(sb + q * kBwdBox, &jb.b0, &full[s], ti.n0 + 64 * q, r);
            for (int q = 0; q < 2; ++q) tma_load_2d(sa + q * kBwdBox, &jb.a, &full[s], ti.m0 + 64 * q, r);
          } else {
            const int half = (KIND == BWD_DX && kb >= KB1) ? 1 : 0;
            const int k0 = (kb - half * KB1) * kBwdBK;
            const CUtensorMap* tb = half ? &jb.b1 : &jb.b0;
            for (int q = 0; q < nbox; ++q) tma_load_3d(sb + q * kBwdBox, tb, &full[s], ti.n0 + 64 * q, k0, ti.g);
            if (KIND == BWD_DX) tma_load_3d(sa, &jb.a, &full[s], k0, half, ti.m0);
            else tma_load_2d(sa, &jb.a, &full[s], k0, ti.m0);
          }
          issued |= 1u << s;
          issued_par = (issued_par & ~(1u << s)) | (ph << s);
          if (++s == kBwdStages) { s = 0; ph ^= 1u; }
        }
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
    // Lane 0 waits and issues.  The whole warp takes part where a DW tile's last block has
    // rows to blank; `ok` is lane 0's until the warp agrees on it at the end of a tile.
    int s = 0, it = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < total; i += gridDim.x, ++it) {
      const BwdTile ti = bwd_tile<KIND>(i, tile_off, goff, args);
      const BwdJob& jb = args.job[ti.job];
      const int KB = k_blocks(ti);
      const int tn = bwd_tile_n(jb.n);
      const uint32_t idesc = make_idesc(kBM, tn, 1u) | (1u << 16) | (KIND == BWD_DW ? 1u << 15 : 0u);
      const uint32_t idesc_ones = make_idesc(kBM, 16, 1u) | (1u << 15);
      const bool sums = KIND == BWD_DW && ti.n0 == 0 && jb.bias_out != nullptr;
      const int acc = it & 1;
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kAccStride);
      if (lane == 0) {
        ok = mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, abort_flag, lim);
        tc_fence_after();
      }
      for (int kb = 0; kb < KB; ++kb) {
        const uint32_t a_addr = smem_u32(smem + s * LY::STAGE_BYTES);
        const uint32_t b_addr = a_addr + LY::A_BYTES;
        int steps = kBwdBK / 16;
        if (KIND == BWD_DW && kb == KB - 1) {
          const int valid = goff[ti.g + 1] - goff[ti.g] - kb * kBwdBK;   // 1..64
          steps = (valid + 15) / 16;
          if ((valid & 15) != 0) {
            const bool got = __all_sync(0xffffffffu, mbar_wait(&full[s], ph, abort_flag, lim));
            if (got) {
              uint8_t* st = smem + s * LY::STAGE_BYTES;
              const int nbox = 2 + (tn + 63) / 64;
              const int blank = 16 * steps - valid;   // rows valid .. 16 steps - 1 of every box
              for (int q = lane; q < nbox * blank * 8; q += 32) {
                const int box = q / (blank * 8), rem = q - box * blank * 8;
                *reinterpret_cast<uint4*>(st + box * kBwdBox + valid * 128 + rem * 16) = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
            }
            __syncwarp();
          }
        }
        if (lane == 0) {
          if (ok) ok = mbar_wait(&full[s], ph, abort_flag, lim);
          if (ok) {
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kBwdBK / 16; ++kk) {
              if (kk < steps) {
                const uint64_t ad = KIND == BWD_DW ? sw128_mnmajor_desc(a_addr + kk * 2048)
                                                   : sw128_kmajor_desc(a_addr + kk * 32);
                const uint32_t accumulate = (kb | kk) != 0 ? 1u : 0u;
                tc_mma<false>(d_tmem, ad, sw128_mnmajor_desc(b_addr + kk * 2048), idesc, accumulate);
                if (sums) tc_mma<false>(d_tmem + kBwdOnesCol, ad, sw128_kmajor_desc(smem_u32(ones)), idesc_ones, accumulate);
              }
            }
            tc_commit(&empty[s]);
          }
        }
        if (++s == kBwdStages) { s = 0; ph ^= 1u; }
      }
      if (lane == 0 && ok) tc_commit(&tfull[acc]);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    }
    if (lane == 0) {
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
      const BwdTile ti = bwd_tile<KIND>(i, tile_off, goff, args);
      const BwdJob& jb = args.job[ti.job];
      const int tn = bwd_tile_n(jb.n);
      const int acc = it & 1;
      const bool got = __all_sync(0xffffffffu, mbar_wait(&tfull[acc], (it >> 1) & 1, abort_flag, lim));
      if (!got) { ok = false; break; }
      tc_fence_after();
      const uint32_t tbase =
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * kAccStride);
      const int row0 = ti.m0 + quarter * 32;
      const bool none = KIND == BWD_DW && goff[ti.g + 1] <= goff[ti.g];   // no rows: the gradient is zero
      const int width = min(tn, jb.n - ti.n0);
      if constexpr (KIND == BWD_DH) {
        const int F = jb.n;
        const int row = row0 + lane;
        const bool rvalid = row < ti.m_end;
        const __nv_bfloat16* g = args.gu + static_cast<size_t>(rvalid ? row : 0) * 2 * F + ti.n0;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(jb.out) + static_cast<size_t>(row) * 2 * F + ti.n0;
#pragma unroll 1
        for (int c = 0; c < width; c += 8) {
          float v[8];
          tmem_ld8(tbase + c, v);
          tmem_ld_wait();
          if (rvalid) {
            float gv[8], uv[8], dg[8], du[8];
            load8<__nv_bfloat16>(g + c, gv);
            load8<__nv_bfloat16>(g + F + c, uv);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              act_grad(v[j], gv[j], uv[j], args.limit, args.alpha, args.gate_lo, dg[j], du[j]);
            store8<__nv_bfloat16>(out + c, dg);
            store8<__nv_bfloat16>(out + F + c, du);
          }
        }
      } else {
        const size_t row_base = KIND == BWD_DW ? static_cast<size_t>(ti.g) * jb.m : 0;
        OutT* out = static_cast<OutT*>(jb.out) + (row_base + row0) * jb.n + ti.n0;
#pragma unroll 1
        for (int c = 0; c < width; c += COLS) {
          float v[COLS];
#pragma unroll
          for (int j = 0; j < COLS; j += 8)
            if (c + j < width) tmem_ld8(tbase + c + j, *reinterpret_cast<float(*)[8]>(v + j));
          tmem_ld_wait();
          if (none) {
#pragma unroll
            for (int j = 0; j < COLS; ++j) v[j] = 0.0f;
          }
          store_rows_staged<OutT>(stage, out + c, jb.n, ti.m_end - row0, width - c, v);
        }
        if (KIND == BWD_DW && ti.n0 == 0 && jb.bias_out != nullptr) {
          float b[8];
          tmem_ld8(tbase + kBwdOnesCol, b);
          tmem_ld_wait();
          if (row0 + lane < ti.m_end) {
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
