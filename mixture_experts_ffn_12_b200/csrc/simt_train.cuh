// The expert block's training pass for fp32 layers, in fp32 FMA (TF32 would truncate the
// operands to 10 mantissa bits): the forward products and the three backward ones of
// train_gemm.cuh as one tiled kernel.
//
// These layers are small, so a launch is a chain of K steps more than a rate.  Tiles of 32
// rows (an expert often has fewer) x 32 columns, 4 x 4 outputs a thread, a three-deep ring of
// cp.async copies of 64 K elements, so that no step waits for the load it has just issued,
// and eight groups of threads that each take a part of a step's K and add up at the end in a
// fixed order: one group alone leaves a scheduler one warp, which issues every third cycle.
// Measured, forward + backward of 128 rows, 8 experts, D = 256, F = 512 (GPU time a pass, in
// a graph): 18.4 + 33.7 us; gate/up and dH on 64 columns and 32 K elements 22.4 + 33.8 us, and
// 129 + 202 against 128 + 199 us at 1024 rows, 4 experts, D = F = 640 (20 TFLOP/s: larger
// tiles would serve such layers better, which the small ones would pay for).
// The weight gradients, whose K is an expert's few rows, are the other way about: few steps
// and many outputs, one group and tiles of 64 x 128 (32 x 64 with four groups: four times the CTAs, of
// one step each, 25 against 13 us).  An operand tile is kept in the order in which it lies in
// memory, [row][K] (16-byte pieces along K) or [K][row] (along the rows), with 16 bytes of
// padding a row; either way a thread takes 4 x 4 of it per four K steps with four 16-byte loads.
//
// No kernel but DX lets its dependents start before it ends: several of these CTAs fit on
// one SM, and a grid launched while another still fills most SMs crowds onto those that come
// free first and runs there two deep (backward of the layer above, passes one after another:
// 46.8 us with early starts throughout, 33.8 without).  DX lets DW start beside it, on the
// half of the SMs that it leaves idle.
#pragma once

#include "train_gemm.cuh"

namespace moe {

enum SimtKind : int { SIMT_GATEUP = 0, SIMT_DOWN = 1, SIMT_DH = 2, SIMT_DX = 3, SIMT_DW = 4 };

constexpr int kStStages = 3, kStThreads = 512;

struct SimtJob {
  const float *a, *b0, *b1;   // GATEUP: b0, b1 = Wg, Wu;  DX: b0 then b1 along K
  const float *bias0, *bias1; // GATEUP, DOWN (null: none)
  float *out, *bias_out;      // DW: bias_out = column sums of A (null: not wanted)
  int lda, ldb;
  int m, n, k;                // DW: m x n gradient;  else n output columns, k (of one half)
};

struct SimtTrainArgs {
  SimtJob job[3];
  const int32_t* group_off;
  int num_groups, m_total;
  const float* gu;            // DH
  float* gu_out;              // GATEUP
  int early;                  // DW: behind a DX launch, starts beside it (as in train_gemm.cuh)
  float limit, alpha, gate_lo;
};

template <int KIND>
struct SimtShape {
  static constexpr int kStM = KIND == SIMT_DW ? 64 : 32;                     // rows of a tile
  static constexpr int kStN = KIND == SIMT_DW ? 128 : 32;                    // columns
  static constexpr int kStK = KIND == SIMT_DW ? 32 : 64;                     // K of a step
  static constexpr int kTX = kStN / 4, kPer = kTX * (kStM / 4), kStGroups = kStThreads / kPer;
  static constexpr bool kAK = KIND != SIMT_DW;                             // A tile [row][K]
  static constexpr bool kBK = KIND == SIMT_GATEUP || KIND == SIMT_DOWN;    // B tile [column][K]
  static constexpr int kNB = KIND == SIMT_GATEUP ? 2 : 1;
  static constexpr int kLdA = kAK ? kStK + 4 : kStM + 4;
  static constexpr int kLdB = kBK ? kStK + 4 : kStN + 4;
  static constexpr int kA = (kAK ? kStM : kStK) * kLdA, kB = (kBK ? kStN : kStK) * kLdB;   // floats
  static constexpr int kStage = kA + kNB * kB;
  static constexpr int kRing = kStStages * kStage, kSums = kStGroups * kNB * kStM * kStN;   // floats, one after the other
  static constexpr int kSmem = (kRing > kSums ? kRing : kSums) * 4;
};

__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(valid ? 16 : 0)
               : "memory");
}

template <int KIND>
__global__ void __launch_bounds__(kStThreads) simt_train_kernel(const SimtTrainArgs args) {
  if (KIND != SIMT_DW || !args.early) pdl_wait();
  if constexpr (KIND == SIMT_DX) pdl_launch_dependents();
  using S = SimtShape<KIND>;
  constexpr int kStM = S::kStM, kStN = S::kStN, kStK = S::kStK, kStGroups = S::kStGroups;
  extern __shared__ __align__(16) float ring[];
  constexpr int kTable = KIND == SIMT_DW ? 1 : kMaxGroups + 1;
  __shared__ int goff[kTable], toff[kTable];
  const int G = args.num_groups;
  if (KIND != SIMT_DW) {
    if (threadIdx.x < 32) group_table(args.group_off, G, args.m_total, kStM, goff, toff);
    __syncthreads();
  }

  const SimtJob& jb = args.job[KIND == SIMT_DW ? blockIdx.z / G : 0];
  const int n0 = blockIdx.y * kStN;
  int g, m0, m_end, r0 = 0, K = jb.k;
  if constexpr (KIND == SIMT_DW) {
    g = blockIdx.z % G;
    m0 = blockIdx.x * kStM;
    m_end = jb.m;
    const int b = args.group_off[g], e = args.group_off[g + 1];
    r0 = min(max(b, 0), args.m_total);
    const int r1 = min(max(e, 0), args.m_total);
    if ((r0 != b || r1 != e || r1 < r0) && threadIdx.x == 0) flag_error(DEVERR_BOUNDS);
    K = max(0, r1 - r0);
    if (m0 >= m_end || n0 >= jb.n) return;     // the grid covers the largest of the gradients
  } else {
    const int mt = blockIdx.x;
    if (mt >= toff[G]) return;
    int lo = 0, hi = G;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (toff[mid] <= mt) lo = mid; else hi = mid;
    }
    g = lo;
    m0 = goff[g] + (mt - toff[g]) * kStM;
    m_end = goff[g + 1];
  }
  const int halves = KIND == SIMT_DX ? 2 : 1;
  const int ksteps = (K + kStK - 1) / kStK, steps = ksteps * halves;

  // K step i into its ring slot; pieces outside the operands read as zeros
  auto load = [&](int i) {
    float* sa = ring + (i % kStStages) * S::kStage;
    const int half = KIND == SIMT_DX && i >= ksteps ? 1 : 0;
    const int k0 = (i - half * ksteps) * kStK;
    if constexpr (S::kAK) {
      for (int p = threadIdx.x; p < kStM * kStK / 4; p += kStThreads) {
        const int r = p / (kStK / 4), c = (p % (kStK / 4)) * 4;
        const bool ok = m0 + r < m_end && k0 + c < K;
        cp_async16(sa + r * S::kLdA + c, ok ? jb.a + static_cast<size_t>(m0 + r) * jb.lda + half * K + k0 + c : jb.a, ok);
      }
    } else {
      for (int p = threadIdx.x; p < kStM * kStK / 4; p += kStThreads) {
        const int r = p / (kStM / 4), c = (p % (kStM / 4)) * 4;
        const bool ok = k0 + r < K && m0 + c < m_end;
        cp_async16(sa + r * S::kLdA + c, ok ? jb.a + static_cast<size_t>(r0 + k0 + r) * jb.lda + m0 + c : jb.a, ok);
      }
    }
#pragma unroll
    for (int b = 0; b < S::kNB; ++b) {
      float* sb = sa + S::kA + b * S::kB;
      const float* src = (b == 1 || half == 1) ? jb.b1 : jb.b0;
      if constexpr (S::kBK) {
        for (int p = threadIdx.x; p < kStN * kStK / 4; p += kStThreads) {
          const int r = p / (kStK / 4), c = (p % (kStK / 4)) * 4;
          const bool ok = n0 + r < jb.n && k0 + c < K;
          cp_async16(sb + r * S::kLdB + c, ok ? src + (static_cast<size_t>(g) * jb.n + n0 + r) * K + k0 + c : src, ok);
        }
      } else {
        const size_t row0 = KIND == SIMT_DW ? r0 : static_cast<size_t>(g) * K;
        for (int p = threadIdx.x; p < kStN * kStK / 4; p += kStThreads) {
          const int r = p / (kStN / 4), c = (p % (kStN / 4)) * 4;
          const bool ok = k0 + r < K && n0 + c < jb.n;
          cp_async16(sb + r * S::kLdB + c, ok ? src + (row0 + k0 + r) * jb.ldb + n0 + c : src, ok);
        }
      }
    }
  };

  const int grp = threadIdx.x / S::kPer, t = threadIdx.x % S::kPer, tx = t % S::kTX, ty = t / S::kTX;
  float acc[S::kNB][4][4] = {}, sum[4] = {};
  for (int i = 0; i < kStStages - 1; ++i) {
    if (i < steps) load(i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  for (int i = 0; i < steps; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStStages - 2) : "memory");
    __syncthreads();
    if (i + kStStages - 1 < steps) load(i + kStStages - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const float* sa = ring + (i % kStStages) * S::kStage;
#pragma unroll
    for (int kk = grp * (kStK / kStGroups); kk < (grp + 1) * (kStK / kStGroups); kk += 4) {
      float a[4][4];   // [row][k]
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (S::kAK) {
          *reinterpret_cast<float4*>(a[q]) = *reinterpret_cast<const float4*>(sa + (ty * 4 + q) * S::kLdA + kk);
        } else {
          const float4 v = *reinterpret_cast<const float4*>(sa + (kk + q) * S::kLdA + ty * 4);
          a[0][q] = v.x;
          a[1][q] = v.y;
          a[2][q] = v.z;
          a[3][q] = v.w;
        }
      }
      if (KIND == SIMT_DW) {
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] += (a[r][0] + a[r][1]) + (a[r][2] + a[r][3]);
      }
#pragma unroll
      for (int b = 0; b < S::kNB; ++b) {
        const float* sb = sa + S::kA + b * S::kB;
        float w[4][4];   // [column][k]
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (S::kBK) {
            *reinterpret_cast<float4*>(w[q]) = *reinterpret_cast<const float4*>(sb + (tx + S::kTX * q) * S::kLdB + kk);
          } else {
            const float4 v = *reinterpret_cast<const float4*>(sb + (kk + q) * S::kLdB + tx * 4);
            w[0][q] = v.x;
            w[1][q] = v.y;
            w[2][q] = v.z;
            w[3][q] = v.w;
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[b][r][c] = fmaf(a[r][q], w[c][q], acc[b][r][c]);
      }
    }
  }

  // the groups' sums through the ring; a group then finishes one row of each thread's four
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  auto slot = [&](int group, int b, int r) { return ring + (((group * S::kNB + b) * 4 + r) * S::kPer + t) * 4; };
#pragma unroll
  for (int b = 0; b < S::kNB; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) *reinterpret_cast<float4*>(slot(grp, b, r)) = *reinterpret_cast<float4*>(acc[b][r]);
  __shared__ float sums[KIND == SIMT_DW ? kStGroups : 1][kStM];
  if (KIND == SIMT_DW && tx == 0)
    for (int r = 0; r < 4; ++r) sums[grp][ty * 4 + r] = sum[r];
  __syncthreads();
  for (int r = grp; r < 4; r += kStGroups) {   // group r (one group: all four rows)
    float tot[S::kNB][4] = {};
#pragma unroll
    for (int b = 0; b < S::kNB; ++b)
#pragma unroll
      for (int q = 0; q < kStGroups; ++q) {
        const float4 v = *reinterpret_cast<const float4*>(slot(q, b, r));
        tot[b][0] += v.x;
        tot[b][1] += v.y;
        tot[b][2] += v.z;
        tot[b][3] += v.w;
      }
    const int row = m0 + ty * 4 + r;
    if (row >= m_end) continue;
    const size_t orow = KIND == SIMT_DW ? static_cast<size_t>(g) * jb.m + row : row;
    if (KIND == SIMT_DW && jb.bias_out != nullptr && n0 == 0 && tx == 0) {
      float s = 0.0f;
      for (int q = 0; q < kStGroups; ++q) s += sums[q][ty * 4 + r];
      jb.bias_out[orow] = s;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int col = n0 + (S::kBK ? tx + S::kTX * c : tx * 4 + c);
      if (col >= jb.n) continue;
      const float v = tot[0][c];
      if constexpr (KIND == SIMT_GATEUP) {
        const size_t bi = static_cast<size_t>(g) * jb.n + col;
        const float gv = jb.bias0 == nullptr ? v : v + jb.bias0[bi];
        const float uv = jb.bias1 == nullptr ? tot[S::kNB - 1][c] : tot[S::kNB - 1][c] + jb.bias1[bi];
        const float gc = clip_nan(gv, args.gate_lo, args.limit), uc = clip_nan(uv, args.limit);
        args.gu_out[orow * 2 * jb.n + col] = gv;
        args.gu_out[orow * 2 * jb.n + jb.n + col] = uv;
        jb.out[orow * jb.n + col] = gc / (1.0f + expf(-args.alpha * gc)) * uc;
      } else if constexpr (KIND == SIMT_DOWN) {
        jb.out[orow * jb.n + col] = jb.bias0 == nullptr ? v : v + jb.bias0[static_cast<size_t>(g) * jb.n + col];
      } else if constexpr (KIND == SIMT_DH) {
        const float gv = args.gu[orow * 2 * jb.n + col], uv = args.gu[orow * 2 * jb.n + jb.n + col];
        const float gc = clip_nan(gv, args.gate_lo, args.limit), uc = clip_nan(uv, args.limit);
        const float s = 1.0f / (1.0f + expf(-args.alpha * gc)), f = gc * s;
        jb.out[orow * 2 * jb.n + col] =
            (gv < args.gate_lo || gv > args.limit) ? 0.0f : v * uc * (s + args.alpha * f * (1.0f - s));
        jb.out[orow * 2 * jb.n + jb.n + col] = fabsf(uv) > args.limit ? 0.0f : v * f;
      } else {
        jb.out[orow * jb.n + col] = v;
      }
    }
  }
  if (KIND == SIMT_DW && args.early) pdl_wait();
}

}  // namespace moe
