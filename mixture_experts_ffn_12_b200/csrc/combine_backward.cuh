// Backward pass of the combine.
#pragma once

#include "mxfp4_quant.cuh"

namespace moe {

// ---------------------------------------------------------------------------
// combine, backward: dy_perm[row(t, j)] = w[t, j] dy[t], dw[t, j] = dy[t] . y_perm[row(t, j)]
// ---------------------------------------------------------------------------
// One CTA a token, as wide as its row where it can be (D / 8 threads), so that all k + 1
// loads of a thread are in flight at once: dy[t] is read once and meets its k rows.  Bound by
// memory, (1 + 2 k) D elements a token.  The dot products are summed per thread, then over
// the warp and the CTA's warps in a fixed order.  KM = 4 or 8 >= k: registers for k rows.
// 4096 tokens, k = 4, D = 2880 bf16: 39 us (5.4 TB/s); 128 threads a token 57 us.
constexpr int kCombineBwdThreads = 384;   // at most
template <typename T, int KM>
__global__ void __launch_bounds__(kCombineBwdThreads)
    combine_backward_kernel(const T* __restrict__ dy, const T* __restrict__ y_perm,
                            const int32_t* __restrict__ row_of_slot, const float* __restrict__ w, int Tn, int k, int D,
                            T* __restrict__ dy_perm, float* __restrict__ dw) {
  pdl_enter();
  __shared__ float part[kCombineBwdThreads / 32][KM];
  constexpr int kWords = sizeof(T) / 2;   // 16-byte words of 8 elements
  const int t = blockIdx.x;
  const int R = Tn * k;
  int row[KM];
  float wt[KM], acc[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    row[j] = j < k ? row_of_slot[static_cast<size_t>(t) * k + j] : -1;
    wt[j] = j < k ? w[static_cast<size_t>(t) * k + j] : 0.0f;
    acc[j] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < KM; ++j)
    if (j < k && (row[j] < 0 || row[j] >= R)) {
      if (threadIdx.x == 0) flag_error(DEVERR_BOUNDS);
      row[j] = -1;
    }
  for (int c = threadIdx.x * 8; c < D; c += blockDim.x * 8) {
    uint4 rd[kWords], ry[KM][kWords];
#pragma unroll
    for (int q = 0; q < kWords; ++q) rd[q] = reinterpret_cast<const uint4*>(dy + static_cast<size_t>(t) * D + c)[q];
#pragma unroll
    for (int j = 0; j < KM; ++j)
      if (row[j] >= 0)
#pragma unroll
        for (int q = 0; q < kWords; ++q)
          ry[j][q] = reinterpret_cast<const uint4*>(y_perm + static_cast<size_t>(row[j]) * D + c)[q];
    float d[8];
    unpack8<T>(rd, d);
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      if (row[j] < 0) continue;
      float y[8], o[8];
      unpack8<T>(ry[j], y);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        acc[j] = fmaf(d[q], y[q], acc[j]);
        o[q] = wt[j] * d[q];
      }
      store8<T>(dy_perm + static_cast<size_t>(row[j]) * D + c, o);
    }
  }
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    if (j >= k) break;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][j] = acc[j];
  }
  __syncthreads();
  if (threadIdx.x < k) {
    float s = 0.0f;
    for (int q = 0; q < static_cast<int>(blockDim.x) / 32; ++q) s += part[q][threadIdx.x];
    dw[static_cast<size_t>(t) * k + threadIdx.x] = s;
  }
}

}  // namespace moe
