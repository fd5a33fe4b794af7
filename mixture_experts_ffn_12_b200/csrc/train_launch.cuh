#pragma once
// Host side of the MXFP4 product and of the expert block's training pass: tensor maps and
// launches (tensor maps as in gemm_launch.cuh: boxes of 128 bytes x rows, 128-byte swizzle,
// zeros out of range).
#include "combine_backward.cuh"
#include "gemm_launch.cuh"
#include "grouped_gemm_mx4.cuh"
#include "simt_train.cuh"
#include "train_gemm.cuh"

namespace moe {

// Sets the kernel's dynamic shared memory once per device.
template <auto kern>
static cudaError_t allow_smem(int smem) {
  int dev = 0;
  cudaGetDevice(&dev);
  static std::mutex mu;
  static uint64_t configured = 0;   // one bit per device
  std::lock_guard<std::mutex> g(mu);
  if (dev < 64 && ((configured >> dev) & 1u)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev < 64) configured |= uint64_t(1) << dev;
  return e;
}

// Rows of bytes [groups, rows, row_bytes]; boxes of 128 B x box_rows, 128-byte swizzle.
static cudaError_t make_tmap_bytes(CUtensorMap* m, const void* ptr, uint64_t row_bytes, uint64_t rows,
                                   uint64_t groups, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {row_bytes, rows, groups ? groups : 1};
  const cuuint64_t strides[2] = {row_bytes, row_bytes * rows};
  const cuuint32_t box[3] = {128, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, groups ? 3 : 2, const_cast<void*>(ptr), dims, strides, box,
                        estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// bf16 rows [groups, rows, cols] that lie ld elements apart (groups 0: one matrix), as a
// K-rows x elements operand (train_gemm.cuh): boxes of 64 columns x 64 rows, alone and in
// pairs (only where the matrix has a whole box: below 64 columns no copy takes pairs).
static cudaError_t make_mn_maps(TrainMaps* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t ld,
                                 uint64_t groups) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  for (int two = 0; two <= (cols >= 64 ? 1 : 0); ++two) {
    const cuuint64_t dims_p[4] = {64, rows, cols / 64, groups}, dims_s[3] = {cols, rows, groups};
    const cuuint64_t strides_p[3] = {ld * 2, 128, rows * ld * 2}, strides_s[2] = {ld * 2, rows * ld * 2};
    const cuuint32_t box_p[4] = {64, 64, 2, 1}, box_s[3] = {64, 64, 1};
    const CUresult r = fn(two ? &m->two : &m->single, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (groups ? 3 : 2) + two,
                          const_cast<void*>(ptr), two ? dims_p : dims_s, two ? strides_p : strides_s,
                          two ? box_p : box_s, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

// ---------------------------------------------------------------------------
// MXFP4 product
// ---------------------------------------------------------------------------
// Runs of bytes as rows of 256 B; boxes of box_rows of them, no swizzle.
static cudaError_t make_tmap_runs(CUtensorMap* m, const void* ptr, uint64_t bytes, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {256, bytes / 256};
  const cuuint64_t strides[1] = {256};
  const cuuint32_t box[2] = {256, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename OutT>
static cudaError_t launch_mx4(const Launch& L, const Mx4Args& args, int64_t max_tiles) {
  const cudaError_t e = allow_smem<grouped_gemm_mx4_kernel<OutT>>(Mx4Layout::SMEM);
  if (e != cudaSuccess) return e;
  auto kern = grouped_gemm_mx4_kernel<OutT>;   // clusters of two CTAs
  pdl_launch(kern, dim3(2 * static_cast<int>(std::min<int64_t>(max_tiles, L.num_sms / 2))), dim3(kMx4Threads),
             Mx4Layout::SMEM, L.stream, args);
  count_launch();
  return cudaGetLastError();
}

cudaError_t mx4_product(const Launch& L, int64_t R, int N, int K, int G, const uint8_t* codes, const uint8_t* tiles,
                        const int32_t* off, const uint8_t* w_codes, const uint8_t* w_tiles, const void* bias,
                        bool out_f32, void* out) {
  Mx4Args a{};
  cudaError_t e;
  if ((e = make_tmap_bytes(&a.w, w_codes, K / 2, N, G, 128)) != cudaSuccess) return e;
  for (int q = 0; q < 3; ++q)
    if ((e = make_tmap_bytes(&a.x[q], codes, K / 2, R, 0, 32 * (q + 1))) != cudaSuccess) return e;
  const uint64_t wt = static_cast<uint64_t>(G) * ((N + 127) / 128) * mx4_chunks(K) * 512;
  if ((e = make_tmap_runs(&a.sw, w_tiles, wt, 4)) != cudaSuccess) return e;
  if ((e = make_tmap_runs(&a.sx, tiles, mx4_row_tiles_bytes(R, G, K), 8)) != cudaSuccess) return e;
  a.group_off = off;
  a.num_groups = G;
  a.m_total = static_cast<int>(R);
  a.n_out = N;
  a.k_dim = K;
  a.row_tiles = static_cast<int>(mx4_row_tiles(R, G));
  a.bias = static_cast<const __nv_bfloat16*>(bias);
  a.out = out;
  a.wait_limit_ns = L.wait_limit_ns;
  const int64_t max_tiles = mx4_row_tiles(R, G) * ((N + kMx4BM - 1) / kMx4BM);
  return out_f32 ? launch_mx4<float>(L, a, max_tiles) : launch_mx4<__nv_bfloat16>(L, a, max_tiles);
}

// ---------------------------------------------------------------------------
// expert block, training pass
// ---------------------------------------------------------------------------
template <int KIND, typename OutT>
static cudaError_t launch_train(const Launch& L, const TrainArgs<KIND>& args, int64_t max_tiles) {
  auto kern = ffn_train_kernel<KIND, OutT>;   // clusters of two CTAs
  const cudaError_t e = allow_smem<ffn_train_kernel<KIND, OutT>>(TrainLayout<KIND>::SMEM);
  if (e != cudaSuccess) return e;
  pdl_launch(kern, dim3(2 * static_cast<int>(std::min<int64_t>(max_tiles, L.num_sms / 2))), dim3(kTrThreads),
             TrainLayout<KIND>::SMEM, L.stream, args);
  count_launch();
  return cudaGetLastError();
}

template <int KIND>
static TrainArgs<KIND> train_args(const Launch& L, int64_t R, int E, int k_dim, const int32_t* off,
                                   const Activation& act) {
  TrainArgs<KIND> a{};
  a.num_jobs = 1;
  a.group_off = off;
  a.num_groups = E;
  a.m_total = static_cast<int>(R);
  a.k_dim = k_dim;
  a.limit = act.limit;
  a.alpha = act.alpha;
  a.gate_lo = act.gate_lo;
  a.wait_limit_ns = L.wait_limit_ns;
  return a;
}

static int64_t train_col_tiles(int n) { return (n + kTrBM - 1) / kTrBM; }

// Rows of a tile: the most the kernel takes, halved (to 64 at least) while the tiles of evenly
// loaded experts would not fill half of the CTA pairs, so that the halves still run at once.
// The host does not know the loads: the estimate gives every expert, empty ones too, the
// average.  (Backward of 8 experts, seven of 143 rows and one empty, D = 1440, F = 720, 74 pairs:
// DH, 24 full tiles by the estimate and 21 in fact, 22.2 us, is quartered to at most 64 rows, 63
// tiles of 48, 17.2 us; DX, 48 and 42, stays full, 15.4 us -- halved, more than a wave, 20.1.)
static int train_tile_rows(const Launch& L, int64_t R, int E, int n, int most) {
  const int64_t avg = std::max<int64_t>(1, (R + E - 1) / E), experts = std::min<int64_t>(E, R);
  while (most > 64 && 2 * experts * ((avg + most - 1) / most) * train_col_tiles(n) <= L.num_sms / 2) most /= 2;
  return most;
}

// Workspace of the backward pass: dgu [R, 2, F], then (bf16) the sums of dg and du by row tile
// (of 64 rows at least) and epilogue half, and the weight gradients' tile counter.
struct BackwardLayout {
  size_t part, counter, total;
};
static BackwardLayout backward_layout(bool bf16, int64_t R, int F, int E) {
  BackwardLayout l{};
  l.part = static_cast<size_t>(R) * 2 * F * (bf16 ? 2 : 4);
  l.total = l.part;
  if (bf16) {
    l.part = (l.part + 255) / 256 * 256;
    l.counter = l.part + static_cast<size_t>((R + 63) / 64 + E) * 2 * 2 * F * 4;
    l.total = l.counter + 16;
  }
  return l;
}
size_t expert_backward_bytes(bool bf16, int64_t R, int F, int E) { return backward_layout(bf16, R, F, E).total; }

// Launches a product with n output columns: tiles of at most `most` rows.
template <int KIND>
static cudaError_t launch_rows(const Launch& L, TrainArgs<KIND>& a, int64_t R, int E, int n) {
  a.tile_rows = train_tile_rows(L, R, E, n, TrainLayout<KIND>::ROWS);
  const int64_t row_tiles = (R + a.tile_rows - 1) / a.tile_rows + E;
  return launch_train<KIND, __nv_bfloat16>(L, a, row_tiles * train_col_tiles(n));
}

// Rows [R, K] in bf16 as the N operand: boxes of 64 elements x 32, 64, .. rows.
static cudaError_t make_row_maps(CUtensorMap* m, int count, const void* ptr, uint64_t K, uint64_t R) {
  for (int q = 0; q < count; ++q) {
    const cudaError_t e = make_tmap(&m[q], ptr, false, K, R, 0, 32 * (q + 1));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t expert_train_bf16(const Launch& L, int64_t R, int D, int F, int E, const void* x_perm,
                              const int32_t* off, const ExpertWeights& w, const Activation& act, void* gu, void* h,
                              void* y_perm) {
  cudaError_t e;
  {
    TrainArgs<TR_GATEUP> a = train_args<TR_GATEUP>(L, R, E, D, off, act);
    TrainJob& j = a.job[0];
    if ((e = make_tmap(&j.a.single, w.w_gate, false, D, F, E, 128)) != cudaSuccess) return e;
    if ((e = make_tmap(&j.a2.single, w.w_up, false, D, F, E, 128)) != cudaSuccess) return e;
    if ((e = make_row_maps(j.b, 2, x_perm, D, R)) != cudaSuccess) return e;
    j.out = h;
    j.bias0 = static_cast<const __nv_bfloat16*>(w.b_gate);
    j.bias1 = static_cast<const __nv_bfloat16*>(w.b_up);
    j.m = F;
    a.gu = static_cast<__nv_bfloat16*>(gu);
    if ((e = launch_rows(L, a, R, E, F)) != cudaSuccess) return e;
  }
  TrainArgs<TR_DOWN> a = train_args<TR_DOWN>(L, R, E, F, off, act);
  TrainJob& j = a.job[0];
  if ((e = make_tmap(&j.a.single, w.w_down, false, F, D, E, 128)) != cudaSuccess) return e;
  if ((e = make_row_maps(j.b, 4, h, F, R)) != cudaSuccess) return e;
  j.out = y_perm;
  j.bias0 = static_cast<const __nv_bfloat16*>(w.b_down);
  j.m = D;
  return launch_rows(L, a, R, E, D);
}

static cudaError_t expert_backward_bf16(const Launch& L, int64_t R, int D, int F, int E, const void* x_perm,
                                        const int32_t* off, const ExpertWeights& w, const Activation& act,
                                        const void* gu, const void* h, const void* dy, void* ws, void* dx,
                                        const ExpertGrads& gr, bool grad_f32) {
  cudaError_t e;
  const BackwardLayout LY = backward_layout(true, R, F, E);
  void* dgu = ws;
  float* part = (gr.b_gate != nullptr || gr.b_up != nullptr) ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + LY.part)
                                                             : nullptr;
  int* counter = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + LY.counter);
  const int dh_rows = train_tile_rows(L, R, E, F, TrainLayout<TR_DH>::ROWS);
  const int part_tiles = static_cast<int>((R + dh_rows - 1) / dh_rows + E);
  __nv_bfloat16* dg = static_cast<__nv_bfloat16*>(dgu);
  if (dx != nullptr || gr.w_gate != nullptr || gr.w_up != nullptr) {
    TrainArgs<TR_DH> a = train_args<TR_DH>(L, R, E, D, off, act);
    TrainJob& j = a.job[0];
    if ((e = make_mn_maps(&j.a, w.w_down, F, D, F, E)) != cudaSuccess) return e;
    if ((e = make_row_maps(j.b, 4, dy, D, R)) != cudaSuccess) return e;
    j.out = dgu;
    j.m = F;
    a.gu = static_cast<__nv_bfloat16*>(const_cast<void*>(gu));   // read only
    a.part = part;
    a.part_tiles = part_tiles;
    a.part_ld = 2 * F;
    a.counter = counter;
    if ((e = launch_rows(L, a, R, E, F)) != cudaSuccess) return e;
  }
  if (dx != nullptr) {
    TrainArgs<TR_DX> a = train_args<TR_DX>(L, R, E, F, off, act);
    TrainJob& j = a.job[0];
    if ((e = make_mn_maps(&j.a, w.w_gate, D, F, D, E)) != cudaSuccess) return e;
    if ((e = make_mn_maps(&j.a2, w.w_up, D, F, D, E)) != cudaSuccess) return e;
    for (int q = 0; q < 4; ++q)
      if ((e = make_tmap_halves(&j.b[q], dgu, F, R, 32 * (q + 1))) != cudaSuccess) return e;
    j.out = dx;
    j.m = D;
    if ((e = launch_rows(L, a, R, E, D)) != cudaSuccess) return e;
  }
  TrainArgs<TR_DW> a = train_args<TR_DW>(L, R, E, 0, off, act);
  a.num_jobs = 0;
  a.early = dx != nullptr;
  a.counter = counter;
  a.tile_rows = dh_rows;
  a.part_tiles = part_tiles;
  a.part_ld = 2 * F;
  int64_t tiles = 0;
  auto add = [&](void* out, void* bias_out, const float* sums, const void* pa, int m, int64_t lda, const void* pb, int n) {
    if (out == nullptr) return cudaSuccess;
    TrainJob& j = a.job[a.num_jobs++];
    j.out = out;
    j.bias_out = bias_out;
    j.part = bias_out == nullptr ? nullptr : sums;
    j.m = m;
    j.n = n;
    j.nt = train_col_blocks(n, bias_out != nullptr && sums == nullptr);
    tiles += int64_t(E) * (train_col_tiles(m)) * j.nt;
    const cudaError_t r = make_mn_maps(&j.a, pa, m, R, lda, 0);
    return r != cudaSuccess ? r : make_mn_maps(&j.bw, pb, n, R, n, 0);
  };
  if ((e = add(gr.w_down, gr.b_down, nullptr, dy, D, D, h, F)) != cudaSuccess) return e;
  if ((e = add(gr.w_gate, gr.b_gate, part, dg, F, 2 * F, x_perm, D)) != cudaSuccess) return e;
  if ((e = add(gr.w_up, gr.b_up, part == nullptr ? nullptr : part + F, dg + F, F, 2 * F, x_perm, D)) != cudaSuccess) return e;
  if (a.num_jobs == 0) return cudaSuccess;
  return grad_f32 ? launch_train<TR_DW, float>(L, a, tiles) : launch_train<TR_DW, __nv_bfloat16>(L, a, tiles);
}

// ---------------------------------------------------------------------------
// fp32 layers
// ---------------------------------------------------------------------------
static SimtTrainArgs simt_args(int64_t R, int E, const int32_t* off, const Activation& act) {
  SimtTrainArgs a{};
  a.group_off = off;
  a.num_groups = E;
  a.m_total = static_cast<int>(R);
  a.limit = act.limit;
  a.alpha = act.alpha;
  a.gate_lo = act.gate_lo;
  return a;
}

static unsigned simt_blocks(int64_t n, int tile) { return static_cast<unsigned>((n + tile - 1) / tile); }

template <int KIND>
static cudaError_t launch_simt(const Launch& L, const SimtTrainArgs& args, dim3 grid) {
  constexpr int smem = SimtShape<KIND>::kSmem;
  const cudaError_t e = allow_smem<simt_train_kernel<KIND>>(smem);
  if (e != cudaSuccess) return e;
  pdl_launch(simt_train_kernel<KIND>, grid, dim3(kStThreads), smem, L.stream, args);
  count_launch();
  return cudaGetLastError();
}

cudaError_t expert_train_f32(const Launch& L, int64_t R, int D, int F, int E, const float* x_perm,
                             const int32_t* off, const ExpertWeights& w, const Activation& act, float* gu, float* h,
                             float* y_perm) {
  const unsigned row_tiles = simt_blocks(R, SimtShape<SIMT_GATEUP>::kStM) + E;
  SimtTrainArgs a = simt_args(R, E, off, act);
  auto f = [](const void* p) { return static_cast<const float*>(p); };
  a.gu_out = gu;
  a.job[0] = SimtJob{x_perm, f(w.w_gate), f(w.w_up), f(w.b_gate), f(w.b_up), h, nullptr, D, D, 0, F, D};
  const cudaError_t e = launch_simt<SIMT_GATEUP>(L, a, dim3(row_tiles, simt_blocks(F, SimtShape<SIMT_GATEUP>::kStN)));
  if (e != cudaSuccess) return e;
  a.job[0] = SimtJob{h, f(w.w_down), nullptr, f(w.b_down), nullptr, y_perm, nullptr, F, F, 0, D, F};
  return launch_simt<SIMT_DOWN>(L, a, dim3(row_tiles, simt_blocks(D, SimtShape<SIMT_DOWN>::kStN)));
}

static cudaError_t expert_backward_f32(const Launch& L, int64_t R, int D, int F, int E, const float* x_perm,
                                       const int32_t* off, const ExpertWeights& w, const Activation& act,
                                       const float* gu, const float* h, const float* dy, float* dgu, float* dx,
                                       const ExpertGrads& gr) {
  const unsigned row_tiles = simt_blocks(R, SimtShape<SIMT_GATEUP>::kStM) + E;
  SimtTrainArgs a = simt_args(R, E, off, act);
  auto f = [](const void* p) { return static_cast<const float*>(p); };
  cudaError_t e;
  if (dx != nullptr || gr.w_gate != nullptr || gr.w_up != nullptr) {
    a.gu = gu;
    a.job[0] = SimtJob{dy, f(w.w_down), nullptr, nullptr, nullptr, dgu, nullptr, D, F, 0, F, D};
    if ((e = launch_simt<SIMT_DH>(L, a, dim3(row_tiles, simt_blocks(F, SimtShape<SIMT_DH>::kStN)))) != cudaSuccess) return e;
  }
  if (dx != nullptr) {
    a.job[0] = SimtJob{dgu, f(w.w_gate), f(w.w_up), nullptr, nullptr, dx, nullptr, 2 * F, D, 0, D, F};
    if ((e = launch_simt<SIMT_DX>(L, a, dim3(row_tiles, simt_blocks(D, SimtShape<SIMT_DX>::kStN)))) != cudaSuccess) return e;
  }
  a.early = dx != nullptr;
  int jobs = 0, most_m = 0, most_n = 0;
  auto add = [&](void* out, void* bias_out, const float* pa, int m, int lda, const float* pb, int n) {
    if (out == nullptr) return;
    a.job[jobs++] = SimtJob{pa, pb, nullptr, nullptr, nullptr, static_cast<float*>(out), static_cast<float*>(bias_out),
                            lda, n, m, n, 0};
    most_m = std::max(most_m, m);
    most_n = std::max(most_n, n);
  };
  add(gr.w_down, gr.b_down, dy, D, D, h, F);
  add(gr.w_gate, gr.b_gate, dgu, F, 2 * F, x_perm, D);
  add(gr.w_up, gr.b_up, dgu + F, F, 2 * F, x_perm, D);
  if (jobs == 0) return cudaSuccess;
  return launch_simt<SIMT_DW>(L, a, dim3(simt_blocks(most_m, SimtShape<SIMT_DW>::kStM), simt_blocks(most_n, SimtShape<SIMT_DW>::kStN), jobs * E));
}

cudaError_t expert_backward(const Launch& L, bool bf16, int64_t R, int D, int F, int E, const void* x_perm,
                            const int32_t* expert_off, const ExpertWeights& w, const Activation& act, const void* gu,
                            const void* h, const void* dy, void* ws, void* dx, const ExpertGrads& grads,
                            bool grad_f32) {
  if (bf16)
    return expert_backward_bf16(L, R, D, F, E, x_perm, expert_off, w, act, gu, h, dy, ws, dx, grads, grad_f32);
  return expert_backward_f32(L, R, D, F, E, static_cast<const float*>(x_perm), expert_off, w, act,
                             static_cast<const float*>(gu), static_cast<const float*>(h),
                             static_cast<const float*>(dy), static_cast<float*>(ws), static_cast<float*>(dx), grads);
}

template <typename T, int KM>
static void launch_combine_backward(const Launch& L, int64_t Tn, int D, int k, const void* dy, const void* y_perm,
                                    const int32_t* row_of_slot, const float* w, void* dy_perm, float* dw) {
  const int threads = std::min(kCombineBwdThreads, (D / 8 + 31) / 32 * 32);
  pdl_launch(combine_backward_kernel<T, KM>, dim3(static_cast<unsigned>(Tn)), dim3(threads), 0, L.stream,
             static_cast<const T*>(dy), static_cast<const T*>(y_perm), row_of_slot, w, static_cast<int>(Tn), k, D,
             static_cast<T*>(dy_perm), dw);
  count_launch();
}

cudaError_t combine_backward(const Launch& L, bool bf16, int64_t T, int D, int k, const void* dy, const void* y_perm,
                             const int32_t* row_of_slot, const float* w, void* dy_perm, float* dw) {
  if (bf16 && k <= 4) launch_combine_backward<__nv_bfloat16, 4>(L, T, D, k, dy, y_perm, row_of_slot, w, dy_perm, dw);
  else if (bf16) launch_combine_backward<__nv_bfloat16, 8>(L, T, D, k, dy, y_perm, row_of_slot, w, dy_perm, dw);
  else if (k <= 4) launch_combine_backward<float, 4>(L, T, D, k, dy, y_perm, row_of_slot, w, dy_perm, dw);
  else launch_combine_backward<float, 8>(L, T, D, k, dy, y_perm, row_of_slot, w, dy_perm, dw);
  return cudaGetLastError();
}

}  // namespace moe
