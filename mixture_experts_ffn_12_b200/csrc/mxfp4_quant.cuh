// MXFP4 quantization: rows of bf16 or fp32 to E2M1 codes with one E8M0 scale per 32
// elements along K, and back.
//
// For a block b of 32 consecutive elements of a row
//   X = the smallest integer >= -127 with max |b| <= 6 * 2^X   (6 = the largest E2M1 value,
//       so no element saturates; -127 for an all-zero block),
//   code = RNE to E2M1 of b / 2^X,   scale byte = X + 127,
// and a block that holds an infinity or a NaN gets scale byte 255 (the E8M0 NaN) and
// zero codes, so that it reads back as NaN instead of as a wrong number.
//
// Bound by memory: 2 (bf16) or 4 (fp32) bytes read and 0.53 written an element, close to
// where its instructions bound it too, so both count: two lanes share a block (16 elements
// each, about 5 instructions an element where 8 each took 9), and their 32 bytes are one
// access where the address allows it (as two accesses of 16 bytes, 32 apart, they ran
// slower than 8 elements a lane).  bf16 maxima and scaling run on packed pairs.
// 92160 x 2880 bf16: quantize 98 us (6.8 TB/s), dequantize 117 us (5.8 TB/s); with 8 elements a
// lane 246 us for both, now 222.  Activations into tiles, 16384 x 2880: 26 us (4.6 TB/s, of which
// some 3 us are the launch's).
//
// Scale layouts.  "Rows": [rows, K/32], what the MXFP4 expert weights of the layer use.
// "Tiles": what the 4-bit x 4-bit product reads: for 128 rows and 128 elements of K one
// 512-byte chunk, in which byte 16 (r % 32) + 4 (r / 32) + b holds row r's scale of block
// b = 0..3 -- the 32-lane x 16-byte image that tcgen05.cp copies to TMEM.  Padding along K
// holds 127 (2^0: it scales codes that read as zero), padding rows are never used.
//   Weights: row blocks of 128 within each group, a block's chunks one after another along
//   K, an even number of them (a pipeline stage of the product covers 256 elements).
//   Activations: a group's rows split evenly into tiles of at most 192 (mx4_rows_per_tile,
//   the product's N), for each tile and 256 elements of K 2 x 2 chunks: of the tile's rows
//   below and above 128 for the first 128 elements, then for the others.
#pragma once

#include "device_util.cuh"
#include "grouped_gemm_mx8.cuh"

namespace moe {

// 128-element chunks of a scale tile row, an even number.
__host__ __device__ constexpr int mx4_chunks(int K) { return 2 * ((K + 255) / 256); }

// Rows of the product's tiles: a group's rows in `tiles` = ceil(rows / kMx4Rows) even parts,
// a multiple of 16 each (never above kMx4Rows, never leaving a tile without rows).
constexpr int kMx4Rows = 192;
__host__ __device__ constexpr int mx4_rows_per_tile(int rows, int tiles) {
  return ((rows + tiles - 1) / tiles + 15) / 16 * 16;
}

// The block scale exponent from the largest |x| as fp32 bits (finite): 6 = 1.5 * 2^2.
__device__ __forceinline__ int mx4_exponent(uint32_t amax_bits) {
  const int ef = static_cast<int>(amax_bits >> 23);
  if (ef == 0) return -127;
  return max(-127, (ef - 127) - 2 + ((amax_bits & 0x7FFFFFu) > 0x400000u ? 1 : 0));
}

// Eight floats to E2M1 codes, round to nearest even, v[0] in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight E2M1 codes (low nibble first) to floats.
__device__ __forceinline__ void e2m1x8_to_f32(uint32_t q, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

// 8 elements as loaded, to floats.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4* raw, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(raw);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __bfloat1622float2(h[j]);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  } else {
    const float* f = reinterpret_cast<const float*>(raw);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f[j];
  }
}

// 32 bytes at once where `kA32` (a 32-byte aligned address), else in two.
template <bool kA32>
__device__ __forceinline__ void load32(uint4 (&v)[2], const uint4* p) {
  if constexpr (kA32) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z),
                   "=r"(v[1].w)
                 : "l"(p));
  } else {
    v[0] = p[0];
    v[1] = p[1];
  }
}
template <bool kA32>
__device__ __forceinline__ void store32(uint4* p, const uint4 (&v)[2]) {
  if constexpr (kA32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0].x), "r"(v[0].y),
                 "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z), "r"(v[1].w)
                 : "memory");
  } else {
    p[0] = v[0];
    p[1] = v[1];
  }
}

// 16 elements of a block that a lane and its neighbour (lane ^ 1) share, as loaded: 16 codes
// and the scale byte.
template <typename T>
__device__ __forceinline__ uint2 mx4_quantize16(const uint4* raw, uint32_t& scale) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(raw);
  uint32_t m;                                 // the largest |x| as fp32 bits: |x| orders as its bits do
  if constexpr (sizeof(T) == 2) {
    uint32_t m2 = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m2 = __vmaxu2(m2, r[j] & 0x7FFF7FFFu);
    m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
    m = max(m2 & 0xFFFFu, m2 >> 16) << 16;
  } else {
    m = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, r[j] & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  }
  if (m >= 0x7F800000u) {                     // an infinity or a NaN in the block
    scale = 255;
    return make_uint2(0, 0);
  }
  const int X = mx4_exponent(m);
  scale = static_cast<uint32_t>(X + 127);
  uint2 q;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float v[8];
    if constexpr (sizeof(T) == 2) {
      const uint16_t ib = static_cast<uint16_t>((127 - X) << 7);    // 2^-X, X in [-127, 126]
      const __nv_bfloat162 inv = __halves2bfloat162(__ushort_as_bfloat16(ib), __ushort_as_bfloat16(ib));
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(raw + w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // exact, or so small that it rounds to zero either way
        const float2 f = __bfloat1622float2(__hmul2(h[j], inv));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    } else {
      const float inv = exp2_int(-X);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[8 * w + j]) * inv;
    }
    (w == 0 ? q.x : q.y) = e2m1x8(v);
  }
  return q;
}

// x [nblk, 32] -> codes [nblk, 16 B], scales [nblk]: rows of any width are runs of blocks.
// A thread loads kMx4Unroll pieces before it uses the first.
constexpr int kMx4Unroll = 2;
template <typename T, bool kA32>
__global__ void __launch_bounds__(256) mx4_quant_rows_kernel(const T* __restrict__ x, int64_t nblk,
                                                             uint2* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
  pdl_enter();
  const int64_t total = nblk * 2;   // lanes; whole warps take part in the shuffles
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256 * kMx4Unroll;
  constexpr int kWords = sizeof(T);   // 16-byte words of 16 elements
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * 256 * kMx4Unroll; base < total; base += step) {
    const uint4* src = reinterpret_cast<const uint4*>(x) + base * kWords;
    uint2* dst = codes + base;
    uint8_t* sdst = scales + (base >> 1);
    const int left = static_cast<int>(min(total - base, static_cast<int64_t>(256 * kMx4Unroll)));
    uint4 raw[kMx4Unroll][kWords / 2][2] = {};
#pragma unroll
    for (int u = 0; u < kMx4Unroll; ++u) {
      const int i = u * 256 + threadIdx.x;
      if (i < left)
#pragma unroll
        for (int w = 0; w < kWords / 2; ++w) load32<kA32>(raw[u][w], src + i * kWords + 2 * w);
    }
#pragma unroll
    for (int u = 0; u < kMx4Unroll; ++u) {
      const int i = u * 256 + threadIdx.x;
      uint32_t s;
      const uint2 q = mx4_quantize16<T>(raw[u][0], s);
      if (i < left) {
        dst[i] = q;
        if ((i & 1) == 0) sdst[i >> 1] = static_cast<uint8_t>(s);
      }
    }
  }
}

// Row-group table of a kernel: goff[g] (clamped into [0, rows]) and the prefix of the groups'
// blocks of at most `most` rows.  Called by one whole warp; G <= kMaxGroups.
__device__ __forceinline__ void group_table(const int32_t* off, int G, int rows, int most, int* goff, int* blk) {
  const int lane = threadIdx.x & 31;
  int bad = 0;
  for (int g = lane; g <= G; g += 32) {
    int v = off == nullptr ? (g == 0 ? 0 : rows) : off[g];
    if (v < 0 || v > rows) { bad = 1; v = min(max(v, 0), rows); }
    goff[g] = v;
  }
  __syncwarp();
  int running = 0;
  if (lane == 0) blk[0] = 0;
  for (int base = 0; base < G; base += 32) {
    const int g = base + lane;
    int cnt = 0;
    if (g < G) {
      const int n = goff[g + 1] - goff[g];
      if (n < 0) bad = 1;
      cnt = n > 0 ? (n + most - 1) / most : 0;
    }
    int incl = cnt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (g < G) blk[g + 1] = running + incl;
    running += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) flag_error(DEVERR_BOUNDS);
}

// x [rows, K] bf16, rows grouped by off (null: one group) -> codes [rows, K/2] and scale
// tiles, the row tiles counted group after group.  Rows outside every group are skipped.
// A warp takes `spans` runs of kMx4QuantSpan elements of a row (blockIdx.y picks which): the
// row's place in the tiles is looked up once, all loads of a run are in flight before the
// first is used, and the scales of 128 elements (four blocks, 8 lanes) leave as one word.
constexpr int kMx4QuantSpan = 1024;
template <bool kA32>
__global__ void __launch_bounds__(256) mx4_quant_tiles_kernel(const __nv_bfloat16* __restrict__ x, int rows, int K,
                                                              const int32_t* __restrict__ off, int G, int max_tiles,
                                                              int spans, uint2* __restrict__ codes,
                                                              uint8_t* __restrict__ tiles) {
  // First the wait, then the dependents: the product that follows starts when everything
  // before this kernel is complete, and may read weights and offsets while this one runs.
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int goff[kMaxGroups + 2];
  __shared__ int tile_off[kMaxGroups + 2];
  if (threadIdx.x < 32) group_table(off, G, rows, kMx4Rows, goff, tile_off);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int kc = mx4_chunks(K);
  const int k_first = blockIdx.y * spans * kMx4QuantSpan;
  const int k_end = min(k_first + spans * kMx4QuantSpan, kc * 128);
  constexpr int IT = kMx4QuantSpan / 512;
  for (int64_t r = blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += gridDim.x * 8) {
    const int row = static_cast<int>(r);
    const __nv_bfloat16* src = x + static_cast<size_t>(row) * K;
    uint2* crow = codes + (static_cast<size_t>(row) * K >> 4);
    uint8_t* dst = nullptr;
    for (int kb = k_first; kb < k_end; kb += kMx4QuantSpan) {
      uint4 raw[IT][2] = {};
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        const int k = kb + 512 * t + lane * 16;
        if (k < K) load32<kA32>(raw[t], reinterpret_cast<const uint4*>(src + k));
      }
      if (kb == k_first) {
        int lo = 0, hi = G;   // goff[lo] <= row < goff[hi] where the row is in a group
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (goff[mid] <= row) lo = mid; else hi = mid;
        }
        const int grows = goff[lo + 1] - goff[lo];
        int p = row - goff[lo];
        if (p >= 0 && p < grows) {
          const int per = mx4_rows_per_tile(grows, tile_off[lo + 1] - tile_off[lo]);
          const int t = p / per;
          p -= t * per;
          const int tile = tile_off[lo] + t;
          if (tile < max_tiles)   // else: offsets that are not ascending (flagged)
            dst = tiles + static_cast<size_t>(tile) * kc * 1024 + 512 * (p >> 7) + 16 * (p & 31) + 4 * ((p & 127) >> 5);
        }
      }
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        const int k = kb + 512 * t + lane * 16;
        uint32_t s;
        const uint2 q = mx4_quantize16<__nv_bfloat16>(raw[t], s);
        if (k < K) crow[k >> 4] = q;
        else s = 127;
        // lanes 0, 2, 4, 6 of each eight hold the scales of a chunk's four blocks
        uint32_t w = s << (8 * ((lane >> 1) & 3));
        w |= __shfl_xor_sync(0xffffffffu, w, 2);
        w |= __shfl_xor_sync(0xffffffffu, w, 4);
        if (dst != nullptr && (lane & 7) == 0 && k < kc * 128)
          *reinterpret_cast<uint32_t*>(dst + static_cast<size_t>(k >> 7) * 1024) = w;
      }
    }
  }
}

// Scales [G, N, nb] as tiles, every group's row blocks on their own.  One thread per 4-byte
// word (four K blocks of one row).
__global__ void __launch_bounds__(256) mx4_scale_tiles_kernel(const uint8_t* __restrict__ scales, int G, int N,
                                                              int nb, uint32_t* __restrict__ tiles) {
  pdl_enter();
  const int kc = 2 * ((nb + 7) / 8), nblk = (N + kBM - 1) / kBM;
  const int64_t total = static_cast<int64_t>(G) * nblk * kc * 128;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
    const int w = static_cast<int>(i & 127);                 // word of the chunk: lane w / 4, row quarter w % 4
    const int64_t chunk = i >> 7;
    const int c = static_cast<int>(chunk % kc);
    const int64_t rbg = chunk / kc;
    const int rb = static_cast<int>(rbg % nblk);
    const int g = static_cast<int>(rbg / nblk);
    const int row = rb * kBM + (w & 3) * 32 + (w >> 2);
    uint32_t v = 0x7F7F7F7Fu;
    if (row < N) {
      const uint8_t* s = scales + (static_cast<size_t>(g) * N + row) * nb;
      v = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) v |= (4 * c + b < nb ? static_cast<uint32_t>(s[4 * c + b]) : 127u) << (8 * b);
    }
    tiles[i] = v;
  }
}

// codes [nblk, 16 B], scales [nblk] -> values; scale byte 255 gives NaN.
template <typename T, bool kA32>
__global__ void __launch_bounds__(256) mx4_dequant_rows_kernel(const uint2* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int64_t nblk,
                                                               T* __restrict__ out) {
  pdl_enter();
  const int64_t total = nblk * 2;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256 * kMx4Unroll;
  constexpr int kWords = sizeof(T);   // 16-byte words of 16 elements
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * 256 * kMx4Unroll; base < total; base += step) {
    const uint2* src = codes + base;
    const uint8_t* ssrc = scales + (base >> 1);
    uint4* dst = reinterpret_cast<uint4*>(out) + base * kWords;
    const int left = static_cast<int>(min(total - base, static_cast<int64_t>(256 * kMx4Unroll)));
    uint2 q[kMx4Unroll];
    int s[kMx4Unroll];
#pragma unroll
    for (int u = 0; u < kMx4Unroll; ++u) {
      const int i = u * 256 + threadIdx.x;
      q[u] = i < left ? src[i] : make_uint2(0, 0);
      s[u] = i < left ? ssrc[i >> 1] : 0;
    }
#pragma unroll
    for (int u = 0; u < kMx4Unroll; ++u) {
      const int i = u * 256 + threadIdx.x;
      const float f = s[u] == 255 ? __uint_as_float(0x7FC00000u) : exp2_int(s[u] - 127);
      float v[16];
      e2m1x8_to_f32(q[u].x, *reinterpret_cast<float(*)[8]>(v));
      e2m1x8_to_f32(q[u].y, *reinterpret_cast<float(*)[8]>(v + 8));
      uint4 o[kWords / 2][2];
      uint32_t* w = reinterpret_cast<uint32_t*>(o);
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j] * f, v[2 * j + 1] * f);
          w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(v[j] * f);
      }
      if (i < left)
#pragma unroll
        for (int p = 0; p < kWords / 2; ++p) store32<kA32>(dst + i * kWords + 2 * p, o[p]);
    }
  }
}

static int mx4_blocks(const Launch& L, int64_t threads) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((threads + 255) / 256, int64_t(L.num_sms) * 8)));
}

static bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

template <typename T>
static void launch_quant_rows(const Launch& L, int64_t nblk, const void* x, uint8_t* codes, uint8_t* scales) {
  auto kern = aligned32(x) ? mx4_quant_rows_kernel<T, true> : mx4_quant_rows_kernel<T, false>;
  pdl_launch(kern, dim3(mx4_blocks(L, nblk * 2 / kMx4Unroll + 1)), dim3(256), 0, L.stream, static_cast<const T*>(x),
             nblk, reinterpret_cast<uint2*>(codes), scales);
}

cudaError_t mx4_quant_rows(const Launch& L, bool bf16, int64_t rows, int K, const void* x, uint8_t* codes,
                           uint8_t* scales) {
  if (bf16) launch_quant_rows<__nv_bfloat16>(L, rows * (K / 32), x, codes, scales);
  else launch_quant_rows<float>(L, rows * (K / 32), x, codes, scales);
  count_launch();
  return cudaGetLastError();
}

template <typename T>
static void launch_dequant_rows(const Launch& L, int64_t nblk, const uint8_t* codes, const uint8_t* scales, void* out) {
  auto kern = aligned32(out) ? mx4_dequant_rows_kernel<T, true> : mx4_dequant_rows_kernel<T, false>;
  pdl_launch(kern, dim3(mx4_blocks(L, nblk * 2 / kMx4Unroll + 1)), dim3(256), 0, L.stream,
             reinterpret_cast<const uint2*>(codes), scales, nblk, static_cast<T*>(out));
}

cudaError_t mx4_dequant_rows(const Launch& L, bool bf16, int64_t rows, int K, const uint8_t* codes,
                             const uint8_t* scales, void* out) {
  if (bf16) launch_dequant_rows<__nv_bfloat16>(L, rows * (K / 32), codes, scales, out);
  else launch_dequant_rows<float>(L, rows * (K / 32), codes, scales, out);
  count_launch();
  return cudaGetLastError();
}

cudaError_t mx4_scale_tiles(const Launch& L, int G, int N, int K, const uint8_t* scales, uint8_t* tiles) {
  const int64_t words = static_cast<int64_t>(G) * ((N + kBM - 1) / kBM) * mx4_chunks(K) * 128;
  pdl_launch(mx4_scale_tiles_kernel, dim3(mx4_blocks(L, words)), dim3(256), 0, L.stream, scales, G, N, K / 32,
             reinterpret_cast<uint32_t*>(tiles));
  count_launch();
  return cudaGetLastError();
}

// Row tiles that R rows in G groups can take: every group may end in a partial one.
int64_t mx4_row_tiles(int64_t R, int G) { return (R + kMx4Rows - 1) / kMx4Rows + std::min<int64_t>(G - 1, R); }
size_t mx4_row_tiles_bytes(int64_t R, int G, int K) {
  return static_cast<size_t>(mx4_row_tiles(R, G)) * mx4_chunks(K) * 1024;
}

cudaError_t mx4_quant_tiles(const Launch& L, int64_t R, int K, const void* x, const int32_t* off, int G,
                            uint8_t* codes, uint8_t* tiles) {
  // many rows: a warp takes whole rows; few: every run of a row is a warp of its own
  const int runs = (K + kMx4QuantSpan - 1) / kMx4QuantSpan;
  const int spans = R >= int64_t(32) * L.num_sms ? runs : 1;
  const unsigned bx = static_cast<unsigned>(std::min<int64_t>((R + 7) / 8, int64_t(L.num_sms) * 8));
  auto kern = aligned32(x) ? mx4_quant_tiles_kernel<true> : mx4_quant_tiles_kernel<false>;
  pdl_launch(kern, dim3(bx, (runs + spans - 1) / spans), dim3(256), 0, L.stream,
             static_cast<const __nv_bfloat16*>(x), static_cast<int>(R), K, off, G,
             static_cast<int>(mx4_row_tiles(R, G)), spans, reinterpret_cast<uint2*>(codes), tiles);
  count_launch();
  return cudaGetLastError();
}

}  // namespace moe
