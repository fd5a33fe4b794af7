// Device helpers of the training and MXFP4 kernels, beside common.cuh.
#pragma once

#include "common.cuh"

namespace moe {

// pdl_enter in two parts, for kernels that set up barriers and TMEM in between: nothing that
// an earlier kernel may have written is read before pdl_wait.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Writes v to another CTA's shared memory and counts its 4 bytes on a barrier there
// (addresses from mapa_shared).
__device__ __forceinline__ void st_async(uint32_t addr, int v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.s32 [%0], %1, [%2];" ::"r"(addr), "r"(v), "r"(bar)
               : "memory");
}

// v clipped into [lo, hi]; a NaN stays one (fminf and fmaxf would drop it, and a diverged
// training step would go unseen).
__device__ __forceinline__ float clip_nan(float v, float lo, float hi) {
  asm("max.NaN.f32 %0, %0, %1;\n\tmin.NaN.f32 %0, %0, %2;" : "+f"(v) : "f"(lo), "f"(hi));
  return v;
}

// The same into [-lim, lim].
__device__ __forceinline__ float clip_nan(float v, float lim) {
  asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(v) : "f"(lim));
  return v;
}

// 1 / (1 + 2^z) of two values, on the approximate units (2 ulp each): the results here are
// rounded to bf16, or to 8 bits more for a sum.
__device__ __forceinline__ float2 sigmoid2_neg_log2(float2 z) {
  float2 e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(z.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(z.y));
  e = __fadd2_rn(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(e.y));
  return s;
}

}  // namespace moe
