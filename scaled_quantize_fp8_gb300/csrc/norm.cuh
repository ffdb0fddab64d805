// Device helpers shared by the norm's forward and backward kernels.
#pragma once

#include "common.cuh"

namespace fp8lin {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// h of two packed elements: bf16(x + residual), one rounding (the packed bf16 add).
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                      *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&s);
}

// gamma of eight consecutive columns as fp32.
__device__ __forceinline__ void load_gamma8(const void* gamma, int gamma_fp32, int c, float* g) {
  if (gamma_fp32) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(gamma) + c);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
    g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(
        reinterpret_cast<const uint16_t*>(gamma) + c));
    g[0] = bf16_lo(v.x); g[1] = bf16_hi(v.x); g[2] = bf16_lo(v.y); g[3] = bf16_hi(v.y);
    g[4] = bf16_lo(v.z); g[5] = bf16_hi(v.z); g[6] = bf16_lo(v.w); g[7] = bf16_hi(v.w);
  }
}

// y of eight elements from their packed h.
__device__ __forceinline__ void norm8(uint4 h, float rstd, const float* g, float* y) {
  const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __fmul_rn(__fmul_rn(bf16_lo(w[i]), rstd), g[2 * i]);
    y[2 * i + 1] = __fmul_rn(__fmul_rn(bf16_hi(w[i]), rstd), g[2 * i + 1]);
  }
}

// Threads per row and vectors (eight columns) a thread for the kernels that keep a row in the
// registers of one thread group: at most 512 threads, 16 or a multiple of 32, and no more
// vectors than that needs.
struct RowPlan {
  int v, tpr, block;
};
inline RowPlan row_plan(int cols, int min_v, int block) {
  const int nv = cols / 8;
  int v = 1;
  while ((nv + v - 1) / v > 512) v *= 2;
  while (v < min_v && (nv + v - 1) / v > 32) v *= 2;
  int tpr = (nv + v - 1) / v;
  tpr = tpr <= 16 ? 16 : (tpr + 31) / 32 * 32;
  return {v, tpr, tpr >= block ? tpr : tpr * (block / tpr)};
}

}  // namespace fp8lin
