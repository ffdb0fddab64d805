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

// Eight bf16 as four pairs of floats.
__device__ __forceinline__ void widen8(uint4 v, float2 (&f)[4]) {
  f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
  f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
  f[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z));
  f[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
}

// gamma (bf16 or fp32) of the eight columns from c on; zeros beyond the tensor.
__device__ __forceinline__ void gamma_pairs(const void* gamma, int gamma_fp32, int cols, int c,
                                            float2 (&g)[4]) {
  if (c >= cols) {
#pragma unroll
    for (int k = 0; k < 4; ++k) g[k] = make_float2(0.0f, 0.0f);
  } else if (gamma_fp32) {
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(gamma) + c);
    const float4 a = __ldg(q), b = __ldg(q + 1);
    g[0] = make_float2(a.x, a.y);
    g[1] = make_float2(a.z, a.w);
    g[2] = make_float2(b.x, b.y);
    g[3] = make_float2(b.z, b.w);
  } else {
    widen8(__ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(gamma) + c)), g);
  }
}

// mx_scale_offset of a tensor with less than 2^31 elements, in 32 bits.
__device__ __forceinline__ uint32_t mx_scale_offset32(uint32_t r, uint32_t kb, uint32_t cols) {
  return ((r >> 7) * (cols >> 7) + (kb >> 2)) * 512u + (r & 31u) * 16u + ((r & 127u) >> 5) * 4u +
         (kb & 3u);
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
