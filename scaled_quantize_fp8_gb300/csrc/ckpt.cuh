// Activation checkpoints in 8 bits: E4M3 codes [rows][cols] and, for every 32 columns of a row, the
// E8M0 byte of the smallest power of two that holds the block in E4M3's range (the MXFP8 rule), in
// the row's order: [rows][4 ceil(cols / 128)], so that 128 columns have one word. A value read back
// is code * 2^e, exact in fp32.
#pragma once

#include "norm.cuh"

namespace fp8lin {

// Bytes of a row's scales.
__host__ __device__ __forceinline__ int64_t ckpt_pitch(int64_t cols) {
  return (cols + 127) / 128 * 4;
}

// 2^(byte - 127); NaN for 0xFF, the byte of a block that held an infinity or a NaN.
__device__ __forceinline__ float ckpt_factor(uint32_t byte) {
  return byte == 0xFFu ? __uint_as_float(0x7FC00000u)
         : byte == 0   ? __uint_as_float(0x00400000u)
                       : __uint_as_float(byte << 23);
}

// Largest magnitude of eight packed bf16 values as the 31 bits of an fp32 (NaN above all).
__device__ __forceinline__ uint32_t bf16x8_mag(uint4 v) {
  const uint32_t a = absmax_bf16x2(absmax_bf16x2(v.x & 0x7FFF7FFFu, v.y), v.z);
  return fold_bf16x2(absmax_bf16x2(a, v.w)) << 16;
}

// Eight codes -> four pairs of floats.
__device__ __forceinline__ void ckpt_widen8(uint2 c, float2 (&f)[4]) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w[i]));
    f[2 * i] = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    f[2 * i + 1] = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  }
}

// The checkpoint of a row that lies in the registers of its threads as norm_row_copy takes it, as
// floats (zeros where a lane has no column); codes: of the thread's first vector, scale: of the row.
template <int V, bool FULL>
__device__ __forceinline__ void ckpt_row(const float2 (&x)[V][4], uint8_t* codes, uint8_t* scale,
                                         int lane, const RowUnits at, int nv, bool live,
                                         uint64_t policy) {
  const int wl = (int(threadIdx.y) * int(blockDim.x) + int(threadIdx.x)) & 31;
  uint32_t m[V];
  float mult[V];
#pragma unroll
  for (int j = 0; j < V; ++j) m[j] = __float_as_uint(max8_abs(x[j]));
  int v;
  const uint32_t word = mx_row_word<V>(m, mult, lane, at, &v);
  if (live && v < nv) *reinterpret_cast<uint32_t*>(scale + (v >> 2)) = word;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float s = mx_mult<V>(mult, j, wl);
    const float2 s2 = make_float2(s, s);
    float2 c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = __fmul2_rn(x[j][k], s2);
    if (FULL || (live && at(j) < nv))
      stg_v2_policy(codes + 8 * j * at.step,
                    make_uint2(cvt_e4m3x4(c[0].x, c[0].y, c[1].x, c[1].y),
                               cvt_e4m3x4(c[2].x, c[2].y, c[3].x, c[3].y)),
                    policy);
  }
}

}  // namespace fp8lin
