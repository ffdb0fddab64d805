// Device helpers shared by the kernels that normalise rows, forward and backward.
#pragma once

#include "common.cuh"
#include "internal.cuh"

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

enum NormOut : int { N_STATS = 0, N_TENSOR = 1, N_MX = 2, N_BW = 3 };

struct NormParams {
  const uint16_t* x;          // [rows][cols], pitch ldx
  const uint16_t* res;        // pitch ldr, or null
  const void* gamma;
  int64_t ldx, ldr;
  int64_t rows, rows_pad;     // rows_pad: a multiple of the recipe's row quantum
  int cols;
  int gamma_fp32;
  float eps, inv_cols;
  uint16_t* h;                // [rows][cols] (written with a residual)
  float* rstd;                // [rows] or null
  uint16_t* y;                // [rows][cols] bf16(y) or null
  uint8_t* row;               // [rows_pad][cols] codes
  void* row_scale;
  uint8_t* col;               // [cols][rows_pad] codes, or bf16 with col_bf16
  void* col_scale;
  const float* scale_in;      // per-tensor scale to cast with (delayed), or null
  uint32_t* part;             // amax partials (31-bit magnitudes), one per CTA, or null
  int n_part;                 // column kernel: partials to reduce
  float* amax_out;            // per-tensor recipes: written by CTA 0 of the last kernel
  float* scale_out;           // tensorwise: written
  float* scale_inv_out;
  int margin;
  int pow2;                   // blockwise: power-of-two scales in the MXFP8 layout
  int col_bf16;
  int keep_h;                 // row kernel: h (x without a residual) is read again, from L2
  const uint8_t* ck;          // the checkpoint of h instead of x and h (ckpt.cuh), or null; then
  const uint8_t* ck_scale;    // rstd and gamma, read only, may both be null: y is h
};

// |a|, |b|, |c|: the largest; NaN if one of them is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// y of a row's eight columns: (h rstd) gamma, each product rounded.
__device__ __forceinline__ void norm_row8(uint4 h, float rstd, const float2 (&g)[4],
                                          float2 (&y)[4]) {
  const float2 r = make_float2(rstd, rstd);
  float2 f[4];
  widen8(h, f);
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] = __fmul2_rn(__fmul2_rn(f[k], r), g[k]);
}
__device__ __forceinline__ float max8_abs(const float2 (&y)[4]) {
  const float m = max3_abs(max3_abs(y[0].x, y[0].y, y[1].x), y[1].y, y[2].x);
  return max3_abs(max3_abs(m, y[2].y, y[3].x), y[3].y, 0.0f);
}

// The sum of a row's threads (a group of tpr: 16, or a whole number of warps), the same in each of
// them: over the lanes, then over the warps in order. One barrier of the group's own; red's two
// halves are used by turns, so the next sum need not wait for the last reader of this one.
template <int N>
__device__ __forceinline__ float row_sum(float v, float (&red)[2][N], int& phase, int warps,
                                         int lane, int grp, int tpr) {
  if (warps != 0) v += __shfl_xor_sync(0xffffffffu, v, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps > 1) {
    float* q = red[phase] + grp * warps;
    if ((lane & 31) == 0) q[lane >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(tpr) : "memory");
    v = 0.0f;
    if ((warps & 3) == 0) {
      for (int i = 0; i < warps; i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(q + i);
        v += (a.x + a.y) + (a.z + a.w);
      }
    } else {
      for (int i = 0; i < warps; ++i) v += q[i];
    }
    phase ^= 1;
  }
  return v;
}

// Largest magnitude over the CTA, in thread 0 (red: one word per warp).
__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  const int t = threadIdx.y * blockDim.x + threadIdx.x;
  __syncthreads();
  if ((t & 31) == 0) red[t >> 5] = v;
  __syncthreads();
  uint32_t m = 0;
  for (int i = 0; i < int((blockDim.x * blockDim.y) >> 5); ++i) m = max(m, red[i]);
  return m;
}

// Reduce the V vectors' values over the lanes that differ in the bits OFF .. 1: as long as there
// is more than one vector, a lane passes on half of them and keeps the half that its bit names.
// With L = 2 OFF lanes: for V >= L lane l ends with the vectors (V / L) (l % L) .. in m[0] ..,
// for V < L with vector (l % L) / (L / V) in m[0].
template <int V, int OFF>
__device__ __forceinline__ void scatter_max(uint32_t (&m)[V]) {
  const int lane = threadIdx.x & 31;
  int n = V;
#pragma unroll
  for (int off = OFF; off > 0; off >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        if (i < n)
          m[i] = max(up ? m[i + n] : m[i],
                     __shfl_xor_sync(0xffffffffu, up ? m[i] : m[i + n], off));
    } else {
      m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], off));
    }
  }
}

// Where a thread's vectors lie in its row: vector j holds the eight columns of unit first + j step.
// The 16 lanes (by their number in the warp, modulo 16) that share a vector have consecutive units.
struct RowUnits {
  int first, step;
  __device__ __forceinline__ int operator()(int j) const { return first + j * step; }
};

// A row's blocks of 32 columns (four lanes to a vector's block): reduces the lanes' magnitudes m (31
// bits) and leaves the multipliers of the blocks that this lane scales in mult (see mx_mult). Four
// blocks, the 16 lanes' share of a vector, make one word of E8M0 bytes: returns a word and in *v
// the first unit of its blocks, or a unit beyond every row where another lane has the word.
template <int V>
__device__ __forceinline__ uint32_t mx_row_word(uint32_t (&m)[V], float (&mult)[V], int lane,
                                                const RowUnits at, int* v) {
  constexpr int T = V >= 4 ? V / 4 : 1;                      // blocks that a lane scales
  scatter_max<V, 2>(m);
  const int q = lane & 3, s = (lane >> 2) & 3;
  uint32_t w[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    w[t] = mx_scale_byte_f32(m[t], &mult[t]) << (8 * s);
    w[t] |= __shfl_xor_sync(0xffffffffu, w[t], 4);
    w[t] |= __shfl_xor_sync(0xffffffffu, w[t], 8);
  }
  uint32_t word = w[0];                                      // of the 16 lanes' vector j
#pragma unroll
  for (int t = 1; t < T; ++t) word = s == t ? w[t] : word;
  const int j = V >= 4 ? T * q + s : V == 2 ? q >> 1 : 0;
  const bool mine = V >= 4 ? s < T : s == 0 && (V == 2 ? (q & 1) == 0 : q == 0);
  *v = mine ? at(j) - (lane & 15) : 0x7fffffff;
  return word;
}
// The multiplier of this lane's block in vector j (wl: the lane in its warp).
template <int V>
__device__ __forceinline__ float mx_mult(const float (&mult)[V], int j, int wl) {
  constexpr int T = V >= 4 ? V / 4 : 1;
  return __shfl_sync(0xffffffffu, mult[j % T], (wl & 28) | (V >= 4 ? j / T : V == 2 ? 2 * j : 0));
}

// What a row kernel writes of a row that lies in the registers of its threads: bf16(y), the row
// copy's codes and block scales, or its part of the tensor's amax. y_of(j, in, y) gives the y of
// vector j, twice: for the maxima and for the codes (in: whether it lies in the row, where that
// matters). FULL: all vectors of the warp lie in a row that is stored, so nothing is tested.
template <int V, int OUT, bool FULL, class Y>
__device__ __forceinline__ void norm_row_copy(const NormParams& p, const Y& y_of, const int64_t r,
                                              const bool live, const bool stored, const int lane,
                                              const RowUnits at, const float tensor_scale,
                                              const uint64_t codes, uint32_t& amax) {
  const int nv = p.cols >> 3;
  const int wl = (int(threadIdx.y) * int(blockDim.x) + int(threadIdx.x)) & 31;

  // ---- the blocks' maxima and multipliers
  uint32_t m[V];
  float mult[V];
  if (OUT == N_MX || OUT == N_BW) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float2 y[4];
      y_of(j, true, y);
      m[j] = __float_as_uint(max8_abs(y));
    }
  }
  if constexpr (OUT == N_MX) {
    int v;
    const uint32_t word = mx_row_word<V>(m, mult, lane, at, &v);
    if (stored && v < nv)
      *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.row_scale) +
                                   mx_scale_offset32(r, v >> 2, p.cols)) = word;
  }
  if constexpr (OUT == N_BW) {
    scatter_max<V, 8>(m);
    float sinv;
    mult[0] = scale_from_amax(__uint_as_float(m[0]), p.margin, &sinv, 448.0f, p.pow2);
    const int j = (lane & 15) / (16 / V), v = at(j) - (lane & 15);
    if (stored && v < nv && (lane & 15) % (16 / V) == 0) {
      if (p.pow2)
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.row_scale) +
                                     mx_scale_offset32(r, v >> 2, p.cols)) =
            e8m0_of_pow2(sinv) * 0x01010101u;
      else
        reinterpret_cast<float*>(p.row_scale)[int64_t(v >> 4) * p.rows_pad + r] = sinv;
    }
  }

  // ---- codes
  // (a quantised tensor has less than 2^31 elements). Padding rows: (0 0) gamma has gamma's sign,
  // their codes are +0.
  const uint32_t kept = live ? 0xffffffffu : 0u;
  uint8_t* row =
      OUT == N_STATS ? nullptr : p.row + (uint32_t(r) * uint32_t(p.cols) + uint32_t(8 * at.first));
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = at(j);
    const bool in = FULL || v < nv;         // uniform over the lanes of a block
    float2 y[4];
    // (for the amax, no NaN where a row's rstd is infinite and a lane has no column)
    y_of(j, (OUT != N_STATS && OUT != N_TENSOR) || in, y);
    // (written apart for FULL: with FULL || (live && in) the norm's row kernels of four vectors that
    // give bf16(y) or statistics alone spill, 8192 x 1024 6.5 us instead of 6.05)
    if (FULL ? p.y != nullptr : p.y != nullptr && live && in)
      *reinterpret_cast<uint4*>(p.y + r * p.cols + 8 * v) =
          make_uint4(pack_bf16(y[0].x, y[0].y), pack_bf16(y[1].x, y[1].y),
                     pack_bf16(y[2].x, y[2].y), pack_bf16(y[3].x, y[3].y));
    if constexpr (OUT == N_STATS || OUT == N_TENSOR)
      amax = max(amax, __float_as_uint(max8_abs(y)));
    if constexpr (OUT != N_STATS) {
      float s = tensor_scale;
      if constexpr (OUT == N_MX) s = mx_mult<V>(mult, j, wl);
      if constexpr (OUT == N_BW)
        s = __shfl_sync(0xffffffffu, mult[0], (wl & 16) | (j * (16 / V)));
      const float2 s2 = make_float2(s, s);
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = __fmul2_rn(y[k], s2);
      if (FULL)
        stg_v2_policy(row + 8 * j * at.step,
                      make_uint2(cvt_e4m3x4(y[0].x, y[0].y, y[1].x, y[1].y),
                                 cvt_e4m3x4(y[2].x, y[2].y, y[3].x, y[3].y)),
                      codes);
      else if (in && stored)
        stg_v2_policy(row + 8 * j * at.step,
                      make_uint2(cvt_e4m3x4(y[0].x, y[0].y, y[1].x, y[1].y) & kept,
                                 cvt_e4m3x4(y[2].x, y[2].y, y[3].x, y[3].y) & kept),
                      codes);
    }
  }
}

// ------------------------------------------------------------------------- host

constexpr int kNormMaxParts = 4096;   // amax partials: one per CTA of the row kernel

// Launches the kernel that writes what a row gives (NormOut says which copy) with the calling
// entry point's own parameters `more`; *ctas (may be null): its CTAs, one amax partial each.
using NormRowLaunch = cudaError_t (*)(int out_kind, const NormParams& p, const void* more,
                                      int* ctas, cudaStream_t st);
NormParams norm_params(const NormArgs& a);
// The copies of a norm's output: rows by `rows`, then columns (and tensorwise rows) from the h
// and rstd that it wrote.
cudaError_t norm_copies_launch(const NormArgs& a, NormParams p, fp8_tensor* out, void* workspace,
                               cudaStream_t st, NormRowLaunch rows, const void* more);

}  // namespace fp8lin
