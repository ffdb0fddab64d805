// RMSNorm in front of the FP8 linear layer: the residual's addition, the norm, and the FP8
// copies of its output (fp8_rmsnorm_quantize).
//
//   h = bf16(x + residual),  rstd = 1 / sqrt(mean h^2 + eps),  y = (h * rstd) * gamma  (fp32)
//
// Kernels:
//   norm_row_kernel   one group of threads per row, the row in registers: h, rstd, and, when
//                     only the row copy is wanted, its codes and scales (blocks along the row
//                     lie in neighbouring lanes). Also the amax partials of per-tensor scales.
//   norm_band_kernel  32 or 128 whole rows per cluster of CTAs, held in registers: both copies
//                     in one pass. The column copy needs 32 or 128 rows of a column at once.
//   norm_cast_kernel  the band kernel's tiles after the row kernel, where one pass cannot do.
// All evaluate y with the same two roundings, so a value has the same y in either copy.
#include <algorithm>

#include "common.cuh"
#include "internal.cuh"
#include "norm.cuh"
#include "sm100_ptx.cuh"

namespace fp8lin {

enum NormOut : int { N_STATS = 0, N_TENSOR = 1, N_MX = 2, N_BW = 3 };

struct NormParams {
  const uint16_t* x;          // [rows][cols], pitch ldx
  const uint16_t* res;        // pitch ldr, or null
  const void* gamma;
  int64_t ldx, ldr;
  int64_t rows, rows_pad;     // rows_pad: a multiple of the recipe's row quantum
  int cols;
  int gamma_fp32;
  float eps;
  uint16_t* h;                // [rows][cols] (written with a residual)
  float* rstd;                // [rows] or null
  uint16_t* y;                // [rows][cols] bf16(y) or null
  uint8_t* row;               // [rows_pad][cols] codes
  void* row_scale;
  uint8_t* col;               // [cols][rows_pad] codes, or bf16 with col_bf16
  void* col_scale;
  const float* scale_in;      // per-tensor scale to cast with (delayed), or null
  uint32_t* part;             // amax partials (31-bit magnitudes), one per CTA, or null
  int n_part;                 // tile kernel: partials to reduce
  float* amax_out;            // per-tensor recipes: written by CTA 0 of the last kernel
  float* scale_out;           // tensorwise: written
  float* scale_inv_out;
  int margin;
  int pow2;                   // blockwise: power-of-two scales in the MXFP8 layout
  int col_bf16;
};

__device__ __forceinline__ uint32_t amax8(const float* y) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag31(y[i]));
  return m;
}

// Eight codes of y * s.
__device__ __forceinline__ uint2 encode8_f32(const float* y, float s) {
  return make_uint2(cvt_e4m3x4(__fmul_rn(y[0], s), __fmul_rn(y[1], s), __fmul_rn(y[2], s),
                               __fmul_rn(y[3], s)),
                    cvt_e4m3x4(__fmul_rn(y[4], s), __fmul_rn(y[5], s), __fmul_rn(y[6], s),
                               __fmul_rn(y[7], s)));
}

// Largest magnitude over the CTA, in thread 0 (red: one word per warp).
__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t m = 0;
  for (int i = 0; i < int(blockDim.x >> 5); ++i) m = max(m, red[i]);
  return m;
}

// ------------------------------------------------------------------------- rows
// tpr threads per row (16, or a multiple of 32), V 16-byte vectors a thread; vector j of lane l
// holds columns 8 (j tpr + l) ..  so a warp reads 512 consecutive bytes and a block of 32 (128)
// columns lies in 4 (16) neighbouring lanes.
template <int V, int OUT>
__global__ void __launch_bounds__(512) norm_row_kernel(const __grid_constant__ NormParams p,
                                                       const int tpr) {
  pdl_wait();
  __shared__ float red[2][16];
  __shared__ uint32_t redm[16];
  const int lane = threadIdx.x % tpr, grp = threadIdx.x / tpr;
  const int rpc = blockDim.x / tpr, nv = p.cols >> 3;
  const int warps = tpr >> 5;                       // warps per row (0: two rows a warp)
  uint32_t amax = 0;
  int phase = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * rpc; r0 < p.rows_pad; r0 += int64_t(gridDim.x) * rpc) {
    const int64_t r = r0 + grp;
    const bool live = r < p.rows, stored = r < p.rows_pad;
    uint4 h[V];
    if (live) {
      uint4 a[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * tpr + lane;
        h[j] = make_uint4(0, 0, 0, 0);
        a[j] = make_uint4(0, 0, 0, 0);
        if (v < nv) {
          h[j] = *reinterpret_cast<const uint4*>(p.x + r * p.ldx + 8 * v);
          if (p.res != nullptr) a[j] = *reinterpret_cast<const uint4*>(p.res + r * p.ldr + 8 * v);
        }
      }
      if (p.res != nullptr) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int v = j * tpr + lane;
          h[j] = make_uint4(add_bf16x2(h[j].x, a[j].x), add_bf16x2(h[j].y, a[j].y),
                            add_bf16x2(h[j].z, a[j].z), add_bf16x2(h[j].w, a[j].w));
          if (v < nv) *reinterpret_cast<uint4*>(p.h + r * p.cols + 8 * v) = h[j];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) h[j] = make_uint4(0, 0, 0, 0);
    }

    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t w[4] = {h[j].x, h[j].y, h[j].z, h[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ss = fmaf(bf16_lo(w[i]), bf16_lo(w[i]), ss);
        ss = fmaf(bf16_hi(w[i]), bf16_hi(w[i]), ss);
      }
    }
    for (int o = (warps == 0 ? tpr : 32) >> 1; o > 0; o >>= 1)
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (warps > 1) {
      if ((threadIdx.x & 31) == 0) red[phase][threadIdx.x >> 5] = ss;
      __syncthreads();
      ss = 0.0f;
      for (int i = 0; i < warps; ++i) ss += red[phase][grp * warps + i];
      phase ^= 1;               // the next row's sums go to the other buffer: one barrier a row
    }
    const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, float(p.cols)), p.eps));
    if (live && lane == 0 && p.rstd != nullptr) p.rstd[r] = rstd;

    if (OUT != N_STATS || p.y != nullptr || p.part != nullptr) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * tpr + lane;
        const bool in = v < nv;               // uniform over the lanes of a block
        float g[8], y[8];
        if (in) load_gamma8(p.gamma, p.gamma_fp32, 8 * v, g);
        else {
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = 0.0f;
        }
        if (live) {
          norm8(h[j], rstd, g, y);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = 0.0f;     // padding rows
        }
        if (p.y != nullptr && live && in)
          *reinterpret_cast<uint4*>(p.y + r * p.cols + 8 * v) =
              make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                         pack_bf16(y[6], y[7]));
        uint32_t m = (in && live) ? amax8(y) : 0u;
        if constexpr (OUT == N_STATS || OUT == N_TENSOR) amax = max(amax, m);
        if constexpr (OUT == N_TENSOR) {
          if (in && stored)
            *reinterpret_cast<uint2*>(p.row + r * p.cols + 8 * v) = encode8_f32(y, *p.scale_in);
        }
        if constexpr (OUT == N_MX) {
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
          float mult;
          uint32_t b = mx_scale_byte_f32(m, &mult);
          if (in && stored)
            *reinterpret_cast<uint2*>(p.row + r * p.cols + 8 * v) = encode8_f32(y, mult);
          // the four bytes of an atom's row in one word
          b <<= 8 * ((lane >> 2) & 3);
          b |= __shfl_xor_sync(0xffffffffu, b, 4);
          b |= __shfl_xor_sync(0xffffffffu, b, 8);
          if (in && stored && (lane & 15) == 0)
            *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.row_scale) +
                                         mx_scale_offset(r, v >> 2, p.cols)) = b;
        }
        if constexpr (OUT == N_BW) {
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          float sinv;
          const float s = scale_from_amax(__uint_as_float(m), p.margin, &sinv, 448.0f, p.pow2);
          if (in && stored) {
            *reinterpret_cast<uint2*>(p.row + r * p.cols + 8 * v) = encode8_f32(y, s);
            if ((lane & 15) == 0) {
              if (p.pow2)
                *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.row_scale) +
                                             mx_scale_offset(r, v >> 2, p.cols)) =
                    e8m0_of_pow2(sinv) * 0x01010101u;
              else
                reinterpret_cast<float*>(p.row_scale)[int64_t(v >> 4) * p.rows_pad + r] = sinv;
            }
          }
        }
      }
    }
  }
  if constexpr (OUT == N_STATS || OUT == N_TENSOR) {
    if (p.part != nullptr) {
      const uint32_t m = cta_max(amax, redm);
      if (threadIdx.x == 0) p.part[blockIdx.x] = m;
    }
  }
  pdl_launch_dependents();
}

// amax = the largest of the row kernel's partials.
__global__ void __launch_bounds__(512) norm_amax_kernel(const uint32_t* part, int n, float* amax) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ uint32_t red[16];
  uint32_t m = 0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) m = max(m, part[i]);
  m = cta_max(m, red);
  if (threadIdx.x == 0) *amax = __uint_as_float(m);
}

// ------------------------------------------------------------------------- tiles of 32 x 128
// A warp holds 32 rows x 128 columns of h in registers, packed bf16: lane l the eight columns
// 8 (l % 16) .. of the 16 rows 16 (l / 16) .. (64 registers). A column's 32-row block lies in
// two lanes, a row's 32-column block in four, so both copies come out of the same registers:
// the column copy is written in 16-byte pieces that pair up to whole 32-byte sectors, the row
// copy in 128-byte rows. Maxima and sums of four rows over the lanes are reduced by halving: a
// lane passes on half of its rows at each step and keeps the other half. y is computed twice
// (for the maxima, then for the codes): two packed multiplies a pair, cheaper than 128 registers
// to keep it.

// |a|, |b|, |c|: the largest; NaN if one of them is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Reduce four rows' values over the lanes that differ in the bits OFF and OFF / 2 by halving.
// The lane ends with row 2 [lane & OFF] + [lane & OFF / 2] in v[0].
template <int OFF, class T, class Op>
__device__ __forceinline__ T reduce4(T (&v)[4], Op op) {
  const int lane = threadIdx.x & 31;
  const bool u = (lane & OFF) != 0, w = (lane & (OFF / 2)) != 0;
  const T s0 = u ? v[0] : v[2], s1 = u ? v[1] : v[3];
  const T a = op(u ? v[2] : v[0], __shfl_xor_sync(0xffffffffu, s0, OFF));
  const T b = op(u ? v[3] : v[1], __shfl_xor_sync(0xffffffffu, s1, OFF));
  return op(w ? b : a, __shfl_xor_sync(0xffffffffu, w ? a : b, OFF / 2));
}
// Over a half-warp: the lanes l with (l >> 2) & 3 == k end with row k's.
template <class T, class Op>
__device__ __forceinline__ T reduce4_half(T (&v)[4], Op op) {
  T r = reduce4<8>(v, op);
  r = op(r, __shfl_xor_sync(0xffffffffu, r, 2));
  return op(r, __shfl_xor_sync(0xffffffffu, r, 1));
}

// y of a row's eight columns: (h rstd) gamma, each product rounded.
__device__ __forceinline__ void norm_row8(uint4 h, float rstd, const float2 (&g)[4],
                                          float2 (&y)[4]) {
  const float2 r = make_float2(rstd, rstd);
  const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    y[k] = __fmul2_rn(__fmul2_rn(make_float2(bf16_lo(w[k]), bf16_hi(w[k])), r), g[k]);
}
__device__ __forceinline__ float max8_abs(const float2 (&y)[4]) {
  const float m = max3_abs(max3_abs(y[0].x, y[0].y, y[1].x), y[1].y, y[2].x);
  return max3_abs(max3_abs(m, y[2].y, y[3].x), y[3].y, 0.0f);
}

// The compiler must not keep floats made from h in one pass for the next (128 registers,
// spilled): h is opaque from here on.
__device__ __forceinline__ void opaque(uint4 (&h)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    asm volatile("" : "+r"(h[i].x), "+r"(h[i].y), "+r"(h[i].z), "+r"(h[i].w));
}

struct NormBandSmem {
  float part[16][32];                  // a warp's row sums
  alignas(16) float csum[8][128];      // the row sums of each CTA of the cluster
  alignas(16) float rstd[128];
  alignas(16) uint32_t cmax[4][512];   // 1x128: column maxima of each 32-row group
  uint32_t red[16];
};

// Codes and scales of one warp tile; returns the lane's share of the tensor's amax (N_TENSOR).
// rg, cw: the warp's 32-row group and 128-column tile in the CTA; r0, c: the tile's first row
// and this lane's first column. FULL: both copies are wanted in FP8 and the tile lies inside
// the padded tensor, so nothing is tested per row.
template <int OUT, bool FULL>
__device__ __forceinline__ uint32_t norm_tile(const NormParams& p, uint4 (&h)[16],
                                              NormBandSmem& S, int rg, int cw, int64_t r0, int c,
                                              float tensor_scale) {
  const int lane = threadIdx.x & 31, half = lane >> 4;
  const bool in = FULL || c < p.cols;
  const bool want_row = FULL || p.row != nullptr, want_col = FULL || p.col != nullptr;
  const bool col_bf16 = !FULL && p.col_bf16;
  const float4* rs = reinterpret_cast<const float4*>(&S.rstd[32 * rg + 16 * half]);
  float2 g[4];
  if (in) {
    float t[8];
    load_gamma8(p.gamma, p.gamma_fp32, c, t);
#pragma unroll
    for (int k = 0; k < 4; ++k) g[k] = make_float2(t[2 * k], t[2 * k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) g[k] = make_float2(0.0f, 0.0f);
  }

  // ---- maxima, and from them the multipliers: mult those of this lane's rows, cs the columns'
  float mult[4];
  float2 cs[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) cs[k] = make_float2(tensor_scale, tensor_scale);
  if constexpr (OUT != N_TENSOR) {
    const auto umax = [](uint32_t a, uint32_t b) { return max(a, b); };
    float2 cm[4];
    uint32_t rowmax[4];              // rows 4j + lane % 4 (MX) or 4j + (lane >> 2) % 4
#pragma unroll
    for (int k = 0; k < 4; ++k) cm[k] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 r4 = rs[j];
      const float r[4] = {r4.x, r4.y, r4.z, r4.w};
      float2 y[4][4];
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        norm_row8(h[4 * j + i], r[i], g, y[i]);
        m[i] = __float_as_uint(max8_abs(y[i]));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        cm[k].x = max3_abs(max3_abs(cm[k].x, y[0][k].x, y[1][k].x), y[2][k].x, y[3][k].x);
        cm[k].y = max3_abs(max3_abs(cm[k].y, y[0][k].y, y[1][k].y), y[2][k].y, y[3][k].y);
      }
      rowmax[j] = OUT == N_MX ? reduce4<2>(m, umax) : reduce4_half(m, umax);
    }
    // Columns: the two halves of the warp hold 16 rows each; the lower half ends with the
    // first four of the eight columns, the upper half with the others.
    uint32_t q[4];
    {
      const uint32_t lo[4] = {__float_as_uint(cm[0].x), __float_as_uint(cm[0].y),
                              __float_as_uint(cm[1].x), __float_as_uint(cm[1].y)};
      const uint32_t hi[4] = {__float_as_uint(cm[2].x), __float_as_uint(cm[2].y),
                              __float_as_uint(cm[3].x), __float_as_uint(cm[3].y)};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        q[k] = max(half ? hi[k] : lo[k], __shfl_xor_sync(0xffffffffu, half ? lo[k] : hi[k], 16));
    }
    const int c4 = c + 4 * half;                     // this lane's four columns
    float s4[4], i4[4];
    if constexpr (OUT == N_MX) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = mx_scale_byte_f32(rowmax[j], &mult[j]) << (2 * (lane & 12));   // block (lane>>2)&3
        w[j] |= __shfl_xor_sync(0xffffffffu, w[j], 4);
        w[j] |= __shfl_xor_sync(0xffffffffu, w[j], 8);
      }
      if (want_row && in) {                          // lane l: row l's four bytes
        const int j = (lane >> 2) & 3;
        const uint32_t v = j == 0 ? w[0] : j == 1 ? w[1] : j == 2 ? w[2] : w[3];
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.row_scale) +
                                     mx_scale_offset(r0 + lane, (c >> 7) * 4, p.cols)) = v;
      }
      uint8_t* d = reinterpret_cast<uint8_t*>(p.col_scale) +
                   mx_scale_offset(c4, r0 >> 5, p.rows_pad);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t b = mx_scale_byte_f32(q[k], &s4[k]);
        if (want_col && !col_bf16 && in) d[16 * k] = uint8_t(b);   // the next column's row
      }
    } else {
      // this lane's row of the 128-column block
      const int j = lane & 3, mine = 16 * half + 4 * j + ((lane >> 2) & 3);
      const uint32_t m = j == 0 ? rowmax[0] : j == 1 ? rowmax[1] : j == 2 ? rowmax[2] : rowmax[3];
      float si;
      mult[0] = scale_from_amax(__uint_as_float(m), p.margin, &si, 448.0f, p.pow2);
      if (want_row && in) {
        if (p.pow2)
          *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.row_scale) +
                                       mx_scale_offset(r0 + mine, (c >> 7) * 4, p.cols)) =
              e8m0_of_pow2(si) * 0x01010101u;
        else
          reinterpret_cast<float*>(p.row_scale)[int64_t(c >> 7) * p.rows_pad + r0 + mine] = si;
      }
      const int at = cw * 128 + 8 * (lane & 15) + 4 * half;
      *reinterpret_cast<uint4*>(&S.cmax[rg][at]) = make_uint4(q[0], q[1], q[2], q[3]);
      __syncthreads();                               // the four row groups of 128 rows
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(&S.cmax[k][at]);
        q[0] = max(q[0], v.x);
        q[1] = max(q[1], v.y);
        q[2] = max(q[2], v.z);
        q[3] = max(q[3], v.w);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        s4[k] = scale_from_amax(__uint_as_float(q[k]), p.margin, &i4[k], 448.0f, p.pow2);
      if (want_col && !col_bf16 && in && rg == 0) {
        if (p.pow2) {
          uint8_t* d = reinterpret_cast<uint8_t*>(p.col_scale) +
                       mx_scale_offset(c4, r0 >> 5, p.rows_pad);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint32_t*>(d + 16 * k) = e8m0_of_pow2(i4[k]) * 0x01010101u;
        } else {
          *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.col_scale) +
                                     (r0 >> 7) * p.cols + c4) =
              make_float4(i4[0], i4[1], i4[2], i4[3]);
        }
      }
    }
    float o4[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o4[k] = __shfl_xor_sync(0xffffffffu, s4[k], 16);
    cs[0] = half ? make_float2(o4[0], o4[1]) : make_float2(s4[0], s4[1]);
    cs[1] = half ? make_float2(o4[2], o4[3]) : make_float2(s4[2], s4[3]);
    cs[2] = half ? make_float2(s4[0], s4[1]) : make_float2(o4[0], o4[1]);
    cs[3] = half ? make_float2(s4[2], s4[3]) : make_float2(o4[2], o4[3]);
    opaque(h);
  }

  // ---- codes, four rows at a time
  uint32_t amax = 0;
  uint32_t code[8][4];                               // 16 codes of each column
  const int64_t rt = r0 + 16 * half;
  const bool stored = in && (FULL || rt < p.rows_pad);      // 16 rows: all or none
  uint8_t* row = p.row + rt * p.cols + c;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 r4 = rs[j];
    const float r[4] = {r4.x, r4.y, r4.z, r4.w};
    float2 y[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      norm_row8(h[4 * j + i], r[i], g, y[i]);
      if constexpr (OUT == N_TENSOR) amax = max(amax, __float_as_uint(max8_abs(y[i])));
      if (want_row) {
        float s = tensor_scale;
        if constexpr (OUT == N_MX) s = __shfl_sync(0xffffffffu, mult[j], (lane & 28) | i);
        if constexpr (OUT == N_BW)
          s = __shfl_sync(0xffffffffu, mult[0], (lane & 16) | (i << 2) | j);
        const float2 ss = make_float2(s, s);
        float2 u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = __fmul2_rn(y[i][k], ss);
        if (stored)
          *reinterpret_cast<uint2*>(row) =
              make_uint2(cvt_e4m3x4(u[0].x, u[0].y, u[1].x, u[1].y),
                         cvt_e4m3x4(u[2].x, u[2].y, u[3].x, u[3].y));
        row += p.cols;
      }
    }
    if (want_col) {
      if (col_bf16) {
        if (stored) {
          uint16_t* d = reinterpret_cast<uint16_t*>(p.col) + int64_t(c) * p.rows_pad + rt + 4 * j;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            *reinterpret_cast<uint2*>(d + 2 * k * p.rows_pad) =
                make_uint2(pack_bf16(y[0][k].x, y[1][k].x), pack_bf16(y[2][k].x, y[3][k].x));
            *reinterpret_cast<uint2*>(d + (2 * k + 1) * p.rows_pad) =
                make_uint2(pack_bf16(y[0][k].y, y[1][k].y), pack_bf16(y[2][k].y, y[3][k].y));
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i][k] = __fmul2_rn(y[i][k], cs[k]);
          code[2 * k][j] = cvt_e4m3x4(y[0][k].x, y[1][k].x, y[2][k].x, y[3][k].x);
          code[2 * k + 1][j] = cvt_e4m3x4(y[0][k].y, y[1][k].y, y[2][k].y, y[3][k].y);
        }
      }
    }
  }
  if (want_col && !col_bf16 && stored) {
    uint8_t* col = p.col + int64_t(c) * p.rows_pad + rt;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      *reinterpret_cast<uint4*>(col) = make_uint4(code[k][0], code[k][1], code[k][2], code[k][3]);
      col += p.rows_pad;
    }
  }
  return amax;
}

// One band of 32 (1x128: 128) rows a cluster: CTA `rank` has the columns of its warps, cg tiles
// side by side, RG row groups one below the other. The row sums of the cluster's CTAs are
// exchanged through distributed shared memory, so the band is read once and never read back.
template <int OUT, bool RES, bool FULL>
__global__ void __launch_bounds__(512) norm_band_kernel(const __grid_constant__ NormParams p,
                                                        const int cg, const int cs) {
  constexpr int RG = OUT == N_BW ? 4 : 1;
  __shared__ NormBandSmem S;
  // every CTA of the cluster has started before one writes into another's shared memory
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, half = lane >> 4;
  const int cw = w % cg, rg = w / cg;
  const int rank = int(blockIdx.x) % cs;
  const int64_t r0 = int64_t(int(blockIdx.x) / cs) * (32 * RG) + 32 * rg;
  const int c = (rank * cg + cw) * 128 + 8 * (lane & 15);
  const bool in = c < p.cols;
  const int live = int(max(int64_t(0), min(int64_t(16), p.rows - r0 - 16 * half)));

  // ---- h and the row sums, four rows' loads at a time
  uint4 h[16];
  const uint16_t* x = p.x + (r0 + 16 * half) * p.ldx + c;
  const uint16_t* res = p.res + (r0 + 16 * half) * p.ldr + c;
  uint16_t* ho = p.h + (r0 + 16 * half) * p.cols + c;
  const auto add = [](float a, float b) { return a + b; };
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 a[4];
    float ss[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[4 * j + i] = a[i] = make_uint4(0, 0, 0, 0);
      if (in && 4 * j + i < live) {
        h[4 * j + i] = *reinterpret_cast<const uint4*>(x);
        if (RES) a[i] = *reinterpret_cast<const uint4*>(res);
      }
      x += p.ldx;
      if (RES) res += p.ldr;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4& v = h[4 * j + i];
      if (RES) {
        v = make_uint4(add_bf16x2(v.x, a[i].x), add_bf16x2(v.y, a[i].y), add_bf16x2(v.z, a[i].z),
                       add_bf16x2(v.w, a[i].w));
        if (in && 4 * j + i < live) *reinterpret_cast<uint4*>(ho) = v;
        ho += p.cols;
      }
      float2 q = make_float2(0.0f, 0.0f);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = make_float2(bf16_lo(u[k]), bf16_hi(u[k]));
        q = __ffma2_rn(f, f, q);
      }
      ss[i] = q.x + q.y;
    }
    const float t = reduce4_half(ss, add);
    if ((lane & 3) == 0) S.part[w][16 * half + 4 * j + ((lane >> 2) & 3)] = t;
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (threadIdx.x < 32 * RG) {
    float t = 0.0f;
    for (int k = 0; k < cg; ++k) t += S.part[(threadIdx.x >> 5) * cg + k][lane];
    for (int k = 0; k < cs; ++k) {
      const uint32_t d = ptx::map_to_rank(&S.csum[rank][threadIdx.x], uint32_t(k));
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(d), "f"(t) : "memory");
    }
  }
  ptx::cluster_sync();
  if (threadIdx.x < 32 * RG) {
    float t = 0.0f;
    for (int k = 0; k < cs; ++k) t += S.csum[k][threadIdx.x];
    const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(t, float(p.cols)), p.eps));
    const int64_t r = r0 - 32 * rg + threadIdx.x;
    S.rstd[threadIdx.x] = r < p.rows ? rstd : 0.0f;      // padding rows: y = (0 0) gamma = 0
    if (rank == 0 && r < p.rows && p.rstd != nullptr) p.rstd[r] = rstd;
  }
  __syncthreads();

  const float scale = OUT == N_TENSOR ? *p.scale_in : 1.0f;
  opaque(h);
  const uint32_t amax = norm_tile<OUT, FULL>(p, h, S, rg, cw, r0, c, scale);
  if constexpr (OUT == N_TENSOR) {
    const uint32_t m = cta_max(amax, S.red);
    if (threadIdx.x == 0) p.part[blockIdx.x] = m;
  }
  pdl_launch_dependents();
}

// The same tiles with h and rstd known (the row kernel ran first): for tensorwise scales, which
// need the whole tensor's amax before any code, and for rows too long for a cluster.
template <int OUT, bool FULL>
__global__ void __launch_bounds__(512) norm_cast_kernel(const __grid_constant__ NormParams p,
                                                        const int cg, const int tiles) {
  constexpr int RG = OUT == N_BW ? 4 : 1;
  __shared__ NormBandSmem S;
  pdl_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, half = lane >> 4;
  const int cw = w % cg, rg = w / cg;
  // Last bands first: the row kernel wrote the last rows of h most recently (L2).
  const int at = int(gridDim.x - 1 - blockIdx.x);
  const int64_t band0 = int64_t(at / tiles) * (32 * RG), r0 = band0 + 32 * rg;
  const int c = ((at % tiles) * cg + cw) * 128 + 8 * (lane & 15);
  const bool in = c < p.cols;
  const int live = int(max(int64_t(0), min(int64_t(16), p.rows - r0 - 16 * half)));
  uint4 h[16];
  const uint16_t* x = p.h + (r0 + 16 * half) * p.ldx + c;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    h[i] = make_uint4(0, 0, 0, 0);
    if (in && i < live) h[i] = *reinterpret_cast<const uint4*>(x);
    x += p.ldx;
  }
  if (threadIdx.x < 32 * RG)
    S.rstd[threadIdx.x] = band0 + threadIdx.x < p.rows ? p.rstd[band0 + threadIdx.x] : 0.0f;
  float scale = 1.0f;
  if constexpr (OUT == N_TENSOR) {
    uint32_t m = 0;
    for (int i = threadIdx.x; i < p.n_part; i += blockDim.x) m = max(m, p.part[i]);
    m = cta_max(m, S.red);
    float sinv;
    scale = p.scale_in != nullptr ? *p.scale_in
                                  : scale_from_amax(__uint_as_float(m), p.margin, &sinv);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      *p.amax_out = __uint_as_float(m);
      if (p.scale_in == nullptr) {
        *p.scale_out = scale;
        *p.scale_inv_out = sinv;
      }
    }
  }
  __syncthreads();
  norm_tile<OUT, FULL>(p, h, S, rg, cw, r0, c, scale);
  pdl_launch_dependents();
}

// ------------------------------------------------------------------------- host

namespace {

constexpr int kNormRowCtas = 8;       // most CTAs of the row kernel per SM (amax partials)

// Rows to stream take four vectors a thread, so that more bytes are in flight; a few rows (one
// per SM or less) take as many threads as there are vectors.
RowPlan fwd_plan(int64_t rows, int cols) { return row_plan(cols, rows > num_sms() ? 4 : 1, 256); }

template <int OUT>
cudaError_t launch_rows(const NormParams& p, int* ctas, cudaStream_t st) {
  const RowPlan pl = fwd_plan(p.rows, p.cols);
  const int rpc = pl.block / pl.tpr;
  const int64_t groups = (p.rows_pad + rpc - 1) / rpc;
  const int grid = int(std::min<int64_t>(groups, int64_t(num_sms()) * kNormRowCtas));
  if (ctas != nullptr) *ctas = grid;
  auto kern = pl.v == 1   ? norm_row_kernel<1, OUT>
              : pl.v == 2 ? norm_row_kernel<2, OUT>
              : pl.v == 4 ? norm_row_kernel<4, OUT>
                          : norm_row_kernel<8, OUT>;
  return launch_kernel(kern, dim3(grid), dim3(pl.block), 0, st, nullptr, p, pl.tpr);
}

// How a band's 128-column tiles are dealt out: cg tiles to a CTA, cs CTAs to a cluster.
struct BandPlan {
  int cg, cs;
};
BandPlan band_plan(int out, int cols) {
  const int tiles = (cols + 127) / 128, most = out == N_BW ? 4 : 8;
  int cs = 1;
  while (cs < 8 && (tiles + cs - 1) / cs > most) cs *= 2;
  return {(tiles + cs - 1) / cs, cs};
}
// Whether a cluster holds a band: at most 16 warps a CTA.
bool band_fits(int out, int cols) {
  return band_plan(out, cols).cg * (out == N_BW ? 4 : 1) <= 16;
}
int64_t band_ctas(int out, int64_t rows_pad, int cols) {
  const int rows = out == N_BW ? 128 : 32;
  return (rows_pad + rows - 1) / rows * band_plan(out, cols).cs;
}

// Whether every warp's tile lies inside the padded tensor and both copies are FP8.
bool full_tiles(int out, const NormParams& p, int across) {
  const int rg = out == N_BW ? 4 : 1;
  return p.row != nullptr && p.col != nullptr && !p.col_bf16 && p.cols % (128 * across) == 0 &&
         p.rows_pad % (32 * rg) == 0;
}

template <int OUT>
cudaError_t launch_band(const NormParams& p, cudaStream_t st) {
  const BandPlan b = band_plan(OUT, p.cols);
  cudaLaunchAttribute cl;
  cl.id = cudaLaunchAttributeClusterDimension;
  cl.val.clusterDim.x = unsigned(b.cs);
  cl.val.clusterDim.y = 1;
  cl.val.clusterDim.z = 1;
  const bool full = full_tiles(OUT, p, b.cg * b.cs), res = p.res != nullptr;
  auto kern = full ? (res ? norm_band_kernel<OUT, true, true> : norm_band_kernel<OUT, false, true>)
                   : (res ? norm_band_kernel<OUT, true, false>
                          : norm_band_kernel<OUT, false, false>);
  return launch_kernel(kern, dim3(unsigned(band_ctas(OUT, p.rows_pad, p.cols))),
                       dim3(32 * b.cg * (OUT == N_BW ? 4 : 1)), 0, st, &cl, p, b.cg, b.cs);
}

template <int OUT>
cudaError_t launch_cast(const NormParams& p, cudaStream_t st) {
  constexpr int RG = OUT == N_BW ? 4 : 1;
  const int tiles = (p.cols + 127) / 128, cg = std::min(tiles, OUT == N_BW ? 4 : 8);
  const int across = (tiles + cg - 1) / cg;
  const int64_t bands = (p.rows_pad + 32 * RG - 1) / (32 * RG);
  auto kern = full_tiles(OUT, p, cg) ? norm_cast_kernel<OUT, true> : norm_cast_kernel<OUT, false>;
  return launch_kernel(kern, dim3(unsigned(bands * across)), dim3(32 * cg * RG), 0, st, nullptr, p,
                       cg, across);
}

}  // namespace

int64_t norm_pad_rows(int kind, int64_t rows) {
  const int64_t q = kind == FP8_RECIPE_MXFP8 || kind == FP8_RECIPE_BLOCKWISE ? 128 : 16;
  return (rows + q - 1) / q * q;
}

size_t norm_workspace_bytes(int kind, int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  // rstd (when the caller keeps none), then the amax partials of the row or the band kernel
  size_t parts = 0;
  if (kind == FP8_RECIPE_TENSORWISE || kind == FP8_RECIPE_DELAYED)
    parts = std::max(size_t(num_sms()) * kNormRowCtas,
                     size_t(band_ctas(N_TENSOR, norm_pad_rows(kind, rows), int(cols))));
  return size_t((rows * 4 + 15) / 16 * 16) + parts * 4;
}

cudaError_t norm_quantize_launch(const NormArgs& a, fp8_tensor* out, void* workspace,
                                 cudaStream_t st) {
  NormParams p{};
  p.x = a.x;
  p.res = a.res;
  p.gamma = a.gamma;
  p.ldx = a.ldx;
  p.ldr = a.ldr;
  p.rows = a.rows;
  p.rows_pad = a.quantise ? norm_pad_rows(a.kind, a.rows) : a.rows;
  p.cols = int(a.cols);
  p.gamma_fp32 = a.gamma_fp32;
  p.eps = a.eps;
  p.h = a.h;
  p.rstd = a.rstd;
  p.y = a.y;
  p.margin = a.margin;
  p.pow2 = a.pow2;
  p.col_bf16 = a.col_bf16;
  if (!a.quantise) return launch_rows<N_STATS>(p, nullptr, st);

  uint32_t* part = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(workspace) +
                                               (a.rows * 4 + 15) / 16 * 16);
  const int out_kind = a.kind == FP8_RECIPE_MXFP8       ? N_MX
                       : a.kind == FP8_RECIPE_BLOCKWISE ? N_BW
                                                        : N_TENSOR;
  const bool delayed = a.kind == FP8_RECIPE_DELAYED, tensorwise = a.kind == FP8_RECIPE_TENSORWISE;
  const auto finish_amax = [&](int n) {
    return launch_kernel(norm_amax_kernel, dim3(1), dim3(512), 0, st, nullptr,
                         static_cast<const uint32_t*>(part), n, out->amax);
  };
  p.row = a.want_row ? out->row : nullptr;
  p.row_scale = out->row_scale;
  p.col = a.want_col ? out->col : nullptr;
  p.col_scale = out->col_scale;

  // The row copy alone: rows.
  if (!a.want_col && !tensorwise) {
    if (out_kind == N_MX) return launch_rows<N_MX>(p, nullptr, st);
    if (out_kind == N_BW) return launch_rows<N_BW>(p, nullptr, st);
    p.scale_in = out->scale;
    p.part = part;
    int ctas = 0;
    const cudaError_t e = launch_rows<N_TENSOR>(p, &ctas, st);
    return e != cudaSuccess ? e : finish_amax(ctas);
  }

  // Both copies in one pass, where the scale needs no more than a band.
  if (!tensorwise && a.y == nullptr && band_fits(out_kind, p.cols)) {
    if (out_kind == N_MX) return launch_band<N_MX>(p, st);
    if (out_kind == N_BW) return launch_band<N_BW>(p, st);
    p.scale_in = out->scale;
    p.part = part;
    const cudaError_t e = launch_band<N_TENSOR>(p, st);
    return e != cudaSuccess ? e : finish_amax(int(band_ctas(N_TENSOR, p.rows_pad, p.cols)));
  }

  // Rows, then tiles.
  if (p.rstd == nullptr) p.rstd = reinterpret_cast<float*>(workspace);
  NormParams q = p;
  if (out_kind == N_TENSOR) q.part = part;
  int ctas = 0;
  cudaError_t e = launch_rows<N_STATS>(q, &ctas, st);
  if (e != cudaSuccess) return e;
  if (a.res == nullptr) p.h = const_cast<uint16_t*>(a.x);     // read only from here on
  else p.ldx = a.cols;
  if (out_kind == N_MX) return launch_cast<N_MX>(p, st);
  if (out_kind == N_BW) return launch_cast<N_BW>(p, st);
  p.part = part;
  p.n_part = ctas;
  p.amax_out = out->amax;
  p.scale_out = out->scale;
  p.scale_inv_out = out->scale_inv;
  if (delayed) p.scale_in = out->scale;
  return launch_cast<N_TENSOR>(p, st);
}

}  // namespace fp8lin
