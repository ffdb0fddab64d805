// RMSNorm in front of the FP8 linear layer: the residual's addition, the norm, and the FP8
// copies of its output (fp8_rmsnorm_quantize).
//
//   h = bf16(x + residual),  rstd = 1 / sqrt(mean h^2 + eps),  y = (h * rstd) * gamma  (fp32)
//
// Two kernels:
//   norm_row_kernel   one group of threads per row, the row in registers: h, rstd, and, when
//                     only the row copy is wanted, its codes and scales (blocks along the row
//                     lie in neighbouring lanes). Also the amax partials of per-tensor scales.
//   norm_tile_kernel  128 x 128 tiles of h with rstd known: codes and scales of both copies.
//                     The column copy needs 32 or 128 rows of one column, which a row's
//                     thread group does not have.
// Both evaluate y with the same two roundings, so a value has the same y in either copy.
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
  int col_v8;                 // the column copy's 32-byte segments are aligned
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
  pdl_launch_dependents();
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

// ------------------------------------------------------------------------- tiles
constexpr int kNormLd = 136;                      // padded row of the bf16 tile (elements)

struct NormTileSmem {
  alignas(16) uint16_t h[128 * kNormLd];
  alignas(16) float rstd[128];
  alignas(16) uint8_t atom_row[512], atom_col[512];   // MXFP8-layout scales of the tile
  float srow[128];                                // 1x128: s_inv of the tile's rows
  uint32_t cmax[4][128];                          // 1x128: column maxima of 32 rows each
  uint32_t red[8];
};

template <int OUT>
__global__ void __launch_bounds__(256, 2) norm_tile_kernel(const __grid_constant__ NormParams p,
                                                           const int tiles_c) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t norm_smem[];
  NormTileSmem& S = *reinterpret_cast<NormTileSmem*>(norm_smem);
  const int t = threadIdx.x;
  // Last tiles first: the row kernel wrote the last rows of h most recently (L2).
  const int tile = int(gridDim.x - 1 - blockIdx.x);
  const int tr = tile / tiles_c, tc = tile % tiles_c;
  const int64_t r0 = int64_t(tr) * 128;
  const int c0 = tc * 128;
  const uint16_t* h = p.h;                        // pitch ldx (x itself) or cols
  const int64_t ldh = p.ldx;

#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int idx = i * 256 + t, r = idx >> 4, v = idx & 15;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (r0 + r < p.rows && c0 + 8 * v < p.cols)
      w = *reinterpret_cast<const uint4*>(h + (r0 + r) * ldh + c0 + 8 * v);
    *reinterpret_cast<uint4*>(&S.h[r * kNormLd + 8 * v]) = w;
  }
  // rstd 0 in the padding rows: y = (0 * 0) * gamma = 0 there for a finite gamma; the passes
  // below do not rely on it and set y to 0 outright.
  if (t < 128) S.rstd[t] = r0 + t < p.rows ? p.rstd[r0 + t] : 0.0f;

  float s = 1.0f, sinv = 1.0f;
  if constexpr (OUT == N_TENSOR) {
    uint32_t m = 0;
    if (p.scale_in == nullptr || blockIdx.x == 0) {
      for (int i = t; i < p.n_part; i += 256) m = max(m, p.part[i]);
      m = cta_max(m, S.red);
    }
    if (p.scale_in != nullptr) s = *p.scale_in;
    else s = scale_from_amax(__uint_as_float(m), p.margin, &sinv);
    if (blockIdx.x == 0 && t == 0) {
      *p.amax_out = __uint_as_float(m);
      if (p.scale_in == nullptr) {
        *p.scale_out = s;
        *p.scale_inv_out = sinv;
      }
    }
  }
  __syncthreads();

  // ---- row copy: eight lanes a row, 16 columns each
  if (p.row != nullptr) {
    const int l8 = t & 7, c = c0 + 16 * l8;
    const bool in = c < p.cols;
    float g[16];
    if (in) {
      load_gamma8(p.gamma, p.gamma_fp32, c, g);
      load_gamma8(p.gamma, p.gamma_fp32, c + 8, g + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) g[i] = 0.0f;
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int r = it * 32 + (t >> 3);
      const bool live = r0 + r < p.rows, stored = r0 + r < p.rows_pad && in;
      const float rstd = S.rstd[r];
      float y[16];
      const uint4* src = reinterpret_cast<const uint4*>(&S.h[r * kNormLd + 16 * l8]);
      norm8(src[0], rstd, g, y);
      norm8(src[1], rstd, g + 8, y + 8);
      if (!live) {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = 0.0f;
      }
      float sc = s;
      if constexpr (OUT == N_MX) {
        uint32_t m = max(amax8(y), amax8(y + 8));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const uint32_t b = mx_scale_byte_f32(m, &sc);
        if ((l8 & 1) == 0) S.atom_row[(r & 31) * 16 + (r >> 5) * 4 + (l8 >> 1)] = uint8_t(b);
      }
      if constexpr (OUT == N_BW) {
        uint32_t m = max(amax8(y), amax8(y + 8));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        sc = scale_from_amax(__uint_as_float(m), p.margin, &sinv, 448.0f, p.pow2);
        if (l8 == 0) {
          if (p.pow2)
            *reinterpret_cast<uint32_t*>(&S.atom_row[(r & 31) * 16 + (r >> 5) * 4]) =
                e8m0_of_pow2(sinv) * 0x01010101u;
          else
            S.srow[r] = sinv;
        }
      }
      if (stored) {
        const uint2 a = encode8_f32(y, sc), b = encode8_f32(y + 8, sc);
        *reinterpret_cast<uint4*>(p.row + (r0 + r) * p.cols + c) =
            make_uint4(a.x, a.y, b.x, b.y);
      }
    }
  }

  // ---- column copy: two columns a thread over 32 rows
  if (p.col != nullptr) {
    const int pr = t & 63, rb = t >> 6, c = c0 + 2 * pr;
    const bool in = c < p.cols;
    float g0 = 0.0f, g1 = 0.0f;
    if (in) {
      if (p.gamma_fp32) {
        g0 = reinterpret_cast<const float*>(p.gamma)[c];
        g1 = reinterpret_cast<const float*>(p.gamma)[c + 1];
      } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(
            reinterpret_cast<const uint16_t*>(p.gamma) + c);
        g0 = bf16_lo(w);
        g1 = bf16_hi(w);
      }
    }
    float y0[32], y1[32];
    const int live = int(max(int64_t(0), min(int64_t(32), p.rows - r0 - 32 * rb)));
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int r = 32 * rb + i;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(&S.h[r * kNormLd + 2 * pr]);
      const float rstd = S.rstd[r];
      y0[i] = i < live ? __fmul_rn(__fmul_rn(bf16_lo(w), rstd), g0) : 0.0f;
      y1[i] = i < live ? __fmul_rn(__fmul_rn(bf16_hi(w), rstd), g1) : 0.0f;
    }
    const int64_t rr = r0 + 32 * rb;
    const bool lo_ok = in && rr < p.rows_pad, hi_ok = in && rr + 16 < p.rows_pad;
    if (p.col_bf16) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(p.col) + int64_t(c) * p.rows_pad + rr;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k < 2 ? lo_ok : hi_ok) {
          reinterpret_cast<uint4*>(dst)[k] = make_uint4(
              pack_bf16(y0[8 * k], y0[8 * k + 1]), pack_bf16(y0[8 * k + 2], y0[8 * k + 3]),
              pack_bf16(y0[8 * k + 4], y0[8 * k + 5]), pack_bf16(y0[8 * k + 6], y0[8 * k + 7]));
          reinterpret_cast<uint4*>(dst + p.rows_pad)[k] = make_uint4(
              pack_bf16(y1[8 * k], y1[8 * k + 1]), pack_bf16(y1[8 * k + 2], y1[8 * k + 3]),
              pack_bf16(y1[8 * k + 4], y1[8 * k + 5]), pack_bf16(y1[8 * k + 6], y1[8 * k + 7]));
        }
      }
    } else {
      float s0 = s, s1 = s;
      if constexpr (OUT != N_TENSOR) {
        uint32_t m0 = 0, m1 = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          m0 = max(m0, mag31(y0[i]));
          m1 = max(m1, mag31(y1[i]));
        }
        const int at = (2 * pr & 31) * 16 + (pr >> 4) * 4;      // the column's row in the atom
        if constexpr (OUT == N_MX) {
          S.atom_col[at + rb] = uint8_t(mx_scale_byte_f32(m0, &s0));
          S.atom_col[at + 16 + rb] = uint8_t(mx_scale_byte_f32(m1, &s1));
        } else {
          S.cmax[rb][2 * pr] = m0;
          S.cmax[rb][2 * pr + 1] = m1;
          __syncthreads();
          m0 = max(max(S.cmax[0][2 * pr], S.cmax[1][2 * pr]),
                   max(S.cmax[2][2 * pr], S.cmax[3][2 * pr]));
          m1 = max(max(S.cmax[0][2 * pr + 1], S.cmax[1][2 * pr + 1]),
                   max(S.cmax[2][2 * pr + 1], S.cmax[3][2 * pr + 1]));
          float i0, i1;
          s0 = scale_from_amax(__uint_as_float(m0), p.margin, &i0, 448.0f, p.pow2);
          s1 = scale_from_amax(__uint_as_float(m1), p.margin, &i1, 448.0f, p.pow2);
          if (rb == 0) {
            if (p.pow2) {
              *reinterpret_cast<uint32_t*>(&S.atom_col[at]) = e8m0_of_pow2(i0) * 0x01010101u;
              *reinterpret_cast<uint32_t*>(&S.atom_col[at + 16]) = e8m0_of_pow2(i1) * 0x01010101u;
            } else {
              *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.col_scale) +
                                         int64_t(tr) * p.cols + c) = make_float2(i0, i1);
            }
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float* y = q == 0 ? y0 : y1;
        const float sc = q == 0 ? s0 : s1;
        const uint2 a = encode8_f32(y, sc), b = encode8_f32(y + 8, sc);
        const uint2 d = encode8_f32(y + 16, sc), e = encode8_f32(y + 24, sc);
        store_seg32(p.col + int64_t(c + q) * p.rows_pad + rr, make_uint4(a.x, a.y, b.x, b.y),
                    make_uint4(d.x, d.y, e.x, e.y), lo_ok, hi_ok, p.col_v8);
      }
    }
  }

  // ---- scales: an atom of a copy is 512 consecutive bytes
  if constexpr (OUT == N_MX || OUT == N_BW) {
    const bool atoms = OUT == N_MX || p.pow2;
    __syncthreads();
    if (p.row != nullptr) {
      if (atoms) {
        if (t < 128)
          reinterpret_cast<uint32_t*>(p.row_scale)[(int64_t(tr) * tiles_c + tc) * 128 + t] =
              reinterpret_cast<const uint32_t*>(S.atom_row)[t];
      } else if (t < 128) {
        reinterpret_cast<float*>(p.row_scale)[int64_t(tc) * p.rows_pad + r0 + t] = S.srow[t];
      }
    }
    if (p.col != nullptr && !p.col_bf16 && atoms && t >= 128)
      reinterpret_cast<uint32_t*>(p.col_scale)[(int64_t(tc) * (p.rows_pad >> 7) + tr) * 128 + t -
                                               128] =
          reinterpret_cast<const uint32_t*>(S.atom_col)[t - 128];
  }
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

template <int OUT>
cudaError_t launch_norm_tiles(const NormParams& p, cudaStream_t st) {
  static ContextOnce attr{};
  const cudaError_t e = once_per_context(attr, [] {
    return cudaFuncSetAttribute(norm_tile_kernel<OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                int(sizeof(NormTileSmem)));
  });
  if (e != cudaSuccess) return e;
  const int tiles_c = (p.cols + 127) / 128;
  const int64_t tiles = (p.rows_pad + 127) / 128 * tiles_c;
  return launch_kernel(norm_tile_kernel<OUT>, dim3(unsigned(tiles)), dim3(256),
                       sizeof(NormTileSmem), st, nullptr, p, tiles_c);
}

}  // namespace

int64_t norm_pad_rows(int kind, int64_t rows) {
  const int64_t q = kind == FP8_RECIPE_MXFP8 || kind == FP8_RECIPE_BLOCKWISE ? 128 : 16;
  return (rows + q - 1) / q * q;
}

size_t norm_workspace_bytes(int kind, int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  // rstd (when the caller keeps none), then the amax partials
  return size_t((rows * 4 + 15) / 16 * 16) +
         (kind == FP8_RECIPE_TENSORWISE || kind == FP8_RECIPE_DELAYED
              ? size_t(num_sms()) * kNormRowCtas * 4
              : 0);
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

  const bool tensor = a.kind == FP8_RECIPE_TENSORWISE || a.kind == FP8_RECIPE_DELAYED;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  uint32_t* part = reinterpret_cast<uint32_t*>(ws + (a.rows * 4 + 15) / 16 * 16);
  const bool two_pass = a.want_col || a.kind == FP8_RECIPE_TENSORWISE;
  int ctas = 0;
  if (!two_pass) {
    p.row = out->row;
    p.row_scale = out->row_scale;
    if (a.kind == FP8_RECIPE_MXFP8) return launch_rows<N_MX>(p, nullptr, st);
    if (a.kind == FP8_RECIPE_BLOCKWISE) return launch_rows<N_BW>(p, nullptr, st);
    p.scale_in = out->scale;
    p.part = part;
    const cudaError_t e = launch_rows<N_TENSOR>(p, &ctas, st);
    if (e != cudaSuccess) return e;
    return launch_kernel(norm_amax_kernel, dim3(1), dim3(512), 0, st, nullptr,
                         static_cast<const uint32_t*>(part), ctas, out->amax);
  }

  if (p.rstd == nullptr) p.rstd = reinterpret_cast<float*>(ws);
  if (tensor) p.part = part;
  cudaError_t e = launch_rows<N_STATS>(p, &ctas, st);
  if (e != cudaSuccess) return e;
  if (a.res == nullptr) {
    p.h = const_cast<uint16_t*>(a.x);             // read only from here on
  } else {
    p.ldx = a.cols;
  }
  p.row = a.want_row ? out->row : nullptr;
  p.row_scale = out->row_scale;
  p.col = a.want_col ? out->col : nullptr;
  p.col_scale = out->col_scale;
  p.col_v8 = p.col != nullptr && reinterpret_cast<uintptr_t>(p.col) % 32 == 0 &&
             p.rows_pad % 32 == 0;
  if (a.kind == FP8_RECIPE_MXFP8) return launch_norm_tiles<N_MX>(p, st);
  if (a.kind == FP8_RECIPE_BLOCKWISE) return launch_norm_tiles<N_BW>(p, st);
  p.n_part = ctas;
  p.scale_in = a.kind == FP8_RECIPE_DELAYED ? out->scale : nullptr;
  p.amax_out = out->amax;
  p.scale_out = out->scale;
  p.scale_inv_out = out->scale_inv;
  return launch_norm_tiles<N_TENSOR>(p, st);
}

}  // namespace fp8lin
