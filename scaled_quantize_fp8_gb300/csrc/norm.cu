// RMSNorm in front of the FP8 linear layer: the residual's addition, the norm, and the FP8
// copies of its output (fp8_rmsnorm_quantize).
//
//   h = bf16(x + residual),  rstd = 1 / sqrt(mean h^2 + eps),  y = (h * rstd) * gamma  (fp32)
//
// Two kernels:
//   norm_row_kernel   one group of threads per row, the row in registers: h, rstd, the row
//                     copy's codes and scales (blocks along the row lie in neighbouring lanes),
//                     and the amax partials of per-tensor scales.
//   norm_col_kernel   the column copy, which needs 32 or 128 rows of a column at once: reads h
//                     again, from L2, where the row kernel left it. With tensorwise scales,
//                     which need the whole tensor's amax before any code, the row copy too.
// Both evaluate y with the same two roundings, so a value has the same y in either copy.
//
// Bound by memory: 8192 x 4096 with a residual and both MXFP8 copies has to move 271 MB, 39.9 us
// at the 6780 GB/s of a copy; the two kernels take 48.7 (the row kernel alone 37.7, 0.92 of that
// rate). Why two: rstd needs a whole row, a column's scale 32 or 128 rows. One kernel that does
// both in one pass (a cluster of CTAs with 32 or 128 whole rows in registers) took 55.7: its
// loads, its exchange and its stores do not overlap, and no room is left to fetch the next rows
// meanwhile. A kernel for the statistics and then one for both copies took 55.8.
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

// ------------------------------------------------------------------------- rows
// tpr threads per row (16, or a multiple of 32), V 16-byte vectors a thread; vector j of lane l
// holds columns 8 (j tpr + l) .. so a warp reads 512 consecutive bytes and a block of 32 (128)
// columns lies in 4 (16) neighbouring lanes. The CTAs stay and walk the rows; each thread copies
// its own elements of the next row to shared memory (cp.async) while it works on the present one,
// and gamma stays in registers (up to four vectors). Sums of squares in fp32, two a thread, then
// over lanes and warps in a fixed order. y is made twice, for the maxima and for the codes: kept
// in between, two vectors are no faster (39.0 us either way, measured at that time) and four
// spill.
//
// What bounds it: memory with a residual (8192 x 4096, MXFP8 row copy: 236 MB in 37.7 us, 6260
// GB/s); without one the instructions as much (21.4 us for 15.0 of memory, of which the second sum
// over the lanes, see there, is 1.2).

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

// Rows on their way while one is worked on: as many as make four vectors a thread. 131072 x 256
// (one vector): both MXFP8 copies with a residual 0.67 -> 0.75 of the measured bandwidth, delayed
// ones without 0.50 -> 0.61; more than four vectors are no faster (two rows of 4096 columns with a
// residual: 41.6 us instead of 38.9).
template <int V, bool RES>
__host__ __device__ constexpr int rows_ahead() {
  return V == 1 ? (RES ? 2 : 4) : V == 2 && !RES ? 2 : 1;
}

template <int V, int OUT, bool RES>
__global__ void __maxnreg__(V <= 2 ? 72 : V == 4 ? 80 : 128)
    norm_row_kernel(const __grid_constant__ NormParams p) {
  constexpr bool kGammaRegs = V <= 4;               // eight vectors: gamma comes from L1
  pdl_wait();
  // Sums of a row's squares: with four vectors, the first and third apart from the second and
  // fourth, so that the order of additions is that of two vectors and twice the threads. (Only
  // where the row is short enough to get two: a branch that costs more than it saves.)
  constexpr int kSums = V == 4 ? 2 : 1;
  __shared__ alignas(16) float red[2][16 * kSums];
  __shared__ uint32_t redm[16];
  extern __shared__ uint4 slots[];                  // each thread's next rows
  const int tpr = blockDim.x, lane = threadIdx.x, grp = threadIdx.y, rpc = blockDim.y;
  const int warp = (grp * tpr + lane) >> 5, wl = (grp * tpr + lane) & 31, nv = p.cols >> 3;
  const int warps = tpr >> 5;                       // warps per row (0: two rows a warp)
  const bool want_y = OUT != N_STATS || p.y != nullptr || p.part != nullptr;
  // x and the residual are read once; h (x without a residual) is read again by the column kernel,
  // which then finds all but 1 % of its 67 MB in L2. With a residual the codes, not read before
  // the kernel is over, go first too. 8192 x 4096, both copies: MXFP8 48.7 us, delayed 46.1; the
  // codes as ordinary lines 49.4 and 47.8 (with a GEMM behind the norm 132.9 and 116.5, else 133.6
  // and 121: it gains nothing from finding the codes in L2); h as ordinary lines 52.0 and 49.0.
  // Without a residual there is room for them, and the GEMM does find them (118 us, else 120).
  const uint64_t first = ptx::l2_evict_first_policy(), last = ptx::l2_evict_last_policy();
  const uint64_t xpol = RES || !p.keep_h ? first : last, hpol = p.keep_h ? last : first;
  const uint64_t codes = RES ? first : ptx::l2_evict_normal_policy();
  const int nt = tpr * rpc, tid = grp * tpr + lane;
  constexpr int kAhead = rows_ahead<V, RES>();

  // Every thread copies its own elements of its next row while it works on the present one.
  const auto prefetch = [&](int64_t r, int buf) {
    uint4* s = slots + buf * (RES ? 2 : 1) * V * nt + tid;
    const uint16_t* x = p.x + r * p.ldx + 8 * lane;
    const uint16_t* res = RES ? p.res + r * p.ldr + 8 * lane : nullptr;
    if (V * tpr == nv && r < p.rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ptx::cp_async_16_hint(s + j * nt, x + 8 * j * tpr, xpol);
        if (RES) ptx::cp_async_16_hint(s + (V + j) * nt, res + 8 * j * tpr, first);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {                  // nothing read beyond the tensor: zeros
        const bool in = r < p.rows && j * tpr + lane < nv;
        const uint32_t n = in ? 16u : 0u;
        ptx::cp_async_16_zfill_hint(s + j * nt, in ? x + 8 * j * tpr : p.x, n, xpol);
        if (RES)
          ptx::cp_async_16_zfill_hint(s + (V + j) * nt, in ? res + 8 * j * tpr : p.res,
                                      n, first);
      }
    }
    ptx::cp_async_commit();
  };
  const int64_t row_step = int64_t(gridDim.x) * rpc;
  prefetch(int64_t(blockIdx.x) * rpc + grp, 0);
#pragma unroll
  for (int k = 1; k < kAhead; ++k) {
    const int64_t r0 = int64_t(blockIdx.x) * rpc + k * row_step;
    if (r0 < p.rows_pad) prefetch(r0 + grp, k);
    else ptx::cp_async_commit();                    // groups are counted: an empty one
  }

  float2 g[kGammaRegs ? V : 1][4];
  if (kGammaRegs && want_y) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * (j * tpr + lane), g[kGammaRegs ? j : 0]);
  }
  const auto gamma_of = [&](int j) -> float2(&)[4] {
    if constexpr (!kGammaRegs)
      gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * (j * tpr + lane), g[0]);
    return g[kGammaRegs ? j : 0];
  };
  const float tensor_scale = OUT == N_TENSOR ? *p.scale_in : 1.0f;
  uint32_t amax = 0;
  int phase = 0, buf = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * rpc; r0 < p.rows_pad; r0 += row_step) {
    const int64_t r = r0 + grp;
    const bool live = r < p.rows, stored = r < p.rows_pad;
    uint4 h[V];
    float ss[kSums];
    {
      uint16_t* ho = RES ? p.h + r * p.cols + 8 * lane : nullptr;
      const bool all = V * tpr == nv && live;                    // nothing to test per vector
      float2 q[kSums];
#pragma unroll
      for (int k = 0; k < kSums; ++k) q[k] = make_float2(0.0f, 0.0f);
      ptx::cp_async_wait<kAhead - 1>();
      const uint4* s = slots + buf * (RES ? 2 : 1) * V * nt + tid;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        h[j] = s[j * nt];
        if (RES) {
          const uint4 e = s[(V + j) * nt];
          h[j] = make_uint4(add_bf16x2(h[j].x, e.x), add_bf16x2(h[j].y, e.y),
                            add_bf16x2(h[j].z, e.z), add_bf16x2(h[j].w, e.w));
        }
      }
      const int64_t next = r0 + kAhead * row_step;
      if (next < p.rows_pad) prefetch(next + grp, buf);
      else if (kAhead > 1) ptx::cp_async_commit();
      if (kAhead > 1) buf = buf + 1 == kAhead ? 0 : buf + 1;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (RES && (all || (live && j * tpr + lane < nv)))
          stg_v4_policy(ho + 8 * j * tpr, h[j], hpol);
        const uint32_t w[4] = {h[j].x, h[j].y, h[j].z, h[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = make_float2(bf16_lo(w[k]), bf16_hi(w[k]));
          q[j % kSums] = __ffma2_rn(f, f, q[j % kSums]);
        }
      }
#pragma unroll
      for (int k = 0; k < kSums; ++k) ss[k] = q[k].x + q[k].y;
    }
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      if (warps != 0) ss[k] += __shfl_xor_sync(0xffffffffu, ss[k], 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss[k] += __shfl_xor_sync(0xffffffffu, ss[k], o);
      sum += ss[k];
    }
    if (warps > 1) {
      const int n = kSums * warps;
      float* q = red[phase] + grp * n;
      if ((lane & 31) == 0) {
#pragma unroll
        for (int k = 0; k < kSums; ++k) q[k * warps + (lane >> 5)] = ss[k];
      }
      __syncthreads();
      sum = 0.0f;
      if ((n & 3) == 0) {
        for (int i = 0; i < n; i += 4) {
          const float4 a = *reinterpret_cast<const float4*>(q + i);
          sum += (a.x + a.y) + (a.z + a.w);
        }
      } else {
        for (int i = 0; i < n; ++i) sum += q[i];
      }
      phase ^= 1;               // the next row's sums go to the other buffer: one barrier a row
    }
    const float rstd = rsqrtf(fmaf(sum, p.inv_cols, p.eps));
    if (live && lane == 0 && p.rstd != nullptr) p.rstd[r] = rstd;
    if (!want_y) continue;
    const float rl = live ? rstd : 0.0f;                         // padding rows: (0 0) gamma = 0

    // ---- the blocks' maxima and multipliers
    uint32_t m[V];
    float mult[V];
    if (OUT == N_MX || OUT == N_BW) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float2 y[4];
        norm_row8(h[j], rl, gamma_of(j), y);
        m[j] = __float_as_uint(max8_abs(y));
      }
    }
    if constexpr (OUT == N_MX) {
      constexpr int T = V >= 4 ? V / 4 : 1;                      // blocks that a lane scales
      scatter_max<V, 2>(m);
      const int q = lane & 3, s = (lane >> 2) & 3;
      uint32_t w[T];
#pragma unroll
      for (int t = 0; t < T; ++t) {
        // the four bytes of an atom's row in one word
        w[t] = mx_scale_byte_f32(m[t], &mult[t]) << (8 * s);
        w[t] |= __shfl_xor_sync(0xffffffffu, w[t], 4);
        w[t] |= __shfl_xor_sync(0xffffffffu, w[t], 8);
      }
      uint32_t word = w[0];                                      // of the 16 lanes' vector j
#pragma unroll
      for (int t = 1; t < T; ++t) word = s == t ? w[t] : word;
      const int j = V >= 4 ? T * q + s : V == 2 ? q >> 1 : 0, v = j * tpr + (lane & ~15);
      if (stored && v < nv && (V >= 4 ? s < T : s == 0 && (V == 2 ? (q & 1) == 0 : q == 0)))
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.row_scale) +
                                     mx_scale_offset32(r, v >> 2, p.cols)) = word;
    }
    if constexpr (OUT == N_BW) {
      scatter_max<V, 8>(m);
      float sinv;
      mult[0] = scale_from_amax(__uint_as_float(m[0]), p.margin, &sinv, 448.0f, p.pow2);
      const int j = (lane & 15) / (16 / V), v = j * tpr + (lane & ~15);
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
        OUT == N_STATS ? nullptr : p.row + (uint32_t(r) * uint32_t(p.cols) + uint32_t(8 * lane));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * tpr + lane;
      const bool in = v < nv;                 // uniform over the lanes of a block
      float2 y[4];
      // (for the amax, no NaN where a row's rstd is infinite and a lane has no column)
      const float rj = OUT == N_STATS || OUT == N_TENSOR ? (in ? rl : 0.0f) : rl;
      norm_row8(h[j], rj, gamma_of(j), y);
      if (p.y != nullptr && live && in)
        *reinterpret_cast<uint4*>(p.y + r * p.cols + 8 * v) =
            make_uint4(pack_bf16(y[0].x, y[0].y), pack_bf16(y[1].x, y[1].y),
                       pack_bf16(y[2].x, y[2].y), pack_bf16(y[3].x, y[3].y));
      if constexpr (OUT == N_STATS || OUT == N_TENSOR)
        amax = max(amax, __float_as_uint(max8_abs(y)));
      if constexpr (OUT != N_STATS) {
        float s = tensor_scale;
        if constexpr (OUT == N_MX) {
          constexpr int T = V >= 4 ? V / 4 : 1;
          s = __shfl_sync(0xffffffffu, mult[j % T],
                          (wl & 28) | (V >= 4 ? j / T : V == 2 ? 2 * j : 0));
        }
        if constexpr (OUT == N_BW)
          s = __shfl_sync(0xffffffffu, mult[0], (wl & 16) | (j * (16 / V)));
        const float2 s2 = make_float2(s, s);
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = __fmul2_rn(y[k], s2);
        if (in && stored)
          stg_v2_policy(row + 8 * j * tpr,
                        make_uint2(cvt_e4m3x4(y[0].x, y[0].y, y[1].x, y[1].y) & kept,
                                   cvt_e4m3x4(y[2].x, y[2].y, y[3].x, y[3].y) & kept),
                        codes);
      }
    }
  }
  if constexpr (OUT == N_STATS || OUT == N_TENSOR) {
    if (p.part != nullptr) {
      const uint32_t m = cta_max(amax, redm);
      if (threadIdx.x == 0 && threadIdx.y == 0) p.part[blockIdx.x] = m;
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

// ------------------------------------------------------------------------- columns
// A CTA of four warps, side by side, walks tiles of 128 rows x 64 columns of one column block.
// Lane l of a warp has the eight columns 8 (l / 16) .. of its 16 and the eight rows 8 (l % 16) ..:
// y stays in 64 registers between the maxima and the codes, and 16 lanes write 128 bytes of a
// column at once. Column maxima over lanes are reduced by halving: at each step a lane passes on
// half of its columns and keeps the other half. While a tile is worked on, the CTA copies the next
// one to the other buffer in shared memory (cp.async); the 16-byte pieces of row r are exchanged
// by (r / 8) % 8 so that the rows eight apart that lanes read at once lie in different banks.
//
// 10.9 us at 8192 x 4096 (MXFP8), where its 35 MB of stores alone would take 5. No one resource
// bounds it: L1, the ALUs and the schedulers are each about half busy; without its loads it took
// 3 us less, without its stores 4 less. Loads by TMA, two and three tiles ahead, column lines put
// together in shared memory, a warp's rows one below the other: all within 0.5 us.
//
// CTAs per SM: five, at 102 registers a thread (MXFP8: 48.7 us for both copies; four 49.2, six,
// which spill, 52.5), but six where there are no maxima (FULL, per-tensor scales: 46.1; five
// 46.4).
template <int OUT, bool FULL>
constexpr int col_ctas() {
  return OUT == N_TENSOR && FULL ? 6 : 5;
}

struct NormColSmem {
  uint4 slots[2][128][8];
  alignas(16) float rstd[2][128];
  uint32_t red[4];
};

// FULL: nothing but the FP8 column copy is wanted and every tile lies inside the padded tensor,
// so nothing is tested per row (8192 x 4096, both copies: 48.7 us, else 52.6, with a few spills).
template <int OUT, bool FULL>
__global__ void __launch_bounds__(128, col_ctas<OUT, FULL>())
    norm_col_kernel(const __grid_constant__ NormParams p, const int tiles_c, const int tiles_r) {
  __shared__ NormColSmem S;
  const int t = threadIdx.x, lane = t & 31, w = t >> 5, l2 = lane >> 4, l16 = lane & 15;
  const int c0 = (int(blockIdx.x) % tiles_c) * 64, c = c0 + 16 * w + 8 * l2;
  const int step = int(gridDim.x) / tiles_c;
  const bool in = FULL || c < p.cols;
  const bool want_row = !FULL && OUT == N_TENSOR && p.row != nullptr;
  const bool want_col = FULL || p.col != nullptr, col_bf16 = !FULL && p.col_bf16;
  pdl_wait();

  // The last read of h. One that was just written becomes an ordinary line: evicted first, its
  // write-back would meet the copies' (both MXFP8 copies, 8192 x 4096: 52.5 us, 48.7). x, which
  // is not dirty, makes room for them (without a residual 32.9 us, as an ordinary line 34.1).
  const uint64_t first = ptx::l2_evict_first_policy();
  const uint64_t policy = p.res != nullptr ? ptx::l2_evict_normal_policy() : first;
  const auto prefetch = [&](int tile, int buf) {
    // thread t copies piece t % 8 of the rows t / 8, t / 8 + 16, ..
    const int64_t r0 = int64_t(tile) * 128, r = r0 + (t >> 3);
    const int piece = t & 7, cp = c0 + 8 * piece;
    const uint16_t* x = p.h + r * p.ldx + cp;
    const bool whole = cp < p.cols && r0 + 128 <= p.rows;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = (t >> 3) + 16 * i;
      uint4* d = &S.slots[buf][row][piece ^ ((row >> 3) & 7)];
      if (whole) {
        ptx::cp_async_16_hint(d, x, policy);
      } else {                                                   // nothing read beyond: zeros
        const uint32_t n = cp < p.cols && r + 16 * i < p.rows ? 16u : 0u;
        ptx::cp_async_16_zfill_hint(d, n ? x : p.h, n, policy);
      }
      x += 16 * p.ldx;
    }
    ptx::cp_async_commit();
    // padding rows: rstd 0, so that y = (0 0) gamma = 0
    return r0 + t < p.rows ? p.rstd[r0 + t] : 0.0f;
  };

  // Last tiles first: the row kernel wrote the last rows of h most recently.
  int tile = tiles_r - 1 - int(blockIdx.x) / tiles_c;
  float next_rstd = tile >= 0 ? prefetch(tile, 0) : 0.0f;
  float2 g[4];
  gamma_pairs(p.gamma, p.gamma_fp32, p.cols, c, g);
  float scale = 1.0f;
  if constexpr (OUT == N_TENSOR) {
    uint32_t m = 0;
    if (p.scale_in == nullptr || blockIdx.x == 0) {
      for (int i = t; i < p.n_part; i += 128) m = max(m, p.part[i]);
      m = cta_max(m, S.red);
    }
    float sinv;
    scale = p.scale_in != nullptr ? *p.scale_in
                                  : scale_from_amax(__uint_as_float(m), p.margin, &sinv);
    if (blockIdx.x == 0 && t == 0) {
      *p.amax_out = __uint_as_float(m);
      if (p.scale_in == nullptr) {
        *p.scale_out = scale;
        *p.scale_inv_out = sinv;
      }
    }
  }

  for (int buf = 0; tile >= 0; tile -= step, buf ^= 1) {
    const int64_t r0 = int64_t(tile) * 128, r = r0 + 8 * l16;
    S.rstd[buf][t] = next_rstd;
    ptx::cp_async_wait<0>();
    __syncthreads();                               // the tile is there, the last one read
    if (tile >= step) next_rstd = prefetch(tile - step, buf ^ 1);
    float2 y[8][4];
    {
      const float4 ra = *reinterpret_cast<const float4*>(&S.rstd[buf][8 * l16]);
      const float4 rb = *reinterpret_cast<const float4*>(&S.rstd[buf][8 * l16 + 4]);
      const float rs[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        norm_row8(S.slots[buf][8 * l16 + i][(2 * w + l2) ^ (l16 & 7)], rs[i], g, y[i]);
    }
    // padding rows: (0 0) gamma has gamma's sign, theirs is +0 (FULL: at the stores)
    if (!FULL && int(r0) + 128 > int(p.rows)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool live = int(r) + i < int(p.rows);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[i][k].x = live ? y[i][k].x : 0.0f;
          y[i][k].y = live ? y[i][k].y : 0.0f;
        }
      }
    }

    // ---- the columns' multipliers
    float2 cs[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) cs[k] = make_float2(scale, scale);
    if (OUT != N_TENSOR && !col_bf16) {
      uint32_t m[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a = max3_abs(y[0][k].x, y[1][k].x, y[2][k].x);
        float b = max3_abs(y[0][k].y, y[1][k].y, y[2][k].y);
        a = max3_abs(max3_abs(a, y[3][k].x, y[4][k].x), y[5][k].x, y[6][k].x);
        b = max3_abs(max3_abs(b, y[3][k].y, y[4][k].y), y[5][k].y, y[6][k].y);
        m[2 * k] = __float_as_uint(max3_abs(a, y[7][k].x, 0.0f));
        m[2 * k + 1] = __float_as_uint(max3_abs(b, y[7][k].y, 0.0f));
      }
      // lane bit 1 names columns 0 - 3 or 4 - 7, bit 0 the first or second pair of those
      const bool u = (lane & 2) != 0, v = (lane & 1) != 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        m[k] = max(u ? m[k + 4] : m[k],
                   __shfl_xor_sync(0xffffffffu, u ? m[k] : m[k + 4], 2));
#pragma unroll
      for (int k = 0; k < 2; ++k)
        m[k] = max(v ? m[k + 2] : m[k], __shfl_xor_sync(0xffffffffu, v ? m[k] : m[k + 2], 1));
      const int c2 = c + 2 * (lane & 3);               // this lane's two columns
      float s0, s1;
      if constexpr (OUT == N_MX) {
        const uint32_t b0 = mx_scale_byte_f32(m[0], &s0), b1 = mx_scale_byte_f32(m[1], &s1);
        uint8_t* d = reinterpret_cast<uint8_t*>(p.col_scale) +
                     mx_scale_offset(c2, r >> 5, p.rows_pad);
        if (want_col && in) {
          d[0] = uint8_t(b0);
          d[16] = uint8_t(b1);                         // the next column's row of the atom
        }
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {                  // 128 rows
          m[k] = max(m[k], __shfl_xor_sync(0xffffffffu, m[k], 4));
          m[k] = max(m[k], __shfl_xor_sync(0xffffffffu, m[k], 8));
        }
        float i0, i1;
        s0 = scale_from_amax(__uint_as_float(m[0]), p.margin, &i0, 448.0f, p.pow2);
        s1 = scale_from_amax(__uint_as_float(m[1]), p.margin, &i1, 448.0f, p.pow2);
        if (want_col && in && l16 < 4) {
          if (p.pow2) {
            uint8_t* d = reinterpret_cast<uint8_t*>(p.col_scale) +
                         mx_scale_offset(c2, r0 >> 5, p.rows_pad);
            *reinterpret_cast<uint32_t*>(d) = e8m0_of_pow2(i0) * 0x01010101u;
            *reinterpret_cast<uint32_t*>(d + 16) = e8m0_of_pow2(i1) * 0x01010101u;
          } else {
            *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.col_scale) +
                                       (r0 >> 7) * p.cols + c2) = make_float2(i0, i1);
          }
        }
      }
      // back to all eight columns of the lane
      const float t0 = __shfl_xor_sync(0xffffffffu, s0, 1);
      const float t1 = __shfl_xor_sync(0xffffffffu, s1, 1);
      const float2 pa = v ? make_float2(t0, t1) : make_float2(s0, s1);
      const float2 pb = v ? make_float2(s0, s1) : make_float2(t0, t1);
      const float2 qa = make_float2(__shfl_xor_sync(0xffffffffu, pa.x, 2),
                                    __shfl_xor_sync(0xffffffffu, pa.y, 2));
      const float2 qb = make_float2(__shfl_xor_sync(0xffffffffu, pb.x, 2),
                                    __shfl_xor_sync(0xffffffffu, pb.y, 2));
      cs[0] = u ? qa : pa;
      cs[1] = u ? qb : pb;
      cs[2] = u ? pa : qa;
      cs[3] = u ? pb : qb;
    }

    // ---- codes
    const bool stored = in && (FULL || r < p.rows_pad);        // 8 rows: all or none
    if (want_col && col_bf16) {
      if (stored) {
        uint16_t* d = reinterpret_cast<uint16_t*>(p.col) + int64_t(c) * p.rows_pad + r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          *reinterpret_cast<uint4*>(d) =
              make_uint4(pack_bf16(y[0][k].x, y[1][k].x), pack_bf16(y[2][k].x, y[3][k].x),
                         pack_bf16(y[4][k].x, y[5][k].x), pack_bf16(y[6][k].x, y[7][k].x));
          d += p.rows_pad;
          *reinterpret_cast<uint4*>(d) =
              make_uint4(pack_bf16(y[0][k].y, y[1][k].y), pack_bf16(y[2][k].y, y[3][k].y),
                         pack_bf16(y[4][k].y, y[5][k].y), pack_bf16(y[6][k].y, y[7][k].y));
          d += p.rows_pad;
        }
      }
    }
    if (want_row || !col_bf16) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i][k] = __fmul2_rn(y[i][k], cs[k]);
    }
    if (want_row) {
      // by way of the tile's buffer (64 bytes a row, 8-byte units exchanged like the pieces), so
      // that four lanes write 64 consecutive bytes
      __syncthreads();
      uint2* codes = reinterpret_cast<uint2*>(&S.slots[buf][0][0]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        codes[(8 * l16 + i) * 8 + ((2 * w + l2) ^ (l16 & 7))] =
            make_uint2(cvt_e4m3x4(y[i][0].x, y[i][0].y, y[i][1].x, y[i][1].y),
                       cvt_e4m3x4(y[i][2].x, y[i][2].y, y[i][3].x, y[i][3].y));
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = (t >> 2) + 32 * i, e = (q >> 3) & 7, at = 2 * (t & 3);
        const uint4 v = reinterpret_cast<const uint4*>(codes)[(q * 8 + (at ^ (e & 6))) >> 1];
        if (r0 + q < p.rows_pad && c0 + 8 * at < p.cols)
          *reinterpret_cast<uint4*>(p.row + (r0 + q) * p.cols + c0 + 8 * at) =
              (e & 1) ? make_uint4(v.z, v.w, v.x, v.y) : v;
      }
    }
    if (want_col && !col_bf16 && stored) {
      const uint32_t pitch = uint32_t(p.rows_pad);    // (less than 2^31 elements)
      uint32_t at = uint32_t(c) * pitch + uint32_t(r);
      const auto store = [&](uint32_t lo, uint32_t hi) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          stg_v2_policy(p.col + at,
                        make_uint2(cvt_e4m3x4(y[0][k].x, y[1][k].x, y[2][k].x, y[3][k].x) & lo,
                                   cvt_e4m3x4(y[4][k].x, y[5][k].x, y[6][k].x, y[7][k].x) & hi),
                        first);
          at += pitch;
          stg_v2_policy(p.col + at,
                        make_uint2(cvt_e4m3x4(y[0][k].y, y[1][k].y, y[2][k].y, y[3][k].y) & lo,
                                   cvt_e4m3x4(y[4][k].y, y[5][k].y, y[6][k].y, y[7][k].y) & hi),
                        first);
          at += pitch;
        }
      };
      // padding rows: (0 0) gamma has gamma's sign, their codes are +0. Where there are maxima,
      // whole tiles go apart (MXFP8 49.1 us, all masked 49.4, none 48.9), else all are masked
      // (delayed 46.3, whole tiles apart 46.6, none 46.2).
      const int live = int(p.rows) - int(r);          // of the lane's eight rows
      if (!FULL || (OUT != N_TENSOR && int(r0) + 128 <= int(p.rows)))
        store(0xffffffffu, 0xffffffffu);
      else
        store(live >= 4 ? 0xffffffffu : live <= 0 ? 0u : (1u << (8 * live)) - 1u,
              live >= 8 ? 0xffffffffu : live <= 4 ? 0u : (1u << (8 * (live - 4))) - 1u);
    }
  }
  pdl_launch_dependents();
}

// ------------------------------------------------------------------------- host

namespace {

constexpr int kNormMaxParts = 4096;   // amax partials: one per CTA of the row kernel

// Vectors a thread: enough loads in flight, but no more registers than that needs. With a residual
// (twice the loads) two, 4096 columns then being 256 threads (8192 x 4096, row copy: 37.7 us; four
// 39.2, one 47.1); without one four (both copies: 33.6; two 36.9); and four for longer rows, of
// which two would make CTAs of 512 threads, one per SM (4096 x 8192, row copy: 38.0; two 42.2;
// widths between the two were not measured).
// A row's sum, and so its last bit, must not depend on how many rows there are (a token served
// alone gives what it gives in a batch) nor on whether the residual was added here: the threads
// are twice as many with two vectors, which are used only where that comes out even, and few rows,
// which one vector would do sooner (64 x 4096: 2.0 us; two 2.2, four 3.0), are no exception.
RowPlan fwd_plan(int cols, bool res) {
  const RowPlan two = row_plan(cols, 2, 256), four = row_plan(cols, 4, 256);
  return res && cols <= 4096 && two.tpr == 2 * four.tpr ? two : four;
}

template <int OUT, bool RES>
cudaError_t launch_rows(const NormParams& p, int* ctas, cudaStream_t st) {
  const RowPlan pl = fwd_plan(p.cols, RES);
  const int rpc = pl.block / pl.tpr;
  // as many CTAs as run at once: a quarter of an SM has registers for seven warps at 72 a thread,
  // six at 80, four at 128. One CTA too many per SM runs alone at the end (6528 x 5120, row copy:
  // 46 us instead of 40).
  const int per_sm = (pl.v <= 2 ? 896 : pl.v == 4 ? 768 : 512) / pl.block;
  const int64_t grid = std::min<int64_t>((p.rows_pad + rpc - 1) / rpc,
                                         int64_t(num_sms()) * std::max(1, per_sm));
  if (ctas != nullptr) *ctas = int(grid);
  auto kern = pl.v == 1   ? norm_row_kernel<1, OUT, RES>
              : pl.v == 2 ? norm_row_kernel<2, OUT, RES>
              : pl.v == 4 ? norm_row_kernel<4, OUT, RES>
                          : norm_row_kernel<8, OUT, RES>;
  const int ahead = pl.v == 1   ? rows_ahead<1, RES>()
                    : pl.v == 2 ? rows_ahead<2, RES>()
                                : 1;
  const size_t smem = size_t(RES ? 2 : 1) * ahead * pl.v * pl.block * 16;
  if (smem > 47 * 1024) {                          // 48 KB with the static part
    static ContextOnce attr[2] = {};               // v = 4 and 8, 512 threads
    const cudaError_t e = once_per_context(attr[pl.v > 4], [&] {
      return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    });
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kern, dim3(unsigned(grid)), dim3(unsigned(pl.tpr), unsigned(rpc)), smem, st,
                       nullptr, p);
}
template <int OUT>
cudaError_t launch_rows(const NormParams& p, int* ctas, cudaStream_t st) {
  return p.res != nullptr ? launch_rows<OUT, true>(p, ctas, st)
                          : launch_rows<OUT, false>(p, ctas, st);
}

template <int OUT>
cudaError_t launch_cols(const NormParams& p, cudaStream_t st) {
  const int tiles_c = (p.cols + 63) / 64;
  const int tiles_r = int((p.rows_pad + 127) / 128);
  const bool full = (OUT != N_TENSOR || p.row == nullptr) && p.col != nullptr && !p.col_bf16 &&
                    p.cols % 64 == 0 && p.rows_pad % 128 == 0;
  auto kern = full ? norm_col_kernel<OUT, true> : norm_col_kernel<OUT, false>;
  // every CTA keeps its column block (and gamma): a whole number of CTAs per block
  const int ctas = full ? col_ctas<OUT, true>() : col_ctas<OUT, false>();
  const int per_block = std::min(tiles_r, std::max(1, num_sms() * ctas / tiles_c));
  return launch_kernel(kern, dim3(unsigned(per_block * tiles_c)), dim3(128), 0, st, nullptr, p,
                       tiles_c, tiles_r);
}

}  // namespace

int64_t norm_pad_rows(int kind, int64_t rows) {
  const int64_t q = kind == FP8_RECIPE_MXFP8 || kind == FP8_RECIPE_BLOCKWISE ? 128 : 16;
  return (rows + q - 1) / q * q;
}

size_t norm_workspace_bytes(int kind, int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  // rstd (when the caller keeps none), then the amax partials
  const bool tensor = kind == FP8_RECIPE_TENSORWISE || kind == FP8_RECIPE_DELAYED;
  return size_t((rows * 4 + 15) / 16 * 16) + (tensor ? size_t(kNormMaxParts) * 4 : 0);
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
  p.inv_cols = 1.0f / float(a.cols);
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
  const bool tensorwise = a.kind == FP8_RECIPE_TENSORWISE;
  p.row = a.want_row ? out->row : nullptr;
  p.row_scale = out->row_scale;
  p.col = a.want_col ? out->col : nullptr;
  p.col_scale = out->col_scale;

  // Rows: h, rstd, the row copy where its scale is known by then.
  const bool cols = a.want_col || tensorwise;
  if (p.rstd == nullptr && cols) p.rstd = reinterpret_cast<float*>(workspace);
  p.keep_h = cols;
  if (out_kind == N_TENSOR) {
    p.part = part;
    if (!tensorwise) p.scale_in = out->scale;
  }
  int ctas = 0;
  cudaError_t e;
  if (p.row == nullptr || tensorwise) e = launch_rows<N_STATS>(p, &ctas, st);
  else if (out_kind == N_MX) e = launch_rows<N_MX>(p, &ctas, st);
  else if (out_kind == N_BW) e = launch_rows<N_BW>(p, &ctas, st);
  else e = launch_rows<N_TENSOR>(p, &ctas, st);
  if (e != cudaSuccess) return e;
  if (!cols) {
    if (out_kind != N_TENSOR) return cudaSuccess;
    return launch_kernel(norm_amax_kernel, dim3(1), dim3(512), 0, st, nullptr,
                         static_cast<const uint32_t*>(part), ctas, out->amax);
  }

  // Columns.
  if (a.res == nullptr) p.h = const_cast<uint16_t*>(a.x);     // read only from here on
  else p.ldx = a.cols;
  if (out_kind == N_MX) return launch_cols<N_MX>(p, st);
  if (out_kind == N_BW) return launch_cols<N_BW>(p, st);
  p.n_part = ctas;
  p.amax_out = out->amax;
  p.scale_out = out->scale;
  p.scale_inv_out = out->scale_inv;
  if (!tensorwise) p.row = nullptr;                           // the row kernel wrote it
  return launch_cols<N_TENSOR>(p, st);
}

}  // namespace fp8lin
