// Activation checkpoints in 8 bits (ckpt.cuh has the format): written from bf16
// (fp8_checkpoint_write), read back (fp8_checkpoint_read), and made into the FP8 copies that the
// linear layer reads, with the norm in front of it or without (fp8_checkpoint_quantize).
//
// The first two are one pass over memory, 3 + 1/32 bytes an element, and run at a copy's rate: 8192 x
// 16384 in 59.7 us written and 59.6 read, 6.8 TB/s (read with two 16-byte stores instead of one of
// 32 bytes: 69.0). A thread has 16 columns (32 bytes of bf16, 16 of codes); two lanes share a block's
// scale, eight a word of scales, so a row counts as a whole number of 128 columns and the lanes
// beyond its end idle.
//
// The third is the norm's column kernel with another source, 16.4 us for the MXFP8 column copy of
// 8192 x 4096 (69 MB: 10.2 at a copy's rate), and checkpoint_row_kernel for the row copy, 17.7. No
// one resource bounds them: DRAM is a quarter busy, of the issue slots 59 and 62 % are used. Their
// registers allow 25 to 30 % of the warps, too few to cover a chain of load, unpacking, maxima,
// shuffles and conversion. Both copies (34.1) read and unpack the checkpoint twice.
#include <algorithm>

#include "ckpt.cuh"
#include "common.cuh"
#include "internal.cuh"
#include "sm100_ptx.cuh"

namespace fp8lin {

struct CkptParams {
  uint16_t* x;                // bf16, pitch ldx (read or written)
  uint8_t* codes;
  uint8_t* scale;
  int64_t ldx, units;         // units: rows * units of a row
  int cols, row_units;        // units of a row: 16 columns each, a multiple of 8
  int step_rows, step_units;  // a CTA's threads in rows and units
  int v8;                     // x is 32-byte aligned (256-bit stores)
};

constexpr int kCkptThreads = 256;
constexpr int kCkptUnits = 4;   // units a thread, all of whose loads are issued first

// The row and the first column of this thread's next unit: one division a thread.
struct CkptAt {
  int64_t row;
  int unit;
  __device__ __forceinline__ CkptAt(const CkptParams& p, int64_t at)
      : row(at / p.row_units), unit(int(at - row * p.row_units)) {}
  __device__ __forceinline__ void next(const CkptParams& p) {
    row += p.step_rows;
    unit += p.step_units;
    if (unit >= p.row_units) {
      unit -= p.row_units;
      ++row;
    }
  }
};

__global__ void __launch_bounds__(kCkptThreads)
    checkpoint_write_kernel(const __grid_constant__ CkptParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const uint64_t first = ptx::l2_evict_first_policy();
  const int64_t at = int64_t(blockIdx.x) * (kCkptThreads * kCkptUnits) + threadIdx.x;
  uint4 v[kCkptUnits][2];
  CkptAt a(p, at);
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i, a.next(p)) {
    v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
    if (at + i * kCkptThreads < p.units && 16 * a.unit < p.cols) {
      const uint16_t* x = p.x + a.row * p.ldx + 16 * a.unit;
      v[i][0] = ldg_nc_v4_policy(x, first);
      v[i][1] = ldg_nc_v4_policy(x + 8, first);
    }
  }
  a = CkptAt(p, at);
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i, a.next(p)) {
    uint32_t m = max(bf16x8_mag(v[i][0]), bf16x8_mag(v[i][1]));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    float mult;
    uint32_t w = mx_scale_byte_f32(m, &mult) << (4 * (threadIdx.x & 6));
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    if (at + i * kCkptThreads >= p.units || 16 * a.unit >= p.cols) continue;
    const uint2 lo = encode8(v[i][0], mult, false), hi = encode8(v[i][1], mult, false);
    *reinterpret_cast<uint4*>(p.codes + a.row * p.cols + 16 * a.unit) =
        make_uint4(lo.x, lo.y, hi.x, hi.y);
    if ((a.unit & 7) == 0)
      *reinterpret_cast<uint32_t*>(p.scale + a.row * (p.row_units >> 1) + (a.unit >> 1)) = w;
  }
}

__global__ void __launch_bounds__(kCkptThreads)
    checkpoint_read_kernel(const __grid_constant__ CkptParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const uint64_t first = ptx::l2_evict_first_policy();
  const int64_t at = int64_t(blockIdx.x) * (kCkptThreads * kCkptUnits) + threadIdx.x;
  uint4 c[kCkptUnits];
  uint32_t e[kCkptUnits];
  CkptAt a(p, at);
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i, a.next(p)) {
    if (at + i * kCkptThreads < p.units && 16 * a.unit < p.cols) {
      c[i] = ldg_nc_v4_policy(p.codes + a.row * p.cols + 16 * a.unit, first);
      e[i] = __ldg(p.scale + a.row * (p.row_units >> 1) + (a.unit >> 1));
    }
  }
  a = CkptAt(p, at);
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i, a.next(p)) {
    if (at + i * kCkptThreads >= p.units || 16 * a.unit >= p.cols) continue;
    const float s = ckpt_factor(e[i]);
    const float2 s2 = make_float2(s, s);
    uint4 x[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float2 f[4];
      ckpt_widen8(k == 0 ? make_uint2(c[i].x, c[i].y) : make_uint2(c[i].z, c[i].w), f);
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] = __fmul2_rn(f[q], s2);
      x[k] = make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y),
                        pack_bf16(f[2].x, f[2].y), pack_bf16(f[3].x, f[3].y));
    }
    store_seg32(p.x + a.row * p.ldx + 16 * a.unit, x[0], x[1], true, true, p.v8);
  }
}

// The row copy of y = (h rstd) gamma (or of h) with h from its checkpoint, or, for per-tensor scales,
// the partials of y's amax; padding rows are zeros. The column copy is the norm's column kernel's.
// `width` lanes (8, 16 or 32) lie side by side on a row's units and stay on them, so gamma stays in
// registers; the CTA walks its share of the rows, four of a thread's at a time, whose loads are all
// issued first. 17.7 us at 8192 x 4096 (MXFP8), 69 MB and 11 instructions an element; threads that
// walk the units of all columns, with a division and gamma's loads for each, took 27.
template <int OUT>
__global__ void __launch_bounds__(kCkptThreads, 3)
    checkpoint_row_kernel(const __grid_constant__ NormParams p, const int width,
                          const uint32_t share) {
  __shared__ uint32_t red[kCkptThreads / 32];
  pdl_wait();
  const uint32_t rows = uint32_t(p.rows), pitch = (p.cols + 127) / 128 * 4;
  const uint32_t unit = blockIdx.x * width + threadIdx.x % width, c = 16 * unit;
  const uint32_t step = kCkptThreads / width;        // rows side by side
  const uint32_t begin = blockIdx.y * share + threadIdx.x / width;
  // (padded rows come by 16, a warp has at most four of them: it ends as a whole)
  const uint32_t end = min(uint32_t(p.rows_pad), (blockIdx.y + 1) * share);
  const bool in = c < uint32_t(p.cols);
  float2 g[2][4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (p.gamma != nullptr) {
      gamma_pairs(p.gamma, p.gamma_fp32, p.cols, c + 8 * k, g[k]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) g[k][q] = make_float2(1.0f, 1.0f);
    }
  }
  const float tensor_scale = OUT == N_TENSOR ? *p.scale_in : 1.0f;
  uint32_t amax = 0;
  for (uint32_t r0 = begin; r0 < end; r0 += kCkptUnits * step) {
    uint4 codes[kCkptUnits];
    uint32_t bytes[kCkptUnits];
    float rstd[kCkptUnits];
#pragma unroll
    for (int i = 0; i < kCkptUnits; ++i) {
      const uint32_t r = r0 + i * step;
      codes[i] = make_uint4(0, 0, 0, 0);             // beyond the tensor: zeros
      bytes[i] = 0;
      rstd[i] = 0.0f;
      if (in && r < min(rows, end)) {
        codes[i] = __ldg(reinterpret_cast<const uint4*>(p.ck + uint64_t(r) * p.cols + c));
        bytes[i] = __ldg(p.ck_scale + uint64_t(r) * pitch + (unit >> 1));
        rstd[i] = p.rstd == nullptr ? 1.0f : p.rstd[r];
      }
    }
#pragma unroll
    for (int i = 0; i < kCkptUnits; ++i) {
      const uint32_t r = r0 + i * step;
      if (r >= end) break;
      float2 y[2][4];
      const float f = ckpt_factor(bytes[i]) * rstd[i];
      const float2 f2 = make_float2(f, f);
      const bool live = r < rows;                    // else +0, whatever gamma's sign
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ckpt_widen8(
            k == 0 ? make_uint2(codes[i].x, codes[i].y) : make_uint2(codes[i].z, codes[i].w), y[k]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          y[k][q] = __fmul2_rn(__fmul2_rn(y[k][q], f2), g[k][q]);
          if (!live) y[k][q] = make_float2(0.0f, 0.0f);
        }
      }
      uint32_t m = max(__float_as_uint(max8_abs(y[0])), __float_as_uint(max8_abs(y[1])));
      if constexpr (OUT == N_STATS || OUT == N_TENSOR) amax = max(amax, m);
      if constexpr (OUT != N_STATS) {
        float s = tensor_scale;
        if constexpr (OUT == N_MX) {
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
          uint32_t w = mx_scale_byte_f32(m, &s) << (4 * (threadIdx.x & 6));
          w |= __shfl_xor_sync(0xffffffffu, w, 2);
          w |= __shfl_xor_sync(0xffffffffu, w, 4);
          if ((unit & 7) == 0 && in)
            *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.row_scale) +
                                         mx_scale_offset32(r, unit >> 1, p.cols)) = w;
        }
        if constexpr (OUT == N_BW) {
#pragma unroll
          for (int o = 1; o < 8; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          float sinv;
          s = scale_from_amax(__uint_as_float(m), p.margin, &sinv, 448.0f, p.pow2);
          if ((unit & 7) == 0 && in) {
            if (p.pow2)
              *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.row_scale) +
                                           mx_scale_offset32(r, unit >> 1, p.cols)) =
                  e8m0_of_pow2(sinv) * 0x01010101u;
            else
              reinterpret_cast<float*>(p.row_scale)[int64_t(unit >> 3) * p.rows_pad + r] = sinv;
          }
        }
        if (in) {
          const float2 s2 = make_float2(s, s);
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 a = __fmul2_rn(y[k >> 1][2 * (k & 1)], s2);
            const float2 b = __fmul2_rn(y[k >> 1][2 * (k & 1) + 1], s2);
            w[k] = cvt_e4m3x4(a.x, a.y, b.x, b.y);
          }
          *reinterpret_cast<uint4*>(p.row + uint64_t(r) * p.cols + c) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  if constexpr (OUT == N_STATS || OUT == N_TENSOR) {
    const uint32_t m = cta_max(amax, red);
    if (threadIdx.x == 0) p.part[blockIdx.y * gridDim.x + blockIdx.x] = m;
  }
  pdl_launch_dependents();
}

namespace {

cudaError_t checkpoint_rows(int out_kind, const NormParams& p, const void*, int* ctas,
                            cudaStream_t st) {
  const int row_units = (p.cols + 127) / 128 * 8;
  const int width = row_units >= 32 ? 32 : row_units == 16 ? 16 : 8;
  const unsigned blocks = (row_units + width - 1) / width;
  // the rows in as many shares as make three CTAs an SM, each some steps of all its threads
  const int64_t quantum = kCkptThreads / width * kCkptUnits;
  const int64_t shares = std::max<int64_t>(
      1, std::min<int64_t>((p.rows_pad + quantum - 1) / quantum, num_sms() * 3 / blocks));
  const int64_t share = ((p.rows_pad + shares - 1) / shares + quantum - 1) / quantum * quantum;
  const unsigned used = unsigned((p.rows_pad + share - 1) / share);
  if (ctas != nullptr) *ctas = int(blocks * used);
  auto kern = out_kind == N_MX       ? checkpoint_row_kernel<N_MX>
              : out_kind == N_BW     ? checkpoint_row_kernel<N_BW>
              : out_kind == N_TENSOR ? checkpoint_row_kernel<N_TENSOR>
                                     : checkpoint_row_kernel<N_STATS>;
  return launch_kernel(kern, dim3(blocks, used), dim3(kCkptThreads), 0, st, nullptr, p, width,
                       uint32_t(share));
}

CkptParams ckpt_params(const uint16_t* x, int64_t ldx, int64_t rows, int64_t cols,
                       const fp8_checkpoint& c, unsigned* grid) {
  CkptParams p{};
  p.x = const_cast<uint16_t*>(x);
  p.codes = c.codes;
  p.scale = c.scale;
  p.ldx = ldx;
  p.cols = int(cols);
  p.row_units = int((cols + 127) / 128 * 8);
  p.units = rows * p.row_units;
  p.v8 = reinterpret_cast<uintptr_t>(x) % 32 == 0;    // (columns come by 16)
  p.step_rows = kCkptThreads / p.row_units;
  p.step_units = kCkptThreads % p.row_units;
  *grid = unsigned((p.units + kCkptThreads * kCkptUnits - 1) / (kCkptThreads * kCkptUnits));
  return p;
}

}  // namespace

cudaError_t checkpoint_write_launch(const uint16_t* x, int64_t ldx, int64_t rows, int64_t cols,
                                    const fp8_checkpoint& out, cudaStream_t st) {
  unsigned grid;
  const CkptParams p = ckpt_params(x, ldx, rows, cols, out, &grid);
  return launch_kernel(checkpoint_write_kernel, dim3(grid), dim3(kCkptThreads), 0, st, nullptr, p);
}

cudaError_t checkpoint_read_launch(const fp8_checkpoint& in, int64_t rows, int64_t cols,
                                   uint16_t* x, cudaStream_t st) {
  unsigned grid;
  const CkptParams p = ckpt_params(x, cols, rows, cols, in, &grid);
  return launch_kernel(checkpoint_read_kernel, dim3(grid), dim3(kCkptThreads), 0, st, nullptr, p);
}

cudaError_t checkpoint_quantize_launch(const NormArgs& a, const fp8_checkpoint& in,
                                       fp8_tensor* out, void* workspace, cudaStream_t st) {
  NormParams p = norm_params(a);
  p.ck = in.codes;
  p.ck_scale = in.scale;
  return norm_copies_launch(a, p, out, workspace, st, checkpoint_rows, nullptr);
}

}  // namespace fp8lin
