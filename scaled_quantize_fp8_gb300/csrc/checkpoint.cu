// Activation checkpoints in 8 bits (ckpt.cuh has the format): written from bf16
// (fp8_checkpoint_write) and read back (fp8_checkpoint_read).
//
// Both are one pass over memory, 3 + 1/32 bytes an element. A thread has 16 columns (32 bytes of
// bf16, 16 of codes); two lanes share a block's scale, eight a word of scales, so a row counts as a
// whole number of 128 columns and the lanes beyond its end idle.
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
    uint4* x = reinterpret_cast<uint4*>(p.x + a.row * p.ldx + 16 * a.unit);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float2 f[4];
      ckpt_widen8(k == 0 ? make_uint2(c[i].x, c[i].y) : make_uint2(c[i].z, c[i].w), f);
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] = __fmul2_rn(f[q], s2);
      x[k] = make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y),
                        pack_bf16(f[2].x, f[2].y), pack_bf16(f[3].x, f[3].y));
    }
  }
}

namespace {

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

}  // namespace fp8lin
