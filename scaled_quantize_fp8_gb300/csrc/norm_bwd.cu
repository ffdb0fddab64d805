// Backward of RMSNorm and of the residual's addition (fp8_rmsnorm_bwd).
//
//   xh = h rstd,  t = dy gamma,  c = mean(t xh),  dh = dres + rstd (t - xh c),
//   dgamma = sum over rows of dy xh
//
// norm_bwd_kernel: a thread group holds a row, so every input is read once; each thread owns the
// same columns in all of its rows and adds their dgamma in registers. The CTAs' sums go to
// the workspace and norm_dgamma_kernel adds them in a fixed order.
//
// Bound by memory: 8 bytes an element. 8192 x 4096: 44.6 us, of which norm_dgamma_kernel 2.3; the
// bytes alone take 39.6 at the 6780 GB/s of a copy (0.89). 2048 x 16384: 46.9, of which 5 for
// dgamma (152 partials of 64 KB). 1024 x 32768: 76: a row of which is 192 KB of slots, so that no
// next one is on its way while it is worked on.
#include <algorithm>

#include "common.cuh"
#include "internal.cuh"
#include "norm.cuh"
#include "sm100_ptx.cuh"

namespace fp8lin {

struct NormBwdParams {
  const uint16_t* dy;
  const uint16_t* h;
  const uint16_t* dres;       // or null
  const void* gamma;
  const float* rstd;
  int64_t ld_dy, ld_h, ld_dres;
  int64_t rows;
  int cols;
  int gamma_fp32;
  float inv_cols;
  uint16_t* dh;               // [rows][cols]
  float* part;                // [CTAs][cols] dgamma sums, or null
};

// tpr threads per row, V vectors of eight columns a thread (vector j of lane l: columns
// 8 (j tpr + l) ..). Every thread copies its own elements of the next row to its own slots of
// shared memory while it works on the present one (cp.async; two buffers up to four vectors a
// thread). Two passes over a row: the dot product c (and dgamma), then dh. Up to two vectors the
// widened dy and xh stay in registers in between, beyond that they are made again from the
// slots. Products and sums are fp32, two an instruction (one at a time: 39 instructions an element
// instead of 21, 55 us at 8192 x 4096).
template <int V, bool DRES>
__global__ void __maxnreg__(V <= 2 ? 104 : 128)
    norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr bool kKeep = V <= 2, kGammaRegs = V <= 4;
  constexpr int kBufs = V <= 4 ? 2 : 1, kIn = DRES ? 3 : 2;
  __shared__ alignas(16) float red[2][16];
  extern __shared__ uint4 slots[];
  const int tpr = blockDim.x, lane = threadIdx.x, grp = threadIdx.y, rpc = blockDim.y;
  const int nt = tpr * rpc, tid = grp * tpr + lane, nv = p.cols >> 3;
  const int warps = tpr >> 5;                       // warps per row (0: two rows a warp)
  if (tid < 32) red[tid >> 4][tid & 15] = 0.0f;     // the unused warps' sums
  if (warps > 1) __syncthreads();
  pdl_wait();

  float next_rstd = 0.0f;
  const auto prefetch = [&](int64_t r, int buf) {
    const uint16_t* dy = p.dy + r * p.ld_dy + 8 * lane;
    const uint16_t* h = p.h + r * p.ld_h + 8 * lane;
    const uint16_t* dr = DRES ? p.dres + r * p.ld_dres + 8 * lane : nullptr;
    uint4* s = slots + buf * kIn * V * nt + tid;
    if (V * tpr == nv && r < p.rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ptx::cp_async_16(s + j * nt, dy + 8 * j * tpr);
        ptx::cp_async_16(s + (V + j) * nt, h + 8 * j * tpr);
        if (DRES) ptx::cp_async_16(s + (2 * V + j) * nt, dr + 8 * j * tpr);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {                  // nothing read beyond the tensor: zeros
        const bool in = r < p.rows && j * tpr + lane < nv;
        const uint32_t n = in ? 16u : 0u;
        ptx::cp_async_16_zfill(s + j * nt, in ? dy + 8 * j * tpr : p.dy, n);
        ptx::cp_async_16_zfill(s + (V + j) * nt, in ? h + 8 * j * tpr : p.h, n);
        if (DRES) ptx::cp_async_16_zfill(s + (2 * V + j) * nt, in ? dr + 8 * j * tpr : p.dres, n);
      }
    }
    ptx::cp_async_commit();
    next_rstd = r < p.rows ? p.rstd[r] : 0.0f;
  };
  const int64_t step = int64_t(gridDim.x) * rpc;
  int64_t r = int64_t(blockIdx.x) * rpc + grp;
  prefetch(r, 0);

  float2 g[kGammaRegs ? V : 1][4], acc[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (kGammaRegs) gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * (j * tpr + lane), g[j]);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[j][k] = make_float2(0.0f, 0.0f);
  }
  const auto gamma_of = [&](int j) -> float2(&)[4] {
    if constexpr (!kGammaRegs)
      gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * (j * tpr + lane), g[0]);
    return g[kGammaRegs ? j : 0];
  };

  for (int n = 0; r - grp < p.rows; r += step, ++n) {
    const int buf = kBufs == 2 ? n & 1 : 0;
    const uint4* s = slots + buf * kIn * V * nt + tid;
    const float2 rs = make_float2(next_rstd, next_rstd);
    ptx::cp_async_wait<0>();
    if (kBufs == 2 && r + step - grp < p.rows) prefetch(r + step, buf ^ 1);

    float2 d[kKeep ? V : 1][4], x[kKeep ? V : 1][4], c2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float2(&dj)[4] = d[kKeep ? j : 0], (&xj)[4] = x[kKeep ? j : 0], (&gj)[4] = gamma_of(j);
      widen8(s[j * nt], dj);
      widen8(s[(V + j) * nt], xj);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        xj[k] = __fmul2_rn(xj[k], rs);
        const float2 t = __fmul2_rn(dj[k], xj[k]);
        acc[j][k] = __fadd2_rn(acc[j][k], t);
        c2 = __ffma2_rn(t, gj[k], c2);
      }
    }
    float c = c2.x + c2.y;
    if (warps != 0) c += __shfl_xor_sync(0xffffffffu, c, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (warps > 1) {
      // by turns in two buffers: one barrier a row; the sums beyond the row's warps are zeros
      if ((lane & 31) == 0) red[n & 1][tid >> 5] = c;
      __syncthreads();
      const float* q = red[n & 1] + grp * warps;
      c = 0.0f;
      if (rpc == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = reinterpret_cast<const float4*>(q)[i];
          c += (v.x + v.y) + (v.z + v.w);
        }
      } else {
        for (int i = 0; i < warps; ++i) c += q[i];
      }
    }
    c *= -p.inv_cols;
    const float2 cc = make_float2(c, c);
    uint16_t* out = p.dh + r * p.cols + 8 * lane;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float2(&dj)[4] = d[kKeep ? j : 0], (&xj)[4] = x[kKeep ? j : 0], (&gj)[4] = gamma_of(j);
      if (!kKeep) {
        widen8(s[j * nt], dj);
        widen8(s[(V + j) * nt], xj);
#pragma unroll
        for (int k = 0; k < 4; ++k) xj[k] = __fmul2_rn(xj[k], rs);
      }
      float2 e[4];
      if (DRES) widen8(s[(2 * V + j) * nt], e);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 t = __ffma2_rn(xj[k], cc, __fmul2_rn(dj[k], gj[k]));
        e[k] = DRES ? __ffma2_rn(rs, t, e[k]) : __fmul2_rn(rs, t);
      }
      if (r < p.rows && j * tpr + lane < nv)
        *reinterpret_cast<uint4*>(out + 8 * j * tpr) =
            make_uint4(pack_bf16(e[0].x, e[0].y), pack_bf16(e[1].x, e[1].y),
                       pack_bf16(e[2].x, e[2].y), pack_bf16(e[3].x, e[3].y));
    }
    if (kBufs == 1 && r + step - grp < p.rows) prefetch(r + step, 0);
  }
  if (p.part != nullptr) {
    // the groups' sums, added by the first group in order (slots: 64 V nt bytes or more up to
    // four vectors a thread, of which 32 V nt are used here; with eight there is one group)
    float4* sums = reinterpret_cast<float4*>(slots);
    if (rpc > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sums[2 * j * nt + tid] = make_float4(acc[j][0].x, acc[j][0].y, acc[j][1].x, acc[j][1].y);
        sums[(2 * j + 1) * nt + tid] =
            make_float4(acc[j][2].x, acc[j][2].y, acc[j][3].x, acc[j][3].y);
      }
      __syncthreads();
    }
    if (grp == 0) {
      for (int i = 1; i < rpc; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float4 a = sums[2 * j * nt + i * tpr + lane];
          const float4 b = sums[(2 * j + 1) * nt + i * tpr + lane];
          acc[j][0] = __fadd2_rn(acc[j][0], make_float2(a.x, a.y));
          acc[j][1] = __fadd2_rn(acc[j][1], make_float2(a.z, a.w));
          acc[j][2] = __fadd2_rn(acc[j][2], make_float2(b.x, b.y));
          acc[j][3] = __fadd2_rn(acc[j][3], make_float2(b.z, b.w));
        }
      }
      float* dst = p.part + int64_t(blockIdx.x) * p.cols + 8 * lane;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j * tpr + lane < nv) {
          float4* q = reinterpret_cast<float4*>(dst + 8 * j * tpr);
          q[0] = make_float4(acc[j][0].x, acc[j][0].y, acc[j][1].x, acc[j][1].y);
          q[1] = make_float4(acc[j][2].x, acc[j][2].y, acc[j][3].x, acc[j][3].y);
        }
      }
    }
  }
  pdl_launch_dependents();
}

// dgamma = sum of n partials: 16 columns by 64 slices of the partials a CTA, a slice's loads four
// at a time; the slices are added in a fixed order. 2.3 us for 152 partials of 4096 columns, most
// of it latency (with 304 partials, a second round of loads, 4.1).
__global__ void __launch_bounds__(256) norm_dgamma_kernel(const float* part, int n, int cols,
                                                          float* dgamma) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float4 red[64][5];          // rows of 80 bytes: the lanes below read other banks
  const int q = threadIdx.x & 3, s = threadIdx.x >> 2;
  const float* at = part + blockIdx.x * 16 + 4 * q;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = s; i < n; i += 256) {
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = i + 64 * k < n ? *reinterpret_cast<const float4*>(at + int64_t(i + 64 * k) * cols)
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a.x += v[k].x;
      a.y += v[k].y;
      a.z += v[k].z;
      a.w += v[k].w;
    }
  }
  red[s][q] = a;
  __syncthreads();
  // column t / 16: four slices a lane, then the 16 lanes
  const int c = threadIdx.x >> 4, l = threadIdx.x & 15;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) t += reinterpret_cast<const float*>(&red[16 * i + l][c >> 2])[c & 3];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (l == 0) dgamma[blockIdx.x * 16 + c] = t;
}

namespace {

struct BwdPlan {
  RowPlan row;
  int grid;
};
// One CTA of up to 512 threads per SM: its row groups' dgamma meet in shared memory, so there are
// at most as many partials as SMs (8192 x 4096: 45.3 us; with two CTAs of 256: 46.4).
// Vectors a thread: many where loads in flight count, few where a row's latency does. Us at
//   rows x 4096:      300    600   1200   4800   8192
//   one              4.9    6.2   11.2   34.1   54.8
//   two              5.9    7.1   10.6   29.0   45.3
//   four             6.6    7.7   11.2   28.7   44.4
// Fewer rows a CTA while there are SMs without any (600 x 1024: 3.5 us, 4.4 with full CTAs).
BwdPlan bwd_plan(int64_t rows, int cols) {
  BwdPlan b;
  const int sms = num_sms();
  b.row = row_plan(cols, rows <= 4 * sms ? 1 : rows <= 32 * sms ? 2 : 4, 512);
  int rpc = b.row.block / b.row.tpr;
  while (rpc > 1 && (rpc / 2) * b.row.tpr >= 128 && rows <= int64_t(rpc / 2) * sms) rpc /= 2;
  b.row.block = rpc * b.row.tpr;
  b.grid = int(std::min<int64_t>((rows + rpc - 1) / rpc, sms));
  return b;
}

template <bool DRES>
cudaError_t launch_bwd(const NormBwdParams& p, const BwdPlan& b, cudaStream_t st) {
  const int v = b.row.v, rpc = b.row.block / b.row.tpr;
  auto kern = v == 1   ? norm_bwd_kernel<1, DRES>
              : v == 2 ? norm_bwd_kernel<2, DRES>
              : v == 4 ? norm_bwd_kernel<4, DRES>
                       : norm_bwd_kernel<8, DRES>;
  const size_t smem = size_t(v <= 4 ? 2 : 1) * (DRES ? 3 : 2) * v * b.row.block * 16;
  if (smem > 47 * 1024) {                                  // 48 KB with the static part
    static ContextOnce attr[4] = {};
    const cudaError_t e = once_per_context(attr[v == 1 ? 0 : v == 2 ? 1 : v == 4 ? 2 : 3], [&] {
      return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    });
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kern, dim3(unsigned(b.grid)), dim3(unsigned(b.row.tpr), unsigned(rpc)),
                       smem, st, nullptr, p);
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return size_t(bwd_plan(rows, int(cols)).grid) * size_t(cols) * 4;
}

cudaError_t norm_bwd_launch(const fp8_norm_grad& a, uint16_t* dh, float* dgamma, void* workspace,
                            cudaStream_t st) {
  const BwdPlan b = bwd_plan(a.rows, int(a.cols));
  NormBwdParams p{};
  p.dy = reinterpret_cast<const uint16_t*>(a.dy);
  p.h = reinterpret_cast<const uint16_t*>(a.h);
  p.dres = reinterpret_cast<const uint16_t*>(a.dres);
  p.gamma = a.gamma;
  p.rstd = a.rstd;
  p.ld_dy = a.ld_dy;
  p.ld_h = a.ld_h;
  p.ld_dres = a.ld_dres;
  p.rows = a.rows;
  p.cols = int(a.cols);
  p.gamma_fp32 = a.gamma_fp32;
  p.inv_cols = 1.0f / float(a.cols);
  p.dh = dh;
  p.part = dgamma == nullptr ? nullptr
           : b.grid == 1    ? dgamma
                             : reinterpret_cast<float*>(workspace);
  const cudaError_t e =
      p.dres != nullptr ? launch_bwd<true>(p, b, st) : launch_bwd<false>(p, b, st);
  if (e != cudaSuccess || dgamma == nullptr || b.grid == 1) return e;
  return launch_kernel(norm_dgamma_kernel, dim3(unsigned(a.cols / 16)), dim3(256), 0, st, nullptr,
                       static_cast<const float*>(p.part), b.grid, p.cols, dgamma);
}

}  // namespace fp8lin
