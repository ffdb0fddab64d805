// Backward of RMSNorm and of the residual's addition (fp8_rmsnorm_bwd).
//
//   xh = h rstd,  t = dy gamma,  c = mean(t xh),  dh = dres + rstd (t - xh c),
//   dgamma = sum over rows of dy xh
//
// norm_bwd_kernel: a thread group holds a row (its dy, h and dres in registers), so every input
// is read once; each thread owns the same columns in all of its rows and adds their dgamma in
// registers. The groups' sums go to the workspace and norm_dgamma_kernel adds them in a fixed
// order.
#include <algorithm>

#include "common.cuh"
#include "internal.cuh"
#include "norm.cuh"

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
  uint16_t* dh;               // [rows][cols]
  float* part;                // [groups of the grid][cols] dgamma sums, or null
};

// V vectors of eight columns a thread, U rows of a group at a time (their sums share one
// barrier).
template <int V, int U>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const __grid_constant__ NormBwdParams p,
                                                       const int tpr) {
  pdl_wait();
  __shared__ float red[2][U][16];
  const int lane = threadIdx.x % tpr, grp = threadIdx.x / tpr;
  const int rpc = blockDim.x / tpr, nv = p.cols >> 3;
  const int warps = tpr >> 5;
  float acc[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
  int phase = 0;
  const int64_t step = int64_t(gridDim.x) * rpc * U;
  for (int64_t base = int64_t(blockIdx.x) * rpc * U; base < p.rows; base += step) {
    const int64_t r0 = base + grp * U;
    uint4 dy[U][V], h[U][V], dr[U][V];
    float rstd[U], c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u;
      rstd[u] = r < p.rows ? p.rstd[r] : 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * tpr + lane;
        dy[u][j] = h[u][j] = dr[u][j] = make_uint4(0, 0, 0, 0);
        if (r < p.rows && v < nv) {
          dy[u][j] = *reinterpret_cast<const uint4*>(p.dy + r * p.ld_dy + 8 * v);
          h[u][j] = *reinterpret_cast<const uint4*>(p.h + r * p.ld_h + 8 * v);
          if (p.dres != nullptr)
            dr[u][j] = *reinterpret_cast<const uint4*>(p.dres + r * p.ld_dres + 8 * v);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) c[u] = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * tpr + lane;
      if (v >= nv) continue;
      float g[8];
      load_gamma8(p.gamma, p.gamma_fp32, 8 * v, g);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t a[4] = {dy[u][j].x, dy[u][j].y, dy[u][j].z, dy[u][j].w};
        const uint32_t b[4] = {h[u][j].x, h[u][j].y, h[u][j].z, h[u][j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = bf16_lo(b[i]) * rstd[u], x1 = bf16_hi(b[i]) * rstd[u];
          const float d0 = bf16_lo(a[i]) * x0, d1 = bf16_hi(a[i]) * x1;
          acc[j][2 * i] += d0;
          acc[j][2 * i + 1] += d1;
          c[u] = fmaf(d0, g[2 * i], c[u]);
          c[u] = fmaf(d1, g[2 * i + 1], c[u]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      for (int o = (warps == 0 ? tpr : 32) >> 1; o > 0; o >>= 1)
        c[u] += __shfl_xor_sync(0xffffffffu, c[u], o);
    if (warps > 1) {
      if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) red[phase][u][threadIdx.x >> 5] = c[u];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        c[u] = 0.0f;
        for (int i = 0; i < warps; ++i) c[u] += red[phase][u][grp * warps + i];
      }
      phase ^= 1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) c[u] = __fdiv_rn(c[u], float(p.cols));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * tpr + lane;
      if (v >= nv) continue;
      float g[8];
      load_gamma8(p.gamma, p.gamma_fp32, 8 * v, g);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u;
        if (r >= p.rows) continue;
        const uint32_t a[4] = {dy[u][j].x, dy[u][j].y, dy[u][j].z, dy[u][j].w};
        const uint32_t b[4] = {h[u][j].x, h[u][j].y, h[u][j].z, h[u][j].w};
        const uint32_t d[4] = {dr[u][j].x, dr[u][j].y, dr[u][j].z, dr[u][j].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = bf16_lo(b[i]) * rstd[u], x1 = bf16_hi(b[i]) * rstd[u];
          const float t0 = fmaf(-x0, c[u], bf16_lo(a[i]) * g[2 * i]);
          const float t1 = fmaf(-x1, c[u], bf16_hi(a[i]) * g[2 * i + 1]);
          o[i] = pack_bf16(fmaf(rstd[u], t0, bf16_lo(d[i])), fmaf(rstd[u], t1, bf16_hi(d[i])));
        }
        *reinterpret_cast<uint4*>(p.dh + r * p.cols + 8 * v) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  if (p.part != nullptr) {
    float* dst = p.part + (int64_t(blockIdx.x) * rpc + grp) * p.cols;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * tpr + lane;
      if (v < nv) {
        float4* q = reinterpret_cast<float4*>(dst + 8 * v);
        q[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        q[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
      }
    }
  }
  pdl_launch_dependents();
}

// dgamma = sum of n partials: 16 columns (four float4) by 64 slices of the partials a CTA; the
// slices are added in order.
__global__ void __launch_bounds__(256) norm_dgamma_kernel(const float* part, int n, int cols,
                                                          float* dgamma) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float4 red[64][4];
  const int q = threadIdx.x & 3, s = threadIdx.x >> 2;
  const int c = blockIdx.x * 16 + 4 * q;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = s; i < n; i += 64) {
    const float4 v = *reinterpret_cast<const float4*>(part + int64_t(i) * cols + c);
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  red[s][q] = a;
  __syncthreads();
  if (threadIdx.x < 16) {
    const int qq = threadIdx.x >> 2, k = threadIdx.x & 3;
    float t = 0.0f;
    for (int i = 0; i < 64; ++i) t += reinterpret_cast<const float*>(&red[i][qq])[k];
    dgamma[blockIdx.x * 16 + threadIdx.x] = t;
  }
}

namespace {

constexpr int kBwdCtas = 2;            // CTAs of 512 threads per SM (and their dgamma partials)
constexpr int kBwdBlock = 512;

struct BwdPlan {
  RowPlan row;
  int u, grid, parts;
};
BwdPlan bwd_plan(int64_t rows, int cols) {
  BwdPlan b;
  b.row = row_plan(cols, 1, kBwdBlock);
  b.u = b.row.v <= 2 ? 2 : 1;
  const int rpc = b.row.block / b.row.tpr;
  const int64_t groups = (rows + rpc * b.u - 1) / (rpc * b.u);
  b.grid = int(std::min<int64_t>(groups, int64_t(num_sms()) * kBwdCtas));
  b.parts = b.grid * rpc;
  return b;
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return size_t(bwd_plan(rows, int(cols)).parts) * size_t(cols) * 4;
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
  p.dh = dh;
  p.part = dgamma == nullptr ? nullptr
           : b.parts == 1    ? dgamma
                             : reinterpret_cast<float*>(workspace);
  auto kern = b.row.v == 1   ? norm_bwd_kernel<1, 2>
              : b.row.v == 2 ? norm_bwd_kernel<2, 2>
              : b.row.v == 4 ? norm_bwd_kernel<4, 1>
                             : norm_bwd_kernel<8, 1>;
  const cudaError_t e =
      launch_kernel(kern, dim3(b.grid), dim3(b.row.block), 0, st, nullptr, p, b.row.tpr);
  if (e != cudaSuccess || dgamma == nullptr || b.parts == 1) return e;
  return launch_kernel(norm_dgamma_kernel, dim3(unsigned(a.cols / 16)), dim3(256), 0, st, nullptr,
                       static_cast<const float*>(p.part), b.parts, p.cols, dgamma);
}

}  // namespace fp8lin
