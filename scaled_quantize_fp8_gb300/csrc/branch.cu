// The end of one block and the start of the next (fp8_branch_rmsnorm_quantize): a block's output o,
// normalised, gated and scaled, joins the residual stream, whose norm is written as the next
// block's FP8 copies.
//
//   xo = o rstd_o,  rstd_o = 1 / sqrt(mean o^2 + eps_o)           (xo = o without a norm after o)
//   h  = bf16(res + (xo t) w),  w = (gamma_o gate) scale            t: the token's gate
//   y  = (h rstd) gamma,  rstd = 1 / sqrt(mean h^2 + eps)
//
// branch_row_kernel holds a row in the registers of a group of threads, as the norm's row kernel
// does, and makes both norms of it, the row copy, and the 8-bit checkpoints of o and h that the
// backward pass reads. The column copy is made by the norm's column kernel from h.
#include <algorithm>

#include "ckpt.cuh"
#include "common.cuh"
#include "internal.cuh"
#include "norm.cuh"
#include "sm100_ptx.cuh"

namespace fp8lin {

struct BranchParams {
  NormParams n;               // x: o, res: the stream
  const void* gamma_post;     // or null: no norm after the block
  const void* gate;           // [cols] or null
  const float* token_gate;    // [rows] or null
  int gamma_post_fp32, gate_fp32;
  float scale, eps_post;
  float* rstd_o;              // [rows] or null
  uint8_t* o_codes;           // checkpoints, or null
  uint8_t* o_scale;
  uint8_t* h_codes;
  uint8_t* h_scale;
};

// Rows on their way: as many as make four vectors a thread, two at least where there is room.
template <int V>
__host__ __device__ constexpr int branch_ahead() {
  return V == 1 ? 4 : V == 8 ? 1 : 2;
}

template <int V, int OUT>
__global__ void __maxnreg__(V <= 2 ? 80 : 128)
    branch_row_kernel(const __grid_constant__ BranchParams b) {
  constexpr bool kRegs = V <= 4;        // eight vectors: gamma and w come from L1 every time
  constexpr int kAhead = branch_ahead<V>();
  const NormParams& p = b.n;
  __shared__ alignas(16) float red[2][16];
  __shared__ uint32_t redm[16];
  extern __shared__ uint4 slots[];                  // each thread's next rows, then w
  const int tpr = blockDim.x, lane = threadIdx.x, grp = threadIdx.y, rpc = blockDim.y;
  const int nv = p.cols >> 3, nt = tpr * rpc, tid = grp * tpr + lane;
  const int warps = tpr >> 5;                       // warps per row (0: two rows a warp)
  const bool post = b.gamma_post != nullptr;
  const bool want_y = OUT != N_STATS || p.y != nullptr || p.part != nullptr;
  pdl_wait();
  // As in the norm's row kernel: o, the stream, and the codes go first, h stays until the column
  // kernel has read it.
  const uint64_t first = ptx::l2_evict_first_policy();
  const uint64_t hpol = p.keep_h ? ptx::l2_evict_last_policy() : first;

  const auto prefetch = [&](int64_t r, int buf) {
    uint4* s = slots + buf * 2 * V * nt + tid;
    const uint16_t* x = p.x + r * p.ldx + 8 * lane;
    const uint16_t* res = p.res + r * p.ldr + 8 * lane;
    if (V * tpr == nv && r < p.rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ptx::cp_async_16_hint(s + j * nt, x + 8 * j * tpr, first);
        ptx::cp_async_16_hint(s + (V + j) * nt, res + 8 * j * tpr, first);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {                  // nothing read beyond the tensor: zeros
        const bool in = r < p.rows && j * tpr + lane < nv;
        const uint32_t n = in ? 16u : 0u;
        ptx::cp_async_16_zfill_hint(s + j * nt, in ? x + 8 * j * tpr : p.x, n, first);
        ptx::cp_async_16_zfill_hint(s + (V + j) * nt, in ? res + 8 * j * tpr : p.res, n, first);
      }
    }
    ptx::cp_async_commit();
  };
  const int64_t row_step = int64_t(gridDim.x) * rpc;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int64_t r0 = int64_t(blockIdx.x) * rpc + k * row_step;
    if (r0 < p.rows_pad) prefetch(r0 + grp, k);
    else ptx::cp_async_commit();                    // groups are counted: an empty one
  }
  // a token's gate: 0 on padding rows
  const auto token = [&](int64_t r) {
    return r >= p.rows ? 0.0f : b.token_gate == nullptr ? 1.0f : __ldg(b.token_gate + r);
  };

  // w of a lane's columns is the same in every row: from shared memory, where there is room, so
  // that gamma may stay in registers
  const auto factor = [&](int j, float2 (&w)[4]) {
    const int c = 8 * (j * tpr + lane);
    float2 g[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = make_float2(1.0f, 1.0f);
    if (post) gamma_pairs(b.gamma_post, b.gamma_post_fp32, p.cols, c, w);
    if (b.gate != nullptr) {
      gamma_pairs(b.gate, b.gate_fp32, p.cols, c, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = __fmul2_rn(w[k], g[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __fmul2_rn(w[k], make_float2(b.scale, b.scale));
  };
  float4* ws = reinterpret_cast<float4*>(slots + kAhead * 2 * V * nt) + lane;
  float2 g[kRegs ? V : 1][4];
  if (kRegs) {
    if (grp == 0) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float2 w[4];
        factor(j, w);
        ws[2 * j * tpr] = make_float4(w[0].x, w[0].y, w[1].x, w[1].y);
        ws[(2 * j + 1) * tpr] = make_float4(w[2].x, w[2].y, w[3].x, w[3].y);
      }
    }
    if (want_y) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * (j * tpr + lane), g[kRegs ? j : 0]);
    }
    __syncthreads();
  }
  const auto gamma_of = [&](int j) -> float2(&)[4] {
    if constexpr (!kRegs)
      gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * (j * tpr + lane), g[0]);
    return g[kRegs ? j : 0];
  };

  const float tensor_scale = OUT == N_TENSOR ? *p.scale_in : 1.0f;
  uint32_t amax = 0;
  int phase = 0, buf = 0;
  float next_t = token(int64_t(blockIdx.x) * rpc + grp);
  for (int64_t r0 = int64_t(blockIdx.x) * rpc; r0 < p.rows_pad; r0 += row_step) {
    const int64_t r = r0 + grp;
    const bool live = r < p.rows, stored = r < p.rows_pad;
    const float t = next_t;
    next_t = token(r + row_step);
    uint4 o[V], h[V];
    ptx::cp_async_wait<kAhead - 1>();
    const uint4* s = slots + buf * 2 * V * nt + tid;
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = s[j * nt];
    float f = t;
    if (post) {
      float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < V; ++j) add_squares8(o[j], q);
      const float sum = row_sum(q.x + q.y, red, phase, warps, lane, grp, tpr);
      const float ro = rsqrtf(fmaf(sum, p.inv_cols, b.eps_post));
      if (live && lane == 0 && b.rstd_o != nullptr) b.rstd_o[r] = ro;
      f = ro * t;
    }
    if (b.o_codes != nullptr)
      ckpt_row<V>(o, b.o_codes + r * p.cols, b.o_scale + r * ckpt_pitch(p.cols), lane, nv, live,
                  first);

    // ---- the stream; a gate of 0 leaves it as it is, whatever o holds
    const float2 f2 = make_float2(f, f);
    uint16_t* ho = p.h + r * p.cols + 8 * lane;
    const bool all = V * tpr == nv && live;                      // nothing to test per vector
    float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      h[j] = s[(V + j) * nt];
      if (t != 0.0f) {
        float2 w[4], x[4], a[4];
        if (kRegs) {
          const float4 u = ws[2 * j * tpr], v = ws[(2 * j + 1) * tpr];
          w[0] = make_float2(u.x, u.y);
          w[1] = make_float2(u.z, u.w);
          w[2] = make_float2(v.x, v.y);
          w[3] = make_float2(v.z, v.w);
        } else {
          factor(j, w);
        }
        widen8(o[j], x);
        widen8(h[j], a);
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = __ffma2_rn(__fmul2_rn(x[k], f2), w[k], a[k]);
        h[j] = make_uint4(pack_bf16(a[0].x, a[0].y), pack_bf16(a[1].x, a[1].y),
                          pack_bf16(a[2].x, a[2].y), pack_bf16(a[3].x, a[3].y));
      }
      if (!all && j * tpr + lane >= nv) h[j] = make_uint4(0, 0, 0, 0);   // (0 inf: no NaN there)
      if (all || (live && j * tpr + lane < nv)) stg_v4_policy(ho + 8 * j * tpr, h[j], hpol);
      add_squares8(h[j], q);
    }
    const int64_t next = r0 + kAhead * row_step;
    if (next < p.rows_pad) prefetch(next + grp, buf);
    else ptx::cp_async_commit();
    buf = buf + 1 == kAhead ? 0 : buf + 1;

    const float sum = row_sum(q.x + q.y, red, phase, warps, lane, grp, tpr);
    const float rstd = rsqrtf(fmaf(sum, p.inv_cols, p.eps));
    if (live && lane == 0 && p.rstd != nullptr) p.rstd[r] = rstd;
    if (b.h_codes != nullptr)
      ckpt_row<V>(h, b.h_codes + r * p.cols, b.h_scale + r * ckpt_pitch(p.cols), lane, nv, live,
                  first);
    if (!want_y) continue;
    const float rl = live ? rstd : 0.0f;                         // padding rows: (0 0) gamma = 0
    norm_row_copy<V, OUT>(p, h, rl, gamma_of, r, live, stored, lane, tensor_scale, first, amax);
  }
  if constexpr (OUT == N_STATS || OUT == N_TENSOR) {
    if (p.part != nullptr) {
      const uint32_t m = cta_max(amax, redm);
      if (threadIdx.x == 0 && threadIdx.y == 0) p.part[blockIdx.x] = m;
    }
  }
  pdl_launch_dependents();
}

namespace {

template <int OUT>
cudaError_t launch_branch(const NormParams& n, const BranchParams& more, int* ctas,
                          cudaStream_t st) {
  BranchParams b = more;
  b.n = n;
  const RowPlan pl = row_plan(n.cols, 2, 256);
  const int rpc = pl.block / pl.tpr;
  const int per_sm = (pl.v <= 2 ? 768 : 512) / pl.block;
  const int64_t grid = std::min<int64_t>((n.rows_pad + rpc - 1) / rpc,
                                         int64_t(num_sms()) * std::max(1, per_sm));
  if (ctas != nullptr) *ctas = int(grid);
  auto kern = pl.v == 1   ? branch_row_kernel<1, OUT>
              : pl.v == 2 ? branch_row_kernel<2, OUT>
              : pl.v == 4 ? branch_row_kernel<4, OUT>
                          : branch_row_kernel<8, OUT>;
  const int ahead = pl.v == 1   ? branch_ahead<1>()
                    : pl.v == 2 ? branch_ahead<2>()
                    : pl.v == 4 ? branch_ahead<4>()
                                : branch_ahead<8>();
  const size_t smem = size_t(pl.v) * 32 * (size_t(ahead) * pl.block + (pl.v <= 4 ? pl.tpr : 0));
  if (smem > 47 * 1024) {                          // 48 KB with the static part
    static ContextOnce attr[4] = {};
    const cudaError_t e =
        once_per_context(attr[pl.v == 1 ? 0 : pl.v == 2 ? 1 : pl.v == 4 ? 2 : 3], [&] {
          return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      200 * 1024);
        });
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kern, dim3(unsigned(grid)), dim3(unsigned(pl.tpr), unsigned(rpc)), smem, st,
                       nullptr, b);
}

cudaError_t branch_rows(int out_kind, const NormParams& p, const void* more, int* ctas,
                        cudaStream_t st) {
  const BranchParams& b = *reinterpret_cast<const BranchParams*>(more);
  return out_kind == N_MX       ? launch_branch<N_MX>(p, b, ctas, st)
         : out_kind == N_BW     ? launch_branch<N_BW>(p, b, ctas, st)
         : out_kind == N_TENSOR ? launch_branch<N_TENSOR>(p, b, ctas, st)
                                : launch_branch<N_STATS>(p, b, ctas, st);
}

}  // namespace

cudaError_t branch_quantize_launch(const NormArgs& a, const fp8_branch_input& in, float* rstd_o,
                                   const fp8_checkpoint* o_ckpt, const fp8_checkpoint* h_ckpt,
                                   fp8_tensor* out, void* workspace, cudaStream_t st) {
  BranchParams b{};
  b.gamma_post = in.gamma_post;
  b.gate = in.gate;
  b.token_gate = in.token_gate;
  b.gamma_post_fp32 = in.gamma_post_fp32;
  b.gate_fp32 = in.gate_fp32;
  b.scale = in.scale;
  b.eps_post = in.eps_post;
  b.rstd_o = rstd_o;
  if (o_ckpt != nullptr) {
    b.o_codes = o_ckpt->codes;
    b.o_scale = o_ckpt->scale;
  }
  if (h_ckpt != nullptr) {
    b.h_codes = h_ckpt->codes;
    b.h_scale = h_ckpt->scale;
  }
  return norm_copies_launch(a, norm_params(a), out, workspace, st, branch_rows, &b);
}

}  // namespace fp8lin
