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
// backward pass reads. The column copy is made by the norm's column kernel from h, in L2.
//
// 8192 x 4096 with both MXFP8 copies and both checkpoints has to move 340 MB, 50.0 us at the 6791
// GB/s of a copy; the two kernels take 68.7, the row kernel alone (305 MB, 44.9) 52.5, 0.86 of that
// rate. What bounds it: the row kernel's time does not follow its instructions (28 to 41 an
// element, all within 3 us); half of its stalls are for shuffles and shared memory, its warps (24
// an SM, by registers) go through two sums of a row with a barrier each. The column kernel adds 17
// us, in which the lines that the row kernel left in L2 are written too. The two side by side (on
// two streams, of different tensors) took as long as in turn.
#include <algorithm>
#include <type_traits>

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

// Buffers for rows, of which what has been read of one takes in the row that comes next to it (o's
// half as soon as o is read, the stream's later). With one vector two are faster, 65536 x 256: 39.3
// us instead of 40.2 with four; else one: 8192 x 4096 69.9, two 72.4, two for whole rows 71.3.
template <int V>
__host__ __device__ constexpr int branch_ahead() {
  return V == 1 ? 2 : 1;
}
// Shared memory of a thread, for the rows on their way, and of a lane, for w and gamma of its
// columns. A warp's pieces lie side by side (cp.async of lanes that write 144 bytes apart: 71 us
// instead of 55).
template <int V>
__host__ __device__ constexpr int branch_slot_bytes() {
  return branch_ahead<V>() * 2 * V * 16;
}
__host__ __device__ constexpr int branch_vec_bytes(int v) { return v <= 4 ? v * 64 : 0; }

// The L2 policies as values that may be made again where they are used (no registers kept).
__device__ __forceinline__ uint64_t policy_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_last() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// tpr threads a row (16, or whole warps); a warp's V vectors a lane follow each other, so that what
// distinguishes them is a constant in every address: lane l of warp w has the units 32 (V w + j) +
// l. (Four vectors a thread: 32 instructions an element, 39 with a thread's vectors tpr units
// apart.) A row is a chain of two sums, with a barrier each, and every element is worked on about
// five times, so instructions count as much as bytes: w and gamma lie in shared memory as floats, o,
// h and y follow each other in the same registers, and whole warps run a form of the row's step in
// which nothing is tested.
template <int V, int OUT>
__global__ void __maxnreg__(V <= 4 ? 80 : 128)
    branch_row_kernel(const __grid_constant__ BranchParams b) {
  constexpr bool kSmem = V <= 4;        // eight vectors: gamma and w come from L1 every time
  constexpr int kAhead = branch_ahead<V>();
  const NormParams& p = b.n;
  __shared__ alignas(16) float red[2][16];
  __shared__ uint32_t redm[16];
  extern __shared__ uint4 slots[];                  // each thread's next rows, then w and gamma
  const int tpr = blockDim.x, lane = threadIdx.x, grp = threadIdx.y, rpc = blockDim.y;
  const int nv = p.cols >> 3, nt = tpr * rpc, tid = grp * tpr + lane;
  const int warps = tpr >> 5;                       // warps per row (0: two rows a warp)
  const RowUnits at = {V == 1 ? lane : (lane >> 5) * 32 * V + (lane & 31), 32};
  const bool whole = at.first - (lane & 31) + 32 * V <= nv && warps != 0;   // of the warp
  const bool post = b.gamma_post != nullptr;
  const bool want_y = OUT != N_STATS || p.y != nullptr || p.part != nullptr;
  pdl_wait();
  // As in the norm's row kernel: o, the stream, and the codes go first, h stays until the column
  // kernel has read it.
  const uint64_t first = policy_first();

  uint4* const slot = slots + (tid >> 5) * (32 * kAhead * 2 * V) + (tid & 31);
  // (less than 2^31 rows, and as many threads at most beyond them)
  const uint32_t rows = uint32_t(p.rows), rows_pad = uint32_t(p.rows_pad), cols = p.cols;
  const uint32_t row_step = gridDim.x * rpc, r_first = blockIdx.x * rpc + grp;
  // Each thread copies its own elements of a row, o and res in groups of their own: what it has
  // read of a buffer makes room for the row that comes next to it.
  const auto prefetch = [&](uint32_t r, int buf, auto res_tag) {
    constexpr bool RES = decltype(res_tag)::value;
    uint4* s = slot + buf * (32 * 2 * V) + (RES ? 32 * V : 0);
    const uint16_t* base = RES ? p.res : p.x;
    const uint16_t* next = base + uint64_t(r) * uint32_t(RES ? p.ldr : p.ldx) + 8 * at.first;
    if (whole && r < rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) ptx::cp_async_16_hint(s + 32 * j, next + 8 * j * at.step, first);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {                  // nothing read beyond the tensor: zeros
        const bool in = r < rows && at(j) < nv;
        ptx::cp_async_16_zfill_hint(s + 32 * j, in ? next + 8 * j * at.step : base, in ? 16u : 0u,
                                    first);
      }
    }
    ptx::cp_async_commit();
  };
  constexpr std::false_type kO{};
  constexpr std::true_type kRes{};
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {                 // (beyond rows: zeros)
    prefetch(r_first + k * row_step, k, kO);
    prefetch(r_first + k * row_step, k, kRes);
  }
  // a token's gate: 0 on padding rows
  const auto token = [&](uint32_t r) {
    return r >= rows ? 0.0f : b.token_gate == nullptr ? 1.0f : __ldg(b.token_gate + r);
  };

  // w and gamma of a lane's columns are the same in every row: as floats from shared memory, where
  // there is room
  const auto factor = [&](int j, float2 (&w)[4]) {
    const int c = 8 * at(j);
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
  float4* const vec = reinterpret_cast<float4*>(slots + ((nt + 31) >> 5) * (32 * kAhead * 2 * V)) +
                      (lane >> 5) * (32 * 4 * V) + (lane & 31);
  if (kSmem) {
    if (grp == 0) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float2 w[4];
        factor(j, w);
        vec[32 * 2 * j] = make_float4(w[0].x, w[0].y, w[1].x, w[1].y);
        vec[32 * (2 * j + 1)] = make_float4(w[2].x, w[2].y, w[3].x, w[3].y);
        gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * at(j), w);
        vec[32 * 2 * (V + j)] = make_float4(w[0].x, w[0].y, w[1].x, w[1].y);
        vec[32 * (2 * (V + j) + 1)] = make_float4(w[2].x, w[2].y, w[3].x, w[3].y);
      }
    }
    __syncthreads();
  }
  const auto from_smem = [&](int j, float2 (&w)[4]) {
    const float4 u = vec[32 * 2 * j], v = vec[32 * (2 * j + 1)];
    w[0] = make_float2(u.x, u.y);
    w[1] = make_float2(u.z, u.w);
    w[2] = make_float2(v.x, v.y);
    w[3] = make_float2(v.z, v.w);
  };

  const float tensor_scale = OUT == N_TENSOR ? *p.scale_in : 1.0f;
  uint32_t amax = 0;
  int phase = 0, buf = 0;
  float next_t = token(r_first);
  uint32_t r = r_first;
  // One row. FULL: the row exists and has columns for all vectors of the warp: nothing is tested.
  const auto one_row = [&](auto full_tag) {
    constexpr bool FULL = decltype(full_tag)::value;
    const bool live = FULL || r < rows, stored = FULL || r < rows_pad;
    const uint64_t elem = uint64_t(r) * cols + 8 * at.first;     // the thread's first of the row
    const uint64_t sc = uint64_t(r) * uint32_t(ckpt_pitch(p.cols));
    const float t = next_t;
    next_t = token(r + row_step);
    float2 x[V][4];                                  // o, then h, then y
    ptx::cp_async_wait<2 * kAhead - 1>();
    const uint4* s = slot + buf * (32 * 2 * V);
    float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      widen8(s[32 * j], x[j]);
#pragma unroll
      for (int k = 0; k < 4; ++k) q = __ffma2_rn(x[j][k], x[j][k], q);
    }
    prefetch(r + kAhead * row_step, buf, kO);
    // (the checkpoints before the sums' barriers: 2048 x 16384 73.3 us, behind them 77.1)
    if (b.o_codes != nullptr)
      ckpt_row<V, FULL>(x, b.o_codes + elem, b.o_scale + sc, lane, at, nv, live, first);
    float f = t;
    if (post) {
      const float sum = row_sum(q.x + q.y, red, phase, warps, lane, grp, tpr);
      const float ro = rsqrtf(fmaf(sum, p.inv_cols, b.eps_post));
      if (live && lane == 0 && b.rstd_o != nullptr) b.rstd_o[r] = ro;
      f = ro * t;
    }

    // ---- the stream; a gate of 0 leaves it as it is, whatever o holds
    const float2 f2 = make_float2(f, f);
    q = make_float2(0.0f, 0.0f);
    ptx::cp_async_wait<2 * kAhead - 1>();
#pragma unroll
    for (int j = 0; j < V; ++j) {
      uint4 h = s[32 * (V + j)];
      if (t != 0.0f) {
        float2 w[4], a[4];
        if (kSmem) from_smem(j, w);
        else factor(j, w);
        widen8(h, a);
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = __ffma2_rn(__fmul2_rn(x[j][k], f2), w[k], a[k]);
        h = make_uint4(pack_bf16(a[0].x, a[0].y), pack_bf16(a[1].x, a[1].y),
                       pack_bf16(a[2].x, a[2].y), pack_bf16(a[3].x, a[3].y));
      }
      if (!FULL && at(j) >= nv) h = make_uint4(0, 0, 0, 0);     // (0 inf: no NaN there)
      if (FULL || (live && at(j) < nv))
        stg_v4_policy(p.h + elem + 8 * j * at.step, h, p.keep_h ? policy_last() : first);
      widen8(h, x[j]);
#pragma unroll
      for (int k = 0; k < 4; ++k) q = __ffma2_rn(x[j][k], x[j][k], q);
    }
    prefetch(r + kAhead * row_step, buf, kRes);
    buf = buf + 1 == kAhead ? 0 : buf + 1;

    if (b.h_codes != nullptr)
      ckpt_row<V, FULL>(x, b.h_codes + elem, b.h_scale + sc, lane, at, nv, live, first);
    const float sum = row_sum(q.x + q.y, red, phase, warps, lane, grp, tpr);
    const float rstd = rsqrtf(fmaf(sum, p.inv_cols, p.eps));
    if (live && lane == 0 && p.rstd != nullptr) p.rstd[r] = rstd;
    if (!want_y) return;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float2 g[4];
      if (kSmem) from_smem(V + j, g);
      else gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * at(j), g);
      // padding rows, and lanes without a column (for the amax): (0 0) gamma = 0
      const float rl = FULL || (live && at(j) < nv) ? rstd : 0.0f;
      const float2 r2 = make_float2(rl, rl);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[j][k] = __fmul2_rn(__fmul2_rn(x[j][k], r2), g[k]);
    }
    const auto y_of = [&](int j, bool, float2 (&y)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = x[j][k];
    };
    norm_row_copy<V, OUT, FULL>(p, y_of, r, live, stored, lane, at, tensor_scale, first, amax);
  };
  // (all warps of a group make the same rows, whichever form of the step they run, for they meet at
  // its barriers)
  if (whole) {
    for (; r < rows; r += row_step) one_row(std::true_type{});
  }
  for (; r - grp < rows_pad; r += row_step) one_row(std::false_type{});
  if constexpr (OUT == N_STATS || OUT == N_TENSOR) {
    if (p.part != nullptr) {
      const uint32_t m = cta_max(amax, redm);
      if (threadIdx.x == 0 && threadIdx.y == 0) p.part[blockIdx.x] = m;
    }
  }
  ptx::cp_async_wait<0>();
  pdl_launch_dependents();
}

namespace {

template <int OUT>
cudaError_t launch_branch(const NormParams& n, const BranchParams& more, int* ctas,
                          cudaStream_t st) {
  BranchParams b = more;
  b.n = n;
  // Two vectors a thread up to 4096 columns, four beyond: us with two / four
  //   1 x 4096, row copy                     4.0 /  6.2
  //   8192 x 4096, row copy                 39.8 / 42.1     with checkpoints 52.5 / 54.2
  //   8192 x 4096, both copies              55.3 / 54.6     with checkpoints 69.0 / 66.7
  //   8192 x 2048, both, with checkpoints   36.2 / 38.2
  //   8192 x 4608, both, with checkpoints   90.9 / 91.5
  //   8192 x 5120, both, with checkpoints   95.5 / 84.7
  // (serving and the training step of the examples want the row copy alone).
  // A row's sums, and so its last bits, must not depend on how many rows there are: the rule goes
  // by the columns alone.
  const RowPlan pl = row_plan(n.cols, n.cols <= 4096 ? 2 : 4, n.cols <= 4096 ? 256 : 384);
  const int rpc = pl.block / pl.tpr;
  auto kern = pl.v == 1   ? branch_row_kernel<1, OUT>
              : pl.v == 2 ? branch_row_kernel<2, OUT>
              : pl.v == 4 ? branch_row_kernel<4, OUT>
                          : branch_row_kernel<8, OUT>;
  const int slot = pl.v == 1   ? branch_slot_bytes<1>()
                   : pl.v == 2 ? branch_slot_bytes<2>()
                   : pl.v == 4 ? branch_slot_bytes<4>()
                               : branch_slot_bytes<8>();
  const int smem = std::max(pl.block, 32) * slot +
                   std::max(pl.tpr, 32) * branch_vec_bytes(pl.v);
  // as many CTAs as run at once, by registers (a quarter of an SM has them for six warps at 80 a
  // thread, four at 128) and by shared memory (an SM has 227 KB, a CTA takes 1 KB more than it asks
  // for)
  const int per_sm =
      std::min((pl.v <= 4 ? 768 : 512) / pl.block, 227 * 1024 / (smem + 1280));
  const int64_t grid = std::min<int64_t>((n.rows_pad + rpc - 1) / rpc,
                                         int64_t(num_sms()) * std::max(1, per_sm));
  if (ctas != nullptr) *ctas = int(grid);
  if (smem > 47 * 1024) {                          // 48 KB with the static part
    static ContextOnce attr[4] = {};
    const cudaError_t e =
        once_per_context(attr[pl.v == 1 ? 0 : pl.v == 2 ? 1 : pl.v == 4 ? 2 : 3], [&] {
          return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      220 * 1024);
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
