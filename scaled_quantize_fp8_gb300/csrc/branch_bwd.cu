// Backward of the branch that joins the stream and of the norm in front of the next block
// (fp8_branch_rmsnorm_bwd). Stream h and branch o each come as bf16 or as an 8-bit checkpoint.
//
//   xh = h rstd,  a = dy gamma,  dh = dres + rstd (a - xh mean(a xh)),  dgamma = sum_r dy xh
//   xo = o rstd_o,  w = (gamma_o gate) scale,  u = dh w,  s[r] = sum_c u xo
//   do = rstd_o t (u - xo s / cols)      without a norm after the block: xo = o, do = t u
//   S[c] = sum_r (t dh) xo:  dgamma_o = scale gate S,  dgate = scale gamma_o S,  dt[r] = s[r]
//
// branch_bwd_kernel: a group of threads holds a row, so every input is read once; each thread owns
// the same columns in all of its rows and adds dgamma and S for them in registers. The CTAs' sums
// go to the workspace and branch_sums_kernel adds them in a fixed order. dh goes on in fp32: its
// rounding to bf16 is the output's alone.
#include <algorithm>

#include "ckpt.cuh"
#include "common.cuh"
#include "internal.cuh"
#include "norm.cuh"
#include "sm100_ptx.cuh"

namespace fp8lin {

struct BranchBwdParams {
  const uint16_t* dy;
  const uint16_t* dres;       // or null
  const uint16_t* h;          // or null: h_codes
  const uint16_t* o;          // or null: o_codes
  const uint8_t* h_codes;
  const uint8_t* h_scale;
  const uint8_t* o_codes;
  const uint8_t* o_scale;
  const void* gamma_post;     // or null
  const void* gate;           // or null
  const float* token_gate;    // or null
  const void* gamma;
  const float* rstd_o;        // with gamma_post
  const float* rstd;
  int64_t ld_dy, ld_dres, ld_h, ld_o;
  int64_t rows;
  int cols;
  int gamma_post_fp32, gate_fp32, gamma_fp32;
  float scale, inv_cols;
  uint16_t* dh;
  uint16_t* d_o;
  float* dtoken;              // or null
  float* part;                // [2][parts][cols]: sums for dgamma, then S; or null
  int parts;
};

// Buffers for a row: one that is worked on, the others on their way.
template <int V, bool HCK, bool OCK>
__host__ __device__ constexpr int bwd_bufs() {
  return V <= 2 ? 2 : HCK && OCK ? 2 : 1;
}
template <int V, bool HCK, bool OCK>
__host__ __device__ constexpr int bwd_row_bytes() {      // of a thread
  return V * (32 + (HCK ? 8 : 16) + (OCK ? 8 : 16));
}

// tpr threads per row, V vectors of eight columns a thread (vector j of lane l: columns 8 (j tpr + l)
// .., in the second CTA of a pair behind those of the first). Every thread copies its own elements
// of the next row to its own slots of shared memory while it works on the present one, and reads
// them once for each of the row's three steps: mean(a xh); dh and s; do. Only dh stays in
// registers in between.
// PAIR: a row of more than 16384 columns, whose two column sums a thread no longer fit in the
// registers of one CTA, lies in two CTAs of a cluster; each adds the other's part of the row's
// sums, which arrive in shared memory.
template <int V, bool HCK, bool OCK, bool PAIR>
__global__ void __maxnreg__(128) branch_bwd_kernel(const __grid_constant__ BranchBwdParams p) {
  constexpr bool kVec = V <= 2;                     // gamma and w kept, else from L1 each time
  constexpr int kBufs = bwd_bufs<V, HCK, OCK>();
  __shared__ alignas(16) float red[2][16];
  __shared__ float other[2];
  extern __shared__ uint4 slots[];
  const int tpr = blockDim.x, lane = threadIdx.x, grp = threadIdx.y, rpc = blockDim.y;
  const int nt = tpr * rpc, tid = grp * tpr + lane;
  const int warps = tpr >> 5;                       // warps per row (0: two rows a warp)
  const uint32_t rank = PAIR ? ptx::cluster_rank() : 0;
  const int all_nv = p.cols >> 3, nv0 = PAIR ? (all_nv + 1) >> 1 : all_nv;
  const int v0 = rank ? nv0 : 0, nv = rank ? all_nv - nv0 : nv0;     // this CTA's vectors
  const bool post = p.gamma_post != nullptr;
  const bool want_s = post || p.dtoken != nullptr;
  uint4* const vec = slots;                                          // [kBufs][dy, dres, (h, o)][V]
  constexpr int kVecs = V * (2 + !HCK + !OCK), kHalves = V * (HCK + OCK);
  uint2* const half = reinterpret_cast<uint2*>(vec + kBufs * kVecs * nt);   // [kBufs][(h, o)][V]
  pdl_wait();

  float next_rstd = 0.0f, next_ro = 0.0f, next_t = 0.0f;
  uint32_t next_he[V], next_oe[V];
  const auto prefetch = [&](int64_t r, int buf) {
    uint4* s = vec + buf * kVecs * nt + tid;
    uint2* q = half + buf * kHalves * nt + tid;
    const bool live = r < p.rows;
#pragma unroll
    for (int j = 0; j < V; ++j) {                    // nothing read beyond the tensor: zeros
      const bool in = live && j * tpr + lane < nv;
      const int c = 8 * (v0 + j * tpr + lane);
      const uint32_t n = in ? 16u : 0u, m = in ? 8u : 0u;
      ptx::cp_async_16_zfill(s + j * nt, in ? p.dy + r * p.ld_dy + c : p.dy, n);
      if (p.dres != nullptr)
        ptx::cp_async_16_zfill(s + (V + j) * nt, in ? p.dres + r * p.ld_dres + c : p.dres, n);
      if (HCK)
        ptx::cp_async_8_zfill(q + j * nt, in ? p.h_codes + r * p.cols + c : p.h_codes, m);
      else
        ptx::cp_async_16_zfill(s + (2 * V + j) * nt, in ? p.h + r * p.ld_h + c : p.h, n);
      if (OCK)
        ptx::cp_async_8_zfill(q + ((HCK ? V : 0) + j) * nt,
                              in ? p.o_codes + r * p.cols + c : p.o_codes, m);
      else
        ptx::cp_async_16_zfill(s + ((HCK ? 2 : 3) * V + j) * nt,
                               in ? p.o + r * p.ld_o + c : p.o, n);
    }
    ptx::cp_async_commit();
  };
  // the row's own numbers, read a row ahead
  const auto scalars = [&](int64_t r) {
    const bool live = r < p.rows;
    next_rstd = live ? p.rstd[r] : 0.0f;
    next_ro = !live ? 0.0f : post ? p.rstd_o[r] : 1.0f;
    next_t = !live ? 0.0f : p.token_gate != nullptr ? p.token_gate[r] : 1.0f;
    const int64_t at = r * ckpt_pitch(p.cols);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool in = live && j * tpr + lane < nv;
      const int b = (v0 + j * tpr + lane) >> 2;
      if (HCK) next_he[j] = in ? __ldg(p.h_scale + at + b) : 0u;
      if (OCK) next_oe[j] = in ? __ldg(p.o_scale + at + b) : 0u;
    }
  };
  const int64_t step = int64_t(PAIR ? gridDim.x >> 1 : gridDim.x) * rpc;
  int64_t r = int64_t(PAIR ? blockIdx.x >> 1 : blockIdx.x) * rpc + grp;
#pragma unroll
  for (int k = 0; k < (kBufs > 1 ? kBufs - 1 : 1); ++k) {
    if (r - grp + k * step < p.rows) prefetch(r + k * step, k);
    else ptx::cp_async_commit();                    // groups are counted: an empty one
  }
  scalars(r);

  const auto factor = [&](int j, float2 (&w)[4]) {
    const int c = 8 * (v0 + j * tpr + lane);
    float2 g[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = make_float2(1.0f, 1.0f);
    if (post) gamma_pairs(p.gamma_post, p.gamma_post_fp32, p.cols, c, w);
    if (p.gate != nullptr) {
      gamma_pairs(p.gate, p.gate_fp32, p.cols, c, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = __fmul2_rn(w[k], g[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __fmul2_rn(w[k], make_float2(p.scale, p.scale));
  };
  float4* ws = reinterpret_cast<float4*>(half + kBufs * kHalves * nt) + lane;
  float2 g[kVec ? V : 1][4], acc_g[V][4], acc_s[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (kVec) {
      gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * (v0 + j * tpr + lane), g[kVec ? j : 0]);
      if (grp == 0) {
        float2 w[4];
        factor(j, w);
        ws[2 * j * tpr] = make_float4(w[0].x, w[0].y, w[1].x, w[1].y);
        ws[(2 * j + 1) * tpr] = make_float4(w[2].x, w[2].y, w[3].x, w[3].y);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) acc_g[j][k] = acc_s[j][k] = make_float2(0.0f, 0.0f);
  }
  __syncthreads();
  if (PAIR) ptx::cluster_sync();                    // the other CTA runs: its memory may be written
  const auto gamma_of = [&](int j) -> float2(&)[4] {
    if constexpr (!kVec)
      gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * (v0 + j * tpr + lane), g[0]);
    return g[kVec ? j : 0];
  };
  const auto w_of = [&](int j, float2 (&w)[4]) {
    if (kVec) {
      const float4 a = ws[2 * j * tpr], b = ws[(2 * j + 1) * tpr];
      w[0] = make_float2(a.x, a.y);
      w[1] = make_float2(a.z, a.w);
      w[2] = make_float2(b.x, b.y);
      w[3] = make_float2(b.z, b.w);
    } else {
      factor(j, w);
    }
  };
  int phase = 0;
  // (row_sum's phase goes by turns; a pair's second number is read before the next barrier of the
  // cluster but one, so two places suffice)
  int turn = 0;
  const auto sum_of = [&](float v) {
    v = row_sum(v, red, phase, warps, lane, grp, tpr);
    if constexpr (PAIR) {
      if (lane == 0) ptx::st_cluster_f32(ptx::map_to_rank(&other[turn], rank ^ 1), v);
      __syncwarp();
      ptx::cluster_sync();
      const float w = other[turn];
      v = rank ? w + v : v + w;                     // the same order in both
      turn ^= 1;
    }
    return v;
  };

  int buf = 0;
  for (; r - grp < p.rows; r += step) {
    const uint4* s = vec + buf * kVecs * nt + tid;
    const uint2* q = half + buf * kHalves * nt + tid;
    const float rs = next_rstd, ro = next_ro, t = next_t;
    float hf[HCK ? V : 1], of[OCK ? V : 1];         // what a code of the row counts in xh and xo
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (HCK) hf[HCK ? j : 0] = ckpt_factor(next_he[j]) * rs;
      if (OCK) of[OCK ? j : 0] = ckpt_factor(next_oe[j]) * ro;
    }
    if (!HCK) hf[0] = rs;
    if (!OCK) of[0] = ro;
    const auto xh_of = [&](int j, float2 (&x)[4]) {
      if constexpr (HCK) ckpt_widen8(q[j * nt], x);
      else widen8(s[(2 * V + j) * nt], x);
      const float2 f = make_float2(hf[HCK ? j : 0], hf[HCK ? j : 0]);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = __fmul2_rn(x[k], f);
    };
    const auto xo_of = [&](int j, float2 (&x)[4]) {
      if constexpr (OCK) ckpt_widen8(q[((HCK ? V : 0) + j) * nt], x);
      else widen8(s[((HCK ? 2 : 3) * V + j) * nt], x);
      const float2 f = make_float2(of[OCK ? j : 0], of[OCK ? j : 0]);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = __fmul2_rn(x[k], f);
    };
    if (kBufs > 1) {
      ptx::cp_async_wait<kBufs - 2>();
      const int64_t ahead = r + (kBufs - 1) * step;
      if (ahead - grp < p.rows) prefetch(ahead, buf + kBufs - 1 >= kBufs ? buf - 1 : buf + kBufs - 1);
      else ptx::cp_async_commit();
    } else {
      ptx::cp_async_wait<0>();
    }
    scalars(r + step);

    // ---- mean(a xh), dgamma
    float2 c2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float2 d[4], x[4], (&gj)[4] = gamma_of(j);
      widen8(s[j * nt], d);
      xh_of(j, x);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = __fmul2_rn(d[k], x[k]);
        acc_g[j][k] = __fadd2_rn(acc_g[j][k], v);
        c2 = __ffma2_rn(v, gj[k], c2);
      }
    }
    const float c = -p.inv_cols * sum_of(c2.x + c2.y);

    // ---- dh, s, S
    const float2 cc = make_float2(c, c), r2 = make_float2(rs, rs), t2 = make_float2(t, t);
    float2 dh[V][4], s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float2 d[4], x[4], w[4], (&gj)[4] = gamma_of(j);
      widen8(s[j * nt], d);
      xh_of(j, x);
      if (p.dres != nullptr) {
        widen8(s[(V + j) * nt], dh[j]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) dh[j][k] = make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        dh[j][k] = __ffma2_rn(r2, __ffma2_rn(x[k], cc, __fmul2_rn(d[k], gj[k])), dh[j][k]);
      if (r < p.rows && j * tpr + lane < nv)
        *reinterpret_cast<uint4*>(p.dh + r * p.cols + 8 * (v0 + j * tpr + lane)) = make_uint4(
            pack_bf16(dh[j][0].x, dh[j][0].y), pack_bf16(dh[j][1].x, dh[j][1].y),
            pack_bf16(dh[j][2].x, dh[j][2].y), pack_bf16(dh[j][3].x, dh[j][3].y));
      xo_of(j, x);
      w_of(j, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = __fmul2_rn(dh[j][k], x[k]);
        // a gate of 0: whatever o holds, nothing of it reaches the sums
        if (t != 0.0f) acc_s[j][k] = __ffma2_rn(t2, v, acc_s[j][k]);
        s2 = __ffma2_rn(v, w[k], s2);
        dh[j][k] = __fmul2_rn(dh[j][k], w[k]);      // u from here on
      }
    }
    float sum = 0.0f;
    if (want_s) {
      sum = sum_of(s2.x + s2.y);
      if (p.dtoken != nullptr && lane == 0 && r < p.rows && rank == 0) p.dtoken[r] = sum;
    }

    // ---- do
    const float rt = ro * t, m = post ? -p.inv_cols * rt * sum : 0.0f;
    const float2 rt2 = make_float2(rt, rt), m2 = make_float2(m, m);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (t == 0.0f) {
#pragma unroll
        for (int k = 0; k < 4; ++k) dh[j][k] = make_float2(0.0f, 0.0f);
      } else if (post) {
        float2 x[4];
        xo_of(j, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) dh[j][k] = __ffma2_rn(x[k], m2, __fmul2_rn(dh[j][k], rt2));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) dh[j][k] = __fmul2_rn(dh[j][k], rt2);
      }
      if (r < p.rows && j * tpr + lane < nv)
        *reinterpret_cast<uint4*>(p.d_o + r * p.cols + 8 * (v0 + j * tpr + lane)) = make_uint4(
            pack_bf16(dh[j][0].x, dh[j][0].y), pack_bf16(dh[j][1].x, dh[j][1].y),
            pack_bf16(dh[j][2].x, dh[j][2].y), pack_bf16(dh[j][3].x, dh[j][3].y));
    }
    if (kBufs == 1) {
      if (r + step - grp < p.rows) prefetch(r + step, 0);
    } else {
      buf = buf + 1 == kBufs ? 0 : buf + 1;
    }
  }

  if (p.part != nullptr) {
    // the groups' sums, added by the first group in order, by way of the slots (96 V nt bytes or
    // more where there are several groups, of which 64 V nt are used)
    float4* sums = reinterpret_cast<float4*>(slots);
    const int n = 2 * V * nt;
    if (rpc > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sums[(2 * j + i) * nt + tid] = make_float4(acc_g[j][2 * i].x, acc_g[j][2 * i].y,
                                                     acc_g[j][2 * i + 1].x, acc_g[j][2 * i + 1].y);
          sums[n + (2 * j + i) * nt + tid] =
              make_float4(acc_s[j][2 * i].x, acc_s[j][2 * i].y, acc_s[j][2 * i + 1].x,
                          acc_s[j][2 * i + 1].y);
        }
      }
      __syncthreads();
    }
    if (grp == 0) {
      for (int i = 1; i < rpc; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float4 a = sums[(2 * j + k) * nt + i * tpr + lane];
            const float4 b = sums[n + (2 * j + k) * nt + i * tpr + lane];
            acc_g[j][2 * k] = __fadd2_rn(acc_g[j][2 * k], make_float2(a.x, a.y));
            acc_g[j][2 * k + 1] = __fadd2_rn(acc_g[j][2 * k + 1], make_float2(a.z, a.w));
            acc_s[j][2 * k] = __fadd2_rn(acc_s[j][2 * k], make_float2(b.x, b.y));
            acc_s[j][2 * k + 1] = __fadd2_rn(acc_s[j][2 * k + 1], make_float2(b.z, b.w));
          }
        }
      }
      const int64_t at = int64_t(PAIR ? blockIdx.x >> 1 : blockIdx.x) * p.cols;
      float* dst = p.part + at + 8 * (v0 + lane);
      const int64_t to_s = int64_t(p.parts) * p.cols;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j * tpr + lane < nv) {
          float4* q = reinterpret_cast<float4*>(dst + 8 * j * tpr);
          q[0] = make_float4(acc_g[j][0].x, acc_g[j][0].y, acc_g[j][1].x, acc_g[j][1].y);
          q[1] = make_float4(acc_g[j][2].x, acc_g[j][2].y, acc_g[j][3].x, acc_g[j][3].y);
          q = reinterpret_cast<float4*>(dst + to_s + 8 * j * tpr);
          q[0] = make_float4(acc_s[j][0].x, acc_s[j][0].y, acc_s[j][1].x, acc_s[j][1].y);
          q[1] = make_float4(acc_s[j][2].x, acc_s[j][2].y, acc_s[j][3].x, acc_s[j][3].y);
        }
      }
    }
  }
  pdl_launch_dependents();
}

struct BranchSumsParams {
  const float* part;          // [2][n][cols]
  int n, cols;
  const void* gamma_post;
  const void* gate;
  int gamma_post_fp32, gate_fp32;
  float scale;
  float* dgamma;              // each may be null
  float* dgamma_post;
  float* dgate;
};

__device__ __forceinline__ float column_of(const void* v, int fp32, int c) {
  return v == nullptr ? 1.0f
         : fp32       ? reinterpret_cast<const float*>(v)[c]
                      : __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(v)[c]) << 16);
}

// The partial sums of 16 columns (blockIdx.x) for dgamma (blockIdx.y 0) or S (1): 64 slices of the
// partials a CTA, a slice's loads four at a time, added in a fixed order.
__global__ void __launch_bounds__(256)
    branch_sums_kernel(const __grid_constant__ BranchSumsParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float4 red[64][5];          // rows of 80 bytes: the lanes below read other banks
  const bool of_s = blockIdx.y != 0;
  if (of_s ? p.dgamma_post == nullptr && p.dgate == nullptr : p.dgamma == nullptr) return;
  const int q = threadIdx.x & 3, s = threadIdx.x >> 2;
  const float* at = p.part + (of_s ? int64_t(p.n) * p.cols : 0) + blockIdx.x * 16 + 4 * q;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = s; i < p.n; i += 256) {
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = i + 64 * k < p.n ? *reinterpret_cast<const float4*>(at + int64_t(i + 64 * k) * p.cols)
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
  if (l != 0) return;
  const int col = blockIdx.x * 16 + c;
  if (!of_s) {
    p.dgamma[col] = t;
    return;
  }
  t *= p.scale;
  if (p.dgamma_post != nullptr) p.dgamma_post[col] = t * column_of(p.gate, p.gate_fp32, col);
  if (p.dgate != nullptr) p.dgate[col] = t * column_of(p.gamma_post, p.gamma_post_fp32, col);
}

namespace {

struct BranchBwdPlan {
  RowPlan row;
  bool pair;
  int parts;                  // CTAs, or pairs of them
};
// One CTA of up to 512 threads per SM, as in the norm's backward pass: its row groups' column sums
// meet in shared memory, so there are at most as many partials as SMs. Few rows: one vector a
// thread, and fewer rows a CTA while there are SMs without any.
BranchBwdPlan branch_bwd_plan(int64_t rows, int64_t cols) {
  BranchBwdPlan b;
  const int sms = num_sms();
  b.pair = cols > 16384;
  const int mine = b.pair ? int(cols / 8 + 1) / 2 * 8 : int(cols);
  b.row = row_plan(mine, rows <= 4 * sms ? 1 : 2, 512);
  int rpc = b.row.block / b.row.tpr;
  while (rpc > 1 && (rpc / 2) * b.row.tpr >= 128 && rows <= int64_t(rpc / 2) * sms) rpc /= 2;
  b.row.block = rpc * b.row.tpr;
  b.parts = int(std::min<int64_t>((rows + rpc - 1) / rpc, b.pair ? sms / 2 : sms));
  return b;
}

template <int V, bool HCK, bool OCK, bool PAIR>
cudaError_t launch_bwd(const BranchBwdParams& p, const BranchBwdPlan& b, cudaStream_t st) {
  auto kern = branch_bwd_kernel<V, HCK, OCK, PAIR>;
  const size_t smem = size_t(bwd_bufs<V, HCK, OCK>()) * bwd_row_bytes<V, HCK, OCK>() * b.row.block +
                      (V <= 2 ? size_t(V) * 32 * b.row.tpr : 0);
  if (smem > 47 * 1024) {                                  // 48 KB with the static part
    static ContextOnce attr = {};
    const cudaError_t e = once_per_context(attr, [&] {
      return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    });
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute cluster = {};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = 2;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  const int rpc = b.row.block / b.row.tpr;
  return launch_kernel(kern, dim3(unsigned(PAIR ? 2 * b.parts : b.parts)),
                       dim3(unsigned(b.row.tpr), unsigned(rpc)), smem, st,
                       PAIR ? &cluster : nullptr, p);
}
template <bool HCK, bool OCK>
cudaError_t launch_bwd(const BranchBwdParams& p, const BranchBwdPlan& b, cudaStream_t st) {
  if (b.pair) return launch_bwd<4, HCK, OCK, true>(p, b, st);
  return b.row.v == 1   ? launch_bwd<1, HCK, OCK, false>(p, b, st)
         : b.row.v == 2 ? launch_bwd<2, HCK, OCK, false>(p, b, st)
                        : launch_bwd<4, HCK, OCK, false>(p, b, st);
}

}  // namespace

size_t branch_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return size_t(branch_bwd_plan(rows, cols).parts) * size_t(cols) * 8;
}

cudaError_t branch_bwd_launch(const fp8_branch_grad& a, const fp8_branch_grad_out& out,
                              void* workspace, cudaStream_t st) {
  const BranchBwdPlan b = branch_bwd_plan(a.rows, a.cols);
  const bool hck = a.h_ckpt.codes != nullptr, ock = a.branch_ckpt.codes != nullptr;
  BranchBwdParams p{};
  p.dy = reinterpret_cast<const uint16_t*>(a.dy);
  p.dres = reinterpret_cast<const uint16_t*>(a.dres);
  p.h = reinterpret_cast<const uint16_t*>(a.h);
  p.o = reinterpret_cast<const uint16_t*>(a.branch);
  p.h_codes = a.h_ckpt.codes;
  p.h_scale = a.h_ckpt.scale;
  p.o_codes = a.branch_ckpt.codes;
  p.o_scale = a.branch_ckpt.scale;
  p.gamma_post = a.gamma_post;
  p.gate = a.gate;
  p.token_gate = a.token_gate;
  p.gamma = a.gamma;
  p.rstd_o = a.rstd_branch;
  p.rstd = a.rstd;
  p.ld_dy = a.ld_dy;
  p.ld_dres = a.ld_dres;
  p.ld_h = a.ld_h;
  p.ld_o = a.ld_branch;
  p.rows = a.rows;
  p.cols = int(a.cols);
  p.gamma_post_fp32 = a.gamma_post_fp32;
  p.gate_fp32 = a.gate_fp32;
  p.gamma_fp32 = a.gamma_fp32;
  p.scale = a.scale;
  p.inv_cols = 1.0f / float(a.cols);
  p.dh = reinterpret_cast<uint16_t*>(out.dh);
  p.d_o = reinterpret_cast<uint16_t*>(out.dbranch);
  p.dtoken = out.dtoken_gate;
  const bool sums = out.dgamma != nullptr || out.dgamma_post != nullptr || out.dgate != nullptr;
  p.part = sums ? reinterpret_cast<float*>(workspace) : nullptr;
  p.parts = b.parts;
  const cudaError_t e = hck ? (ock ? launch_bwd<true, true>(p, b, st)
                                   : launch_bwd<true, false>(p, b, st))
                            : (ock ? launch_bwd<false, true>(p, b, st)
                                   : launch_bwd<false, false>(p, b, st));
  if (e != cudaSuccess || !sums) return e;
  BranchSumsParams s{};
  s.part = p.part;
  s.n = b.parts;
  s.cols = p.cols;
  s.gamma_post = p.gamma_post;
  s.gate = p.gate;
  s.gamma_post_fp32 = p.gamma_post_fp32;
  s.gate_fp32 = p.gate_fp32;
  s.scale = p.scale;
  s.dgamma = out.dgamma;
  s.dgamma_post = out.dgamma_post;
  s.dgate = out.dgate;
  return launch_kernel(branch_sums_kernel, dim3(unsigned(p.cols / 16), 2), dim3(256), 0, st,
                       nullptr, s);
}

}  // namespace fp8lin
