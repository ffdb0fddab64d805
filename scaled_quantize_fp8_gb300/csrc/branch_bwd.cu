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
//
// 8192 x 4096 from both checkpoints, with dres, moves 338 MB: 60.8 us (49.8 at a copy's rate), of
// which branch_sums_kernel about 3; from bf16 403 MB in 66.6 (59.4). What bounds it: 16 warps an
// SM, by registers, for rows that are chains of two sums; 36 instructions an element from
// checkpoints (29.5 from bf16). A CTA of three groups with four vectors and 168 registers a thread
// took 121; dy and h copied apart from dres and o, each refilled as soon as read, 67; gamma in shared
// memory 61.7; one exchange a row, of its second sum and the next row's first, for which dy and h
// are widened twice and three rows lie in shared memory, 66.0. Wide rows have one group an SM and
// nothing beside it: 4096 x 8192 65.7 us, 8192 x 5120 91 (62), 2048 x 16384 (clusters of two) 116,
// 1024 x 32768 (of four) 202; with four vectors a thread in one CTA the last two took 182 and more,
// with one exchange a row 95 and 181.
#include <algorithm>
#include <type_traits>

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

// Units of eight columns that each CTA of a cluster has of a row's, whole blocks of 32 columns (the
// last one fewer): 1024 at most.
__host__ __device__ __forceinline__ int bwd_share(int units, int cluster) {
  return ((units + 3) / 4 + cluster - 1) / cluster * 4;
}

// Buffers for a row: one that is worked on, one on its way.
constexpr int kBwdBufs = 2;
template <int V, bool HCK, bool OCK>
__host__ __device__ constexpr int bwd_row_bytes() {      // of a thread
  return V * (32 + (HCK ? 8 : 16) + (OCK ? 8 : 16));
}

// tpr threads per row (16, or whole warps), V vectors of eight columns a thread, laid out as in
// branch_row_kernel. Every thread copies its own elements of the next row to its own slots of
// shared memory while it works on the present one, whose three steps, mean(a xh), dh and s, and do,
// it makes in the same registers. rstd or rstd_o times a checkpoint's power of two is a factor of
// whole vectors: it is applied to a vector's sums and to its other factors, not to its elements
// (69.7 us -> 65.1 with dy, h and o kept in registers), and whole warps run a form of the row's
// step in which nothing is tested (-> 61.4). From bf16 the elements are scaled (see there), within
// 1 % of the time without at most widths, 3 % at 4112 columns.
// CL: a row of more than 8192 columns, whose two column sums a thread no longer fit in the
// registers of one CTA, lies in the two or four CTAs of a cluster, each of which adds the others'
// parts of the row's sums, which arrive in shared memory.
// REGS: registers a thread, 128, or 96 for CTAs of more than 512 threads.
template <int V, bool HCK, bool OCK, int CL, int REGS>
__global__ void __maxnreg__(REGS) branch_bwd_kernel(const __grid_constant__ BranchBwdParams p) {
  constexpr int kBufs = kBwdBufs;
  __shared__ alignas(16) float red[2][REGS < 128 ? 32 : 16];     // (20 words for 20 warps: 93 us, not 91)
  __shared__ float other[2][CL];
  extern __shared__ uint4 slots[];
  const int tpr = blockDim.x, lane = threadIdx.x, grp = threadIdx.y, rpc = blockDim.y;
  const int nt = tpr * rpc, tid = grp * tpr + lane;
  const int warps = tpr >> 5;                       // warps per row (0: two rows a warp)
  const uint32_t rank = CL > 1 ? ptx::cluster_rank() : 0;
  // this CTA's vectors: from v0 on (the beginning of a block), nv of them
  const int all_nv = p.cols >> 3, per = CL > 1 ? bwd_share(all_nv, CL) : all_nv;
  const int v0 = rank * per, nv = min(per, all_nv - v0);
  const RowUnits at = {V == 1 ? lane : (lane >> 5) * 32 * V + (lane & 31), 32};   // from v0 on
  const bool whole = at.first - (lane & 31) + 32 * V <= nv && warps != 0;         // of the warp
  const bool post = p.gamma_post != nullptr, dres = p.dres != nullptr;
  const bool want_s = post || p.dtoken != nullptr;
  constexpr int kVecs = V * (2 + !HCK + !OCK), kHalves = V * (HCK + OCK);
  const int all_warps = (nt + 31) >> 5;
  // a warp's pieces side by side: [kBufs][dy, dres, (h, o)][V][32], then [kBufs][(h, o)][V][32]
  uint4* const vec = slots + (tid >> 5) * (32 * kBufs * kVecs) + (tid & 31);
  uint2* const half = reinterpret_cast<uint2*>(slots + all_warps * (32 * kBufs * kVecs)) +
                      (tid >> 5) * (32 * kBufs * kHalves) + (tid & 31);
  const uint32_t rows = uint32_t(p.rows), cols = p.cols, c0 = 8 * (v0 + at.first);
  pdl_wait();

  float next_rstd = 0.0f, next_ro = 0.0f, next_t = 0.0f;
  uint32_t next_he[V], next_oe[V];
  const auto prefetch = [&](uint32_t r, int buf) {
    uint4* s = vec + buf * (32 * kVecs);
    uint2* q = half + buf * (32 * kHalves);
    const uint16_t* dy = p.dy + (uint64_t(r) * uint32_t(p.ld_dy) + c0);
    const uint16_t* dr = p.dres + (uint64_t(r) * uint32_t(p.ld_dres) + c0);
    const uint16_t* h = HCK ? nullptr : p.h + (uint64_t(r) * uint32_t(p.ld_h) + c0);
    const uint16_t* o = OCK ? nullptr : p.o + (uint64_t(r) * uint32_t(p.ld_o) + c0);
    const uint64_t e = uint64_t(r) * cols + c0;
    if (whole && r < rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ptx::cp_async_16(s + 32 * j, dy + 8 * j * at.step);
        if (dres) ptx::cp_async_16(s + 32 * (V + j), dr + 8 * j * at.step);
        if (HCK) ptx::cp_async_8(q + 32 * j, p.h_codes + e + 8 * j * at.step);
        else ptx::cp_async_16(s + 32 * (2 * V + j), h + 8 * j * at.step);
        if (OCK)
          ptx::cp_async_8(q + 32 * ((HCK ? V : 0) + j), p.o_codes + e + 8 * j * at.step);
        else
          ptx::cp_async_16(s + 32 * ((HCK ? 2 : 3) * V + j), o + 8 * j * at.step);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {                  // nothing read beyond the tensor: zeros
        const bool in = r < rows && at(j) < nv;
        const uint32_t n = in ? 16u : 0u, m = in ? 8u : 0u, d = 8 * j * at.step;
        ptx::cp_async_16_zfill(s + 32 * j, in ? dy + d : p.dy, n);
        if (dres) ptx::cp_async_16_zfill(s + 32 * (V + j), in ? dr + d : p.dres, n);
        if (HCK) ptx::cp_async_8_zfill(q + 32 * j, in ? p.h_codes + e + d : p.h_codes, m);
        else ptx::cp_async_16_zfill(s + 32 * (2 * V + j), in ? h + d : p.h, n);
        if (OCK)
          ptx::cp_async_8_zfill(q + 32 * ((HCK ? V : 0) + j), in ? p.o_codes + e + d : p.o_codes,
                                m);
        else
          ptx::cp_async_16_zfill(s + 32 * ((HCK ? 2 : 3) * V + j), in ? o + d : p.o, n);
      }
    }
    ptx::cp_async_commit();
  };
  // the row's own numbers, read a row ahead
  const auto scalars = [&](auto full_tag, uint32_t r) {
    constexpr bool FULL = decltype(full_tag)::value;
    const bool live = r < rows;
    next_rstd = live ? p.rstd[r] : 0.0f;
    next_ro = !live ? 0.0f : post ? p.rstd_o[r] : 1.0f;
    next_t = !live ? 0.0f : p.token_gate != nullptr ? p.token_gate[r] : 1.0f;
    const uint64_t e = uint64_t(r) * uint32_t(ckpt_pitch(p.cols)) + ((v0 + at.first) >> 2);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool in = live && (FULL || at(j) < nv);
      const uint32_t b = j * at.step / 4;
      if (HCK) next_he[j] = in ? __ldg(p.h_scale + e + b) : 0u;
      if (OCK) next_oe[j] = in ? __ldg(p.o_scale + e + b) : 0u;
    }
  };
  const uint32_t step = gridDim.x / CL * rpc;
  uint32_t r = blockIdx.x / CL * rpc + grp;
#pragma unroll
  for (int k = 0; k < kBufs - 1; ++k) prefetch(r + k * step, k);
  scalars(std::false_type{}, r);

  const auto factor = [&](int j, float2 (&w)[4]) {
    const int c = 8 * (v0 + at(j));
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
  float4* const ws = reinterpret_cast<float4*>(
                         slots + all_warps * (32 * kBufs * kVecs + 16 * kBufs * kHalves)) +
                     (lane >> 5) * (32 * 2 * V) + (lane & 31);
  float2 g[V][4], acc_g[V][4], acc_s[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    gamma_pairs(p.gamma, p.gamma_fp32, p.cols, 8 * (v0 + at(j)), g[j]);
    if (grp == 0) {
      float2 w[4];
      factor(j, w);
      ws[32 * 2 * j] = make_float4(w[0].x, w[0].y, w[1].x, w[1].y);
      ws[32 * (2 * j + 1)] = make_float4(w[2].x, w[2].y, w[3].x, w[3].y);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) acc_g[j][k] = acc_s[j][k] = make_float2(0.0f, 0.0f);
  }
  __syncthreads();
  if (CL > 1) ptx::cluster_sync();                  // the others run: their memory may be written
  const auto w_of = [&](int j, float2 (&w)[4]) {
    const float4 a = ws[32 * 2 * j], b = ws[32 * (2 * j + 1)];
    w[0] = make_float2(a.x, a.y);
    w[1] = make_float2(a.z, a.w);
    w[2] = make_float2(b.x, b.y);
    w[3] = make_float2(b.z, b.w);
  };
  int phase = 0;
  // A cluster's sum: every CTA's part comes to every CTA, by turns to two places. (What is written
  // two sums later was read before the barrier in between.)
  int turn = 0;
  const auto sum_of = [&](float v) {
    v = row_sum(v, red, phase, warps, lane, grp, tpr);
    if constexpr (CL > 1) {
      if (lane < CL) ptx::st_cluster_f32(ptx::map_to_rank(&other[turn][rank], lane), v);
      __syncwarp();
      ptx::cluster_sync();
      v = other[turn][0];
#pragma unroll
      for (int i = 1; i < CL; ++i) v += other[turn][i];
      turn ^= 1;
    }
    return v;
  };

  // One row. FULL: the row exists and has columns for all vectors of the warp: nothing is tested.
  int buf = 0;
  const auto one_row = [&](auto full_tag) {
    constexpr bool FULL = decltype(full_tag)::value;
    const uint4* s = vec + buf * (32 * kVecs);
    const uint2* q = half + buf * (32 * kHalves);
    const uint64_t elem = uint64_t(r) * cols + c0;
    const float rs = next_rstd, ro = next_ro, t = next_t;
    float hf[HCK ? V : 1], of[OCK ? V : 1];         // what a code of the row counts in xh and xo
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (HCK) hf[HCK ? j : 0] = ckpt_factor(next_he[j]) * rs;
      if (OCK) of[OCK ? j : 0] = ckpt_factor(next_oe[j]) * ro;
    }
    if (!HCK) hf[0] = 1.0f;
    if (!OCK) of[0] = 1.0f;
    // what h and o hold. A code's factors are applied to sums and to other factors; bf16 is made xh
    // and xo where it is read, for a row whose squares overflow has an rstd of 0 and elements
    // whose products with a gradient may be infinite.
    const auto h_of = [&](int j, float2 (&x)[4]) {
      if constexpr (HCK) ckpt_widen8(q[32 * j], x);
      else widen8(s[32 * (2 * V + j)], x);
    };
    const auto o_of = [&](int j, float2 (&x)[4]) {
      if constexpr (OCK) ckpt_widen8(q[32 * ((HCK ? V : 0) + j)], x);
      else widen8(s[32 * ((HCK ? 2 : 3) * V + j)], x);
    };
    ptx::cp_async_wait<kBufs - 2>();
    prefetch(r + (kBufs - 1) * step, buf == 0 ? kBufs - 1 : buf - 1);
    scalars(full_tag, r + step);

    // ---- mean(a xh), dgamma
    const float2 r2 = make_float2(rs, rs), ro2 = make_float2(ro, ro);
    float2 d[V][4], x[V][4];                        // dy, then dh, then u; h, then o
    float c = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float2(&xj)[4] = x[j], (&gj)[4] = g[j];
      widen8(s[32 * j], d[j]);
      h_of(j, xj);
      const float f = hf[HCK ? j : 0];
      const float2 f2 = make_float2(f, f);
      float2 c2 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!HCK) xj[k] = __fmul2_rn(xj[k], r2);
        const float2 v = __fmul2_rn(d[j][k], xj[k]);
        acc_g[j][k] = __ffma2_rn(v, f2, acc_g[j][k]);
        c2 = __ffma2_rn(v, gj[k], c2);
      }
      c = fmaf(c2.x + c2.y, f, c);
    }
    uint4 er[V];                                    // read before the barrier (61.4 -> 60.8)
#pragma unroll
    for (int j = 0; j < V; ++j) er[j] = dres ? s[32 * (V + j)] : make_uint4(0, 0, 0, 0);
    c = -p.inv_cols * sum_of(c);

    // ---- dh, s, S
    float s1 = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float2 w[4], e[4], (&xj)[4] = x[j], (&gj)[4] = g[j];
      widen8(er[j], e);
      const float fc = hf[HCK ? j : 0] * c;
      const float2 fc2 = make_float2(fc, fc);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        d[j][k] = __ffma2_rn(r2, __ffma2_rn(xj[k], fc2, __fmul2_rn(d[j][k], gj[k])), e[k]);
      if (FULL || (r < rows && at(j) < nv))
        *reinterpret_cast<uint4*>(p.dh + elem + 8 * j * at.step) = make_uint4(
            pack_bf16(d[j][0].x, d[j][0].y), pack_bf16(d[j][1].x, d[j][1].y),
            pack_bf16(d[j][2].x, d[j][2].y), pack_bf16(d[j][3].x, d[j][3].y));
      o_of(j, xj);
      w_of(j, w);
      const float f = of[OCK ? j : 0], ft = f * t;
      const float2 ft2 = make_float2(ft, ft);
      float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!OCK) xj[k] = __fmul2_rn(xj[k], ro2);
        const float2 v = __fmul2_rn(d[j][k], xj[k]);
        // a gate of 0: whatever o holds, nothing of it reaches the sums
        if (t != 0.0f) acc_s[j][k] = __ffma2_rn(v, ft2, acc_s[j][k]);
        s2 = __ffma2_rn(v, w[k], s2);
        d[j][k] = __fmul2_rn(d[j][k], w[k]);        // u from here on
      }
      s1 = fmaf(s2.x + s2.y, f, s1);
    }
    float sum = 0.0f;
    if (want_s) {
      sum = sum_of(s1);
      if (p.dtoken != nullptr && lane == 0 && (FULL || r < rows) && rank == 0) p.dtoken[r] = sum;
    }

    // ---- do
    const float rt = ro * t, m = post ? -p.inv_cols * rt * sum : 0.0f;
    const float2 rt2 = make_float2(rt, rt);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (t == 0.0f) {
#pragma unroll
        for (int k = 0; k < 4; ++k) d[j][k] = make_float2(0.0f, 0.0f);
      } else if (post) {
        float2(&xj)[4] = x[j];
        const float fm = of[OCK ? j : 0] * m;
        const float2 fm2 = make_float2(fm, fm);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          d[j][k] = __ffma2_rn(xj[k], fm2, __fmul2_rn(d[j][k], rt2));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) d[j][k] = __fmul2_rn(d[j][k], rt2);
      }
      if (FULL || (r < rows && at(j) < nv))
        *reinterpret_cast<uint4*>(p.d_o + elem + 8 * j * at.step) = make_uint4(
            pack_bf16(d[j][0].x, d[j][0].y), pack_bf16(d[j][1].x, d[j][1].y),
            pack_bf16(d[j][2].x, d[j][2].y), pack_bf16(d[j][3].x, d[j][3].y));
    }
    buf = buf + 1 == kBufs ? 0 : buf + 1;
  };
  // All warps of a group make the same rows, the existing ones, for they meet at its barriers; the
  // two groups of a warp go on together.
  if (whole) {
    for (; r < rows; r += step) one_row(std::true_type{});
  } else {
    for (; warps != 0 ? r < rows : r - grp < rows; r += step) one_row(std::false_type{});
  }
  ptx::cp_async_wait<0>();
  if (p.part != nullptr) {
    // the groups' sums, added by the first group in order, by way of the slots (96 V nt bytes or
    // more where there are several groups, of which 64 V nt are used)
    static_assert(kBwdBufs * bwd_row_bytes<V, HCK, OCK>() >= 64 * V, "the slots hold both sums");
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
      const int64_t part = int64_t(blockIdx.x / CL) * p.cols;
      float* dst = p.part + part + c0;
      const int64_t to_s = int64_t(p.parts) * p.cols;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (at(j) < nv) {
          float4* q = reinterpret_cast<float4*>(dst + 8 * j * at.step);
          q[0] = make_float4(acc_g[j][0].x, acc_g[j][0].y, acc_g[j][1].x, acc_g[j][1].y);
          q[1] = make_float4(acc_g[j][2].x, acc_g[j][2].y, acc_g[j][3].x, acc_g[j][3].y);
          q = reinterpret_cast<float4*>(dst + to_s + 8 * j * at.step);
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
  RowPlan row;                // of a CTA's part of a row
  int cluster;                // CTAs that share a row
  int parts;                  // CTAs, or clusters of them
};
// One CTA of up to 512 threads per SM, as in the norm's backward pass: its row groups' column sums
// meet in shared memory, so there are at most as many partials as SMs. Few rows: one vector a
// thread, and fewer rows a CTA while there are SMs without any.
// Rows of 577 to 640 vectors, of which two vectors a thread would make one group of ten warps and
// nothing beside it, have twenty with one vector at 96 registers. From checkpoints / bf16, us, with
// two and with one: 8192 x 5120 103 and 91 / 93.8 and 89.8, 8192 x 5104 111 and 94, 300 x 5120 13.0
// and 11.5; 8192 x 4608 101 and 104 / 91 and 99, 8192 x 6144 (at 80 registers) 96.7 and 110. Two
// groups of ten warps with two vectors, at 96 registers, spill: 120 / 89.8.
BranchBwdPlan branch_bwd_plan(int64_t rows, int64_t cols) {
  BranchBwdPlan b;
  const int sms = num_sms(), nv = int(cols / 8);
  b.cluster = cols > 16384 ? 4 : cols > 8192 ? 2 : 1;
  const int mine = b.cluster > 1 ? bwd_share(nv, b.cluster) : nv;
  if (b.cluster == 1 && nv > 576 && nv <= 640) {
    const int tpr = (nv + 31) / 32 * 32;
    b.row = {1, tpr, tpr};
  } else {
    b.row = row_plan(8 * mine, rows <= 4 * sms ? 1 : 2, 512);
  }
  int rpc = b.row.block / b.row.tpr;
  while (rpc > 1 && (rpc / 2) * b.row.tpr >= 128 && rows <= int64_t(rpc / 2) * sms) rpc /= 2;
  b.row.block = rpc * b.row.tpr;
  b.parts = int(std::min<int64_t>((rows + rpc - 1) / rpc, sms / b.cluster));
  return b;
}

template <int V, bool HCK, bool OCK, int CL, int REGS>
cudaError_t launch_bwd(const BranchBwdParams& p, const BranchBwdPlan& b, cudaStream_t st) {
  auto kern = branch_bwd_kernel<V, HCK, OCK, CL, REGS>;
  const size_t smem = size_t(kBwdBufs) * bwd_row_bytes<V, HCK, OCK>() * std::max(b.row.block, 32) +
                      size_t(V) * 32 * std::max(b.row.tpr, 32);
  if (smem > 47 * 1024) {                                  // 48 KB with the static part
    static ContextOnce attr = {};
    const cudaError_t e = once_per_context(attr, [&] {
      return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    });
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute cluster = {};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = CL;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  const int rpc = b.row.block / b.row.tpr;
  return launch_kernel(kern, dim3(unsigned(CL * b.parts)), dim3(unsigned(b.row.tpr), unsigned(rpc)),
                       smem, st, CL > 1 ? &cluster : nullptr, p);
}
template <bool HCK, bool OCK>
cudaError_t launch_bwd(const BranchBwdParams& p, const BranchBwdPlan& b, cudaStream_t st) {
  if (b.cluster == 4) return launch_bwd<2, HCK, OCK, 4, 128>(p, b, st);
  if (b.cluster == 2) return launch_bwd<2, HCK, OCK, 2, 128>(p, b, st);
  if (b.row.tpr > 512) return launch_bwd<1, HCK, OCK, 1, 96>(p, b, st);
  return b.row.v == 1 ? launch_bwd<1, HCK, OCK, 1, 128>(p, b, st)
                      : launch_bwd<2, HCK, OCK, 1, 128>(p, b, st);
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
