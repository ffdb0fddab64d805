// The gradients of a step before the optimizer: global norm and clipping (fp8_grad_norm,
// fp8_grad_clip).
//
// A list of tensors of any sizes is cut into chunks, so that a CTA's work does not depend on the
// tensors' sizes; the CTA of a chunk looks its tensor up in the prefix sums of the chunk counts.
// The list travels in the kernel's parameters: nothing is copied to the device and the call can
// be captured in a graph.
//
// Norm: bytes read once, eight 16-byte loads a thread in flight. Squares are added in fp32 in two
// levels (four sums a thread for a chunk, each at most 18 squares; those sums over at most 16
// chunks), then over the warp; the warps' sums in fp64, all in a fixed order. The levels are for
// precision: a bf16 square has few bits, so that adding it to a long sum often ends in a tie, and
// the ties do not cancel out. With 256 squares to a sum, 268M normal bf16 gave a norm that was
// 1.1e-7 too small in the mean, now 4e-9 (a result's own rounding: up to 6e-8), in the same
// time. fp64 is slow on this GPU (two additions a clock and SM), hence so little of it:
// with every thread's sum in fp64, 134M fp32 took 79.5 us instead of 77.9. A vector whose largest
// magnitude lies outside [2^-50, 2^50], where squares would leave fp32's range or lose bits, is
// added in fp64. 134M fp32 in 77.9 us is 6.9 TB/s: memory bound. Up to 1 MB: one launch instead of
// two (see there).
// Clip: one multiply, read once and written once: 134M fp32 in 153.5 us, 7.0 TB/s. One CTA a
// chunk: CTAs that stay and walk chunks measured 20 us more (262 against 242 with the norm). Four
// elements a thread: with eight, each fp32 sector is asked for twice.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.cuh"
#include "norm.cuh"
#include "sm100_ptx.cuh"

namespace fp8lin {

constexpr int kGradThreads = 256;
constexpr int kGradCtas = 4;             // CTAs per SM of the norm
constexpr int kNormChunk = 16384;        // elements a chunk of the norm
constexpr int kClipChunk = 8192;         // ... of clipping
constexpr int kGradUnroll = 8;           // loads in flight a thread
constexpr int kSmallCtas = 8;            // the cluster that takes a short list
constexpr int kSmallThreads = 512;
constexpr int kSmallBytes = 4096;        // bytes a warp takes at once
constexpr int kSmallPieces = 256;        // pieces at most
constexpr int kGradFlush = 16;           // chunks between flushes of the fp32 sums

// Up to N tensors in the kernel parameters (28 bytes each).
template <int N>
struct GradList {
  const void* g[N];
  void* out[N];
  int64_t numel[N];                      // bit 62: grad is fp32, bit 61: out is fp32
  uint32_t first[N + 1];                 // chunks before tensor i
  int n;
};
constexpr int64_t kGradF32 = int64_t(1) << 62, kOutF32 = int64_t(1) << 61;
constexpr int64_t kNumelMask = kOutF32 - 1;
// Two lengths of the list: 64 tensors are 1.8 KB of parameters, 1024 are 29 KB (of 32 that a launch
// may have), which costs the host 0.75 us a launch (grad_clip of 12 tensors: 3.4 against 4.15) and
// the GPU 0.1.
constexpr int kGradSmall = 64, kGradLarge = 1024;

// The tensor that holds chunk c.
template <int N>
__device__ __forceinline__ int grad_find(const GradList<N>& l, uint32_t c) {
  int lo = 0, hi = l.n;                  // first[lo] <= c < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float grad_at(const void* p, bool f32, int64_t i) {
  return f32 ? reinterpret_cast<const float*>(p)[i]
             : __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(p)[i]) << 16);
}

struct GradSum {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  double d = 0.0;
  __device__ __forceinline__ void flush() {
    d += double((s[0] + s[1]) + (s[2] + s[3]));
    s[0] = s[1] = s[2] = s[3] = 0.0f;
  }
};

// Magnitudes (31-bit patterns) whose squares are added in fp64: not zero and outside
// [2^-50, 2^50]; infinities and NaN among them.
__device__ __forceinline__ bool grad_far(uint32_t m) {
  return m - 0x26800000u > 0x58800000u - 0x26800000u && m != 0u;
}

__device__ __forceinline__ void add_one(GradSum& a, float v) {
  if (grad_far(mag31(v))) a.d += double(v) * double(v);
  else a.s[0] = fmaf(v, v, a.s[0]);
}

__device__ __forceinline__ void add_vec(GradSum& a, uint4 v, bool f32) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (f32) {
    const uint32_t m = max(max(w[0] & 0x7FFFFFFFu, w[1] & 0x7FFFFFFFu),
                           max(w[2] & 0x7FFFFFFFu, w[3] & 0x7FFFFFFFu));
    if (grad_far(m)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double x = double(__uint_as_float(w[i]));
        a.d += x * x;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a.s[i] = fmaf(__uint_as_float(w[i]), __uint_as_float(w[i]), a.s[i]);
    }
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = absmax_bf16x2(m, w[i]);
    m = fold_bf16x2(m) << 16;
    if (grad_far(m)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double x = double(bf16_lo(w[i])), y = double(bf16_hi(w[i]));
        a.d += x * x;
        a.d += y * y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a.s[i] = fmaf(bf16_lo(w[i]), bf16_lo(w[i]), a.s[i]);
        a.s[i] = fmaf(bf16_hi(w[i]), bf16_hi(w[i]), a.s[i]);
      }
    }
  }
}

// Sum over the warp in a fixed order, in every lane. fp64 additions are slow (two a clock and SM),
// so the fp32 sums are added as such; the fp64 ones only where there are any.
__device__ __forceinline__ double warp_sum(const GradSum& a) {
  float s = (a.s[0] + a.s[1]) + (a.s[2] + a.s[3]);
  double d = a.d;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (__any_sync(0xffffffffu, d != 0.0)) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  }
  return d + double(s);
}

// Sum of n doubles in shared memory, 32 to a step, by one warp.
__device__ __forceinline__ double sum_of(const double* red, int n, int lane) {
  double s = lane < n ? red[lane] : 0.0;
  for (int i = 32 + lane; i < n; i += 32) s += red[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// norm and coef from the sum of squares; NaN and infinity pass through. fp64 is slow here too, so
// the root of sum = m 4^k, 1 <= m < 4, is taken in fp32 and corrected by one Newton step.
__device__ __forceinline__ void grad_finish(double sum, float max_norm, float scale, float* norm,
                                            float* coef) {
  double root = sum;
  if (sum > 0.0 && !isinf(sum)) {                    // no subnormal: a square is 2^-298 or more
    const uint32_t hi = uint32_t(__double2hiint(sum)), lo = uint32_t(__double2loint(sum));
    const int e = int(hi >> 20) - 1023, k = e >> 1;
    const double m = __hiloint2double(int((hi & 0xFFFFFu) | uint32_t(1023 + (e & 1)) << 20),
                                      int(lo));
    const float r = __fsqrt_rn(float(m));
    const double rest = fma(-double(r), double(r), m);
    root = (double(r) + double(float(rest) / (2.0f * r))) * __hiloint2double((1023 + k) << 20, 0);
  }
  const float n = float(double(scale) * root);
  *norm = n;
  if (coef != nullptr) {
    float c = max_norm / (n + 1e-6f);
    if (c > 1.0f || isinf(max_norm)) c = 1.0f;
    *coef = scale * c;
  }
}

// The squares of n elements from p on, by THREADS threads (a CTA or a warp): the elements before
// the first 16-byte boundary, whole vectors, the rest. Their sums are made apart and then added.
template <int THREADS>
__device__ __forceinline__ void add_chunk(GradSum& a, const uint8_t* p, bool f32, int n, int tid) {
  const int size = f32 ? 4 : 2, per = f32 ? 4 : 8;
  const int head = min(n, int((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / size);
  const int nvec = (n - head) / per;
  const uint4* v = reinterpret_cast<const uint4*>(p + head * size);
  const float before[4] = {a.s[0], a.s[1], a.s[2], a.s[3]};
#pragma unroll
  for (int k = 0; k < 4; ++k) a.s[k] = 0.0f;
  for (int i = tid; i < nvec; i += kGradUnroll * THREADS) {
    uint4 w[kGradUnroll];
#pragma unroll
    for (int k = 0; k < kGradUnroll; ++k) {
      const int at = i + k * THREADS;
      w[k] = at < nvec ? ldg_nc_v4_sched(v + at) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kGradUnroll; ++k) add_vec(a, w[k], f32);
  }
  const int rest = head + nvec * per + tid;
  if (tid < head) add_one(a, grad_at(p, f32, tid));
  if (rest < n) add_one(a, grad_at(p, f32, rest));
#pragma unroll
  for (int k = 0; k < 4; ++k) a.s[k] += before[k];
}

template <int N>
__global__ void __launch_bounds__(kGradThreads)
    grad_norm_kernel(const __grid_constant__ GradList<N> l, double* part) {
  pdl_wait();
  __shared__ double red[kGradThreads / 32];
  const uint32_t total = l.first[l.n];
  GradSum a;
  int since = 0;
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    const int t = grad_find(l, c);
    const bool f32 = (l.numel[t] & kGradF32) != 0;
    const int64_t e0 = int64_t(c - l.first[t]) * kNormChunk;
    const int n = int(min(int64_t(kNormChunk), (l.numel[t] & kNumelMask) - e0));
    add_chunk<kGradThreads>(
        a, reinterpret_cast<const uint8_t*>(l.g[t]) + e0 * (f32 ? 4 : 2), f32, n, threadIdx.x);
    if (++since == kGradFlush) {
      a.flush();
      since = 0;
    }
  }
  const double s = warp_sum(a);
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    const double t = sum_of(red, kGradThreads / 32, lane);
    if (lane == 0) part[blockIdx.x] = t;
  }
  pdl_launch_dependents();
}

__global__ void __launch_bounds__(kGradThreads)
    grad_finish_kernel(const double* part, int n, float max_norm, float scale, float* norm,
                       float* coef) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ double red[kGradThreads];
  double s = threadIdx.x < n ? part[threadIdx.x] : 0.0;
  for (int i = threadIdx.x + kGradThreads; i < n; i += kGradThreads) s += part[i];
  red[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = sum_of(red, kGradThreads, threadIdx.x);
    if (threadIdx.x == 0) grad_finish(s, max_norm, scale, norm, coef);
  }
}

// Norm of a short list in one launch: a cluster of kSmallCtas CTAs whose warps take a piece of 4
// KB (one round of loads) each; the warps' sums meet in the shared memory of the first CTA. The
// pieces themselves are in the parameters: there is nothing to look up (a binary search in the
// constant bank took 0.8 us). Latency bound: 64 tensors of 1024 in 3.0 us and one launch, 3.9 in
// two; at 1 MB the two take the same time on the GPU (4.6 and 4.8 us), beyond it the cluster is
// too few SMs. 16 CTAs would be 0.7 us faster at 1 MB and no faster below, and are more than a
// cluster may count on.
struct GradPieces {
  const void* p[kSmallPieces];
  uint32_t n[kSmallPieces];              // elements; bit 31: fp32
  int total;
};
__global__ void __cluster_dims__(kSmallCtas) __launch_bounds__(kSmallThreads)
    grad_norm_small_kernel(const __grid_constant__ GradPieces l, float max_norm, float scale,
                           float* norm, float* coef) {
  constexpr int kWarps = kSmallThreads / 32;
  __shared__ double red[kSmallCtas * kWarps];
  ptx::cluster_arrive_relaxed();                   // the first CTA runs: its memory is there
  pdl_wait();
  const int lane = threadIdx.x & 31;
  // neighbouring pieces go to different CTAs
  const int warp = int(threadIdx.x >> 5) * kSmallCtas + int(blockIdx.x);
  GradSum a;
  for (int c = warp; c < l.total; c += kSmallCtas * kWarps)
    add_chunk<32>(a, reinterpret_cast<const uint8_t*>(l.p[c]), (l.n[c] >> 31) != 0,
                  int(l.n[c] & 0x7FFFFFFFu), lane);
  const double s = warp_sum(a);
  ptx::cluster_wait();
  if (lane == 0) ptx::st_cluster(ptx::map_to_rank(&red[warp], 0), s);
  ptx::cluster_sync();
  if (warp == 0) {
    const double t = sum_of(red, kSmallCtas * kWarps, lane);
    if (lane == 0) grad_finish(t, max_norm, scale, norm, coef);
  }
  pdl_launch_dependents();
}

__device__ __forceinline__ void grad_put(void* p, bool f32, int64_t i, float v) {
  if (f32) {
    reinterpret_cast<float*>(p)[i] = v;
  } else {
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  }
}

// Four elements, on a boundary of four, as a thread's share: neighbouring threads then read and
// write neighbouring bytes whatever the two types (with eight, an fp32 sector would be asked for
// twice).
__device__ __forceinline__ uint4 load4(const uint8_t* src, bool f32) {
  if (f32) return *reinterpret_cast<const uint4*>(src);
  const uint2 v = *reinterpret_cast<const uint2*>(src);
  return make_uint4(v.x << 16, v.x & 0xFFFF0000u, v.y << 16, v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(uint8_t* dst, uint4 v, bool o32, float k) {
  const float a = __uint_as_float(v.x) * k, b = __uint_as_float(v.y) * k;
  const float c = __uint_as_float(v.z) * k, d = __uint_as_float(v.w) * k;
  if (o32) *reinterpret_cast<float4*>(dst) = make_float4(a, b, c, d);
  else *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
}

template <int N>
__global__ void __launch_bounds__(kGradThreads)
    grad_clip_kernel(const __grid_constant__ GradList<N> l, const float* coef) {
  pdl_wait();
  const float k = *coef;
  // last chunk first: the norm read the last ones most recently, so some are still in L2
  const uint32_t c = gridDim.x - 1 - blockIdx.x;
  const int t = grad_find(l, c);
  const bool f32 = (l.numel[t] & kGradF32) != 0, o32 = (l.numel[t] & kOutF32) != 0;
  if (k == 1.0f && l.out[t] == l.g[t]) return;
  const int64_t e0 = int64_t(c - l.first[t]) * kClipChunk;
  const int n = int(min(int64_t(kClipChunk), (l.numel[t] & kNumelMask) - e0));
  const int size = f32 ? 4 : 2, osize = o32 ? 4 : 2;
  const uint8_t* p = reinterpret_cast<const uint8_t*>(l.g[t]) + e0 * size;
  uint8_t* q = reinterpret_cast<uint8_t*>(l.out[t]) + e0 * osize;
  // elements before p's first boundary of four; the groups from there on need q on one too,
  // otherwise all are done one by one
  const int gs = 4 * size, gq = 4 * osize;
  int head = min(n, int((gs - (reinterpret_cast<uintptr_t>(p) & (gs - 1))) & (gs - 1)) / size);
  const bool both = ((reinterpret_cast<uintptr_t>(q) + head * osize) & (gq - 1)) == 0;
  const int ng = both ? (n - head) / 4 : 0;
  if (!both) head = n;
  const uint8_t* src = p + head * size;
  uint8_t* dst = q + head * osize;
  for (int i = threadIdx.x; i < ng; i += kGradUnroll * kGradThreads) {
    uint4 v[kGradUnroll];
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
      const int at = i + u * kGradThreads;
      if (at < ng) v[u] = load4(src + at * gs, f32);
    }
#pragma unroll
    for (int u = 0; u < kGradUnroll; ++u) {
      const int at = i + u * kGradThreads;
      if (at < ng) store4(dst + at * gq, v[u], o32, k);
    }
  }
  for (int e = threadIdx.x; e < head; e += kGradThreads)
    grad_put(q, o32, e, grad_at(p, f32, e) * k);
  const int rest = head + 4 * ng + int(threadIdx.x);
  if (rest < n) grad_put(q, o32, rest, grad_at(p, f32, rest) * k);
  pdl_launch_dependents();
}

// ------------------------------------------------------------------------- host

namespace {

int grad_grid(uint32_t chunks) {
  return int(std::min<int64_t>(chunks, int64_t(num_sms()) * kGradCtas));
}

// The next tensors of the list, from item *at on, as one launch's parameters; empty tensors are
// left out. Returns their number of chunks.
template <int N>
uint32_t grad_pack(int n, const fp8_grad_item* items, int chunk, int* at, GradList<N>* l) {
  uint64_t chunks = 0;
  l->n = 0;
  for (; *at < n && l->n < N; ++*at) {
    const fp8_grad_item& it = items[*at];
    if (it.numel == 0) continue;
    l->g[l->n] = it.grad;
    l->out[l->n] = it.out;
    l->numel[l->n] = it.numel | (it.dtype == FP8_GRAD_FP32 ? kGradF32 : 0) |
                     (it.out_dtype == FP8_GRAD_FP32 ? kOutF32 : 0);
    l->first[l->n] = uint32_t(chunks);
    chunks += (uint64_t(it.numel) + chunk - 1) / chunk;      // < 2^31: the caller checked
    ++l->n;
  }
  l->first[l->n] = uint32_t(chunks);
  return uint32_t(chunks);
}

template <int N>
cudaError_t norm_lists(int n, const fp8_grad_item* items, double* part, int* parts,
                       cudaStream_t st) {
  for (int at = 0; at < n;) {
    GradList<N> l;
    const uint32_t chunks = grad_pack<N>(n, items, kNormChunk, &at, &l);
    if (chunks == 0) break;
    const int grid = grad_grid(chunks);
    const cudaError_t e = launch_kernel(grad_norm_kernel<N>, dim3(grid), dim3(kGradThreads), 0, st,
                                        nullptr, l, part + *parts);
    if (e != cudaSuccess) return e;
    *parts += grid;
  }
  return cudaSuccess;
}

// The pieces of a short list; false when there are too many.
bool grad_pieces(int n, const fp8_grad_item* items, GradPieces* l) {
  int c = 0;
  for (int i = 0; i < n; ++i) {
    const bool f32 = items[i].dtype == FP8_GRAD_FP32;
    const int size = f32 ? 4 : 2, per = kSmallBytes / size;
    if (items[i].numel > int64_t(kSmallPieces - c) * per) return false;
    const uint8_t* p = reinterpret_cast<const uint8_t*>(items[i].grad);
    for (int64_t left = items[i].numel; left > 0; left -= per, p += kSmallBytes, ++c) {
      l->p[c] = p;
      l->n[c] = uint32_t(std::min<int64_t>(left, per)) | (f32 ? 0x80000000u : 0u);
    }
  }
  l->total = c;
  return true;
}

template <int N>
cudaError_t clip_lists(int n, const fp8_grad_item* items, const float* coef, cudaStream_t st) {
  for (int at = 0; at < n;) {
    GradList<N> l;
    const uint32_t chunks = grad_pack<N>(n, items, kClipChunk, &at, &l);
    if (chunks == 0) break;
    const cudaError_t e = launch_kernel(grad_clip_kernel<N>, dim3(chunks), dim3(kGradThreads), 0,
                                        st, nullptr, l, coef);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_workspace_bytes(int n) {
  if (n < 0) return 0;
  return size_t(n / kGradLarge + 1) * num_sms() * kGradCtas * sizeof(double);
}

cudaError_t grad_norm_launch(int n, const fp8_grad_item* items, const fp8_clip_rule& rule,
                             float* norm, float* coef, void* workspace, cudaStream_t st) {
  GradPieces pieces;
  if (grad_pieces(n, items, &pieces))
    return launch_kernel(grad_norm_small_kernel, dim3(kSmallCtas), dim3(kSmallThreads), 0, st,
                         nullptr, pieces, rule.max_norm, rule.scale, norm, coef);
  double* part = reinterpret_cast<double*>(workspace);
  int parts = 0;
  const cudaError_t e = n <= kGradSmall ? norm_lists<kGradSmall>(n, items, part, &parts, st)
                                        : norm_lists<kGradLarge>(n, items, part, &parts, st);
  if (e != cudaSuccess) return e;
  return launch_kernel(grad_finish_kernel, dim3(1), dim3(kGradThreads), 0, st, nullptr,
                       static_cast<const double*>(part), parts, rule.max_norm, rule.scale, norm,
                       coef);
}

cudaError_t grad_clip_launch(int n, const fp8_grad_item* items, const float* coef,
                             cudaStream_t st) {
  return n <= kGradSmall ? clip_lists<kGradSmall>(n, items, coef, st)
                         : clip_lists<kGradLarge>(n, items, coef, st);
}

}  // namespace fp8lin
