// The gradients of a step before the optimizer: global norm and clipping (fp8_grad_norm,
// fp8_grad_clip).
//
// A list of tensors of any sizes is cut into chunks, so that a CTA's work does not depend on the
// tensors' sizes; the CTA of a chunk looks its tensor up in the prefix sums of the chunk counts.
// The list travels in the kernel's parameters: nothing is copied to the device and the call can
// be captured in a graph.
//
// Norm: bytes read once, eight 16-byte loads a thread in flight. Squares are added in fp32 (four
// sums a thread, at most 16 chunks each), those sums in fp64, in a fixed order. A vector whose
// largest magnitude lies outside [2^-50, 2^50], where squares would leave fp32's range or lose
// bits, is added in fp64 instead.
// Clip: one multiply, read once and written once. One CTA a chunk: CTAs that stay and walk
// chunks measured 20 us more for 134M fp32 (262 against 242 with the norm).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.cuh"
#include "norm.cuh"

namespace fp8lin {

constexpr int kGradThreads = 256;
constexpr int kGradCtas = 4;             // CTAs per SM of the norm
constexpr int kNormChunk = 16384;        // elements a chunk of the norm
constexpr int kClipChunk = 8192;         // ... of clipping
constexpr int kGradUnroll = 8;           // loads in flight a thread
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

// Sum over the CTA in a fixed order, in thread 0.
__device__ __forceinline__ double cta_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
  for (int i = 0; i < int(blockDim.x >> 5); ++i) t += red[i];
  return t;
}

// norm and coef from the sum of squares; NaN and infinity pass through.
__device__ __forceinline__ void grad_finish(double sum, float max_norm, float scale, float* norm,
                                            float* coef) {
  const float n = float(double(scale) * sqrt(sum));
  *norm = n;
  if (coef != nullptr) {
    float c = max_norm / (n + 1e-6f);
    if (c > 1.0f || isinf(max_norm)) c = 1.0f;
    *coef = scale * c;
  }
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
    const int size = f32 ? 4 : 2, per = f32 ? 4 : 8;
    const uint8_t* p = reinterpret_cast<const uint8_t*>(l.g[t]) + e0 * size;
    // elements before the first 16-byte boundary, whole vectors, the rest
    const int head = min(n, int((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / size);
    const int nvec = (n - head) / per;
    const uint4* v = reinterpret_cast<const uint4*>(p + head * size);
    for (int i = threadIdx.x; i < nvec; i += kGradUnroll * kGradThreads) {
      uint4 w[kGradUnroll];
#pragma unroll
      for (int k = 0; k < kGradUnroll; ++k) {
        const int at = i + k * kGradThreads;
        w[k] = at < nvec ? ldg_nc_v4_sched(v + at) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < kGradUnroll; ++k) add_vec(a, w[k], f32);
    }
    const int rest = head + nvec * per + int(threadIdx.x);
    if (int(threadIdx.x) < head) add_one(a, grad_at(p, f32, threadIdx.x));
    if (rest < n) add_one(a, grad_at(p, f32, rest));
    if (++since == kGradFlush) {
      a.flush();
      since = 0;
    }
  }
  a.flush();
  const double s = cta_sum(a.d, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
  pdl_launch_dependents();
}

__global__ void __launch_bounds__(kGradThreads)
    grad_finish_kernel(const double* part, int n, float max_norm, float scale, float* norm,
                       float* coef) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ double red[kGradThreads / 32];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kGradThreads) s += part[i];
  s = cta_sum(s, red);
  if (threadIdx.x == 0) grad_finish(s, max_norm, scale, norm, coef);
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
