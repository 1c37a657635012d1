// Global gradient norm and clipping over many tensors.
//   norm = sqrt(sum x^2),  coef = min(1, max_norm / (norm + 1e-6)),  dst = coef * src
// Two passes over the values: the sum needs all of them before the first is scaled.  The
// tensors are cut into chunks of 8192 elements, dealt to the CTAs in turn; the descriptors
// travel as kernel parameters (no copy to the device, so a captured call replays).  The
// second pass walks the chunks backwards: it begins with those the first pass left in L2.
#include <cuda_bf16.h>

#include <algorithm>

#include "pdl.cuh"
#include "ptx.cuh"
#include "train.cuh"

namespace dspark {
namespace clip {
namespace {

struct Tensor {
  const void* src;
  void* dst;
  int64_t n;
  int32_t bf16;
  int32_t chunk0;  // index of the tensor's first chunk
};
// The descriptors of one launch, in three sizes: they are copied with every launch.
template <int N>
struct Batch {
  Tensor t[N];
  int32_t count, chunks;
};
static_assert(sizeof(Batch<kMaxTensors>) < 32000, "kernel parameters");

// The tensor a chunk belongs to: the last whose first chunk is not after it (tensors without
// elements share their successor's first chunk and are never the last).
template <int N>
__device__ __forceinline__ int find(const Batch<N>& b, int chunk) {
  int lo = 0, hi = b.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (b.t[mid].chunk0 <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Sum of squares of up to eight values: in FP32 where that is exact enough, which is
// whenever the sum is far from overflow and from the subnormals; else in FP64.
template <int N>
__device__ __forceinline__ double squares(const float* v) {
  float s = 0.f, m = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf(v[i], v[i], s), m = fmaxf(m, fabsf(v[i]));
  if ((s > 1e-20f && s < 1e37f) || (s == 0.f && m == 0.f)) return double(s);
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) d = fma(double(v[i]), double(v[i]), d);
  return d;
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
  else return static_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void unpack(const uint4& q, float* v) {
  if constexpr (BF16) {
    v[0] = bf16lo(q.x), v[1] = bf16hi(q.x), v[2] = bf16lo(q.y), v[3] = bf16hi(q.y);
    v[4] = bf16lo(q.z), v[5] = bf16hi(q.z), v[6] = bf16lo(q.w), v[7] = bf16hi(q.w);
  } else {
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
  }
}

// Elements before the first 16-byte boundary of p (at most n).
template <bool BF16>
__device__ __forceinline__ int64_t head_of(const void* p, int64_t n) {
  constexpr int es = BF16 ? 2 : 4;
  const int64_t h = int64_t((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / es;
  return h < n ? h : n;
}

// Sum of squares of elements [0, n) at p; whole vectors from the first 16-byte boundary on,
// the ends element by element.
template <bool BF16>
__device__ double chunk_squares(const void* p, int64_t n) {
  // vectors in flight: a whole chunk of fp32 (311 MB: 54.7 -> 49.6 us against 4), but 4 of
  // bf16, whose eight values each cost registers (1.2 GB: 209 us, with 8 249)
  constexpr int N = BF16 ? 8 : 4, es = BF16 ? 2 : 4, U = BF16 ? 4 : 8;
  const int64_t head = head_of<BF16>(p, n), nv = (n - head) / N;
  const uint4* vp = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + head * es);
  double acc = 0.0;
  for (int64_t i0 = threadIdx.x; i0 < nv; i0 += U * kThreads) {
    uint4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) q[u] = i0 + u * kThreads < nv ? vp[i0 + u * kThreads] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[N];
      unpack<BF16>(q[u], v);
      acc += squares<N>(v);
    }
  }
  const int64_t rest = n - head - nv * N;
  if (threadIdx.x < head + rest) {
    const int64_t i = threadIdx.x < head ? threadIdx.x : nv * N + threadIdx.x;
    const double x = load1<BF16>(p, i);
    acc += x * x;
  }
  return acc;
}

// Sum over the CTA in a fixed order; every thread gets it.
__device__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x / 32] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) t += sh[w];
  __syncthreads();
  return t;
}

template <int N>
__global__ void __launch_bounds__(kThreads) sumsq_kernel(const __grid_constant__ Batch<N> b, double* part,
                                                         uint32_t* status) {
  pdl_trigger();
  if (status && blockIdx.x == 0 && threadIdx.x == 0) *status = 0u;  // this call's status word
  __shared__ double sh[kThreads / 32];
  double acc = 0.0;
  for (int c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const Tensor& t = b.t[find(b, c)];
    const int64_t at = int64_t(c - t.chunk0) * kChunk, n = min(kChunk, t.n - at);
    if (t.bf16) acc += chunk_squares<true>(static_cast<const uint16_t*>(t.src) + at, n);
    else acc += chunk_squares<false>(static_cast<const float*>(t.src) + at, n);
  }
  acc = block_sum(acc, sh);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

__device__ __forceinline__ double total_of(const double* part, int64_t n, double* sh) {
  double a = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) a += part[i];
  return block_sum(a, sh);
}

__global__ void __launch_bounds__(kThreads) total_kernel(const double* part, int64_t n, double* sumsq) {
  pdl_wait();
  pdl_trigger();
  __shared__ double sh[kThreads / 32];
  const double t = total_of(part, n, sh);
  if (threadIdx.x == 0) *sumsq = t;
}

template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t i, float x) {
  if constexpr (BF16) static_cast<uint16_t*>(p)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
  else static_cast<float*>(p)[i] = x;
}

template <bool BF16>
__device__ void chunk_scale(const void* src, void* dst, int64_t n, float coef) {
  constexpr int N = BF16 ? 8 : 4, es = BF16 ? 2 : 4, U = BF16 ? 4 : 8;
  if (((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15u) != 0) {
    // the two sides meet their 16-byte boundaries at different elements
    for (int64_t i = threadIdx.x; i < n; i += kThreads) store1<BF16>(dst, i, load1<BF16>(src, i) * coef);
    return;
  }
  const int64_t head = head_of<BF16>(src, n), nv = (n - head) / N;
  const uint4* vp = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(src) + head * es);
  uint4* vd = reinterpret_cast<uint4*>(static_cast<uint8_t*>(dst) + head * es);
  for (int64_t i0 = threadIdx.x; i0 < nv; i0 += U * kThreads) {
    uint4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kThreads < nv) q[u] = vp[i0 + u * kThreads];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * kThreads >= nv) break;
      float v[N];
      unpack<BF16>(q[u], v);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= coef;
      uint4 o;
      if constexpr (BF16)
        o = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
      else
        o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      vd[i0 + u * kThreads] = o;
    }
  }
  const int64_t rest = n - head - nv * N;
  if (threadIdx.x < head + rest) {
    const int64_t i = threadIdx.x < head ? threadIdx.x : nv * N + threadIdx.x;
    store1<BF16>(dst, i, load1<BF16>(src, i) * coef);
  }
}

// The same with the product taken in FP64: a coefficient below FP32's normal range (a norm of
// 1e38 and more, a tiny max_norm) has lost its bits there, though the product need not be small.
// No call for speed here: one element at a time.
template <bool BF16>
__device__ void chunk_scale_wide(const void* src, void* dst, int64_t n, double coef) {
#pragma unroll 1
  for (int64_t i = threadIdx.x; i < n; i += kThreads) store1<BF16>(dst, i, float(double(load1<BF16>(src, i)) * coef));
}

template <int N>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Batch<N> b, const double* sumsq,
                                                         const double* part, int64_t n_part, float max_norm,
                                                         float* norm_out, float* coef_out, uint32_t* status) {
  pdl_wait();
  pdl_trigger();
  __shared__ double sh[kThreads / 32];
  const double ss = sumsq ? *sumsq : total_of(part, n_part, sh);
  const double root = sqrt(ss);
  const float norm = float(root);
  // In FP32 (an FP64 division here costs calls of small tensors 2.6 of 13.6 us) where norm and
  // coefficient are in its range, else in FP64.
  float coef = isfinite(norm) ? fminf(max_norm / (norm + 1e-6f), 1.f) : 1.f;
  const bool wide = isfinite(root) && (!isfinite(norm) || coef < 0x1p-126f);
  double coef_wide = 1.0;
  if (wide) {
    coef_wide = fmin(double(max_norm) / (root + 1e-6), 1.0);
    coef = float(coef_wide);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (status) *status = 0u;
    if (norm_out) *norm_out = norm;
    if (coef_out) *coef_out = coef;
  }
  for (int c = b.chunks - 1 - int(blockIdx.x); c >= 0; c -= gridDim.x) {
    const Tensor& t = b.t[find(b, c)];
    if (coef == 1.f && t.src == t.dst) continue;  // in place and unchanged
    const int64_t at = int64_t(c - t.chunk0) * kChunk, n = min(kChunk, t.n - at);
    const uint8_t* src = static_cast<const uint8_t*>(t.src) + at * (t.bf16 ? 2 : 4);
    uint8_t* dst = static_cast<uint8_t*>(t.dst) + at * (t.bf16 ? 2 : 4);
    if (wide) t.bf16 ? chunk_scale_wide<true>(src, dst, n, coef_wide) : chunk_scale_wide<false>(src, dst, n, coef_wide);
    else t.bf16 ? chunk_scale<true>(src, dst, n, coef) : chunk_scale<false>(src, dst, n, coef);
  }
}

// The descriptors of one launch, and the CTAs it gets.
template <int N>
int fill(Batch<N>& b, const dspark_tensor_t* t, int64_t count) {
  b.count = int32_t(count);
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) {
    b.t[i] = Tensor{t[i].src, t[i].dst, t[i].n, t[i].dtype == DSPARK_BF16, int32_t(chunks)};
    chunks += (t[i].n + kChunk - 1) / kChunk;
  }
  b.chunks = int32_t(chunks);
  return int(std::max<int64_t>(1, std::min<int64_t>(chunks, kGrid)));
}

inline double* partials_of(void* ws) { return reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + 256); }

// One launch over `count` tensors; *grid: its CTAs (and partial sums).
template <int N>
cudaError_t sumsq_batch(const dspark_tensor_t* t, int64_t count, double* part, uint32_t* status, cudaStream_t s,
                        int* grid) {
  Batch<N> b;
  *grid = fill(b, t, count);
  sumsq_kernel<N><<<*grid, kThreads, 0, s>>>(b, part, status);
  return cudaGetLastError();
}

template <int N>
cudaError_t scale_batch(const dspark_tensor_t* t, int64_t count, bool first_of_call, const double* sumsq,
                        const double* part, int64_t partials, float max_norm, float* norm, float* coef,
                        uint32_t* status, cudaStream_t s) {
  Batch<N> b;
  const int grid = fill(b, t, count);
  PdlLaunch l(grid, kThreads, 0, s);
  if (first_of_call) l.cfg.numAttrs = 0;  // after all work before the call
  return cudaLaunchKernelEx(&l.cfg, scale_kernel<N>, b, sumsq, part, partials, max_norm, norm, coef, status);
}

}  // namespace

cudaError_t launch_sumsq(const dspark_tensor_t* t, int64_t count, void* ws, cudaStream_t s, int64_t* partials) {
  int64_t at = 0;
  for (int64_t i = 0; i < count; i += kMaxTensors) {
    const int64_t n = std::min<int64_t>(kMaxTensors, count - i);
    uint32_t* status = i == 0 ? static_cast<uint32_t*>(ws) : nullptr;
    auto run = n <= 16 ? sumsq_batch<16> : n <= 256 ? sumsq_batch<256> : sumsq_batch<kMaxTensors>;
    int grid = 0;
    const cudaError_t e = run(t + i, n, partials_of(ws) + at, status, s, &grid);
    if (e != cudaSuccess) return e;
    at += grid;
  }
  *partials = at;
  return cudaSuccess;
}

cudaError_t launch_total(const void* ws, int64_t partials, double* sumsq, cudaStream_t s) {
  PdlLaunch l(1, kThreads, 0, s);
  return cudaLaunchKernelEx(&l.cfg, total_kernel,
                            reinterpret_cast<const double*>(static_cast<const uint8_t*>(ws) + 256), partials, sumsq);
}

cudaError_t launch_scale(const dspark_tensor_t* t, int64_t count, const double* sumsq, int64_t partials,
                         float max_norm, float* norm, float* coef, void* ws, cudaStream_t s) {
  for (int64_t i = 0; i < count; i += kMaxTensors) {
    const int64_t n = std::min<int64_t>(kMaxTensors, count - i);
    const bool head = i == 0;
    auto run = n <= 16 ? scale_batch<16> : n <= 256 ? scale_batch<256> : scale_batch<kMaxTensors>;
    const cudaError_t e = run(t + i, n, sumsq && head, sumsq, partials_of(ws), partials, max_norm,
                              head ? norm : nullptr, head ? coef : nullptr,
                              sumsq && head ? static_cast<uint32_t*>(ws) : nullptr, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace clip
}  // namespace dspark
