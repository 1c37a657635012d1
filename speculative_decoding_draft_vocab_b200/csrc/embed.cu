// Scaled embedding lookup, and its gradient summed over sorted ids.
//   lookup     out_r = scale * table[id_r], rounded once
//   gradient   dtable_i = scale * sum_{r: id_r = i} dout_r
// The gradient sorts (id, row) by id with a stable radix sort, so an id's rows come in row
// order, then sums windows of consecutive sorted rows.  A segment (the rows of one id) that
// lies inside a window is finished there; one that crosses a window's end leaves a partial
// sum, and the partial sums of a segment are added in window order.  Every sum has a fixed
// order whatever runs when: no floating-point atomics.
#include <cuda_bf16.h>

#include <algorithm>

#include "pdl.cuh"
#include "ptx.cuh"
#include "train.cuh"

namespace dspark {
namespace embed {
namespace {

// 16 bytes of a row as FP32 values, and back (one rounding).
template <bool F32>
struct Vec;
template <>
struct Vec<true> {
  static constexpr int N = 4;
  __device__ static void get(const uint4& q, float* v) {
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
  }
  __device__ static uint4 put(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Vec<false> {
  static constexpr int N = 8;
  __device__ static void get(const uint4& q, float* v) {
    v[0] = bf16lo(q.x), v[1] = bf16hi(q.x), v[2] = bf16lo(q.y), v[3] = bf16hi(q.y);
    v[4] = bf16lo(q.z), v[5] = bf16hi(q.z), v[6] = bf16lo(q.w), v[7] = bf16hi(q.w);
  }
  __device__ static uint4 put(const float* v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};

__device__ __forceinline__ bool dropped(const dspark_embed_problem_t& p, int64_t r) {
  return p.valid != nullptr && p.valid[r] == 0;
}
__device__ __forceinline__ bool in_table(const dspark_embed_problem_t& p, int64_t id) { return id >= 0 && id < p.Vt; }

// Whether any row that counts has an id outside the table; by one CTA, which also makes the
// status word this call's.
__device__ void check_ids(const dspark_embed_problem_t& p, WsEmbedHeader* hdr) {
  int bad = 0;
  for (int64_t r = threadIdx.x; r < p.R; r += blockDim.x)
    if (!dropped(p, r) && !in_table(p, p.ids[r])) bad = 1;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) hdr->status = bad ? kFlagIdOutOfRange : 0u;
}

// ------------------------------------------------------------------ lookup
// A warp takes one row's run of 4 x 32 16-byte vectors at a time; the last CTA checks the ids.
constexpr int kFwdVecs = 4;

template <bool F32>
__global__ void __launch_bounds__(256) lookup_kernel(const FwdArgs a) {
  if (blockIdx.x == gridDim.x - 1) {
    check_ids(a.p, a.hdr);
    return;
  }
  using V = Vec<F32>;
  const int lane = threadIdx.x & 31;
  const int64_t nv = a.p.D / V::N, parts = (nv + 32 * kFwdVecs - 1) / (32 * kFwdVecs);
  const int64_t items = a.p.R * parts, step = int64_t(gridDim.x - 1) * 8;
  for (int64_t w = int64_t(blockIdx.x) * 8 + threadIdx.x / 32; w < items; w += step) {
    const int64_t r = w / parts, j0 = (w - r * parts) * 32 * kFwdVecs + lane;
    const int64_t id = a.p.ids[r];
    const bool live = !dropped(a.p, r) && in_table(a.p, id);
    const uint4* src = static_cast<const uint4*>(a.table) + (live ? id : 0) * (a.table_ld / V::N);
    uint4* dst = static_cast<uint4*>(a.out) + r * (a.out_ld / V::N);
    uint4 q[kFwdVecs];
#pragma unroll
    for (int k = 0; k < kFwdVecs; ++k)
      if (live && j0 + 32 * k < nv) q[k] = src[j0 + 32 * k];
#pragma unroll
    for (int k = 0; k < kFwdVecs; ++k) {
      if (j0 + 32 * k >= nv) break;
      uint4 o = make_uint4(0u, 0u, 0u, 0u);
      if (live) {
        float v[V::N];
        V::get(q[k], v);
#pragma unroll
        for (int i = 0; i < V::N; ++i) v[i] *= a.p.scale;
        o = V::put(v);
      }
      dst[j0 + 32 * k] = o;
    }
  }
}

// ------------------------------------------------------------------ sort
// One radix pass over digit [shift, shift + kDigitBits) is two kernels: each CTA counts the
// digits of its run of rows; then each CTA finds where its rows of each digit go (all
// smaller digits, the same digit in the CTAs before it) and moves them in order.  The first
// pass reads the ids themselves.
struct Pass {
  int shift, first;
  const uint32_t* key_in;
  const uint32_t* row_in;
  uint32_t* key_out;
  uint32_t* row_out;
};

__device__ __forceinline__ uint32_t load_key(const BwdArgs& a, const Pass& ps, int64_t i) {
  if (!ps.first) return ps.key_in[i];
  const int64_t id = a.p.ids[i];
  return !dropped(a.p, i) && in_table(a.p, id) ? uint32_t(id) : uint32_t(a.p.Vt);
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(const BwdArgs a, const Pass ps) {
  pdl_wait();
  pdl_trigger();
  if (int(blockIdx.x) == a.plan.ctas) {  // first pass only: one CTA more
    check_ids(a.p, a.ws.hdr);
    return;
  }
  __shared__ uint32_t c[kDigits];
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) c[d] = 0;
  __syncthreads();
  const int64_t i0 = int64_t(blockIdx.x) * a.plan.run, i1 = min(i0 + a.plan.run, a.p.R);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads)
    atomicAdd(&c[(load_key(a, ps, i) >> ps.shift) & (kDigits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) a.ws.counts[size_t(blockIdx.x) * kDigits + d] = c[d];
}

__global__ void __launch_bounds__(kSortThreads) move_kernel(const BwdArgs a, const Pass ps) {
  pdl_wait();
  pdl_trigger();
  static_assert(kSortThreads == kDigits, "one thread per digit");
  constexpr int kWarps = kSortThreads / 32;
  __shared__ uint32_t base[kDigits];
  __shared__ uint16_t cnt[kWarps][kDigits];
  __shared__ uint32_t wsum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  {  // thread = digit
    uint32_t before = 0, total = 0;
    for (int c = 0; c < a.plan.ctas; ++c) {
      const uint32_t n = a.ws.counts[size_t(c) * kDigits + tid];
      if (c < int(blockIdx.x)) before += n;
      total += n;
    }
    uint32_t incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    uint32_t lower = 0;
    for (int w = 0; w < warp; ++w) lower += wsum[w];
    base[tid] = lower + incl - total + before;
  }
  const int64_t i0 = int64_t(blockIdx.x) * a.plan.run, i1 = min(i0 + a.plan.run, a.p.R);
  for (int64_t c0 = i0; c0 < i1; c0 += kSortChunk) {
    for (int d = lane; d < kDigits; d += 32) cnt[warp][d] = 0;
    __syncwarp();
    uint32_t key[kSortItems], row[kSortItems], rank[kSortItems];
    // a warp's items are 32 * kSortItems consecutive rows, taken 32 at a time: row order
    const int64_t w0 = c0 + warp * 32 * kSortItems + lane;
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
      const int64_t i = w0 + 32 * k;
      const bool on = i < i1;
      key[k] = on ? load_key(a, ps, i) : 0u;
      row[k] = on ? (ps.first ? uint32_t(i) : ps.row_in[i]) : 0u;
    }
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
      const bool on = w0 + 32 * k < i1;
      const uint32_t d = on ? (key[k] >> ps.shift) & (kDigits - 1) : uint32_t(kDigits);
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      const int lead = __ffs(same) - 1;
      if (on) rank[k] = cnt[warp][d] + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (on && lane == lead) cnt[warp][d] += uint16_t(__popc(same));
      __syncwarp();
    }
    __syncthreads();
    {  // thread = digit: the warps' counts become offsets within the digit
      uint32_t at = 0;
      for (int w = 0; w < kWarps; ++w) {
        const uint32_t n = cnt[w][tid];
        cnt[w][tid] = uint16_t(at);
        at += n;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kSortItems; ++k) {
        if (w0 + 32 * k >= i1) continue;
        const uint32_t d = (key[k] >> ps.shift) & (kDigits - 1);
        const uint32_t to = base[d] + cnt[warp][d] + rank[k];
        ps.key_out[to] = key[k];
        ps.row_out[to] = row[k];
      }
      __syncthreads();
      base[tid] += at;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ zero rows
template <bool TF32>
__global__ void __launch_bounds__(256) zero_kernel(const BwdArgs a) {
  pdl_trigger();
  constexpr int N = Vec<TF32>::N;
  const int64_t nv = a.p.D / N, total = a.p.Vt * nv, ldv = a.dtable_ld / N;
  uint4* t = static_cast<uint4*>(a.dtable);
  if (ldv == nv) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) t[i] = make_uint4(0u, 0u, 0u, 0u);
  } else {
    for (int64_t r = blockIdx.x; r < a.p.Vt; r += gridDim.x)
      for (int64_t j = threadIdx.x; j < nv; j += 256) t[r * ldv + j] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// ------------------------------------------------------------------ sums
// dtable row `id`, the vector's columns from `col`: scale * acc, stored or added.
template <bool TF32, int N>
__device__ __forceinline__ void write_row(const BwdArgs& a, uint32_t id, int64_t col, const float* acc) {
  if constexpr (TF32) {
    float* d = static_cast<float*>(a.dtable) + size_t(id) * a.dtable_ld + col;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      float4 o = make_float4(acc[i] * a.p.scale, acc[i + 1] * a.p.scale, acc[i + 2] * a.p.scale, acc[i + 3] * a.p.scale);
      float4* at = reinterpret_cast<float4*>(d + i);
      if (a.accumulate) {
        const float4 old = *at;
        o.x += old.x, o.y += old.y, o.z += old.z, o.w += old.w;
      }
      *at = o;
    }
  } else {
    uint16_t* d = static_cast<uint16_t*>(a.dtable) + size_t(id) * a.dtable_ld + col;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      *reinterpret_cast<uint2*>(d + i) = make_uint2(pack_bf16(acc[i] * a.p.scale, acc[i + 1] * a.p.scale),
                                                    pack_bf16(acc[i + 2] * a.p.scale, acc[i + 3] * a.p.scale));
    }
  }
}

// A warp sums one window's rows over 32 vectors of columns.
template <bool F32, bool TF32>
__global__ void __launch_bounds__(256) sum_kernel(const BwdArgs a, const uint32_t* key, const uint32_t* row) {
  pdl_wait();
  pdl_trigger();
  using V = Vec<F32>;
  constexpr int N = V::N, U = 8;  // rows in flight
  const int lane = threadIdx.x & 31;
  const int64_t nv = a.p.D / N, blocks = (nv + 31) / 32;
  const uint32_t none = uint32_t(a.p.Vt);
  const int64_t w = int64_t(blockIdx.x) * 8 + threadIdx.x / 32;
  if (w >= a.plan.windows * blocks) return;
  const int64_t win = w / blocks, j = (w - win * blocks) * 32 + lane;
  const bool on = j < nv;
  const int64_t p0 = win * a.plan.window, p1 = min(p0 + a.plan.window, a.p.R);
  const uint32_t prev = p0 > 0 ? key[p0 - 1] : ~0u, next = p1 < a.p.R ? key[p1] : ~0u;
  const uint4* src = static_cast<const uint4*>(a.dout) + j;
  const int64_t ldv = a.dout_ld / N;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  uint32_t cur = key[p0];
  bool head = cur == prev;  // the segment began in an earlier window
  auto partial = [&](int slot) {
    float* d = a.ws.part + (size_t(win) * 2 + slot) * a.p.D + j * N;
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(d + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
  };
  for (int64_t c0 = p0; c0 < p1 && cur != none; c0 += 32) {
    const int n = int(min(int64_t(32), p1 - c0));
    const uint32_t k_l = lane < n ? key[c0 + lane] : none;
    const uint32_t r_l = lane < n ? row[c0 + lane] : 0u;
    for (int u0 = 0; u0 < n; u0 += U) {
      uint4 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t k = __shfl_sync(0xffffffffu, k_l, (u0 + u) & 31), r = __shfl_sync(0xffffffffu, r_l, (u0 + u) & 31);
        q[u] = make_uint4(0u, 0u, 0u, 0u);
        if (on && u0 + u < n && k != none) q[u] = src[int64_t(r) * ldv];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u0 + u >= n) break;
        const uint32_t k = __shfl_sync(0xffffffffu, k_l, u0 + u);
        if (k != cur) {  // the whole warp: the segment before this row is complete
          if (on) {
            if (head) partial(0);
            else write_row<TF32, N>(a, cur, j * N, acc);
          }
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] = 0.f;
          cur = k, head = false;
        }
        float v[N];
        V::get(q[u], v);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += v[i];
      }
    }
  }
  if (!on || cur == none) return;
  if (head) partial(0);
  else if (cur == next) partial(1);
  else write_row<TF32, N>(a, cur, j * N, acc);
}

// The segments that cross windows: the window a segment begins in adds the parts that the
// windows after it left.
template <bool F32, bool TF32>
__global__ void __launch_bounds__(256) join_kernel(const BwdArgs a, const uint32_t* key) {
  pdl_wait();
  pdl_trigger();
  constexpr int N = Vec<F32>::N;
  const int lane = threadIdx.x & 31;
  const int64_t nv = a.p.D / N, blocks = (nv + 31) / 32;
  const int64_t w = int64_t(blockIdx.x) * 8 + threadIdx.x / 32;
  if (w >= a.plan.windows * blocks) return;
  const int64_t win = w / blocks, j = (w - win * blocks) * 32 + lane;
  const int64_t p0 = win * a.plan.window, p1 = p0 + a.plan.window;
  if (p1 >= a.p.R) return;
  const uint32_t id = key[p1 - 1];
  if (id == uint32_t(a.p.Vt) || key[p1] != id) return;                 // nothing goes on
  if (p0 > 0 && key[p0 - 1] == id) return;                            // nor begins here
  // the last window that begins with the id (the keys are sorted: bisection)
  int64_t last = win + 1, past = a.plan.windows;
  while (past - last > 1) {
    const int64_t mid = (last + past) / 2;
    if (key[mid * a.plan.window] == id) last = mid;
    else past = mid;
  }
  if (j >= nv) return;
  float acc[N];
  const float* src = a.ws.part + (size_t(win) * 2 + 1) * a.p.D + j * N;
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = src[i];
#pragma unroll 4
  for (int64_t x = win + 1; x <= last; ++x) {
    const float* q = a.ws.part + size_t(x) * 2 * a.p.D + j * N;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(q + i);
      acc[i] += f.x, acc[i + 1] += f.y, acc[i + 2] += f.z, acc[i + 3] += f.w;
    }
  }
  write_row<TF32, N>(a, id, j * N, acc);
}

template <bool F32, bool TF32>
cudaError_t sums(const BwdArgs& a, const uint32_t* key, const uint32_t* row, cudaStream_t s) {
  const int64_t nv = a.p.D / Vec<F32>::N, warps = a.plan.windows * ((nv + 31) / 32);
  PdlLaunch l((warps + 7) / 8, 256, 0, s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, sum_kernel<F32, TF32>, a, key, row);
  if (e != cudaSuccess) return e;
  PdlLaunch l2((warps + 7) / 8, 256, 0, s);
  return cudaLaunchKernelEx(&l2.cfg, join_kernel<F32, TF32>, a, key);
}

}  // namespace

cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t s) {
  const bool f32 = a.p.dtype == DSPARK_F32;
  const int64_t nv = a.p.D / (f32 ? 4 : 8), parts = (nv + 32 * kFwdVecs - 1) / (32 * kFwdVecs);
  const int64_t ctas = std::min<int64_t>((a.p.R * parts + 7) / 8, 148 * 8);
  if (f32) lookup_kernel<true><<<unsigned(ctas + 1), 256, 0, s>>>(a);
  else lookup_kernel<false><<<unsigned(ctas + 1), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_bwd(const BwdArgs& a, cudaStream_t s) {
  cudaError_t e;
  const bool f32 = a.p.dtype == DSPARK_F32;
  if (!a.accumulate) {
    if (a.table_f32) zero_kernel<true><<<148 * 8, 256, 0, s>>>(a);
    else zero_kernel<false><<<148 * 8, 256, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  int from = 0;
  for (int k = 0; k < a.plan.passes; ++k) {
    Pass ps{k * kDigitBits, k == 0, a.ws.key[from], a.ws.row[from], a.ws.key[1 - from], a.ws.row[1 - from]};
    if (k == 0 && a.accumulate) {  // the first kernel of the call waits for all work before it
      count_kernel<<<unsigned(a.plan.ctas + 1), kSortThreads, 0, s>>>(a, ps);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    } else {
      PdlLaunch l(a.plan.ctas + (k == 0), kSortThreads, 0, s);
      if ((e = cudaLaunchKernelEx(&l.cfg, count_kernel, a, ps)) != cudaSuccess) return e;
    }
    PdlLaunch l(a.plan.ctas, kSortThreads, 0, s);
    if ((e = cudaLaunchKernelEx(&l.cfg, move_kernel, a, ps)) != cudaSuccess) return e;
    from = 1 - from;
  }
  const uint32_t *key = a.ws.key[from], *row = a.ws.row[from];
  if (f32) return a.table_f32 ? sums<true, true>(a, key, row, s) : sums<true, false>(a, key, row, s);
  return a.table_f32 ? sums<false, true>(a, key, row, s) : sums<false, false>(a, key, row, s);
}

}  // namespace embed
}  // namespace dspark
