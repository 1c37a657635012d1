// Scaled embedding lookup, and its gradient summed over sorted ids.
//   lookup     out_r = scale * table[id_r], rounded once
//   gradient   dtable_i = scale * sum_{r: id_r = i} dout_r
// The gradient sorts (id, row) by id with a stable radix sort, so an id's rows come in row
// order, then sums windows of consecutive sorted rows.  A segment (the rows of one id) that
// lies inside a window is finished there; one that crosses a window's end leaves a partial
// sum, and the partial sums of a segment are added in window order.  Every sum has an order
// that the sizes and the ids fix, whatever runs when.  The one floating-point atomic is the
// addition to an accumulated table, one per element and call.
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
// status word this call's.  Eight rows per thread in flight.
__device__ void check_ids(const dspark_embed_problem_t& p, WsEmbedHeader* hdr) {
  constexpr int U = 8;
  int bad = 0;
  for (int64_t r0 = threadIdx.x; r0 < p.R; r0 += U * blockDim.x) {
    int64_t id[U];
    uint8_t on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * blockDim.x;
      id[u] = r < p.R ? p.ids[r] : 0;
      on[u] = p.valid && r < p.R ? p.valid[r] : 1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) bad |= on[u] && !in_table(p, id[u]);
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) hdr->status = bad ? kFlagIdOutOfRange : 0u;
}

// ------------------------------------------------------------------ lookup
// Whether the ids are checked by one CTA more, beside the lookup (its time, about 1.2 us per
// 2048 rows, is then hidden by rows of 2 KB and more, or short anyway), or by the lookup's own
// threads, behind a kernel that clears the status word.
inline bool check_beside(const dspark_embed_problem_t& p) {
  return p.R <= 8192 || p.D * (p.dtype == DSPARK_F32 ? 4 : 2) >= 2048;
}

__global__ void clear_status_kernel(WsEmbedHeader* hdr) {
  pdl_trigger();
  if (threadIdx.x == 0) hdr->status = 0u;
}

template <bool F32>
__device__ __forceinline__ uint4 scaled(const uint4& q, float scale) {
  using V = Vec<F32>;
  float v[V::N];
  V::get(q, v);
#pragma unroll
  for (int i = 0; i < V::N; ++i) v[i] *= scale;
  return V::put(v);
}

// Rows of 32 vectors and more: a warp takes one row's run of 2 x 32 16-byte vectors at a time.
// Shorter rows: a thread takes two vectors, wherever in the rows they fall, so that no lane
// idles.
constexpr int kFwdVecs = 2;

template <bool F32, bool NARROW>
__global__ void __launch_bounds__(256, 8) lookup_kernel(const FwdArgs a, const int beside) {
  if (beside && blockIdx.x == gridDim.x - 1) {
    check_ids(a.p, a.hdr);
    return;
  }
  pdl_wait();
  using V = Vec<F32>;
  const int ctas = int(gridDim.x) - beside;
  const int64_t nv = a.p.D / V::N, ldt = a.table_ld / V::N, ldo = a.out_ld / V::N;
  const uint4* table = static_cast<const uint4*>(a.table);
  uint4* out = static_cast<uint4*>(a.out);
  // the row's place in the table, or -1; its first thread reports an id outside
  auto place = [&](int64_t r, bool first) -> int64_t {
    const int64_t id = a.p.ids[r];
    if (dropped(a.p, r)) return -1;
    if (in_table(a.p, id)) return id;
    if (!beside && first) atomicOr(&a.hdr->status, kFlagIdOutOfRange);
    return -1;
  };
  if constexpr (NARROW) {
    const int64_t total = a.p.R * nv, step = int64_t(ctas) * 256;
    const uint32_t n = uint32_t(nv);
    for (int64_t i0 = int64_t(blockIdx.x) * 256 + threadIdx.x; i0 < total; i0 += kFwdVecs * step) {
      uint4 q[kFwdVecs];
      int64_t to[kFwdVecs];
#pragma unroll
      for (int k = 0; k < kFwdVecs; ++k) {
        const int64_t i = i0 + k * step;
        q[k] = make_uint4(0u, 0u, 0u, 0u);
        to[k] = -1;
        if (i >= total) continue;
        const int64_t r = uint32_t(i) / n, j = i - r * n;  // total is below 2^29: rows below 2^24, vectors below 32
        const int64_t id = place(r, j == 0);
        to[k] = r * ldo + j;
        if (id >= 0) q[k] = table[id * ldt + j];
      }
#pragma unroll
      for (int k = 0; k < kFwdVecs; ++k)
        if (to[k] >= 0) __stcs(out + to[k], scaled<F32>(q[k], a.p.scale));
    }
  } else {
    const int lane = threadIdx.x & 31;
    const int64_t parts = (nv + 32 * kFwdVecs - 1) / (32 * kFwdVecs);
    const int64_t items = a.p.R * parts, step = int64_t(ctas) * 8;
    for (int64_t w = int64_t(blockIdx.x) * 8 + threadIdx.x / 32; w < items; w += step) {
      const int64_t r = w / parts, j0 = (w - r * parts) * 32 * kFwdVecs + lane;
      const int64_t id = place(r, j0 == 0);
      const bool live = id >= 0;
      const uint4* src = table + (live ? id : 0) * ldt;
      uint4* dst = out + r * ldo;
      uint4 q[kFwdVecs];
#pragma unroll
      for (int k = 0; k < kFwdVecs; ++k)
        if (live && j0 + 32 * k < nv) q[k] = src[j0 + 32 * k];
#pragma unroll
      for (int k = 0; k < kFwdVecs; ++k) {
        if (j0 + 32 * k >= nv) break;
        const uint4 o = live ? scaled<F32>(q[k], a.p.scale) : make_uint4(0u, 0u, 0u, 0u);
        __stcs(dst + j0 + 32 * k, o);  // written once: the table's rows keep their place in L2
      }
    }
  }
}

template <bool F32>
cudaError_t lookup(const FwdArgs& a, cudaStream_t s) {
  const int64_t nv = a.p.D / Vec<F32>::N;
  const bool narrow = nv < 32, beside = check_beside(a.p);
  const int64_t parts = (nv + 32 * kFwdVecs - 1) / (32 * kFwdVecs);
  const int64_t work = narrow ? (a.p.R * nv + 511) / 512 : (a.p.R * parts + 7) / 8;
  PdlLaunch l(std::min<int64_t>(work, 148 * 8) + beside, 256, 0, s);
  if (beside) {
    l.cfg.numAttrs = 0;  // the call's only kernel: after all work before it
  } else {
    clear_status_kernel<<<1, 32, 0, s>>>(a.hdr);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return narrow ? cudaLaunchKernelEx(&l.cfg, lookup_kernel<F32, true>, a, int(beside))
                : cudaLaunchKernelEx(&l.cfg, lookup_kernel<F32, false>, a, int(beside));
}

// ------------------------------------------------------------------ zero rows
// The table rows that no id touches.  While the ids are sorted, what is touched is not known
// and the memory is idle: the sorting kernels' spare CTAs zero the first plan.fill rows
// whatever their ids (a touched one is written again later); the sums' kernel zeroes the
// others, looking each row up in the sorted keys.  (8192 rows, table 151936 x 256 FP32: all
// rows beside the sort 45.5 us, all beside the sums 53.9, 64 MB beside the sort 41.4; a share
// beside the joins as well 45.5.)  The zeros are streamed past L2, which holds the keys and
// the partial sums.
template <bool TF32>
__device__ void zero_rows(const BwdArgs& a, int64_t r0, int64_t r1, int64_t thread, int64_t threads) {
  constexpr int N = Vec<TF32>::N;
  const int64_t nv = a.p.D / N, ldv = a.dtable_ld / N;
  uint4* t = static_cast<uint4*>(a.dtable);
  if (ldv == nv) {
    for (int64_t i = r0 * nv + thread; i < r1 * nv; i += threads) __stcs(t + i, make_uint4(0u, 0u, 0u, 0u));
  } else {
    for (int64_t i = thread; i < (r1 - r0) * nv; i += threads) {
      const int64_t r = i / nv;
      __stcs(t + (r0 + r) * ldv + (i - r * nv), make_uint4(0u, 0u, 0u, 0u));
    }
  }
}

// CTA `cta` of `ctas` zeroes its share of part `part` of `parts` of the first plan.fill rows.
__device__ __forceinline__ void zero_share(const BwdArgs& a, int part, int parts, int cta, int ctas) {
  const int64_t r0 = a.plan.fill * part / parts, r1 = a.plan.fill * (part + 1) / parts;
  const int64_t thread = int64_t(cta) * blockDim.x + threadIdx.x, threads = int64_t(ctas) * blockDim.x;
  if (a.table_f32) zero_rows<true>(a, r0, r1, thread, threads);
  else zero_rows<false>(a, r0, r1, thread, threads);
}

// ------------------------------------------------------------------ sort
// Keys are the ids, Vt for rows that do not count; 9-bit digits, least first.  Ranks within a
// warp come from ballots, in row order, so every pass is stable.
__device__ __forceinline__ uint32_t key_of(const BwdArgs& a, int64_t i, bool& bad) {
  const int64_t id = a.p.ids[i];
  if (dropped(a.p, i)) return uint32_t(a.p.Vt);
  if (in_table(a.p, id)) return uint32_t(id);
  bad = true;
  return uint32_t(a.p.Vt);
}

// Ranks of a warp's items among the earlier ones of the same digit; `cnt`: its digit counts.
template <int ITEMS>
__device__ __forceinline__ void warp_ranks(const uint32_t (&digit)[ITEMS], uint16_t* cnt, uint32_t (&rank)[ITEMS],
                                           int lane) {
  for (int d = lane; d < kDigits / 2; d += 32) reinterpret_cast<uint32_t*>(cnt)[d] = 0;
  __syncwarp();
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    uint32_t same = 0xffffffffu;  // the lanes with this digit, bit by bit
#pragma unroll
    for (int b = 0; b <= kDigitBits; ++b) {
      const bool one = (digit[k] >> b) & 1u;
      const uint32_t m = __ballot_sync(0xffffffffu, one);
      same &= one ? m : ~m;
    }
    const bool on = digit[k] < kDigits;
    if (on) rank[k] = cnt[digit[k]] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (on && lane == __ffs(same) - 1) cnt[digit[k]] += uint16_t(__popc(same));
    __syncwarp();
  }
}

// Up to kRankRows rows: a row's place is the number of rows before it in the order, and
// every row can count that for itself.  kRankThreads / 32 warps each take a stretch of the keys
// (in shared memory, four to a load) for the CTA's 32 rows, one per lane.  R^2 comparisons,
// spread over the whole GPU and without any exchange (the gradient of 448 rows into a table of
// 256 columns takes 10.2 us so, 17.4 with the cluster's sort; of 4096 rows 14.3 and 20.1; of
// 8192 rows 24.5 and 23.2); the other CTAs zero table rows meanwhile.
__global__ void __launch_bounds__(kRankThreads) rank_kernel(const BwdArgs a) {
  pdl_trigger();
  const int R = int(a.p.R), ranking = (R + 31) / 32;
  if (int(blockIdx.x) >= ranking) {
    zero_share(a, 0, 1, int(blockIdx.x) - ranking, int(gridDim.x) - ranking);
    return;
  }
  extern __shared__ uint4 smem_rank[];
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem_rank);  // R rounded up to 4, then the counts
  constexpr int kWarps = kRankThreads / 32;
  __shared__ uint32_t count[kWarps][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  const int padded = (R + 3) / 4 * 4;
#pragma unroll 8
  for (int i = tid; i < padded; i += kRankThreads) keys[i] = i < R ? key_of(a, i, bad) : ~0u;
  const int any_bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && tid == 0) a.ws.hdr->status = any_bad ? kFlagIdOutOfRange : 0u;
  const int row = int(blockIdx.x) * 32 + lane;
  const uint32_t key = row < R ? keys[row] : 0u;
  // before row: every earlier row with a key not above, every later one with a key below
  const int quads = padded / 4, per = (quads + kWarps - 1) / kWarps;
  const int q0 = warp * per, q1 = min(q0 + per, quads);
  const int own = int(blockIdx.x) * 8;  // the quads [own, own + 8) hold the CTA's rows themselves
  uint32_t n = 0;
  const uint32_t upto = key + 1;  // (keys are at most 2^30)
#pragma unroll 8
  for (int q = q0; q < min(q1, own); ++q) {
    const uint4 k = reinterpret_cast<const uint4*>(keys)[q];
    n += (k.x < upto) + (k.y < upto) + (k.z < upto) + (k.w < upto);
  }
  for (int q = max(q0, own); q < min(q1, own + 8); ++q) {
    const uint4 k = reinterpret_cast<const uint4*>(keys)[q];
    n += (k.x < key + (4 * q < row)) + (k.y < key + (4 * q + 1 < row)) + (k.z < key + (4 * q + 2 < row)) +
         (k.w < key + (4 * q + 3 < row));
  }
#pragma unroll 8
  for (int q = max(q0, own + 8); q < q1; ++q) {
    const uint4 k = reinterpret_cast<const uint4*>(keys)[q];
    n += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
  }
  count[warp][lane] = n;
  __syncthreads();
  if (warp == 0 && row < R) {
    uint32_t at = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) at += count[w][lane];
    a.ws.key[0][at] = key;
    a.ws.row[0][at] = uint32_t(row);
  }
}

cudaError_t rank_sort(const BwdArgs& a, cudaStream_t s) {
  const size_t smem = size_t(a.p.R + 3) / 4 * 16;
  const int spare = fill_ctas(a.plan, a.p.D * (a.table_f32 ? 4 : 2), 1, 148 * 4);
  PdlLaunch l((a.p.R + 31) / 32 + spare, kRankThreads, smem, s);
  l.cfg.numAttrs = 0;  // the first kernel of the call waits for all work before it
  return cudaLaunchKernelEx(&l.cfg, rank_kernel, a);
}

// More rows, up to kSmallRows: one cluster of eight CTAs keeps them in registers, one, two or four
// per thread, and moves them through its distributed shared memory; the other clusters zero
// table rows meanwhile.  (8192 rows: 20 us in one CTA, whose issue slots the ranking fills.)
struct SmallSort {
  uint64_t item[kSmallThreads * kSmallItems];  // key, row: one remote store each
  uint16_t cnt[kSmallThreads / 32][kDigits];
  uint32_t mine[kDigits];  // digit counts of this CTA, read by the others
  uint32_t wsum[kSmallThreads / 32];
  uint32_t bad;
};

__device__ __forceinline__ uint32_t ld_dsmem(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int ITEMS>
__global__ void __launch_bounds__(kSmallThreads) small_sort_kernel(const BwdArgs a) {
  pdl_trigger();
  if (blockIdx.x >= kSmallCtas) {  // whole clusters
    zero_share(a, 0, 1, int(blockIdx.x) - kSmallCtas, int(gridDim.x) - kSmallCtas);
    return;
  }
  extern __shared__ uint4 smem_small[];
  SmallSort& sm = *reinterpret_cast<SmallSort*>(smem_small);
  constexpr int kWarps = kSmallThreads / 32, CAP = kSmallThreads * ITEMS;  // rows per CTA
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = int(cluster_ctarank());
  const int l0 = warp * 32 * ITEMS + lane;  // a warp's items are consecutive rows, 32 at a time
  const int R = int(a.p.R);
  uint32_t key[ITEMS], row[ITEMS];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    row[k] = uint32_t(cta * CAP + l0 + 32 * k);
    key[k] = int(row[k]) < R ? key_of(a, row[k], bad) : ~0u;  // past the rows: last in every pass
  }
  const int any_bad = __syncthreads_or(bad);
  if (tid == 0) sm.bad = any_bad ? kFlagIdOutOfRange : 0u;
  for (int p = 0; p < a.plan.passes; ++p) {
    uint32_t digit[ITEMS], rank[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) digit[k] = (key[k] >> (p * kDigitBits)) & (kDigits - 1);
    warp_ranks<ITEMS>(digit, sm.cnt[warp], rank, lane);
    __syncthreads();
    // two threads per digit, sixteen warps each
    const int d = tid >> 1, half = tid & 1, w0 = half * (kWarps / 2);
    uint32_t own = 0;
#pragma unroll
    for (int w = 0; w < kWarps / 2; ++w) own += sm.cnt[w0 + w][d];
    const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
    if (half == 0) sm.mine[d] = own + other;
    cluster_sync();  // every CTA's counts are there, and its items in registers
    uint32_t before = 0, total = 0;
#pragma unroll
    for (int c = 0; c < kSmallCtas / 2; ++c) {
      const int from = half * (kSmallCtas / 2) + c;
      const uint32_t n = ld_dsmem(dsmem_map(smem_u32(&sm.mine[d]), uint32_t(from)));
      if (from < cta) before += n;
      total += n;
    }
    before += __shfl_xor_sync(0xffffffffu, before, 1);
    total += __shfl_xor_sync(0xffffffffu, total, 1);
    uint32_t incl = half ? total : 0u;  // a digit counts once, at its second thread
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) sm.wsum[warp] = incl;
    __syncthreads();
    uint32_t lower = lane < warp ? sm.wsum[lane] : 0u;
    lower = __reduce_add_sync(0xffffffffu, lower);
    uint32_t at = lower + incl - (half ? total : 0u) + before + (half ? other : 0u);
#pragma unroll
    for (int w = 0; w < kWarps / 2; ++w) {  // counts become places
      const uint32_t n = sm.cnt[w0 + w][d];
      sm.cnt[w0 + w][d] = uint16_t(at);
      at += n;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const uint32_t to = sm.cnt[warp][digit[k]] + rank[k];
      const uint32_t there = to / CAP, slot = to % CAP;
      asm volatile("st.shared::cluster.u64 [%0], %1;"
                   ::"r"(dsmem_map(smem_u32(&sm.item[slot]), there)), "l"(uint64_t(row[k]) << 32 | key[k]) : "memory");
    }
    if (p == 0 && cta == 0 && warp == 0) {  // the call's status from the eight CTAs'
      uint32_t f = lane < kSmallCtas ? ld_dsmem(dsmem_map(smem_u32(&sm.bad), uint32_t(lane))) : 0u;
      f = __reduce_or_sync(0xffffffffu, f);
      if (lane == 0) a.ws.hdr->status = f;
    }
    cluster_sync();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) key[k] = uint32_t(sm.item[l0 + 32 * k]), row[k] = uint32_t(sm.item[l0 + 32 * k] >> 32);
    // the next pass writes these places only after its first cluster barrier
  }
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int i = cta * CAP + l0 + 32 * k;
    if (i < R) a.ws.key[0][i] = key[k], a.ws.row[0][i] = row[k];
  }
}

template <int ITEMS>
cudaError_t small_sort(const BwdArgs& a, cudaStream_t s) {
  auto kern = small_sort_kernel<ITEMS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(SmallSort)));
  if (e != cudaSuccess) return e;
  const int spare =
      (fill_ctas(a.plan, a.p.D * (a.table_f32 ? 4 : 2), 1, 148 * 2) + kSmallCtas - 1) / kSmallCtas * kSmallCtas;
  PdlLaunch l(kSmallCtas + spare, kSmallThreads, sizeof(SmallSort), s, kSmallCtas);
  l.at[0].val.programmaticStreamSerializationAllowed = 0;  // the first kernel of the call waits for all work before it
  return cudaLaunchKernelEx(&l.cfg, kern, a);
}

// Still more rows: a pass is two kernels.  Each CTA counts the digits of its run of rows; then each
// CTA finds where its rows of each digit go (all smaller digits, the same digit in the CTAs
// before it) and moves them in order.  The first pass reads the ids themselves.
struct Pass {
  int shift, index;
  const uint32_t* key_in;
  const uint32_t* row_in;
  uint32_t* key_out;
  uint32_t* row_out;
};

__global__ void __launch_bounds__(kSortThreads) count_kernel(const BwdArgs a, const Pass ps) {
  pdl_wait();
  pdl_trigger();
  if (int(blockIdx.x) >= a.plan.ctas) {
    zero_share(a, 2 * ps.index, 2 * a.plan.passes, int(blockIdx.x) - a.plan.ctas, int(gridDim.x) - a.plan.ctas);
    return;
  }
  __shared__ uint32_t c[kDigits];
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) c[d] = 0;
  __syncthreads();
  const int64_t i0 = int64_t(blockIdx.x) * a.plan.run, i1 = min(i0 + a.plan.run, a.p.R);
  bool bad = false;
  for (int64_t c0 = i0 + threadIdx.x; c0 < i1; c0 += kSortChunk) {
    uint32_t key[kSortItems];
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
      const int64_t i = c0 + k * kSortThreads;
      key[k] = i >= i1 ? 0u : ps.index == 0 ? key_of(a, i, bad) : ps.key_in[i];
    }
#pragma unroll
    for (int k = 0; k < kSortItems; ++k)
      if (c0 + k * kSortThreads < i1) atomicAdd(&c[(key[k] >> ps.shift) & (kDigits - 1)], 1u);
  }
  const int any_bad = __syncthreads_or(bad);
  if (threadIdx.x == 0 && ps.index == 0) a.ws.flags[blockIdx.x] = any_bad ? kFlagIdOutOfRange : 0u;
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) a.ws.counts[size_t(blockIdx.x) * kDigits + d] = c[d];
}

__global__ void __launch_bounds__(kSortThreads) move_kernel(const BwdArgs a, const Pass ps) {
  pdl_wait();
  pdl_trigger();
  if (int(blockIdx.x) >= a.plan.ctas) {
    zero_share(a, 2 * ps.index + 1, 2 * a.plan.passes, int(blockIdx.x) - a.plan.ctas, int(gridDim.x) - a.plan.ctas);
    return;
  }
  static_assert(kSortThreads == kDigits, "one thread per digit");
  constexpr int kWarps = kSortThreads / 32;
  __shared__ uint32_t base[kDigits];
  __shared__ uint16_t cnt[kWarps][kDigits];
  __shared__ uint32_t wsum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0 && warp == 0 && ps.index == 0) {  // the call's status from the runs'
    uint32_t f = 0;
    for (int c = lane; c < a.plan.ctas; c += 32) f |= a.ws.flags[c];
    f = __reduce_or_sync(0xffffffffu, f);
    if (lane == 0) a.ws.hdr->status = f;
  }
  {  // thread = digit
    uint32_t before = 0, total = 0;
#pragma unroll 8
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
    uint32_t key[kSortItems], row[kSortItems], digit[kSortItems], rank[kSortItems];
    // a warp's items are 32 * kSortItems consecutive rows, taken 32 at a time: row order
    const int64_t w0 = c0 + warp * 32 * kSortItems + lane;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
      const int64_t i = w0 + 32 * k;
      const bool on = i < i1;
      key[k] = !on ? 0u : ps.index == 0 ? key_of(a, i, bad) : ps.key_in[i];
      row[k] = !on ? 0u : ps.index == 0 ? uint32_t(i) : ps.row_in[i];
      digit[k] = on ? (key[k] >> ps.shift) & (kDigits - 1) : uint32_t(kDigits);
    }
    warp_ranks<kSortItems>(digit, cnt[warp], rank, lane);
    __syncthreads();
    uint32_t at = 0;  // thread = digit: the warps' counts become offsets within the digit
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t n = cnt[w][tid];
      cnt[w][tid] = uint16_t(at);
      at += n;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
      if (digit[k] == uint32_t(kDigits)) continue;
      const uint32_t to = base[digit[k]] + cnt[warp][digit[k]] + rank[k];
      ps.key_out[to] = key[k];
      ps.row_out[to] = row[k];
    }
    __syncthreads();
    base[tid] += at;
    __syncthreads();
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
      const float4 o = make_float4(acc[i] * a.p.scale, acc[i + 1] * a.p.scale, acc[i + 2] * a.p.scale, acc[i + 3] * a.p.scale);
      // an element gets one addition per call, so its value does not depend on any order;
      // the reduction does not wait for the old value
      if (a.accumulate)
        asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(d + i), "f"(o.x), "f"(o.y), "f"(o.z), "f"(o.w) : "memory");
      else
        *reinterpret_cast<float4*>(d + i) = o;
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

// The first of the n sorted keys that is not below `id`; a warp looks at 32 at a time.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* key, int64_t n, uint32_t id, int lane) {
  int64_t lo = 0;
  while (n > 0) {
    const int64_t step = (n + 31) / 32, at = (lane + 1) * step - 1;
    const int below = __popc(__ballot_sync(0xffffffffu, at < n && key[lo + at] < id));
    lo += below * step;
    n = min(step - 1, n - below * step);  // the probe that was not below is itself a candidate
  }
  return lo;
}

// A warp zeroes those of at most 32 table rows, from `r0` and below `r1`, that no sorted key
// names.
template <bool TF32>
__device__ void zero_untouched(const BwdArgs& a, const uint32_t* key, int64_t r0, int64_t r1, int lane) {
  constexpr int N = Vec<TF32>::N;
  const int64_t nv = a.p.D / N, ldv = a.dtable_ld / N;
  uint32_t free = r1 - r0 < 32 ? (1u << (r1 - r0)) - 1u : 0xffffffffu;
  for (uint32_t from = uint32_t(r0);;) {  // again only where more than 32 keys name these rows
    const int64_t at = lower_bound(key, a.p.R, from, lane) + lane;
    const uint32_t k = at < a.p.R ? key[at] : ~0u, off = k - uint32_t(r0);
    free &= ~__reduce_or_sync(0xffffffffu, off < 32u ? 1u << off : 0u);
    const uint32_t top = __shfl_sync(0xffffffffu, off, 31);
    if (top >= 31u) break;
    from = uint32_t(r0) + top + 1;
  }
  uint4* t = static_cast<uint4*>(a.dtable);
  for (uint32_t m = free; m != 0; m &= m - 1) {
    uint4* d = t + (r0 + __ffs(m) - 1) * ldv;
    for (int64_t j = lane; j < nv; j += 32) __stcs(d + j, make_uint4(0u, 0u, 0u, 0u));
  }
}

// A warp sums one window's rows over 32 vectors of columns; warps past the windows zero
// untouched table rows.
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
  if (w >= a.plan.windows * blocks) {
    const int64_t r0 = a.plan.fill + (w - a.plan.windows * blocks) * a.plan.zero_rows;
    if (!a.accumulate && r0 < a.p.Vt)
      zero_untouched<TF32>(a, key, r0, min(r0 + a.plan.zero_rows, a.p.Vt), lane);
    return;
  }
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

// (volatile: the compiler would sink each load to its addition and wait for one at a time)
__device__ __forceinline__ float4 load_part(const float* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}

// The segments that cross windows: the window a segment begins in adds the parts that the
// windows after it left.
template <bool F32, bool TF32>
__global__ void __launch_bounds__(256) join_kernel(const BwdArgs a, const uint32_t* key) {
  pdl_wait();
  pdl_trigger();
  constexpr int N = Vec<F32>::N, U = F32 ? 16 : 8;  // parts in flight
  const int lane = threadIdx.x & 31;
  const int64_t nv = a.p.D / N, blocks = (nv + 31) / 32;
  const int64_t w = int64_t(blockIdx.x) * 8 + threadIdx.x / 32;
  if (w >= a.plan.windows * blocks) return;
  const int64_t win = w / blocks, j = (w - win * blocks) * 32 + lane;
  const int64_t p0 = win * a.plan.window, p1 = p0 + a.plan.window;
  if (p1 >= a.p.R) return;
  const uint32_t id = key[p1 - 1], next = key[p1], prev = p0 > 0 ? key[p0 - 1] : ~0u;
  if (id == uint32_t(a.p.Vt) || next != id || prev == id) return;  // nothing goes on, or nothing begins here
  // the last window that begins with the id, 32 windows a look
  int64_t last = win + 1;
  for (;;) {
    const int64_t x = last + 1 + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, x < a.plan.windows && key[x * a.plan.window] == id);
    last += __popc(m);
    if (m != 0xffffffffu) break;
  }
  if (j >= nv) return;
  float acc[N];
  const float* src = a.ws.part + (size_t(win) * 2 + 1) * a.p.D + j * N;
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = src[i];
  const int64_t stride = 2 * a.p.D;
  for (int64_t x = win + 1; x <= last; x += U) {
    const float* q = a.ws.part + size_t(x) * stride + j * N;
    float4 f[U][N / 4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        f[u][i] = load_part(q + (x + u <= last ? u : 0) * stride + 4 * i);  // (past the last: not added)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (x + u > last) break;
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        acc[4 * i] += f[u][i].x, acc[4 * i + 1] += f[u][i].y, acc[4 * i + 2] += f[u][i].z, acc[4 * i + 3] += f[u][i].w;
    }
  }
  write_row<TF32, N>(a, id, j * N, acc);
}

template <bool F32, bool TF32>
cudaError_t sums(const BwdArgs& a, const uint32_t* key, const uint32_t* row, cudaStream_t s) {
  const int64_t nv = a.p.D / Vec<F32>::N, warps = a.plan.windows * ((nv + 31) / 32);
  const int64_t zeros = a.accumulate ? 0 : (a.p.Vt - a.plan.fill + a.plan.zero_rows - 1) / a.plan.zero_rows;
  PdlLaunch l((warps + zeros + 7) / 8, 256, 0, s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, sum_kernel<F32, TF32>, a, key, row);
  if (e != cudaSuccess) return e;
  PdlLaunch l2((warps + 7) / 8, 256, 0, s);
  return cudaLaunchKernelEx(&l2.cfg, join_kernel<F32, TF32>, a, key);
}

}  // namespace

cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t s) {
  return a.p.dtype == DSPARK_F32 ? lookup<true>(a, s) : lookup<false>(a, s);
}

cudaError_t launch_bwd(const BwdArgs& a, cudaStream_t s) {
  cudaError_t e;
  int from = 0;
  if (a.p.R <= kRankRows) {
    if ((e = rank_sort(a, s)) != cudaSuccess) return e;
  } else if (a.p.R <= kSmallRows) {
    e = a.p.R <= kSmallRows / 4   ? small_sort<kSmallItems / 4>(a, s)
        : a.p.R <= kSmallRows / 2 ? small_sort<kSmallItems / 2>(a, s)
                                  : small_sort<kSmallItems>(a, s);
    if (e != cudaSuccess) return e;
  } else {
    const int spare = fill_ctas(a.plan, a.p.D * (a.table_f32 ? 4 : 2), 2 * a.plan.passes, 148 * 3);
    for (int k = 0; k < a.plan.passes; ++k) {
      const Pass ps{k * kDigitBits, k, a.ws.key[from], a.ws.row[from], a.ws.key[1 - from], a.ws.row[1 - from]};
      PdlLaunch l(a.plan.ctas + spare, kSortThreads, 0, s);
      if (k == 0) l.cfg.numAttrs = 0;  // the first kernel of the call waits for all work before it
      if ((e = cudaLaunchKernelEx(&l.cfg, count_kernel, a, ps)) != cudaSuccess) return e;
      PdlLaunch l2(a.plan.ctas + spare, kSortThreads, 0, s);
      if ((e = cudaLaunchKernelEx(&l2.cfg, move_kernel, a, ps)) != cudaSuccess) return e;
      from = 1 - from;
    }
  }
  const uint32_t *key = a.ws.key[from], *row = a.ws.row[from];
  const bool f32 = a.p.dtype == DSPARK_F32;
  if (f32) return a.table_f32 ? sums<true, true>(a, key, row, s) : sums<true, false>(a, key, row, s);
  return a.table_f32 ? sums<false, true>(a, key, row, s) : sums<false, false>(a, key, row, s);
}

}  // namespace embed
}  // namespace dspark
