// Linear cross entropy: softmax cross entropy of z = hidden . weight^T over the whole
// vocabulary and its gradients.  Of the logits only 8 bytes per row and 128 columns reach
// memory, but where they are few (keep_pays).
//   forward   prep:  the labelled rows' places, their hidden rows gathered compact
//             fwd:   product tiles; each row's (maximum, sum of exponentials) in the tile
//             merge: logsumexp, CE and the loss from the tiles' pairs
//   backward, a piece of the vocabulary at a time:
//             dz:    dL/dz of the piece, bf16: from the product again, or from the logits
//                    where they are few enough to have stayed in the workspace
//             dw:    dweight rows of the piece = dz^T . hidden
//             dh:    partial sums of dhidden = dz . weight, FP32
//             then dhidden from the partial sums, scattered to the labelled rows
//   Where no head gradient follows (hidden_grad_only), the forward gathers the hidden
//   gradient as it goes, like attention's softmax: sum_v exp(z_v - ref) weight_v beside
//   sum_v exp(z_v - ref), with one product less (1600 labelled rows of 4096 against 151936
//   columns, passes queued: 5180 us without, 3700 us with it).
// A label's row appears in no product unless it is labelled (ignore_index rows are neither
// read nor computed), so masked batches pay for their labels only.
//
// The four products share one kernel: tcgen05.mma (bf16 in, FP32 in TMEM), fed by TMA.
// CG CTAs (one, or a cluster of two sharing a 256-row tile through cta_group::2) form a
// tile; 320 threads each:
//   warp 0      one thread issues the TMA loads into a ring of 64-wide K stages
//   warp 1      allocates TMEM; one thread (of the tile's first CTA) issues the MMAs
//   warps 2..9  read the accumulator (a thread: one tile row, half the columns), finish it
// The accumulator is double-buffered in TMEM: a tile's epilogue runs beside the next
// tile's MMAs.
#include <cuda_bf16.h>

#include <algorithm>

#include "lce.cuh"
#include "pdl.cuh"
#include "tc_host.cuh"

namespace dspark {
namespace lce {
namespace {

using tc::BK;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint64_t kDrainNs = 1000000;

// ------------------------------------------------------------------ prep
// Each CTA takes a contiguous run of rows, counts the labelled rows before it (the labels
// are small and in L2) and writes its rows' places; then it copies its labelled hidden
// rows.  The last CTA, which sees every row, writes the counts and the status and
// zero-fills the compact rows up to a whole 64-row K chunk: the dweight product reads
// those, and zero is what they have to add.
constexpr int kPrepThreads = 256;

__global__ void __launch_bounds__(kPrepThreads) prep_kernel(const dspark_lce_problem_t p, const View ws,
                                                            int64_t* num_tokens, int64_t rows_per_cta,
                                                            int keep) {
  pdl_trigger();
  __shared__ int sh_warp[kPrepThreads / 32];
  __shared__ int sh_before, sh_bad, sh_row[kPrepThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r0 = int64_t(blockIdx.x) * rows_per_cta;
  const int64_t r1 = r0 + rows_per_cta < p.R ? r0 + rows_per_cta : p.R;
  const bool last = blockIdx.x == gridDim.x - 1;
  if (tid == 0) sh_before = 0, sh_bad = 0;
  __syncthreads();
  // labelled rows before r0 (and, in the last CTA, any label out of range)
  int n = 0, bad = 0;
  const int64_t seen = last ? r1 : r0;
  for (int64_t r8 = tid; r8 < seen; r8 += 8 * kPrepThreads) {
    int64_t t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) t[u] = r8 + u * kPrepThreads < seen ? p.targets[r8 + u * kPrepThreads] : p.ignore_index;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = t[u] >= 0 && t[u] < p.V;
      if (t[u] != p.ignore_index) {
        if (!in) bad = 1;
        else if (r8 + u * kPrepThreads < r0) ++n;
      }
    }
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) atomicAdd(&sh_before, n);
  if (bad) sh_bad = 1;
  __syncthreads();
  int base = sh_before;
  for (int64_t c0 = r0; c0 < r1; c0 += kPrepThreads) {
    const int64_t r = c0 + tid;
    int64_t t = -1;
    bool live = false;
    if (r < r1) {
      t = p.targets[r];
      live = t != p.ignore_index && t >= 0 && t < p.V;
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, live);
    if (lane == 0) sh_warp[warp] = __popc(mask);
    __syncthreads();
    int at = base + __popc(mask & ((1u << lane) - 1u));
    int total = 0;
    for (int w = 0; w < kPrepThreads / 32; ++w) {
      if (w < warp) at += sh_warp[w];
      total += sh_warp[w];
    }
    if (r < r1) ws.index[r] = live ? at : -1;
    if (live) {
      ws.tok[at] = int32_t(t);
      ws.w[at] = p.row_weight ? p.row_weight[r] : 1.f;
    }
    if (live) sh_row[at - base] = tid;
    __syncthreads();
    // this run's labelled rows, four 16-byte vectors per thread in flight
    const int h8 = int(p.H / 8);
    const int64_t n_vec = int64_t(total) * h8;
    uint4* dst = reinterpret_cast<uint4*>(ws.hsup + size_t(base) * p.H);
    for (int64_t j0 = tid; j0 < n_vec; j0 += 4 * kPrepThreads) {
      uint4 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t j = j0 + u * kPrepThreads;
        if (j >= n_vec) break;
        const int k = int(j / h8), v = int(j - int64_t(k) * h8);
        q[u] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.hidden) +
                                              size_t(c0 + sh_row[k]) * p.hidden_ld)[v];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t j = j0 + u * kPrepThreads;
        if (j >= n_vec) break;
        dst[j] = q[u];
      }
    }
    __syncthreads();
    base += total;
  }
  if (last) {
    const int64_t pad = (int64_t(base) + 63) / 64 * 64;
    uint4* z0 = reinterpret_cast<uint4*>(ws.hsup + size_t(base) * p.H);
    const int64_t nz = (pad - base) * p.H / 8;
    for (int64_t j = tid; j < nz; j += kPrepThreads) z0[j] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) {
      ws.hdr->status = sh_bad ? kFlagIdOutOfRange : 0u;
      ws.hdr->n_valid = base;
      ws.hdr->done = 0;
      ws.hdr->redo = 0;
      ws.hdr->kept = uint32_t(keep);
      if (num_tokens) *num_tokens = base;
    }
  }
}

// ------------------------------------------------------------------ the products
// Work item w -> (m tile, n tile, K split).  Items run through groups of `group` m tiles,
// m fastest inside a group: the tiles in flight at one time share both operands in L2.
struct Work {
  int m_tiles, n_tiles, kchunks, group;
  int bound_m, bound_k;  // the number of labelled rows bounds the tile rows / the K range
  int beside;            // runs beside the kernel launched before it
  const int32_t* n_valid;
  uint64_t span_inv, group_inv;  // ceil(2^64 / divisor): n / d = the high half of n * inverse
};

__host__ __device__ inline uint64_t inverse(uint32_t d) { return d == 1 ? 0 : ~uint64_t(0) / d + 1; }
__device__ __forceinline__ int div_by(int n, uint64_t inv) { return inv == 0 ? n : int(__umul64hi(uint64_t(n), inv)); }

struct Item {
  int mt, nt, s, kc0, kc1;
};

// (A division costs about a hundred cycles here, and the epilogue warps of short products
// pass through this once per 2048 cycles: the common ones are multiplications.)
__device__ __forceinline__ Item decode(const Work& wk, int w, int me, int kch, int ksplit) {
  Item it;
  it.s = 0, it.kc0 = 0, it.kc1 = kch;
  int t = w;
  if (ksplit > 1) {
    const int per = me * wk.n_tiles;
    it.s = w / per;
    t = w - it.s * per;
    it.kc0 = int((int64_t(it.s) * kch) / ksplit);
    it.kc1 = int((int64_t(it.s + 1) * kch) / ksplit);
  }
  const int g = div_by(t, wk.span_inv);
  t -= g * wk.group * wk.n_tiles;
  const int m0 = g * wk.group, gm = min(wk.group, me - m0);
  it.nt = gm == wk.group ? div_by(t, wk.group_inv) : gm == 1 ? t : t / gm;
  it.mt = m0 + (t - it.nt * gm);
  return it;
}

// When a product runs: what only the device knows may turn it off.
enum : int { kAlways = 0, kIfRedo = 1, kIfNotKept = 2 };

enum : int { kFwd = 0, kDz = 1, kDh = 2, kDwBf16 = 3, kDwF32 = 4, kGather = 5, kFwdKeep = 6 };

struct EpiArgs {
  View ws;
  Plan plan;
  int32_t rows, n_cols;      // rows and columns of the product that exist
  int32_t col0;              // first vocabulary id of the piece
  float z_alpha;
  const float* grad_scale;
  int32_t add;               // dh: add to the planes; dw: add to dweight
  int32_t watch;             // dh of a gathered forward: a plane that nears FP32's range asks for the other way
  int32_t when;              // kIfRedo: only where a gathered forward has to be done the other way;
                             // kIfNotKept: only where the forward did not keep its logits
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// TMA tile load completing on the barrier of the tile's first CTA.
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CG == 1) {
    tc::tma_load_2d(dst, map, x, y, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
  }
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 1) {
    tc::mma_bf16(d, a, b, idesc, acc);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
  }
}

// Arrive on `bar` (in every CTA of the tile) once this thread's MMAs so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1) {
    tc::mma_commit(bar);
  } else {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(bar), "h"(uint16_t(3)) : "memory");
  }
}

__device__ __forceinline__ void st_shared_u4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 or 32 consecutive fp32 columns of this thread's TMEM lane (warp-collective).  The values
// are there after tmem_wait, which names them, so that no use of them moves before it.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                 "+f"(v[15])::"memory");
}
// This warp's share of an accumulator, 128 columns: all loads in flight, then one wait.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&v)[128]) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) tmem_ld16(taddr + uint32_t(16 * i), v + 16 * i);
#pragma unroll
  for (int i = 0; i < 8; ++i) tmem_wait16(v + 16 * i);
}

template <int CG>
constexpr uint32_t stage_bytes() { return uint32_t(kBM * BK * 2 + 256 / CG * BK * 2); }
// The bf16 dweight product has a short K range and much to write: its epilogue warps get two
// staging tiles each, at the price of a stage.
constexpr int staging_tiles(int epi) { return epi == kDwBf16 ? 2 : 1; }
template <int CG>
constexpr int stages(int epi) { return (CG == 1 ? 4 : 6) - (staging_tiles(epi) - 1); }
template <int CG>
constexpr size_t smem_bytes(int epi) {
  return size_t(stages<CG>(epi)) * stage_bytes<CG>() + 1024 + size_t(staging_tiles(epi)) * kEpiWarps * 4096 + 1024;
}

// One epilogue warp's share of a tile: 32 rows (row = this thread's lane, `m0 + lane`) and
// `cols` columns of the tile from c0 on.  `n0`: first product column of the tile.
struct Share {
  uint32_t sbuf;   // this warp's 4 KB staging tile (or two of them)
  int m0, n0, c0, cols;
  int nt, half;
  int plane0;      // first row of the K split's plane
  bool empty;      // no K range: the product is zero and the accumulator was not written
  int n_valid, lane;
  int boxes;       // boxes this warp has stored (picks one of two staging tiles)
};

// Forward: (maximum, sum) of the row's exponentials over this share, base 2, and the logit
// at the label, from the row's logits in registers.
__device__ __forceinline__ void fwd_finish(const EpiArgs& a, const Share& sh, const float (&z)[128]) {
  const int row = sh.m0 + sh.lane;
  const int tgt = row < sh.n_valid ? a.ws.tok[row] - sh.n0 - sh.c0 : -1;
  const int cols = min(sh.cols, a.n_cols - sh.n0 - sh.c0);  // <= 0: wholly past the vocabulary
  float zt = 0.f;
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (uint32_t(tgt - 32 * c) < 32u && tgt < cols) {
#pragma unroll
      for (int i = 0; i < 32; ++i) zt = tgt - 32 * c == i ? z[32 * c + i] : zt;
      a.ws.zt[row] = zt;
    }
    if (cols - 32 * c >= 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], z[32 * c + i]);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (32 * c + i < cols) m4[i & 3] = fmaxf(m4[i & 3], z[32 * c + i]);
    }
  }
  const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * kLog2e;
  const float ref = mx == -INFINITY ? 0.f : mx;
  float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (cols - 32 * c >= 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i) s4[i & 3] += ex2(fmaf(z[32 * c + i], kLog2e, -ref));
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (32 * c + i < cols) s4[i & 3] += ex2(fmaf(z[32 * c + i], kLog2e, -ref));
    }
  }
  if (row < sh.n_valid)
    a.ws.part[size_t(2 * sh.nt + sh.half) * a.plan.Rp + row] = make_float2(mx, (s4[0] + s4[1]) + (s4[2] + s4[3]));
}

// 32 rows x 64 bf16 columns of the share, from packed words, to the output at (x, y)
__device__ __forceinline__ void store_box(Share& sh, const CUtensorMap& out, const uint32_t* o, int x, int y, int mode,
                                          int tiles) {
  const uint32_t buf = sh.sbuf + (tiles == 2 ? uint32_t(sh.boxes++ & 1) * 4096u : 0u);
  if (sh.lane == 0) {  // the store that last used this staging tile has read it
    if (tiles == 2) tc::bulk_wait_read<1>();
    else tc::bulk_wait_read<0>();
  }
  __syncwarp();
  // 16-byte chunk k of row `lane` at chunk k ^ (lane % 8): the 128-byte swizzle
#pragma unroll
  for (int k = 0; k < 8; ++k)
    st_shared_u4(buf + uint32_t(sh.lane) * 128u + uint32_t((k ^ (sh.lane & 7)) * 16), o[4 * k], o[4 * k + 1],
                 o[4 * k + 2], o[4 * k + 3]);
  tc::fence_proxy_async_smem();
  __syncwarp();
  if (sh.lane == 0) {
    if (mode) tc::tma_reduce_add_2d(&out, buf, x, y);
    else tc::tma_store_2d(&out, buf, x, y);
    tc::bulk_commit();
  }
}

// dL/dz = w g (p (1 + 2 z_alpha lse) - onehot), rounded once to bf16, the type that the gradient
// products' tensor cores take (bf16 gradients are then off by 1.8e-3 to 2.2e-3 of their norm,
// with the results' own rounding alone by 1.7e-3; two bf16 parts of dz would double the
// products); zero past the last labelled row and past the vocabulary (those enter the products).
__device__ __forceinline__ void dz_finish(const EpiArgs& a, const CUtensorMap& out, Share& sh, float (&z)[128]) {
  if (sh.m0 >= a.rows) return;  // the whole warp
  const int row = sh.m0 + sh.lane;
  const bool live = row < sh.n_valid;
  const int n0 = sh.n0 + sh.c0;
  const int tgt = live ? a.ws.tok[row] - a.col0 - n0 : -1;
  const float lse2 = live ? a.ws.lse2[row] : 0.f;
  const float gw = live ? a.ws.w[row] * (a.grad_scale ? *a.grad_scale : 1.f) : 0.f;
  const float scale = gw * fmaf(2.f * a.z_alpha, lse2 * kLn2, 1.f);
  const int cols = live ? a.n_cols - n0 : 0;
#pragma unroll
  for (int c = 0; c < 128; c += 64) {
    uint32_t o[32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int cc = c + 32 * h;
      float* v = z + cc;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = ex2(fmaf(v[i], kLog2e, -lse2)) * scale;
      if (uint32_t(tgt - cc) < 32u) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = tgt - cc == i ? v[i] - gw : v[i];
      }
      if (cols - cc < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < cols - cc ? v[i] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) o[16 * h + i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
    store_box(sh, out, o, n0 + c, sh.m0, 0, staging_tiles(kDz));
  }
}

// Gathered forward: the row's exponentials relative to its reference, as bf16 for the product
// with the head (one rounding in dz's stead) and summed in FP32; the logit at the label.  The label's column is left out
// of the product: its factor in the gradient is p - 1, which for a row that is nearly right
// is far below the rounding of p.  A logit 96 octaves above the reference (66 above the
// largest of the sampled columns) is reported, and the call goes the other way: below that
// the sum of 2^30 exponentials stays in FP32's range.
__device__ __forceinline__ void gather_finish(const EpiArgs& a, const CUtensorMap& out, Share& sh, float (&z)[128]) {
  if (sh.m0 >= a.rows) return;  // the whole warp
  const int row = sh.m0 + sh.lane;
  const bool live = row < sh.n_valid;
  const int n0 = sh.n0 + sh.c0;
  const int tgt = live ? a.ws.tok[row] - a.col0 - n0 : -1;
  const float ref = live ? a.ws.ref[row] : 0.f;
  const int cols = live ? a.n_cols - n0 : 0;
  float s4[4] = {0.f, 0.f, 0.f, 0.f}, top = -INFINITY;
#pragma unroll
  for (int c = 0; c < 128; c += 64) {
    uint32_t o[32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int cc = c + 32 * h;
      float* v = z + cc;
      const int at = tgt < cols ? tgt - cc : -1;
      if (uint32_t(at) < 32u) {
        float zt = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) zt = at == i ? v[i] : zt;
        a.ws.zt[row] = zt;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = fmaf(v[i], kLog2e, -ref);
        const bool in = cols - cc >= 32 || i < cols - cc;
        top = in ? fmaxf(top, x) : top;
        v[i] = in ? ex2(x) : 0.f;
        s4[i & 3] += v[i];
      }
      if (uint32_t(at) < 32u) {  // the label's own term is not rounded: it is added at the end
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = at == i ? 0.f : v[i];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) o[16 * h + i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
    store_box(sh, out, o, n0 + c, sh.m0, 0, staging_tiles(kGather));
  }
  if (!live) return;
  if (top > kGatherRange) a.ws.hdr->redo = 1;  // every writer writes the same
  a.ws.part[size_t(2 * (a.col0 / kBN + sh.nt) + sh.half) * a.plan.Rp + row] =
      make_float2(ref, (s4[0] + s4[1]) + (s4[2] + s4[3]));
}

// FP32 results: kept logits, dhidden's partial sums (one plane per K split; a plane's element gets one
// addition per piece, in stream order, so the sums have a fixed order), or dweight.
template <int EPI>
__device__ __forceinline__ void f32_finish(const EpiArgs& a, const CUtensorMap& out, Share& sh, const float (&z)[128]) {
  if (sh.m0 >= (EPI == kDh || EPI == kFwdKeep ? sh.n_valid : a.rows) || (sh.empty && a.add)) return;
  if constexpr (EPI == kDh) {
    // 32 splits of at most 2^22 pieces of the vocabulary, each below this, add up to less than
    // 2^127 (columns past the hidden size are zeros)
    if (a.watch && !sh.empty && sh.m0 + sh.lane < sh.n_valid) {
      bool in = true;
#pragma unroll
      for (int i = 0; i < 128; ++i) in = in && (i >= sh.cols || fabsf(z[i]) < 1e30f);
      if (!in) a.ws.hdr->redo = 1;  // every writer writes the same
    }
  }
#pragma unroll
  for (int c = 0; c < 128; c += 32) {
    if (c >= sh.cols || sh.n0 + sh.c0 + c >= a.n_cols) break;
    uint32_t o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = sh.empty ? 0u : __float_as_uint(z[c + i]);
    store_box(sh, out, o, sh.n0 + sh.c0 + c, (EPI == kDh ? sh.plane0 : 0) + sh.m0, a.add, staging_tiles(EPI));
  }
}

// dweight, rounded once to bf16
__device__ __forceinline__ void bf16_finish(const EpiArgs& a, const CUtensorMap& out, Share& sh, const float (&z)[128]) {
  if (sh.m0 >= a.rows) return;
#pragma unroll
  for (int c = 0; c < 128; c += 64) {
    if (c >= sh.cols || sh.n0 + sh.c0 + c >= a.n_cols) break;
    uint32_t o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = sh.empty ? 0u : pack_bf16(z[c + 2 * i], z[c + 2 * i + 1]);
    store_box(sh, out, o, sh.n0 + sh.c0 + c, sh.m0, 0, staging_tiles(kDwBf16));
  }
}

// Operand majors of each product: K-major = rows of 64 K values, MN-major = rows of 64
// M (N) values per K index.  Boxes: K-major {64 K, rows}; MN-major {64 M/N, 64 K}.
template <int CG, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmO, const Work wk, const EpiArgs ea, const int bn) {
  constexpr bool A_MN = EPI == kDwBf16 || EPI == kDwF32;
  constexpr bool B_MN = EPI == kDh || A_MN;
  constexpr int STAGES = stages<CG>(EPI);
  // The tensor cores' FP32 accumulation rounds towards zero: over K = 4096 the logits come
  // out 2.2e-6 short (relative), over K = 512 3e-7, and sums over K rows or columns about
  // K 2e-9.  So no accumulator runs over a whole K range: it is handed over in segments, which
  // the epilogue adds in registers, rounding to nearest.  The forward's logits, whose errors
  // the exponentials magnify, take segments of 512 values; dz, the planes and dweight, which
  // pass through bf16 factors of 2^-9, take 4096.
  constexpr bool LOGITS = EPI == kFwd || EPI == kFwdKeep || EPI == kGather;
  constexpr int SEG = (LOGITS ? 512 : 4096) / BK;
  constexpr uint32_t SA = kBM * BK * 2, SS = stage_bytes<CG>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + size_t(STAGES) * SS);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * STAGES;
  const uint32_t accf0 = empty0 + 8 * STAGES;
  const uint32_t acce0 = accf0 + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 4);
  uint8_t* stage = smem + size_t(STAGES) * SS + 1024;  // 1024-byte aligned

  if (ea.when != kAlways) {  // the same in all CTAs; before anything is set up
    pdl_wait();
    if (ea.when == kIfRedo ? ea.ws.hdr->redo == 0 : ea.ws.hdr->kept != 0) return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = CG == 1 ? 0u : cluster_ctarank();
  const int tile0 = int(blockIdx.x) / CG, tiles_step = int(gridDim.x) / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, kEpiWarps * CG);
    }
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {  // fetched while the kernel before this one runs
    prefetch_map(&tmA);
    prefetch_map(&tmB);
    prefetch_map(&tmO);
  }
  if (warp == 1) {
    __syncwarp();
    if constexpr (CG == 1) {
      tc::tmem_alloc(smem_u32(tmem_slot), 512);
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;"
                   ::"r"(smem_u32(tmem_slot)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  tc::fence_before_sync();
  if constexpr (CG == 1) __syncthreads();
  else cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  // What the kernel before it wrote.  The hidden gradient may run beside the head gradient
  // launched before it (`beside`): that one let it start only once it had dz itself; it is
  // waited for at the end, so that what follows finds both done.
  if (!wk.beside) pdl_wait();
  pdl_trigger();

  const int n_valid = *wk.n_valid;
  const int me = wk.bound_m ? min(wk.m_tiles, (n_valid + kBM * CG - 1) / (kBM * CG)) : wk.m_tiles;
  const int kch = wk.bound_k ? min(wk.kchunks, (n_valid + BK - 1) / BK) : wk.kchunks;
  const int ks = EPI == kDh ? splits_of(ea.plan, me) : 1;
  const int W = me * wk.n_tiles * ks;  // the same in every role
  bool timed_out = false;

  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer: this CTA's 128 rows of A, its 1/CG of B's columns
    const int bnc = bn / CG;
    const uint32_t tx = CG * (SA + uint32_t(bnc) * BK * 2);
    // operands that the kernels before wrote by ordinary stores (the gathered rows, dz)
    asm volatile("fence.proxy.async.global;" ::: "memory");
    int it = 0;
    for (int w = tile0; w < W && !timed_out; w += tiles_step) {
      const Item t = decode(wk, w, me, kch, ks);
      const int am = (t.mt * CG + int(rank)) * kBM, bn0 = t.nt * bn + int(rank) * bnc;
      for (int kc = t.kc0; kc < t.kc1; ++kc, ++it) {
        const int st = it % STAGES;
        const uint32_t round = uint32_t(it / STAGES);
        if (!mbar_wait_bounded(empty0 + 8 * st, (round & 1u) ^ 1u)) {
          timed_out = true;
          break;
        }
        uint32_t fb = full0 + 8 * st;
        if (rank == 0) mbar_arrive_expect_tx(fb, tx);
        else fb = dsmem_map(fb, 0);
        const uint32_t sa = smem_u32(smem + size_t(st) * SS), sb = sa + SA;
        const int k0 = kc * BK;
        if constexpr (!A_MN) {
          load_2d<CG>(sa, &tmA, k0, am, fb);
        } else {
#pragma unroll
          for (int c = 0; c < kBM / 64; ++c) load_2d<CG>(sa + c * 8192, &tmA, am + c * 64, k0, fb);
        }
        if constexpr (!B_MN) {
          load_2d<CG>(sb, &tmB, k0, bn0, fb);
        } else {
          for (int c = 0; c < bnc / 64; ++c) load_2d<CG>(sb + c * 8192, &tmB, bn0 + c * 64, k0, fb);
        }
      }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---------------- MMA issuer
    const uint32_t idesc = tc::idesc_bf16(kBM * CG, bn, A_MN, B_MN);
    int it = 0, tl = 0;
    for (int w = tile0; w < W && !timed_out; w += tiles_step) {
      const Item t = decode(wk, w, me, kch, ks);
      int kc = t.kc0;
      do {  // one accumulator per segment (an empty K range still hands one over)
        const int b = tl & 1;
        if (!mbar_wait_bounded(acce0 + 8 * b, (uint32_t(tl >> 1) & 1u) ^ 1u)) timed_out = true;
        tc::fence_after_sync();
        if (timed_out) break;
        const uint32_t d_tmem = tmem_base + uint32_t(b * 256);
        const int k1 = min(t.kc1, kc + SEG), kfirst = kc;
        for (; kc < k1; ++kc, ++it) {
          const int st = it % STAGES;
          if (!mbar_wait_bounded(full0 + 8 * st, uint32_t(it / STAGES) & 1u)) timed_out = true;
          tc::fence_after_sync();
          if (timed_out) break;
          const uint32_t sa = smem_u32(smem + size_t(st) * SS), sb = sa + SA;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k) {
            const uint64_t ad = A_MN ? tc::sdesc(sa + k * 2048, 8192, 1024) : tc::sdesc(sa + k * 32, 16, 1024);
            const uint64_t bd = B_MN ? tc::sdesc(sb + k * 2048, 8192, 1024) : tc::sdesc(sb + k * 32, 16, 1024);
            mma<CG>(d_tmem, ad, bd, idesc, (kc > kfirst || k > 0) ? 1u : 0u);
          }
          commit<CG>(empty0 + 8 * st);  // frees the stage once these MMAs have read it
        }
        if (timed_out) break;
        commit<CG>(accf0 + 8 * b);  // accumulator ready
        ++tl;
      } while (kc < t.kc1);
    }
  } else if (warp >= 2) {
    // ---------------- epilogue: warp w reads TMEM lanes 32 * (w % 4) .. + 31 of its half
    // of the columns
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes = uint32_t(q * 32) << 16;
    Share sh;
    sh.sbuf = smem_u32(stage + (warp - 2) * staging_tiles(EPI) * 4096);
    sh.boxes = 0;
    sh.half = half, sh.n_valid = n_valid, sh.lane = lane;
    sh.c0 = half * (bn / 2), sh.cols = bn / 2;
    // Hands an accumulator back to the MMA thread.  What is ordered is TMEM, by the loads'
    // wait and the tcgen05 fences on both sides of the barrier, and no other memory: the
    // barrier operations stay at CTA scope also between the pair (a cluster-scope release
    // waits for this thread's stores, 1300 cycles a tile; a cluster-scope acquire empties
    // the MMA thread's queue).
    auto release = [&](int b) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) tc::mbar_arrive(acce0 + 8 * b);
        else asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];"
                          ::"r"(dsmem_map(acce0 + 8 * b, 0)) : "memory");
      }
    };
    // Waits for the accumulator of segment `tl`; the warp gives up as one.
    auto arrived = [&](int tl) {
      const bool ok = mbar_wait_bounded(accf0 + 8 * (tl & 1), uint32_t(tl >> 1) & 1u);
      if (!__all_sync(0xffffffffu, ok)) timed_out = true;
      tc::fence_after_sync();
      return !timed_out;
    };
    // Adds the accumulator of segment `tl` to this warp's share.
    auto add_segment = [&](int tl, float (&z)[128]) {
      const int b = tl & 1;
      if (!arrived(tl)) return;
      const uint32_t taddr = tmem_base + lanes + uint32_t(b * 256 + sh.c0);
      constexpr int N = LOGITS ? 16 : 4;  // columns at a time (8 spill in some of the gradient products)
#pragma unroll
      for (int c = 0; c < 128; c += N) {
        float v[N];
        __syncwarp();
        if constexpr (N == 16) {
          tmem_ld16(taddr + uint32_t(c), v);
          tmem_wait16(v);
        } else {
          tm::ld<N>(taddr + uint32_t(c), v);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) z[c + i] += v[i];
      }
      release(b);
    };
    int tl = 0;
    for (int w = tile0; w < W; w += tiles_step) {
      const Item t = decode(wk, w, me, kch, ks);
      sh.m0 = (t.mt * CG + int(rank)) * kBM + q * 32, sh.n0 = t.nt * bn;
      sh.nt = t.nt, sh.plane0 = t.s * me * kBM * CG, sh.empty = t.kc0 == t.kc1;
      if constexpr (LOGITS) {
        float z[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) z[i] = 0.f;
        for (int kc = t.kc0; kc < t.kc1 && !timed_out; kc += SEG, ++tl) add_segment(tl, z);
        if (timed_out) break;
        if constexpr (EPI == kGather) gather_finish(ea, tmO, sh, z);
        else fwd_finish(ea, sh, z);
        if constexpr (EPI == kFwdKeep) f32_finish<EPI>(ea, tmO, sh, z);
      } else {
        const int b = tl & 1;
        if (!arrived(tl)) break;
        // to registers at once, so that the next tile's MMAs have the accumulator early
        float z[128];
        tmem_ld128(tmem_base + lanes + uint32_t(b * 256 + sh.c0), z);
        release(b);
        for (int kc = t.kc0 + SEG; kc < t.kc1 && !timed_out; kc += SEG) add_segment(++tl, z);
        if (timed_out) break;
        if constexpr (EPI == kDz) dz_finish(ea, tmO, sh, z);
        else if constexpr (EPI == kDwBf16) bf16_finish(ea, tmO, sh, z);
        else f32_finish<EPI>(ea, tmO, sh, z);
        ++tl;
      }
    }
    if (lane == 0) tc::bulk_wait_read<0>();  // the staging stays until the TMA engine has read it
  }
  if (timed_out) atomicOr(&ea.ws.hdr->status, kFlagTimeout);
  if (wk.beside) pdl_wait();
  tc::fence_before_sync();
  // A role whose wait has run out leaves its loop, and the roles that wait for it run out in
  // turn.  What they have in flight (copies into shared memory, MMAs) waits for nobody and
  // lands in microseconds: it gets a millisecond before memory and TMEM are given back.
  if (__syncthreads_or(timed_out)) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < kDrainNs) {}
  }
  if constexpr (CG == 2) cluster_sync();  // the pair's barriers and TMEM stay until both are done
  tc::fence_after_sync();
  if (warp == 1) {
    if constexpr (CG == 1) tc::tmem_dealloc(tmem_base, 512);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem_base) : "memory");
  }
}

// ------------------------------------------------------------------ merge
// 32 rows per CTA, the tiles of a row spread over 32 slices (one warp each, the rows its
// lanes); then a warp per row combines the slices' pairs.  Loss terms in FP64, summed per
// CTA and by the last CTA in CTA order: a fixed order, so repeated calls agree bit by bit.
constexpr int kSlices = 32;

__global__ void __launch_bounds__(kSlices * 32) merge_kernel(const View ws, const Plan pl, const float z_alpha,
                                                             const dspark_lce_out_t out, const int if_redo) {
  pdl_wait();
  pdl_trigger();
  if (if_redo && ws.hdr->redo == 0) return;
  __shared__ float2 sp[kSlices][kMergeRows];
  __shared__ double sd[32];
  __shared__ int is_last;
  const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int64_t r = int64_t(blockIdx.x) * kMergeRows + lane;
  const int i = r < pl.R ? ws.index[r] : -1;
  float m = -INFINITY, s = 0.f;
  if (i >= 0) {
    constexpr int U = 8;  // pairs in flight
    for (int64_t t = sl; t < 2 * pl.fwd_tiles; t += U * kSlices) {
      float2 p[U];
      float nm = m;
#pragma unroll
      for (int u = 0; u < U; ++u)
        p[u] = t + u * kSlices < 2 * pl.fwd_tiles ? ws.part[size_t(t + u * kSlices) * pl.Rp + i] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int u = 0; u < U; ++u) nm = fmaxf(nm, p[u].x);
      const float ref = nm == -INFINITY ? 0.f : nm;
      s *= ex2(m - ref);
#pragma unroll
      for (int u = 0; u < U; ++u) s += p[u].y * ex2(p[u].x - ref);
      m = nm;
    }
  }
  sp[sl][lane] = make_float2(m, s);
  __syncthreads();
  // now warp = row, lane = slice: a fixed tree over the slices
  const int64_t row = int64_t(blockIdx.x) * kMergeRows + sl;
  const int k = row < pl.R ? ws.index[row] : -1;
  const float2 p = sp[lane][sl];
  m = p.x;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  s = p.y * ex2(p.x - (m == -INFINITY ? 0.f : m));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (lane == 0) {
    float ce = 0.f, lse = 0.f;
    double term = 0.0;
    if (k >= 0) {
      const float lse2 = m + log2f(s);
      ws.lse2[k] = lse2;
      lse = lse2 * kLn2;
      ce = fmaf(lse2, kLn2, -ws.zt[k]);
      term = double(ws.w[k]) * (double(ce) + double(z_alpha) * double(lse) * double(lse));
    }
    if (row < pl.R) {
      if (out.ce_rows) out.ce_rows[row] = ce;
      if (out.lse_rows) out.lse_rows[row] = lse;
    }
    sd[sl] = term;
  }
  __syncthreads();
  if (sl == 0) {
    double term = sd[lane];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) term += __shfl_xor_sync(0xffffffffu, term, off);
    if (lane == 0) {
      if (gridDim.x == 1) {  // nothing to add up
        if (out.loss_num) *out.loss_num = float(term);
        is_last = 0;
      } else {
        ws.loss_part[blockIdx.x] = term;
        __threadfence();
        is_last = atomicAdd(&ws.hdr->done, 1u) == gridDim.x - 1;
      }
    }
  }
  __syncthreads();
  if (!is_last) return;
  if (threadIdx.x == 0) ws.hdr->done = 0;  // for a second merge of the call
  if (out.loss_num == nullptr) return;
  __threadfence();
  double acc = 0.0;
  for (int64_t k = threadIdx.x; k < gridDim.x; k += blockDim.x) acc += __ldcg(ws.loss_part + k);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if (lane == 0) sd[sl] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int k = 0; k < kSlices; ++k) t += sd[k];
    *out.loss_num = float(t);
  }
}

// ------------------------------------------------------------------ dz of kept logits
// As dz_finish, from the logits that the forward kept: eight columns per thread.  Rows up to a
// whole 64-row K chunk and columns up to a whole 64-column one are zeros.
__global__ void __launch_bounds__(256) dz_kernel(const View ws, const Plan pl, const float z_alpha,
                                                 const float* grad_scale) {
  pdl_wait();
  pdl_trigger();
  if (ws.hdr->kept == 0) return;  // the product has formed dz
  const int n = ws.hdr->n_valid, rows = (n + 63) / 64 * 64;
  const int c8 = int((pl.V + 63) / 64 * 8);
  const float g = grad_scale ? *grad_scale : 1.f;
  for (int i = blockIdx.y; i < rows; i += gridDim.y) {
    const bool live = i < n;
    const int tgt = live ? ws.tok[i] : -1;
    const float lse2 = live ? ws.lse2[i] : 0.f, gw = live ? g * ws.w[i] : 0.f;
    const float scale = gw * fmaf(2.f * z_alpha, lse2 * kLn2, 1.f);
    const float4* src = reinterpret_cast<const float4*>(ws.z + size_t(i) * pl.piece);
    uint4* dst = reinterpret_cast<uint4*>(ws.dz + size_t(i) * pl.piece);
    for (int j = int(blockIdx.x) * 256 + threadIdx.x; j < c8; j += int(gridDim.x) * 256) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) {
        const float4 a = __ldcs(src + 2 * j), b = __ldcs(src + 2 * j + 1);
        const float z[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float p = ex2(fmaf(z[u], kLog2e, -lse2)) * scale;
          v[u] = 8 * j + u >= pl.V ? 0.f : 8 * j + u == tgt ? p - gw : p;
        }
      }
      dst[j] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
  }
}

// ------------------------------------------------------------------ reference
// A gathered row's reference: the largest logit of the sampled columns (one that is not a
// number, or infinite, is left to the exponentials to show).
__global__ void __launch_bounds__(256) reference_kernel(const View ws, const Plan pl) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= ws.hdr->n_valid) return;
  float m = -INFINITY;
#pragma unroll
  for (int t = 0; t < 2 * kSampleCols / kBN; ++t) m = fmaxf(m, ws.part[size_t(t) * pl.Rp + i].x);
  ws.ref[i] = fabsf(m) < INFINITY ? m : 0.f;
}

// ------------------------------------------------------------------ dhidden
// The planes' sums in plane order, rounded once; rows without a label are zero.  After a
// gathered forward the planes hold the sum over v != target of 2^(z log2 e - ref) weight_v,
// and here, with c = 1 + 2 z_alpha lse,
//   dhidden_r = g w (c 2^(ref - lse2) that + (c 2^(z_target log2 e - lse2) - 1) weight[target])
__global__ void __launch_bounds__(256) dhidden_kernel(const View ws, const Plan pl, const dspark_lce_problem_t p,
                                                      const float* grad_scale, uint16_t* dh, int64_t ld) {
  pdl_wait();
  pdl_trigger();
  const int64_t h8 = pl.H / 8, n = pl.R * h8;
  const int tile = kBM * pl.cg, me = (ws.hdr->n_valid + tile - 1) / tile, splits = splits_of(pl, me);
  const size_t plane = size_t(me) * tile * pl.H;
  const bool gathered = pl.gathered && ws.hdr->redo == 0;
  const float g = pl.gathered && grad_scale ? *grad_scale : 1.f;  // else dz has it
  for (int64_t k = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; k < n; k += int64_t(gridDim.x) * blockDim.x) {
    const int64_t r = k / h8, j = (k - r * h8) * 8;
    const int i = ws.index[r];
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (i >= 0) {
      float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      const float* src = ws.planes + size_t(i) * pl.H + j;
#pragma unroll 4
      for (int s = 0; s < splits; ++s, src += plane) {
        const float4 x = *reinterpret_cast<const float4*>(src), y = *reinterpret_cast<const float4*>(src + 4);
        a[0] += x.x, a[1] += x.y, a[2] += x.z, a[3] += x.w;
        a[4] += y.x, a[5] += y.y, a[6] += y.z, a[7] += y.w;
      }
      if (gathered) {
        const float lse2 = ws.lse2[i], gw = g * ws.w[i];
        const float c = gw * fmaf(2.f * p.z_alpha, lse2 * kLn2, 1.f);
        const float f = c * ex2(ws.ref[i] - lse2), ft = ex2(fmaf(ws.zt[i], kLog2e, -lse2)) * c - gw;
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.weight) +
                                                        size_t(ws.tok[i]) * p.weight_ld + j);
        const float t[8] = {bf16lo(q.x), bf16hi(q.x), bf16lo(q.y), bf16hi(q.y),
                            bf16lo(q.z), bf16hi(q.z), bf16lo(q.w), bf16hi(q.w)};
#pragma unroll
        for (int u = 0; u < 8; ++u) a[u] = fmaf(f, a[u], ft * t[u]);
      } else if (pl.gathered) {
#pragma unroll
        for (int u = 0; u < 8; ++u) a[u] *= g;
      }
      o = make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7]));
    }
    *reinterpret_cast<uint4*>(dh + size_t(r) * ld + j) = o;
  }
}

// ------------------------------------------------------------------ host side
// A bf16 output written by tensor stores of 32-row, 64-column boxes (128-byte swizzle).
bool make_out16_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t ld) {
  return tc::make_map(m, base, rows, cols, ld, 64, 32);
}

template <int CG, int EPI>
cudaError_t product_cg(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o, const Work& wk,
                       const EpiArgs& ea, int bn, cudaStream_t s) {
  auto kern = product_kernel<CG, EPI>;
  constexpr size_t smem = smem_bytes<CG>(EPI);
  // per device, so set on every call (it is a host-side table entry)
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  // K splits (hidden gradient) make more items of few tiles
  const int64_t W = int64_t(wk.m_tiles) * wk.n_tiles * (EPI == kDh ? kMaxSplit : 1);
  const int64_t grid = std::min<int64_t>(W, std::max(1, tc::sm_count() / CG)) * CG;
  PdlLaunch l(grid, kThreads, smem, s, CG);
  return cudaLaunchKernelEx(&l.cfg, kern, a, b, o, wk, ea, bn);
}

template <int EPI>
cudaError_t product(const Plan& pl, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o, const Work& wk,
                    const EpiArgs& ea, int bn, cudaStream_t s) {
  return pl.cg == 2 ? product_cg<2, EPI>(a, b, o, wk, ea, bn, s) : product_cg<1, EPI>(a, b, o, wk, ea, bn, s);
}

int tiles(int64_t n, int64_t t) { return int(ceil_div(n, t)); }

// `over_rows`: the labelled rows are the K range (else the tile rows).
Work make_work(int m_tiles, int n_tiles, int kchunks, int group, bool over_rows, const View& ws) {
  return Work{m_tiles, n_tiles, kchunks, group, !over_rows, over_rows, 0, &ws.hdr->n_valid,
              inverse(uint32_t(group) * uint32_t(n_tiles)), inverse(uint32_t(group))};
}

cudaError_t launch_merge(const dspark_lce_problem_t& p, const dspark_lce_out_t& out, const Plan& pl, const View& ws,
                         bool if_redo, cudaStream_t s) {
  PdlLaunch l(pl.merge_blocks, kSlices * 32, 0, s);
  return cudaLaunchKernelEx(&l.cfg, merge_kernel, ws, pl, p.z_alpha, out, int(if_redo));
}

// The forward product over the first `cols` columns, then the rows' logsumexps (all columns)
// or references (a sample of them).
cudaError_t launch_logsumexp(const dspark_lce_problem_t& p, const dspark_lce_out_t& out, const Plan& pl, const View& ws,
                             int64_t cols, bool keep, bool if_redo, cudaStream_t s) {
  CUtensorMap ma, mb, mo;
  if (!tc::make_map(&ma, ws.hsup, pl.Rp, p.H, p.H, 64, kBM) ||
      !tc::make_map(&mb, p.weight, p.V, p.H, p.weight_ld, 64, kBN / pl.cg))
    return cudaErrorInvalidValue;
  const Work wk = make_work(tiles(p.R, kBM * pl.cg), tiles(cols, kBN), tiles(p.H, BK), 16, false, ws);
  EpiArgs ea{};
  ea.ws = ws;
  ea.plan = pl;
  ea.rows = int32_t(pl.Rp);
  ea.n_cols = int32_t(cols);
  ea.when = if_redo ? kIfRedo : kAlways;
  if (keep && !tc::make_out_map(&mo, ws.z, pl.Rp, pl.piece, pl.piece)) return cudaErrorInvalidValue;
  const cudaError_t e = keep ? product<kFwdKeep>(pl, ma, mb, mo, wk, ea, kBN, s)
                             : product<kFwd>(pl, ma, mb, ma, wk, ea, kBN, s);
  if (e != cudaSuccess) return e;
  if (cols == p.V) return launch_merge(p, out, pl, ws, if_redo, s);
  PdlLaunch l(ceil_div(p.R, 256), 256, 0, s);
  return cudaLaunchKernelEx(&l.cfg, reference_kernel, ws, pl);
}

// A piece of the vocabulary at a time: dL/dz (kDz) or a gathered forward's exponentials
// (kGather) into the workspace, and the products with them.  In a gathered call kDz is the
// other way, taken only where a row asked for it.
cudaError_t launch_pieces(const dspark_lce_problem_t& p, const dspark_lce_grads_t& g, const Plan& pl, const View& ws,
                          int what, bool dhidden, cudaStream_t s) {
  const bool f32 = g.dweight_dtype == DSPARK_F32;
  cudaError_t e;
  CUtensorMap h_k, h_mn;
  if (!tc::make_map(&h_k, ws.hsup, pl.Rp, p.H, p.H, 64, kBM) || !tc::make_map(&h_mn, ws.hsup, pl.Rp, p.H, p.H, 64, 64))
    return cudaErrorInvalidValue;
  for (int i = 0; i < pl.pieces; ++i) {
    const int64_t v0 = int64_t(i) * pl.piece, n = std::min<int64_t>(pl.piece, p.V - v0);
    const int64_t ldz = pl.piece;
    const uint16_t* w0 = static_cast<const uint16_t*>(p.weight) + size_t(v0) * p.weight_ld;
    CUtensorMap w_k, w_mn, z_out, z_k, z_mn, o;
    if (!tc::make_map(&w_k, w0, n, p.H, p.weight_ld, 64, kBN / pl.cg) ||
        !make_out16_map(&z_out, ws.dz, pl.Rp, ldz, ldz))
      return cudaErrorInvalidValue;
    EpiArgs ea{};
    ea.ws = ws;
    ea.plan = pl;
    ea.rows = int32_t(pl.Rp);
    ea.n_cols = int32_t(n);
    ea.col0 = int32_t(v0);
    ea.z_alpha = p.z_alpha;
    ea.grad_scale = g.grad_scale;
    ea.watch = what == kGather;
    ea.when = what != kDz ? kAlways : pl.gathered ? kIfRedo : pl.keep ? kIfNotKept : kAlways;
    const Work wz = make_work(tiles(p.R, kBM * pl.cg), tiles(n, kBN), tiles(p.H, BK), 16, false, ws);
    // Of the product and dz_kernel one returns at once: only the device knows what the forward
    // kept (1.0 us of a call of 56 rows; with dz_kernel first 2.4).
    e = what == kGather ? product<kGather>(pl, h_k, w_k, z_out, wz, ea, kBN, s)
                        : product<kDz>(pl, h_k, w_k, z_out, wz, ea, kBN, s);
    if (e != cudaSuccess) return e;
    if (ea.when == kIfNotKept) {
      const int64_t x = std::min<int64_t>(ceil_div(p.V, 2048), 64), y = std::min<int64_t>(pl.Rp, ceil_div(16 * kSlots, x));
      PdlLaunch l(x, 256, 0, s);
      l.cfg.gridDim.y = unsigned(y);
      if ((e = cudaLaunchKernelEx(&l.cfg, dz_kernel, ws, pl, p.z_alpha, g.grad_scale)) != cudaSuccess) return e;
      ea.when = kAlways;
    }
    if (g.dweight) {
      void* d0 = static_cast<uint8_t*>(g.dweight) + size_t(v0) * g.dweight_ld * (f32 ? 4 : 2);
      if (!tc::make_map(&z_mn, ws.dz, pl.Rp, ldz, ldz, 64, 64) ||
          !(f32 ? tc::make_out_map(&o, d0, n, p.H, g.dweight_ld) : make_out16_map(&o, d0, n, p.H, g.dweight_ld)))
        return cudaErrorInvalidValue;
      ea.rows = int32_t(n);
      ea.n_cols = int32_t(p.H);
      ea.add = g.accumulate ? 1 : 0;
      const Work ww = make_work(tiles(n, kBM * pl.cg), tiles(p.H, pl.bn_h), tiles(p.R, BK), 1, true, ws);
      e = f32 ? product<kDwF32>(pl, z_mn, h_mn, o, ww, ea, pl.bn_h, s)
              : product<kDwBf16>(pl, z_mn, h_mn, o, ww, ea, pl.bn_h, s);
      if (e != cudaSuccess) return e;
    }
    if (dhidden) {
      if (!tc::make_map(&w_mn, w0, n, p.H, p.weight_ld, 64, 64) || !tc::make_map(&z_k, ws.dz, pl.Rp, ldz, ldz, 64, kBM) ||
          !tc::make_out_map(&o, ws.planes, pl.plane_rows, p.H, p.H))
        return cudaErrorInvalidValue;
      // the sums last: the kernel after the last piece finds them in L2
      ea.rows = int32_t(pl.Rp);
      ea.n_cols = int32_t(p.H);
      ea.add = i > 0;
      Work wh = make_work(tiles(p.R, kBM * pl.cg), tiles(p.H, pl.bn_h), tiles(n, BK), 8, false, ws);
      wh.beside = g.dweight != nullptr;
      if ((e = product<kDh>(pl, z_k, w_mn, o, wh, ea, pl.bn_h, s)) != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_fwd(const dspark_lce_problem_t& p, const dspark_lce_out_t& out, const Plan& pl, const View& ws,
                       bool keep, cudaStream_t s) {
  const int64_t ctas = std::min<int64_t>(p.R, 4 * kSlots);
  const int64_t rows_per_cta = ceil_div(p.R, ctas);
  PdlLaunch first(ceil_div(p.R, rows_per_cta), kPrepThreads, 0, s);
  first.cfg.numAttrs = 0;  // the first kernel of the call waits for all work before it
  cudaError_t e = cudaLaunchKernelEx(&first.cfg, prep_kernel, p, ws, out.num_tokens, rows_per_cta, int(keep));
  if (e != cudaSuccess) return e;
  if (!pl.gathered) return launch_logsumexp(p, out, pl, ws, p.V, keep, false, s);
  // the reference from a few columns, then the logsumexp and the hidden gradient in one pass
  if ((e = launch_logsumexp(p, out, pl, ws, kSampleCols, false, false, s)) != cudaSuccess) return e;
  dspark_lce_grads_t none{};
  if ((e = launch_pieces(p, none, pl, ws, kGather, true, s)) != cudaSuccess) return e;
  if ((e = launch_merge(p, out, pl, ws, false, s)) != cudaSuccess) return e;
  // and where a row left the range of its reference, both again from its own maximum
  if ((e = launch_logsumexp(p, out, pl, ws, p.V, false, true, s)) != cudaSuccess) return e;
  return launch_pieces(p, none, pl, ws, kDz, true, s);
}

cudaError_t launch_bwd(const dspark_lce_problem_t& p, const dspark_lce_grads_t& g, const Plan& pl, const View& ws,
                       cudaStream_t s) {
  cudaError_t e;
  if (!pl.gathered && (e = launch_pieces(p, g, pl, ws, kDz, g.dhidden != nullptr, s)) != cudaSuccess) return e;
  if (!g.dhidden) return cudaSuccess;
  const int64_t blocks = std::min<int64_t>(ceil_div(p.R * (p.H / 8), 256), 8 * kSlots);
  PdlLaunch l(blocks, 256, 0, s);
  if (pl.gathered) l.cfg.numAttrs = 0;  // the first kernel of the call
  return cudaLaunchKernelEx(&l.cfg, dhidden_kernel, ws, pl, p, g.grad_scale, static_cast<uint16_t*>(g.dhidden),
                            g.dhidden_ld);
}

}  // namespace lce
}  // namespace dspark
