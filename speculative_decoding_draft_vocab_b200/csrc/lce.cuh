// Linear cross entropy (softmax cross entropy of hidden . weight^T): the plan a shape gets,
// its workspace map and the launchers.
#pragma once
#include "internal.cuh"

namespace dspark {
namespace lce {

constexpr int kBM = 128;                             // tile rows per CTA (TMEM lanes)
// Vocabulary columns per tile.  Narrower tiles (192, 208) that fill the last wave of tiles
// better were measured no faster: on a pair of CTAs an MMA of N = 192 takes the time of 256.
constexpr int kBN = 256;
constexpr int kSlots = 148;                          // SMs the plan assumes
constexpr size_t kPieceBytes = size_t(256) << 20;    // bound on the kept piece of dz
constexpr int kMaxSplitTiles = 32;                   // more row tiles than this are not split
constexpr int kMaxSplit = 32;
constexpr size_t kPlaneBytes = size_t(96) << 20;     // bound on split planes (they stay in L2)
// A workspace with room for a backward has room for FP32 logits up to this size; where they
// stay, the backward is spared a product.
constexpr size_t kKeepBytes = size_t(320) << 20;
// Whether that pays: the product spared grows with the hidden size, the traffic added does not,
// and logits that stay in L2 cost little.  Both gradients, kept against formed again, us:
//   24 MiB, H 64 (41 x 151936)      89 /  93     140 MiB, H 640 (1146 x 32003)   236 /  236
//   63 MiB, H 64 (524 x 32003)      93 /  93     140 MiB, H 768 (241 x 151936)   299 /  308
//   96 MiB, H 256 (165 x 151936)   162 / 152     300 MiB, H 64 (517 x 151936)    310 /  254
//   96 MiB, H 512 (786 x 32003)    146 / 149     300 MiB, H 640 (2457 x 32003)   452 /  439
//  140 MiB, H 512 (1146 x 32003)   193 / 184     300 MiB, H 768 (517 x 151936)   596 /  619
//                                                260 MiB, H 4096 (448 x 151936) 1826 / 2247
inline bool keep_pays(size_t bytes, int64_t H) {
  return bytes <= size_t(40) << 20 || (bytes <= size_t(100) << 20 && H >= 512) || H > 640;
}
// A gathered forward takes the reference of a row's exponentials from this many columns (1024,
// 2048, 4096 of 32003, 1600 rows of 1000: 276, 278, 285 us; fewer leave rows out of range
// sooner).
constexpr int kSampleCols = 2048;
// A logit more than this many octaves above a row's reference sends the call the other way.
constexpr float kGatherRange = 96.f;
// It saves one of three products and adds the sample and kernels that mostly return at once.
// Against forming the logits again it pays from this vocabulary on, but for few rows of a small
// hidden size; where logits of at most about 100 MiB could have been kept instead (which this
// rule does not look at) that was faster still.  Hidden gradient alone, gathered / kept /
// formed again, us:
//   rows x columns x H     448 x   8192 x 4096   128 /   90 /  116   (forced)
//                          448 x  16384 x 4096   190 /  157 /  213
//                         4096 x  16384 x 4096  1005 / 1044 / 1348
//                           56 x  32003 x 1000    80 /   61 /   71
//                         1600 x  32003 x 1000   282 /  322 /  358
//                           56 x 151936 x 4096   498 /  472 /  675
//                          448 x 151936 x  512   224 /  292 /  269
//                         1600 x 151936 x 4096  3760 /    - / 5182
constexpr int64_t kGatherFrom = 16384;
constexpr int kMergeRows = 32;                       // rows per CTA of the merge kernel

struct WsLceHeader {
  uint32_t status;     // device error bits
  int32_t n_valid;     // labelled rows
  uint32_t done;       // merge CTAs finished
  uint32_t redo;       // gathered forward: exponentials, or their products with the head, left their range
  uint32_t kept;       // the forward left its logits in the workspace
  uint32_t pad[59];
};
static_assert(sizeof(WsLceHeader) == 256, "header is one 256-byte line");

// Everything about a call that follows from its sizes alone.
struct Plan {
  int64_t R, V, H;
  int64_t Rp;          // R rounded up to a whole 64-row K chunk
  int cg;              // CTAs per tile: 1, or a pair sharing one 256-row tile
  int bn_h;            // hidden columns per tile of the gradient products
  int64_t fwd_tiles;   // vocabulary tiles of the forward product
  int64_t piece;       // vocabulary columns per piece of the backward
  int pieces;
  int64_t plane_rows;  // rows of the hidden gradient's partial sums, all planes together
  uint8_t ksplit[kMaxSplitTiles + 1];  // its K splits (planes) by the number of row tiles
  int64_t merge_blocks;
  int room;            // a backward's workspace has room for the logits
  int keep;            // they stay there if the forward was given that room
  int gathered;        // the forward also gathers the hidden gradient (no head gradient follows)
};

struct View {
  WsLceHeader* hdr;
  double* loss_part;   // [merge_blocks]
  int32_t* index;      // [R] position of a row among the labelled ones, -1 without a label
  int32_t* tok;        // [R] label of the i-th labelled row
  float* w;            // [R] weight of the i-th labelled row
  float* lse2;         // [R] base-2 logsumexp of the i-th labelled row
  float* zt;           // [R] logit at the label
  float* ref;          // [R] base-2 exponent that a gathered row's exponentials are relative to
  uint16_t* hsup;      // [Rp][H] bf16 labelled hidden rows, compact, zeros up to a whole chunk
  float2* part;        // [2 fwd_tiles][Rp] (base-2 maximum, sum) of a row's columns in half a tile
  float* z;            // [Rp][piece] kept logits
  uint16_t* dz;        // [Rp][piece] bf16 piece of dL/dlogits
  float* planes;       // [splits][row tiles' rows][H] partial sums of the hidden gradient
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline Plan make_plan(int64_t R, int64_t V, int64_t H, bool hidden_grad_only) {
  Plan p{};
  p.R = R, p.V = V, p.H = H;
  p.Rp = ceil_div(R, 64) * 64;
  p.cg = R > kBM ? 2 : 1;
  const int64_t slots = kSlots / p.cg, m_tiles = ceil_div(R, kBM * p.cg);
  p.bn_h = H > 128 ? 256 : 128;
  p.fwd_tiles = ceil_div(V, kBN);
  const int64_t most = std::max<int64_t>(256, int64_t(kPieceBytes / (2 * size_t(p.Rp))) / 256 * 256);
  p.pieces = int(ceil_div(V, most));
  p.piece = ceil_div(ceil_div(V, p.pieces), 256) * 256;
  p.pieces = int(ceil_div(V, p.piece));
  // Few row and hidden tiles: the K range (the piece's vocabulary) is split so that the waves
  // of tiles over the SMs are full.  How many row tiles there are only the device knows (they
  // hold the labelled rows), so there is a number of splits for each count.
  const int64_t n_tiles = ceil_div(H, p.bn_h), chunks = ceil_div(std::min(V, p.piece), 64);
  p.plane_rows = R;
  for (int64_t m = 1; m <= std::min<int64_t>(kMaxSplitTiles, m_tiles); ++m) {
    int best = 1;
    int64_t cost = INT64_MAX;
    for (int k = 1; k <= kMaxSplit && (k == 1 || chunks / k >= 8); ++k) {
      if (k > 1 && size_t(m * k * kBM * p.cg) * size_t(H) * 4 > kPlaneBytes) break;
      const int64_t c = ceil_div(m * n_tiles * k, slots) * (ceil_div(chunks, k) + 12);  // 12: writing the sums
      if (c < cost) cost = c, best = k;
    }
    p.ksplit[m] = uint8_t(best);
    if (best > 1) p.plane_rows = std::max(p.plane_rows, m * best * kBM * p.cg);
  }
  p.merge_blocks = ceil_div(R, kMergeRows);
  p.gathered = hidden_grad_only && V >= kGatherFrom;
  p.room = !p.gathered && p.pieces == 1 && 4 * size_t(p.Rp) * size_t(p.piece) <= kKeepBytes;
  p.keep = p.room && keep_pays(4 * size_t(R) * size_t(V), H);
  return p;
}

// K splits and rows per plane of the hidden gradient for n labelled rows.
__host__ __device__ inline int splits_of(const Plan& p, int row_tiles) {
  return row_tiles >= 1 && row_tiles <= kMaxSplitTiles ? p.ksplit[row_tiles] : 1;
}

struct Offsets {
  size_t hdr, loss_part, index, tok, w, lse2, zt, ref, hsup, part, z, dz, planes, bytes;
};

inline Offsets offsets(const Plan& p, bool bwd, bool dhidden) {
  if (p.gathered) bwd = dhidden = true;
  Offsets o{};
  size_t off = 0;
  const size_t R = size_t(p.R), Rp = size_t(p.Rp);
  auto take = [&](size_t& at, size_t n) { at = off; off = align256(off + n); };
  take(o.hdr, sizeof(WsLceHeader));
  take(o.loss_part, sizeof(double) * size_t(p.merge_blocks));
  take(o.index, 4 * R);
  take(o.tok, 4 * R);
  take(o.w, 4 * R);
  take(o.lse2, 4 * R);
  take(o.zt, 4 * R);
  take(o.ref, 4 * R);
  take(o.hsup, 2 * Rp * size_t(p.H));
  take(o.part, sizeof(float2) * 2 * size_t(p.fwd_tiles) * Rp);
  take(o.z, bwd && p.room ? 4 * Rp * size_t(p.piece) : 0);
  take(o.dz, bwd ? 2 * Rp * size_t(p.piece) : 0);
  take(o.planes, bwd && dhidden ? sizeof(float) * size_t(p.plane_rows) * size_t(p.H) : 0);
  o.bytes = off;
  return o;
}

inline View view(void* base, const Plan& p) {
  const Offsets o = offsets(p, true, true);
  uint8_t* b = static_cast<uint8_t*>(base);
  View v{};
  v.hdr = reinterpret_cast<WsLceHeader*>(b + o.hdr);
  v.loss_part = reinterpret_cast<double*>(b + o.loss_part);
  v.index = reinterpret_cast<int32_t*>(b + o.index);
  v.tok = reinterpret_cast<int32_t*>(b + o.tok);
  v.w = reinterpret_cast<float*>(b + o.w);
  v.lse2 = reinterpret_cast<float*>(b + o.lse2);
  v.zt = reinterpret_cast<float*>(b + o.zt);
  v.ref = reinterpret_cast<float*>(b + o.ref);
  v.hsup = reinterpret_cast<uint16_t*>(b + o.hsup);
  v.part = reinterpret_cast<float2*>(b + o.part);
  v.z = reinterpret_cast<float*>(b + o.z);
  v.dz = reinterpret_cast<uint16_t*>(b + o.dz);
  v.planes = reinterpret_cast<float*>(b + o.planes);
  return v;
}

// `keep`: the workspace has room for the plan's kept logits.  The header says whether the
// last forward kept them; the backward goes by that, whatever room it was given itself.
cudaError_t launch_fwd(const dspark_lce_problem_t& p, const dspark_lce_out_t& out, const Plan& plan, const View& ws,
                       bool keep, cudaStream_t s);
cudaError_t launch_bwd(const dspark_lce_problem_t& p, const dspark_lce_grads_t& g, const Plan& plan, const View& ws,
                       cudaStream_t s);

}  // namespace lce
}  // namespace dspark
