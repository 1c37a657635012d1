// The embedding and gradient-clipping operators: workspace maps and launchers.
#pragma once
#include "internal.cuh"

namespace dspark {

// ------------------------------------------------------------------ embedding
namespace embed {

constexpr int kSortThreads = 512;
constexpr int kSortItems = 2;                          // per thread and chunk
constexpr int kSortChunk = kSortThreads * kSortItems;  // rows ranked at a time
constexpr int kSortCtas = 128;                         // at most: a CTA sorts a run of chunks
constexpr int kRankThreads = 512;
constexpr int kRankRows = 4096;                        // placed by counting
constexpr int kSmallThreads = 1024;
constexpr int kSmallItems = 4;                         // rows per thread, at most
constexpr int kSmallCtas = 8;
constexpr int kSmallRows = kSmallThreads * kSmallItems * kSmallCtas;  // sorted by one cluster
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;

struct WsEmbedHeader {
  uint32_t status;  // device error bits
  uint32_t pad[63];
};
static_assert(sizeof(WsEmbedHeader) == 256, "header is one 256-byte line");

struct Plan {
  int64_t R, Vt, D;
  int bits, passes;    // key bits and radix passes
  int64_t run;         // rows per sorting CTA (whole chunks)
  int ctas;            // sorting CTAs
  int window;          // sorted rows per partial sum
  int64_t windows;
  int64_t fill;        // table rows [0, fill) are zeroed beside the sort (0 when accumulating)
  int64_t zero_rows;   // rows of the others that a warp looks up and zeroes
};

inline Plan make_plan(int64_t R, int64_t Vt, int64_t D, bool f32) {
  Plan p{};
  p.R = R, p.Vt = Vt, p.D = D;
  p.bits = 1;
  while ((int64_t(1) << p.bits) <= Vt) ++p.bits;  // keys 0 .. Vt (Vt: dropped rows)
  p.passes = (p.bits + kDigitBits - 1) / kDigitBits;
  const int64_t chunks = (R + kSortChunk - 1) / kSortChunk;
  p.run = (chunks + kSortCtas - 1) / kSortCtas * kSortChunk;
  p.ctas = int((R + p.run - 1) / p.run);
  // windows of 16 to 512 sorted rows: longer ones as long as 32 warps per SM still have one
  // each (32749 rows of 4096 columns: 64 rows 128 us, 256 rows 200 us).  Beyond 16384 rows at
  // least 32, for the sake of the segments that cross windows (131072 rows of 256 columns:
  // 16 rows 175 us, 32 rows 118 us)
  const int64_t cols = f32 ? 128 : 256, blocks = (D + cols - 1) / cols;  // a warp's columns
  p.window = R > 16384 ? 32 : 16;
  while (p.window < 512 && (R / (2 * p.window)) * blocks >= 148 * 32) p.window *= 2;
  p.windows = (R + p.window - 1) / p.window;
  return p;
}

// Table rows zeroed beside the sort: as many as its kernels' latencies hide.  With 0, 32, 64 and
// 128 MB, us: 20 rows into 151936 x 256 FP32 33.3, 35.2, 31.0, 30.4; 4096 rows 38.9, 40.3, 32.0,
// 33.2; 8192 rows 43.3, 45.1, 37.2, 43.0; 32768 rows 51.3, 50.0, 48.9, 49.9; 8192 rows into
// 32003 x 1024 40.4, 40.2, 36.1, 43.1, into 151936 x 4096 438, 435, 434, 430.
inline int64_t fill_rows(const Plan& p, int64_t row_bytes) {
  const int64_t bytes = p.R <= kSmallRows ? 64000000 : 48000000 * p.passes;
  return std::min(p.Vt, bytes / row_bytes);
}

// Rows per warp of those left: 32 share a look into the keys, but few rows are spread over
// more warps (16 MB in rows of 4 KB: 18 us by 125 warps).
inline int64_t zero_rows(int64_t left) { return left >= 32 * 148 * 16 ? 32 : left >= 8 * 148 * 16 ? 8 : 2; }

// CTAs that zero those rows: one per 16 KB of each of `parts` kernels, up to `most`.
inline int fill_ctas(const Plan& p, int64_t row_bytes, int parts, int most) {
  return int(std::min<int64_t>(most, (p.fill * row_bytes / parts + 16383) / 16384));
}

struct View {
  WsEmbedHeader* hdr;
  uint32_t* flags;    // [ctas] error bits of the sorting CTAs' runs
  uint32_t* counts;   // [ctas][kDigits] digit counts of the sorting CTAs' runs
  uint32_t* key[2];   // [R] ids, sorted back and forth
  uint32_t* row[2];   // [R] the rows they came with
  float* part;        // [windows][2][D] sums of the segments that cross a window's ends
  size_t bytes;
};

inline View view(void* base, const Plan& p) {
  View v{};
  size_t off = 0;
  uint8_t* b = static_cast<uint8_t*>(base);
  auto take = [&](size_t n) { uint8_t* at = b + off; off = align256(off + n); return at; };
  v.hdr = reinterpret_cast<WsEmbedHeader*>(take(sizeof(WsEmbedHeader)));
  v.flags = reinterpret_cast<uint32_t*>(take(4 * size_t(p.ctas)));
  v.counts = reinterpret_cast<uint32_t*>(take(4 * size_t(p.ctas) * kDigits));
  for (int i = 0; i < 2; ++i) v.key[i] = reinterpret_cast<uint32_t*>(take(4 * size_t(p.R)));
  for (int i = 0; i < 2; ++i) v.row[i] = reinterpret_cast<uint32_t*>(take(4 * size_t(p.R)));
  v.part = reinterpret_cast<float*>(take(sizeof(float) * 2 * size_t(p.windows) * size_t(p.D)));
  v.bytes = off;
  return v;
}

struct FwdArgs {
  dspark_embed_problem_t p;
  const void* table;
  int64_t table_ld;
  void* out;
  int64_t out_ld;
  WsEmbedHeader* hdr;
};
struct BwdArgs {
  dspark_embed_problem_t p;
  const void* dout;
  int64_t dout_ld;
  void* dtable;
  int64_t dtable_ld;
  int32_t table_f32, accumulate;
  Plan plan;
  View ws;
};
cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t s);
cudaError_t launch_bwd(const BwdArgs& a, cudaStream_t s);

}  // namespace embed

// ------------------------------------------------------------------ gradient clipping
namespace clip {

constexpr int kMaxTensors = 900;   // descriptors per launch (kernel parameters)
constexpr int kGrid = 148 * 8;     // CTAs of a launch, at most
constexpr int kThreads = 256;
constexpr int64_t kChunk = 8192;   // elements a CTA takes at a time

inline int64_t launches(int64_t count) { return (count + kMaxTensors - 1) / kMaxTensors; }
// workspace: 256-byte header (status word, the total at byte 8), then one FP64 partial sum per
// CTA and launch
inline double* total_of_call(void* ws) { return reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + 8); }
inline size_t ws_bytes(int64_t count) { return align256(256 + sizeof(double) * size_t(launches(count)) * kGrid); }

cudaError_t launch_sumsq(const dspark_tensor_t* t, int64_t count, void* ws, cudaStream_t s, int64_t* partials);
cudaError_t launch_total(const void* ws, int64_t partials, double* sumsq, cudaStream_t s);
// by sumsq, or (null) by the partial sums in ws
cudaError_t launch_scale(const dspark_tensor_t* t, int64_t count, const double* sumsq, int64_t partials,
                         float max_norm, float* norm, float* coef, void* ws, cudaStream_t s);

}  // namespace clip
}  // namespace dspark
