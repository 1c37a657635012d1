// Entry points of the training-step operators beside the loss (include/dspark.h): host-side
// validation, workspace carving and the launches.  No allocation, no synchronisation.
#include "internal.cuh"
#include "lce.cuh"
#include "train.cuh"

using namespace dspark;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

dspark_status_t check_lce(const dspark_lce_problem_t* p) {
  if (p == nullptr) return DSPARK_ERR_INVALID_ARG;
  if (p->R <= 0 || p->V <= 0 || p->H <= 0) return DSPARK_ERR_INVALID_ARG;
  if (p->R > (int64_t(1) << 24) || p->V > (int64_t(1) << 30) || p->H > (int64_t(1) << 20)) return DSPARK_ERR_UNSUPPORTED;
  if (lce::ceil_div(p->R, 128) * lce::ceil_div(p->V, 128) > (int64_t(1) << 31) - 1) return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

dspark_status_t check_lce_call(const dspark_lce_problem_t* p) {
  dspark_status_t st = check_lce(p);
  if (st != DSPARK_OK) return st;
  if (!p->hidden || !p->weight || !p->targets) return DSPARK_ERR_INVALID_ARG;
  if (p->hidden_ld < p->H || p->weight_ld < p->H) return DSPARK_ERR_INVALID_ARG;
  if (!(p->z_alpha >= 0.f) || (p->hidden_grad_only != 0 && p->hidden_grad_only != 1)) return DSPARK_ERR_INVALID_ARG;
  if (p->H % 8 || p->hidden_ld % 8 || p->weight_ld % 8 || !aligned16(p->hidden) || !aligned16(p->weight))
    return DSPARK_ERR_ALIGNMENT;
  return DSPARK_OK;
}

lce::Plan lce_plan(const dspark_lce_problem_t* p) { return lce::make_plan(p->R, p->V, p->H, p->hidden_grad_only != 0); }

dspark_status_t check_ws(const void* ws, size_t have, size_t need) {
  if (ws == nullptr) return DSPARK_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return DSPARK_ERR_ALIGNMENT;
  return have < need ? DSPARK_ERR_WORKSPACE : DSPARK_OK;
}

inline bool is_dtype(int64_t d) { return d == DSPARK_F32 || d == DSPARK_BF16; }
inline int64_t elem_size(int64_t d) { return d == DSPARK_BF16 ? 2 : 4; }

dspark_status_t check_embed(const dspark_embed_problem_t* p) {
  if (p == nullptr || p->R <= 0 || p->Vt <= 0 || p->D <= 0 || !is_dtype(p->dtype)) return DSPARK_ERR_INVALID_ARG;
  if (p->R > (int64_t(1) << 24) || p->Vt > (int64_t(1) << 30) || p->D > (int64_t(1) << 20)) return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

dspark_status_t check_matrix(const void* m, int64_t ld, int64_t cols, int64_t dtype) {
  if (m == nullptr || ld < cols) return DSPARK_ERR_INVALID_ARG;
  const int64_t es = elem_size(dtype);
  return !aligned16(m) || (ld * es) % 16 || (cols * es) % 16 ? DSPARK_ERR_ALIGNMENT : DSPARK_OK;
}

embed::Plan embed_plan(const dspark_embed_problem_t* p) {
  return embed::make_plan(p->R, p->Vt, p->D, p->dtype == DSPARK_F32);
}

dspark_status_t check_tensors(const dspark_tensor_t* t, int64_t count, bool dst) {
  if (t == nullptr || count < 1) return DSPARK_ERR_INVALID_ARG;
  if (count > (int64_t(1) << 20)) return DSPARK_ERR_UNSUPPORTED;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n < 0 || !is_dtype(t[i].dtype)) return DSPARK_ERR_INVALID_ARG;
    if (t[i].n > (int64_t(1) << 40)) return DSPARK_ERR_UNSUPPORTED;
    if (t[i].n == 0) continue;
    if (t[i].src == nullptr || (dst && t[i].dst == nullptr)) return DSPARK_ERR_INVALID_ARG;
    const uintptr_t m = uintptr_t(elem_size(t[i].dtype) - 1);
    if ((reinterpret_cast<uintptr_t>(t[i].src) & m) || (dst && (reinterpret_cast<uintptr_t>(t[i].dst) & m)))
      return DSPARK_ERR_ALIGNMENT;
  }
  // a launch numbers the chunks of its tensors in 32 bits
  for (int64_t i = 0; i < count; i += clip::kMaxTensors) {
    int64_t chunks = 0;
    for (int64_t k = i; k < count && k < i + clip::kMaxTensors; ++k) chunks += (t[k].n + clip::kChunk - 1) / clip::kChunk;
    if (chunks > (int64_t(1) << 30)) return DSPARK_ERR_UNSUPPORTED;
  }
  return DSPARK_OK;
}

}  // namespace

extern "C" {

size_t dspark_lce_workspace_size(const dspark_lce_problem_t* prob, const dspark_lce_grads_t* grads) {
  if (check_lce(prob) != DSPARK_OK) return 0;
  const bool bwd = grads && (grads->dhidden || grads->dweight);
  return lce::offsets(lce_plan(prob), bwd, bwd && grads->dhidden).bytes;
}

dspark_status_t dspark_lce_fwd(const dspark_lce_problem_t* prob, const dspark_lce_out_t* out, void* ws,
                               size_t ws_bytes, dspark_stream_t stream) {
  if (out == nullptr) return DSPARK_ERR_INVALID_ARG;
  dspark_status_t st = check_lce_call(prob);
  if (st != DSPARK_OK) return st;
  if ((st = check_ws(ws, ws_bytes, dspark_lce_workspace_size(prob, nullptr))) != DSPARK_OK) return st;
  const lce::Plan plan = lce_plan(prob);
  // a workspace that a backward could use is one that a backward may follow on
  const bool keep = plan.keep && ws_bytes >= lce::offsets(plan, true, false).bytes;
  return cuda_status(
      lce::launch_fwd(*prob, *out, plan, lce::view(ws, plan), keep, reinterpret_cast<cudaStream_t>(stream)));
}

dspark_status_t dspark_lce_bwd(const dspark_lce_problem_t* prob, const dspark_lce_grads_t* grads, void* ws,
                               size_t ws_bytes, dspark_stream_t stream) {
  if (grads == nullptr || (!grads->dhidden && !grads->dweight)) return DSPARK_ERR_INVALID_ARG;
  dspark_status_t st = check_lce_call(prob);
  if (st != DSPARK_OK) return st;
  if (grads->dhidden) {
    if (grads->dhidden_ld < prob->H) return DSPARK_ERR_INVALID_ARG;
    if (!aligned16(grads->dhidden) || grads->dhidden_ld % 8) return DSPARK_ERR_ALIGNMENT;
  }
  if (grads->dweight) {
    if (prob->hidden_grad_only) return DSPARK_ERR_INVALID_ARG;
    const bool f32 = grads->dweight_dtype == DSPARK_F32;
    if (!f32 && grads->dweight_dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARG;
    if (grads->dweight_ld < prob->H) return DSPARK_ERR_INVALID_ARG;
    if (grads->accumulate && !f32) return DSPARK_ERR_UNSUPPORTED;  // a bf16 sum over calls would lose its small terms
    if (!aligned16(grads->dweight) || grads->dweight_ld % (f32 ? 4 : 8)) return DSPARK_ERR_ALIGNMENT;
  }
  if ((st = check_ws(ws, ws_bytes, dspark_lce_workspace_size(prob, grads))) != DSPARK_OK) return st;
  const lce::Plan plan = lce_plan(prob);
  return cuda_status(lce::launch_bwd(*prob, *grads, plan, lce::view(ws, plan), reinterpret_cast<cudaStream_t>(stream)));
}

size_t dspark_embed_workspace_size(const dspark_embed_problem_t* prob, int64_t grads) {
  if (check_embed(prob) != DSPARK_OK) return 0;
  return grads ? embed::view(nullptr, embed_plan(prob)).bytes : sizeof(embed::WsEmbedHeader);
}

dspark_status_t dspark_embed_fwd(const dspark_embed_problem_t* prob, const void* table, int64_t table_ld, void* out,
                                 int64_t out_ld, void* ws, size_t ws_bytes, dspark_stream_t stream) {
  dspark_status_t st = check_embed(prob);
  if (st != DSPARK_OK) return st;
  if (prob->ids == nullptr) return DSPARK_ERR_INVALID_ARG;
  if ((st = check_matrix(table, table_ld, prob->D, prob->dtype)) != DSPARK_OK) return st;
  if ((st = check_matrix(out, out_ld, prob->D, prob->dtype)) != DSPARK_OK) return st;
  if ((st = check_ws(ws, ws_bytes, dspark_embed_workspace_size(prob, 0))) != DSPARK_OK) return st;
  const embed::FwdArgs a{*prob, table, table_ld, out, out_ld, static_cast<embed::WsEmbedHeader*>(ws)};
  return cuda_status(embed::launch_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

dspark_status_t dspark_embed_bwd(const dspark_embed_problem_t* prob, const void* dout, int64_t dout_ld, void* dtable,
                                 int64_t dtable_ld, int64_t dtable_dtype, int64_t accumulate, void* ws,
                                 size_t ws_bytes, dspark_stream_t stream) {
  dspark_status_t st = check_embed(prob);
  if (st != DSPARK_OK) return st;
  if (prob->ids == nullptr || !is_dtype(dtable_dtype)) return DSPARK_ERR_INVALID_ARG;
  if (accumulate && dtable_dtype != DSPARK_F32) return DSPARK_ERR_UNSUPPORTED;
  if ((st = check_matrix(dout, dout_ld, prob->D, prob->dtype)) != DSPARK_OK) return st;
  if ((st = check_matrix(dtable, dtable_ld, prob->D, dtable_dtype)) != DSPARK_OK) return st;
  if ((st = check_ws(ws, ws_bytes, dspark_embed_workspace_size(prob, 1))) != DSPARK_OK) return st;
  embed::BwdArgs a{};
  a.p = *prob;
  a.dout = dout, a.dout_ld = dout_ld;
  a.dtable = dtable, a.dtable_ld = dtable_ld;
  a.table_f32 = dtable_dtype == DSPARK_F32;
  a.accumulate = accumulate ? 1 : 0;
  a.plan = embed_plan(prob);
  if (!accumulate) a.plan.fill = embed::fill_rows(a.plan, prob->D * elem_size(dtable_dtype));
  a.plan.zero_rows = embed::zero_rows(prob->Vt - a.plan.fill);
  a.ws = embed::view(ws, a.plan);
  return cuda_status(embed::launch_bwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dspark_grad_workspace_size(int64_t count) {
  return count < 1 || count > (int64_t(1) << 20) ? 0 : clip::ws_bytes(count);
}

dspark_status_t dspark_grad_sumsq(const dspark_tensor_t* tensors, int64_t count, double* sumsq, void* ws,
                                  size_t ws_bytes, dspark_stream_t stream) {
  dspark_status_t st = check_tensors(tensors, count, false);
  if (st != DSPARK_OK) return st;
  if (sumsq == nullptr) return DSPARK_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, clip::ws_bytes(count))) != DSPARK_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int64_t n = 0;
  const cudaError_t e = clip::launch_sumsq(tensors, count, ws, s, &n);
  return cuda_status(e != cudaSuccess ? e : clip::launch_total(ws, n, sumsq, s));
}

dspark_status_t dspark_grad_scale(const dspark_tensor_t* tensors, int64_t count, const double* sumsq, float max_norm,
                                  float* norm, float* coef, void* ws, size_t ws_bytes, dspark_stream_t stream) {
  dspark_status_t st = check_tensors(tensors, count, true);
  if (st != DSPARK_OK) return st;
  if (sumsq == nullptr || !(max_norm > 0.f)) return DSPARK_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, clip::ws_bytes(count))) != DSPARK_OK) return st;
  return cuda_status(clip::launch_scale(tensors, count, sumsq, 0, max_norm, norm, coef, ws,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

dspark_status_t dspark_grad_clip(const dspark_tensor_t* tensors, int64_t count, float max_norm, float* norm,
                                 float* coef, void* ws, size_t ws_bytes, dspark_stream_t stream) {
  dspark_status_t st = check_tensors(tensors, count, true);
  if (st != DSPARK_OK) return st;
  if (!(max_norm > 0.f)) return DSPARK_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, clip::ws_bytes(count))) != DSPARK_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int64_t n = 0;
  cudaError_t e = clip::launch_sumsq(tensors, count, ws, s, &n);
  if (e != cudaSuccess) return cuda_status(e);
  // One launch's partial sums are few: every CTA of the scaling adds them up for itself.  Those
  // of several are added up once (or each CTA of each launch would read all of them: 20000
  // tensors of 9000 bf16 elements 668 against 429 us).
  double* total = nullptr;
  if (clip::launches(count) > 1) {
    total = clip::total_of_call(ws);
    if ((e = clip::launch_total(ws, n, total, s)) != cudaSuccess) return cuda_status(e);
  }
  return cuda_status(clip::launch_scale(tensors, count, total, n, max_norm, norm, coef, ws, s));
}

}  // extern "C"
