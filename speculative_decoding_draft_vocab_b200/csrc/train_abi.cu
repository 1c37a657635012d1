// Entry points of the training-step operators beside the loss (include/dspark.h): host-side
// validation, workspace carving and the launches.  No allocation, no synchronisation.
#include "internal.cuh"
#include "lce.cuh"

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
  if (!(p->z_alpha >= 0.f)) return DSPARK_ERR_INVALID_ARG;
  if (p->H % 8 || p->hidden_ld % 8 || p->weight_ld % 8 || !aligned16(p->hidden) || !aligned16(p->weight))
    return DSPARK_ERR_ALIGNMENT;
  return DSPARK_OK;
}

dspark_status_t check_ws(const void* ws, size_t have, size_t need) {
  if (ws == nullptr) return DSPARK_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return DSPARK_ERR_ALIGNMENT;
  return have < need ? DSPARK_ERR_WORKSPACE : DSPARK_OK;
}

}  // namespace

extern "C" {

size_t dspark_lce_workspace_size(const dspark_lce_problem_t* prob, const dspark_lce_grads_t* grads) {
  if (check_lce(prob) != DSPARK_OK) return 0;
  const bool bwd = grads && (grads->dhidden || grads->dweight);
  return lce::offsets(lce::make_plan(prob->R, prob->V, prob->H), bwd, bwd && grads->dhidden).bytes;
}

dspark_status_t dspark_lce_fwd(const dspark_lce_problem_t* prob, const dspark_lce_out_t* out, void* ws,
                               size_t ws_bytes, dspark_stream_t stream) {
  if (out == nullptr) return DSPARK_ERR_INVALID_ARG;
  dspark_status_t st = check_lce_call(prob);
  if (st != DSPARK_OK) return st;
  if ((st = check_ws(ws, ws_bytes, dspark_lce_workspace_size(prob, nullptr))) != DSPARK_OK) return st;
  const lce::Plan plan = lce::make_plan(prob->R, prob->V, prob->H);
  return cuda_status(lce::launch_fwd(*prob, *out, plan, lce::view(ws, plan), reinterpret_cast<cudaStream_t>(stream)));
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
    const bool f32 = grads->dweight_dtype == DSPARK_F32;
    if (!f32 && grads->dweight_dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARG;
    if (grads->dweight_ld < prob->H) return DSPARK_ERR_INVALID_ARG;
    if (grads->accumulate && !f32) return DSPARK_ERR_UNSUPPORTED;  // a bf16 sum over calls would lose its small terms
    if (!aligned16(grads->dweight) || grads->dweight_ld % (f32 ? 4 : 8)) return DSPARK_ERR_ALIGNMENT;
  }
  if ((st = check_ws(ws, ws_bytes, dspark_lce_workspace_size(prob, grads))) != DSPARK_OK) return st;
  const lce::Plan plan = lce::make_plan(prob->R, prob->V, prob->H);
  return cuda_status(lce::launch_bwd(*prob, *grads, plan, lce::view(ws, plan), reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
