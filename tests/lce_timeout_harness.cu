// Test harness for waits that run out inside the linear cross entropy's products (compiled by
// tests/test_train_ops_timeout_gpu.py with a wait limit of a nanosecond, so that ordinary
// waits run out).  Nothing is broken: every copy and every MMA that was begun ends by itself.
#include "lce.cu"

// Forward and backward, whatever the waits did; returns the launches' error.
extern "C" int lce_timeout_run(const dspark_lce_problem_t* p, const dspark_lce_out_t* out, const dspark_lce_grads_t* g,
                               void* ws, cudaStream_t s) {
  using namespace dspark::lce;
  const Plan plan = make_plan(p->R, p->V, p->H, p->hidden_grad_only != 0);
  const cudaError_t e = launch_fwd(*p, *out, plan, view(ws, plan), false, s);
  return int(e != cudaSuccess ? e : launch_bwd(*p, *g, plan, view(ws, plan), s));
}

extern "C" uint64_t lce_timeout_limit_ns() { return dspark::kWaitLimitNs; }
