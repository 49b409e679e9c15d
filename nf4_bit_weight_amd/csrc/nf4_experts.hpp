// Launch interface of the expert kernels (nf4_experts.hip), between the C ABI of
// nf4_experts.h and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4 {

struct RouteArgs {
  const void* logits;
  bool bf16;
  int64_t stride;
  int32_t T, E, k;
  const float* bias;
  bool sigmoid, top2, renorm;
  int32_t groups, top_groups;
  float scale;
  float* weights;
  int32_t* experts;
  int32_t lanes = 0, group_lds = 0, plan_lds = 0;               // of the launch
};

struct PlanArgs {
  const int32_t* experts;
  int32_t T, k, E;
  int32_t *offsets, *tokens, *slots;
};

struct RowsArgs {
  bool bf16;
  int64_t H;
  int32_t T, k;
  const int32_t* slots;
  const int32_t* end;
  bool fill;
};

size_t plan_ws_bytes(int64_t T, int32_t k, int32_t E);
hipError_t launch_route(const RouteArgs& a, const PlanArgs& plan, void* ws, hipStream_t stream);   // plan.offsets NULL: no plan
hipError_t launch_route_bwd(const RouteArgs& a, const float* grad_weights, void* grad_logits, hipStream_t stream);
hipError_t launch_plan(const PlanArgs& a, void* ws, hipStream_t stream);
hipError_t launch_gather(const RowsArgs& a, const void* x, int64_t stride, void* rows, hipStream_t stream);
hipError_t launch_gather_bwd(const RowsArgs& a, const void* grad_rows, void* grad_x, hipStream_t stream);
hipError_t launch_combine(const RowsArgs& a, const void* rows, const float* weights, void* out, hipStream_t stream);
hipError_t launch_combine_bwd(const RowsArgs& a, const void* grad_out, int64_t stride, const void* rows,
                              const float* weights, void* grad_rows, float* grad_weights, hipStream_t stream);

}  // namespace nf4
