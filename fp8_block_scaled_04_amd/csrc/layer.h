// Internal interface of the norm, routing and expert kernels: launch arguments
// and the launchers.  Arguments are checked by the C ABI layer (layer_api.hip);
// definitions are in include/fp8bs_layer.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {

struct NormArgs {
  const void* x;
  const void* residual;      // may be nullptr
  const void* weight;
  bool weight_f32;
  float eps;
  int64_t M;
  int32_t K;
  void* h;                   // nullptr with residual
  void* y;                   // may be nullptr
  uint8_t* q;
  float* s;
  float* rstd;               // may be nullptr
};

struct NormBackArgs {
  const void* dy;
  const void* h;
  const float* rstd;
  const void* weight;
  bool weight_f32;
  const void* dh;            // may be nullptr
  int64_t M;
  int32_t K;
  void* dx;
  float* dweight;
  bool accumulate;
  int32_t groups;            // row groups, one partial dweight each
  float* part;               // [groups][K]
};

struct RouteArgs {
  const void* logits;
  bool logits_f32, renorm;
  int64_t T;
  int32_t E, topk;
  int32_t* ids;              // backward: input
  float* weights;            // backward: the weights' gradients
  void* dlogits;             // backward only
};

struct ExpertArgs {
  const uint8_t* x;
  const float* sx;
  const int32_t* ids;
  const float* weights;
  const uint8_t* w13;
  const float* s13;
  const uint8_t* w2;
  const float* s2;
  void* out;
  bool out_f32;
  int32_t T, H, I, E, topk;
  // workspace
  uint16_t* hi;              // [T topk][I] BF16, weighted activations
  uint16_t* lo;              // what hi leaves
  float* part;               // [T topk][H] second product, by place
  uint32_t* image;           // jobs, their number, rows
};

int32_t norm_back_groups(int64_t M, int64_t K);
// How a call of these sizes runs: rows per pass, columns of the two products,
// waves that share the second's.
struct ExpertTile {
  int32_t rows, up, down, waves;
};
ExpertTile experts_tile(const ExpertArgs& a);
// Bytes of the workspace; lays it out from `base`.
int64_t experts_workspace(ExpertArgs& a, void* base);

hipError_t launch_rms_norm(const NormArgs& a, bool pow2, hipStream_t stream);
hipError_t launch_rms_norm_back(const NormBackArgs& a, hipStream_t stream);
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream);
hipError_t launch_moe_route_back(const RouteArgs& a, hipStream_t stream);
hipError_t launch_moe_experts(const ExpertArgs& a, hipStream_t stream);

}  // namespace fp8bs
