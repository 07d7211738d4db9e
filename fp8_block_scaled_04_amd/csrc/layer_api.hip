// C ABI of the norm, routing and expert calls (include/fp8bs_layer.h): argument
// checks and dispatch.
#include <algorithm>
#include <cmath>

#include "abi_common.h"
#include "fp8bs_layer.h"
#include "layer.h"

namespace {

using fp8bs::aligned16;
using fp8bs::aligned4;
using fp8bs::check_device;
using fp8bs::launched;

constexpr int64_t kMaxRows = 0x7FFFFFFF;

bool norm_sizes_fit(int64_t M, int64_t K) { return M >= 0 && M <= kMaxRows && K > 0 && K <= 16384 && K % 128 == 0; }

bool known_type(int32_t t) { return t == FP8BS_BF16 || t == FP8BS_FP32; }

bool route_sizes_fit(int64_t T, int32_t E, int32_t topk) {
  return T >= 0 && T <= kMaxRows && E > 0 && E <= 1024 && topk > 0 && topk <= std::min(E, 64);
}

bool width_fits(int64_t n) { return n > 0 && n <= 32768 && n % 128 == 0; }

bool expert_sizes_fit(int64_t T, int64_t H, int64_t I, int32_t E, int32_t topk) {
  return T >= 0 && T <= 128 && width_fits(H) && width_fits(I) && 2 * H * I < ((int64_t)1 << 31) && E > 0 && E <= 1024 &&
         topk > 0 && topk <= 16;
}

}  // namespace

extern "C" {

fp8bs_status fp8bs_rms_norm_quantize(const void* x, const void* residual, const void* weight, int32_t weight_type,
                                     float eps, int64_t M, int64_t K, void* h, void* y, uint8_t* q, float* s,
                                     float* rstd, uint32_t flags, fp8bs_stream_t stream) {
  if (!norm_sizes_fit(M, K)) return FP8BS_ERR_SHAPE;
  if ((flags & ~(uint32_t)FP8BS_SCALE_POW2) || !known_type(weight_type)) return FP8BS_ERR_FLAGS;
  if (!std::isfinite(eps) || eps < 0x1p-126f) return FP8BS_ERR_FLAGS;
  if (M == 0) return FP8BS_OK;
  if (!x || !weight || !q || !s || !residual != !h) return FP8BS_ERR_NULL;
  for (const void* p : {x, residual, weight, (const void*)h, (const void*)y, (const void*)q, (const void*)s})
    if (!aligned16(p)) return FP8BS_ERR_ALIGN;
  if (!aligned4(rstd)) return FP8BS_ERR_ALIGN;
  if (fp8bs_status e = check_device()) return e;
  const fp8bs::NormArgs a{x, residual, weight, weight_type == FP8BS_FP32, eps, M, (int32_t)K, h, y, q, s, rstd};
  (void)hipGetLastError();
  return launched(fp8bs::launch_rms_norm(a, (flags & FP8BS_SCALE_POW2) != 0, (hipStream_t)stream));
}

fp8bs_status fp8bs_rms_norm_backward_workspace(int64_t M, int64_t K, int64_t* bytes) {
  if (!norm_sizes_fit(M, K)) return FP8BS_ERR_SHAPE;
  if (!bytes) return FP8BS_ERR_NULL;
  *bytes = (int64_t)fp8bs::norm_back_groups(M, K) * K * 4;
  return FP8BS_OK;
}

fp8bs_status fp8bs_rms_norm_backward(const void* dy, const void* h, const float* rstd, const void* weight,
                                     int32_t weight_type, const void* dh, int64_t M, int64_t K, void* dx,
                                     float* dweight, int32_t accumulate, void* workspace, int64_t workspace_bytes,
                                     fp8bs_stream_t stream) {
  if (!norm_sizes_fit(M, K)) return FP8BS_ERR_SHAPE;
  const int32_t groups = fp8bs::norm_back_groups(M, K);
  if (workspace_bytes < (int64_t)groups * K * 4) return FP8BS_ERR_SHAPE;
  if (!known_type(weight_type) || (accumulate != 0 && accumulate != 1)) return FP8BS_ERR_FLAGS;
  if (M == 0 && accumulate) return FP8BS_OK;
  if (!dweight || (M > 0 && (!dy || !h || !rstd || !weight || !dx || !workspace))) return FP8BS_ERR_NULL;
  for (const void* p : {dy, h, weight, dh, (const void*)dx, (const void*)dweight, (const void*)workspace})
    if (!aligned16(p)) return FP8BS_ERR_ALIGN;
  if (!aligned4(rstd)) return FP8BS_ERR_ALIGN;
  if (fp8bs_status e = check_device()) return e;
  const fp8bs::NormBackArgs a{dy, h, rstd, weight, weight_type == FP8BS_FP32, dh, M, (int32_t)K, dx, dweight,
                              accumulate == 1, groups, static_cast<float*>(workspace)};
  (void)hipGetLastError();
  return launched(fp8bs::launch_rms_norm_back(a, (hipStream_t)stream));
}

fp8bs_status fp8bs_moe_route(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t topk,
                             int32_t* ids, float* weights, uint32_t flags, fp8bs_stream_t stream) {
  if (!route_sizes_fit(T, E, topk)) return FP8BS_ERR_SHAPE;
  if ((flags & ~(uint32_t)FP8BS_ROUTE_RENORM) || !known_type(logits_type)) return FP8BS_ERR_FLAGS;
  if (T == 0) return FP8BS_OK;
  if (!logits || !ids || !weights) return FP8BS_ERR_NULL;
  if (!aligned16(logits) || !aligned4(ids) || !aligned4(weights)) return FP8BS_ERR_ALIGN;
  if (fp8bs_status e = check_device()) return e;
  const fp8bs::RouteArgs a{logits, logits_type == FP8BS_FP32, (flags & FP8BS_ROUTE_RENORM) != 0, T, E, topk, ids,
                           weights, nullptr};
  (void)hipGetLastError();
  return launched(fp8bs::launch_moe_route(a, (hipStream_t)stream));
}

fp8bs_status fp8bs_moe_route_backward(const void* logits, int32_t logits_type, const int32_t* ids,
                                      const float* dweights, int64_t T, int32_t E, int32_t topk, void* dlogits,
                                      uint32_t flags, fp8bs_stream_t stream) {
  if (!route_sizes_fit(T, E, topk)) return FP8BS_ERR_SHAPE;
  if ((flags & ~(uint32_t)FP8BS_ROUTE_RENORM) || !known_type(logits_type)) return FP8BS_ERR_FLAGS;
  if (T == 0) return FP8BS_OK;
  if (!logits || !ids || !dweights || !dlogits) return FP8BS_ERR_NULL;
  if (!aligned16(logits) || !aligned4(ids) || !aligned4(dweights) || !aligned16(dlogits)) return FP8BS_ERR_ALIGN;
  if (fp8bs_status e = check_device()) return e;
  const fp8bs::RouteArgs a{logits, logits_type == FP8BS_FP32, (flags & FP8BS_ROUTE_RENORM) != 0, T, E, topk,
                           const_cast<int32_t*>(ids), const_cast<float*>(dweights), dlogits};
  (void)hipGetLastError();
  return launched(fp8bs::launch_moe_route_back(a, (hipStream_t)stream));
}

fp8bs_status fp8bs_moe_experts_tile(int64_t T, int64_t H, int64_t I, int32_t E, int32_t topk, int32_t* rows,
                                    int32_t* up_columns, int32_t* down_columns, int32_t* down_waves) {
  if (!expert_sizes_fit(T, H, I, E, topk)) return FP8BS_ERR_SHAPE;
  if (!rows || !up_columns || !down_columns || !down_waves) return FP8BS_ERR_NULL;
  fp8bs::ExpertArgs a{};
  a.T = (int32_t)T, a.H = (int32_t)H, a.I = (int32_t)I, a.E = E, a.topk = topk;
  const fp8bs::ExpertTile t = experts_tile(a);
  *rows = t.rows, *up_columns = t.up, *down_columns = t.down, *down_waves = t.waves;
  return FP8BS_OK;
}

fp8bs_status fp8bs_moe_experts_workspace(int64_t T, int64_t H, int64_t I, int32_t E, int32_t topk, int64_t* bytes) {
  if (!expert_sizes_fit(T, H, I, E, topk)) return FP8BS_ERR_SHAPE;
  if (!bytes) return FP8BS_ERR_NULL;
  fp8bs::ExpertArgs a{};
  a.T = (int32_t)T, a.H = (int32_t)H, a.I = (int32_t)I, a.E = E, a.topk = topk;
  *bytes = T == 0 ? 0 : experts_workspace(a, nullptr);
  return FP8BS_OK;
}

fp8bs_status fp8bs_moe_experts(const uint8_t* x, const float* sx, const int32_t* ids, const float* weights,
                               const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2, void* out,
                               int64_t T, int64_t H, int64_t I, int32_t E, int32_t topk, int32_t out_dtype,
                               void* workspace, int64_t workspace_bytes, fp8bs_stream_t stream) {
  if (!expert_sizes_fit(T, H, I, E, topk)) return FP8BS_ERR_SHAPE;
  fp8bs::ExpertArgs a{x, sx, ids, weights, w13, s13, w2, s2, out, out_dtype == FP8BS_OUT_FP32, (int32_t)T, (int32_t)H,
                      (int32_t)I, E, topk, nullptr, nullptr, nullptr, nullptr};
  if (workspace_bytes < (T == 0 ? 0 : experts_workspace(a, workspace))) return FP8BS_ERR_SHAPE;
  if (out_dtype != FP8BS_OUT_BF16 && out_dtype != FP8BS_OUT_FP32) return FP8BS_ERR_FLAGS;
  if (T == 0) return FP8BS_OK;
  if (!x || !sx || !ids || !weights || !w13 || !s13 || !w2 || !s2 || !out || !workspace) return FP8BS_ERR_NULL;
  for (const void* p : {(const void*)x, (const void*)w13, (const void*)w2, (const void*)out, (const void*)workspace})
    if (!aligned16(p)) return FP8BS_ERR_ALIGN;
  for (const void* p : {(const void*)sx, (const void*)ids, (const void*)weights, (const void*)s13, (const void*)s2})
    if (!aligned4(p)) return FP8BS_ERR_ALIGN;
  if (fp8bs_status e = check_device()) return e;
  (void)hipGetLastError();
  return launched(fp8bs::launch_moe_experts(a, (hipStream_t)stream));
}

}  // extern "C"
