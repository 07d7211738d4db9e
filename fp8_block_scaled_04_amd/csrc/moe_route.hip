// The router's choice of experts and its gradient (include/fp8bs_layer.h,
// fp8bs_moe_route and fp8bs_moe_route_backward).
//
// A wave holds one token's logits, expert 64 n + lane at v[n] of a lane.
#include <algorithm>

#include "layer.h"
#include "quant_common.h"

namespace fp8bs {
namespace {

constexpr int kWaves = 4;   // tokens per workgroup

__device__ __forceinline__ float logit(const RouteArgs& a, int64_t at) {
  if (a.logits_f32) return static_cast<const float*>(a.logits)[at];
  return __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t*>(a.logits)[at] << 16);
}

// Logits as whole numbers of the same order; 0 for an expert that is left out
// (-inf, NaN), as no other logit has it.  -0 counts as 0.
__device__ __forceinline__ uint32_t rank_of(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  return x > -__builtin_inff() ? ((b & 0x80000000u) ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float logit_of(uint32_t rank) {
  return __builtin_bit_cast(float, (rank & 0x80000000u) ? rank & 0x7FFFFFFFu : ~rank);
}

// exp(x - top), top the largest logit of those that count: 0 for one that is
// left out, and where top is +inf 1 for the logits equal to it.
__device__ __forceinline__ float weight_of(float x, float top) {
  return x > -__builtin_inff() ? (x == top ? 1.0f : expf(x - top)) : 0.0f;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
// The largest of the wave's values, by DPP (a shuffle through LDS costs several
// times as much, and topk of these follow one another).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t max_step(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max_step<0x111, 0xF>(v);                       // row_shr 1, 2, 4, 8: a row's last lane has its largest
  v = max_step<0x112, 0xF>(v);
  v = max_step<0x114, 0xF>(v);
  v = max_step<0x118, 0xF>(v);
  v = max_step<0x142, 0xA>(v);                       // row_bcast 15, 31: into the rows after
  v = max_step<0x143, 0xC>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// N: experts per lane.
template <int N>
__global__ __launch_bounds__(64 * kWaves) void k_route(RouteArgs a) {
  const int lane = threadIdx.x % 64;
  const int64_t step = (int64_t)gridDim.x * kWaves;
  float next[N];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int e = 64 * n + lane;
      next[n] = e < a.E ? logit(a, t * a.E + e) : -__builtin_inff();
    }
  };
  int64_t t = (int64_t)blockIdx.x * kWaves + threadIdx.x / 64;
  if (t < a.T) fetch(t);
  for (; t < a.T; t += step) {
    uint32_t v[N];
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = rank_of(next[n]);
    if (t + step < a.T) fetch(t + step);
    float all = 0.0f, top = 0.0f;
    // lane j keeps place j
    int id = -1;
    float x = -__builtin_inff();
    for (int j = 0; j < a.topk; ++j) {
      uint32_t best = v[0];
#pragma unroll
      for (int n = 1; n < N; ++n) best = max(best, v[n]);
      best = wave_max(best);
      if (j == 0) {
        top = logit_of(best);
        if (!a.renorm && best) {
#pragma unroll
          for (int n = 0; n < N; ++n) all += v[n] ? weight_of(logit_of(v[n]), top) : 0.0f;
          all = wave_sum(all);
        }
      }
      if (!best) break;
      int e = 0;
#pragma unroll
      for (int n = N - 1; n >= 0; --n) {
        const uint64_t hit = __builtin_amdgcn_ballot_w64(v[n] == best);
        if (hit) e = 64 * n + __builtin_ctzll(hit);
      }
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (e == 64 * n + lane) v[n] = 0u;
      if (lane == j) id = e, x = logit_of(best);
    }
    const float w = id >= 0 ? weight_of(x, top) : 0.0f;
    const float sum = a.renorm ? wave_sum(w) : all;
    if (lane < a.topk) {
      a.ids[t * a.topk + lane] = id;
      a.weights[t * a.topk + lane] = id >= 0 ? w / sum : 0.0f;
    }
  }
}

template <int N>
__global__ __launch_bounds__(64 * kWaves) void k_route_back(RouteArgs a) {
  const int lane = threadIdx.x % 64;
  for (int64_t t = (int64_t)blockIdx.x * kWaves + threadIdx.x / 64; t < a.T; t += (int64_t)gridDim.x * kWaves) {
    // place `lane`: its expert, logit and gradient
    int id = lane < a.topk ? a.ids[t * a.topk + lane] : -1;
    const bool there = (uint32_t)id < (uint32_t)a.E;
    float x = there ? logit(a, t * a.E + id) : -__builtin_inff();
    if (!(x > -__builtin_inff())) x = -__builtin_inff();
    const float g = there ? a.weights[t * a.topk + lane] : 0.0f;
    float p[N], add[N];                              // p_i of each expert, and p_i G_i
    float mean, place;                               // place: p of this place's expert
    if (a.renorm) {
      const float top = wave_max(x);
      const float w = weight_of(x, top), sum = wave_sum(w);
      place = sum > 0.0f ? w / sum : 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n) p[n] = 0.0f;
    } else {
      float l[N], top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int e = 64 * n + lane;
        l[n] = e < a.E ? logit(a, t * a.E + e) : -__builtin_inff();
        if (!(l[n] > -__builtin_inff())) l[n] = -__builtin_inff();
        top = fmaxf(top, l[n]);
      }
      top = wave_max(top);
#pragma unroll
      for (int n = 0; n < N; ++n) p[n] = weight_of(l[n], top), sum += p[n];
      sum = wave_sum(sum);
#pragma unroll
      for (int n = 0; n < N; ++n) p[n] = sum > 0.0f ? p[n] / sum : 0.0f;
      place = sum > 0.0f ? weight_of(x, top) / sum : 0.0f;
    }
    if (place == 0.0f) id = -1;
    mean = wave_sum(place > 0.0f ? place * g : 0.0f);
    const float mine = place > 0.0f ? place * (a.renorm ? g - mean : g) : 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) add[n] = a.renorm ? 0.0f : -(p[n] * mean);
    for (int j = 0; j < a.topk; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float d = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mine), j));
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (e == 64 * n + lane) add[n] += d;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int e = 64 * n + lane;
      if (e >= a.E) continue;
      if (a.logits_f32) static_cast<float*>(a.dlogits)[t * a.E + e] = add[n];
      else static_cast<__bf16*>(a.dlogits)[t * a.E + e] = (__bf16)add[n];
    }
  }
}

// As many workgroups as run at once: starting one takes longer than a token.
unsigned grid_of(int64_t T) { return (unsigned)std::min<int64_t>((T + kWaves - 1) / kWaves, 2048); }

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
  const auto k = a.E <= 64 ? k_route<1> : a.E <= 128 ? k_route<2> : a.E <= 256 ? k_route<4> : k_route<16>;
  k<<<grid_of(a.T), 64 * kWaves, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_moe_route_back(const RouteArgs& a, hipStream_t stream) {
  const auto k =
      a.E <= 64 ? k_route_back<1> : a.E <= 128 ? k_route_back<2> : a.E <= 256 ? k_route_back<4> : k_route_back<16>;
  k<<<grid_of(a.T), 64 * kWaves, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace fp8bs
