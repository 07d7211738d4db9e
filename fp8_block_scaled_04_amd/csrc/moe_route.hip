// The router's choice of experts and its gradient (include/fp8bs_layer.h,
// fp8bs_moe_route and fp8bs_moe_route_backward).
//
// Bound by instructions: each choice is a maximum over a token's logits, and one
// wave instruction takes four cycles.  So 16 lanes hold a token where they can
// (up to 256 experts and 16 places): each lane has a 16th of the experts, four tokens
// share each instruction, and a maximum over 16 lanes is four DPP steps.  Otherwise a
// wave holds one token, expert 64 n + lane at v[n] of a lane.
//
// 16384 tokens, 256 experts, 8 places: 7.5 us (BF16 logits, 9 MB), the gradient 7.3
// (FP32, 18 MB); 64 tokens 3.8 us, all of it latency.  (One token per wave against 16
// lanes, logits read one by one: 14.7 and 10.4 us, the gradient 12.6 and 8.1.)
// 16384 tokens of 384, 512 and 1024 experts, BF16, one token per wave: 39, 40 and 50 us,
// the gradient (over the chosen) 22, 23 and 24; by bytes 2, 3 and 6 each.  All three have
// 16 logits per lane, however many of them there are.
#include <algorithm>
#include <type_traits>

#include "layer.h"
#include "quant_common.h"

namespace fp8bs {
namespace {

constexpr int kWaves = 4;   // tokens per workgroup

__device__ __forceinline__ float logit(const RouteArgs& a, int64_t at) {
  if (a.logits_f32) return static_cast<const float*>(a.logits)[at];
  return __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t*>(a.logits)[at] << 16);
}

__device__ __forceinline__ void put(const RouteArgs& a, int64_t at, float v) {
  if (a.logits_f32) static_cast<float*>(a.dlogits)[at] = v;
  else static_cast<__bf16*>(a.dlogits)[at] = (__bf16)v;
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
      put(a, t * a.E + e, add[n]);
    }
  }
}

// ---- four tokens per wave ----

// A value of every lane of the row of 16, joined by f, on all of its lanes.
template <class T, class F>
__device__ __forceinline__ T row_join(T v, F f) {
  const auto other = [](T x, auto ctrl) {
    return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v = f(v, other(v, std::integral_constant<int, 0xB1>()));    // quad_perm 1,0,3,2
  v = f(v, other(v, std::integral_constant<int, 0x4E>()));    // quad_perm 2,3,0,1
  v = f(v, other(v, std::integral_constant<int, 0x141>()));   // row_half_mirror
  return f(v, other(v, std::integral_constant<int, 0x140>()));  // row_mirror
}
__device__ __forceinline__ float row_sum(float v) {
  return row_join(v, [](float x, float y) { return x + y; });
}
__device__ __forceinline__ float row_max(float v) {
  return row_join(v, [](float x, float y) { return fmaxf(x, y); });
}

constexpr int kTokens = 4 * kWaves;   // per workgroup

// A logit's rank and its expert as one whole number, exact in a double: keys of
// a token all differ, the lower expert first among equal logits, and v_max_f64
// takes the larger of two in one instruction.  Keys below kFirst are left out.
constexpr double kFirst = 1024.0;
__device__ __forceinline__ double key_of(uint32_t rank, int e) {
  return __builtin_fma((double)rank, kFirst, rank ? (double)(1023 - e) : 0.0);
}
__device__ __forceinline__ uint32_t rank_in(double key) { return (uint32_t)(key * 0x1p-10); }
__device__ __forceinline__ int expert_in(double key) {
  return 1023 - (int)(key - (double)rank_in(key) * kFirst);
}

__device__ __forceinline__ double row_max(double v) {
  const auto step = [](double x, auto ctrl) {
    constexpr int kCtrl = decltype(ctrl)::value;
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, kCtrl, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), kCtrl, 0xF, 0xF, true);
    return __builtin_fmax(x, __builtin_bit_cast(double, (uint64_t)hi << 32 | lo));
  };
  v = step(v, std::integral_constant<int, 0xB1>());
  v = step(v, std::integral_constant<int, 0x4E>());
  v = step(v, std::integral_constant<int, 0x141>());
  return step(v, std::integral_constant<int, 0x140>());
}

// Falling order, by Batcher's odd-even merge sort (N a power of two; all indexes are
// known when compiled).
template <int N>
__device__ __forceinline__ void sort_falling(double (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int d = p; d >= 1; d /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int j = i + d;
        if (j >= N || i < d % p || (i - d % p) / d % 2 || i / (2 * p) != j / (2 * p)) continue;
        const double hi = __builtin_fmax(k[i], k[j]), lo = __builtin_fmin(k[i], k[j]);
        k[i] = hi;
        k[j] = lo;
      }
}

// Rows are read and written in pieces of P values, up to 16 bytes (piece_of below): a
// lane has every 16th piece, so that a wave's access is whole lines.  16384 tokens,
// 256 experts, in us, single values -> pieces: BF16 9.9 -> 7.5, its gradient (softmax
// over all) 13.0 -> 10.1; FP32 8.8 -> 8.2, its gradient (over the chosen) 7.5 -> 7.3, but
// 10.6 with a lane's values one after the other.
template <int P>
__device__ __forceinline__ int expert_at(int n, int l) {
  return n / P * (16 * P) + l * P + n % P;
}

// Lane l's logits of token t; -inf where there is none.
template <int N, int P>
__device__ __forceinline__ void read_row(float (&x)[N], const RouteArgs& a, int64_t t, int l) {
#pragma unroll
  for (int n = 0; n < N; ++n) x[n] = -__builtin_inff();
  if (t >= a.T) return;
#pragma unroll
  for (int n = 0; n < N; n += P) {
    const int e = expert_at<P>(n, l);
    if (e >= a.E) break;
    const int64_t at = t * a.E + e;
    if constexpr (P == 1) {
      x[n] = logit(a, at);
    } else {
      typedef uint32_t Piece __attribute__((ext_vector_type(P / 2)));
      if (P == 4 && a.logits_f32) {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + at);
        x[n] = v.x, x[n + 1] = v.y, x[n + 2] = v.z, x[n + 3] = v.w;
      } else {
        const Piece v = *reinterpret_cast<const Piece*>(static_cast<const uint16_t*>(a.logits) + at);
#pragma unroll
        for (int i = 0; i < P / 2; ++i) x[n + 2 * i] = bf16_lo(v[i]), x[n + 2 * i + 1] = bf16_hi(v[i]);
      }
    }
  }
}

// And its gradients.
template <int N, int P>
__device__ __forceinline__ void write_row(const float (&x)[N], const RouteArgs& a, int64_t t, int l) {
  if (t >= a.T) return;
#pragma unroll
  for (int n = 0; n < N; n += P) {
    const int e = expert_at<P>(n, l);
    if (e >= a.E) break;
    const int64_t at = t * a.E + e;
    if constexpr (P == 1) {
      put(a, at, x[n]);
    } else {
      typedef uint32_t Piece __attribute__((ext_vector_type(P / 2)));
      if (P == 4 && a.logits_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + at) = make_float4(x[n], x[n + 1], x[n + 2], x[n + 3]);
      } else {
        Piece v;
#pragma unroll
        for (int i = 0; i < P / 2; ++i) v[i] = pack2_bf16(x[n + 2 * i], x[n + 2 * i + 1]);
        *reinterpret_cast<Piece*>(static_cast<uint16_t*>(a.dlogits) + at) = v;
      }
    }
  }
}

// Each lane sorts its own N logits and keeps them in LDS; a choice is then the
// largest of the 16 lists' heads, and one list moves on.
template <int N, int P>
__global__ __launch_bounds__(64 * kWaves) void k_route_rows(RouteArgs a) {
  __shared__ double lists[N + 1][64 * kWaves];
  const int l = threadIdx.x % 16, tid = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * kTokens;
  float x[N];
  lists[N][tid] = 0.0;                               // (each lane reads and writes its own column only)
  // (the four rows of a wave go on together, so that their DPP steps see live lanes)
  int64_t t = (int64_t)blockIdx.x * kTokens + tid / 16;
  read_row<N, P>(x, a, t, l);
  for (int64_t first = (int64_t)blockIdx.x * kTokens; first < a.T; first += step, t += step) {
    double k[N];
#pragma unroll
    for (int n = 0; n < N; ++n) k[n] = key_of(rank_of(x[n]), expert_at<P>(n, l));
    float sum = 0.0f, top = 0.0f;
    if (!a.renorm) {
      double best = k[0];
#pragma unroll
      for (int n = 1; n < N; ++n) best = __builtin_fmax(best, k[n]);
      best = row_max(best);
      if (best >= kFirst) top = logit_of(rank_in(best));
#pragma unroll
      for (int n = 0; n < N; ++n) sum += weight_of(x[n], top);
    }
    read_row<N, P>(x, a, t + step, l);
    sort_falling(k);
#pragma unroll
    for (int n = 0; n < N; ++n) lists[n][tid] = k[n];
    // lane j keeps place j
    double head = k[0], mine = 0.0;
    int at = 0;
    for (int j = 0; j < a.topk; ++j) {
      const double best = row_max(head);
      if (l == j) mine = best;
      if (j == 0 && a.renorm && best >= kFirst) top = logit_of(rank_in(best));
      if (head == best && at < N) head = lists[++at][tid];
    }
    const bool there = mine >= kFirst;
    const float w = there ? weight_of(logit_of(rank_in(mine)), top) : 0.0f;
    sum = row_sum(a.renorm ? w : sum);
    if (l < a.topk && t < a.T) {
      a.ids[t * a.topk + l] = there ? expert_in(mine) : -1;
      a.weights[t * a.topk + l] = there ? w / sum : 0.0f;
    }
  }
}

template <int N, int P>
__global__ __launch_bounds__(64 * kWaves) void k_route_back_rows(RouteArgs a) {
  const int l = threadIdx.x % 16;
  const int64_t step = (int64_t)gridDim.x * kTokens;
  int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / 16;
  for (int64_t first = (int64_t)blockIdx.x * kTokens; first < a.T; first += step, t += step) {
    const bool live = t < a.T;
    // place l: its expert, logit and gradient
    const int id = live && l < a.topk ? a.ids[t * a.topk + l] : -1;
    const bool there = (uint32_t)id < (uint32_t)a.E;
    float x = there ? logit(a, t * a.E + id) : -__builtin_inff();
    if (!(x > -__builtin_inff())) x = -__builtin_inff();
    const float g = there ? a.weights[t * a.topk + l] : 0.0f;
    float p[N], place;                               // p_i of each expert; of this place's
    if (a.renorm) {
      const float w = weight_of(x, row_max(x)), sum = row_sum(w);
      place = sum > 0.0f ? w / sum : 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n) p[n] = 0.0f;
    } else {
      float top = -__builtin_inff(), sum = 0.0f;
      read_row<N, P>(p, a, t, l);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (!(p[n] > -__builtin_inff())) p[n] = -__builtin_inff();
        top = fmaxf(top, p[n]);
      }
      top = row_max(top);
#pragma unroll
      for (int n = 0; n < N; ++n) p[n] = weight_of(p[n], top), sum += p[n];
      sum = row_sum(sum);
#pragma unroll
      for (int n = 0; n < N; ++n) p[n] = sum > 0.0f ? p[n] / sum : 0.0f;
      place = sum > 0.0f ? weight_of(x, top) / sum : 0.0f;
    }
    const float mean = row_sum(place > 0.0f ? place * g : 0.0f);
    const int key = place > 0.0f ? id : -1;          // (places that count)
    const float d = place > 0.0f ? place * (a.renorm ? g - mean : g) : 0.0f;
    // an expert that stands in several places gets the sum of theirs, the same on
    // each of their lanes
    float total = 0.0f;
    for (int j = 0; j < a.topk; ++j) {
      const int from = (threadIdx.x & ~15) + j;      // (lane of the wave: shuffles take it modulo 64)
      const int other = __shfl(key, from);
      const float add = __shfl(d, from);
      total += other == key ? add : 0.0f;
    }
    if (!a.renorm) total -= place * mean;
#pragma unroll
    for (int n = 0; n < N; ++n) p[n] = -(p[n] * mean);
    write_row<N, P>(p, a, t, l);
    // the places' own experts, over what other lanes of this wave have just
    // written there (a wave's stores to one address stay in order)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (key >= 0) put(a, t * a.E + key, total);
  }
}

// As many workgroups as run at once.
unsigned grid_of(int64_t T, int tokens) { return (unsigned)std::min<int64_t>((T + tokens - 1) / tokens, 2048); }

bool by_rows(const RouteArgs& a) { return a.E <= 256 && a.topk <= 16; }
// Values of a piece: as many as 16 bytes and a lane hold, of rows that are whole pieces
// (arrays start at multiples of 16 bytes).
int piece_of(const RouteArgs& a) {
  if (!a.logits_f32 && a.E > 64 && a.E % 8 == 0) return 8;
  return a.E % 4 == 0 ? 4 : 1;
}
// f(N, P), both known when compiled.
template <class F>
void with_shape(const RouteArgs& a, F f) {
  const auto with_piece = [&](auto n) {
    const int p = piece_of(a);
    if constexpr (decltype(n)::value > 4)
      if (p == 8) return f(n, std::integral_constant<int, 8>());
    if (p == 4) return f(n, std::integral_constant<int, 4>());
    return f(n, std::integral_constant<int, 1>());
  };
  if (a.E <= 64) return with_piece(std::integral_constant<int, 4>());
  if (a.E <= 128) return with_piece(std::integral_constant<int, 8>());
  return with_piece(std::integral_constant<int, 16>());
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
  if (by_rows(a)) {
    with_shape(a, [&](auto n, auto p) {
      k_route_rows<decltype(n)::value, decltype(p)::value><<<grid_of(a.T, kTokens), 64 * kWaves, 0, stream>>>(a);
    });
  } else {
    const auto k = a.E <= 256 ? k_route<4> : k_route<16>;
    k<<<grid_of(a.T, kWaves), 64 * kWaves, 0, stream>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_moe_route_back(const RouteArgs& a, hipStream_t stream) {
  if (by_rows(a)) {
    with_shape(a, [&](auto n, auto p) {
      k_route_back_rows<decltype(n)::value, decltype(p)::value><<<grid_of(a.T, kTokens), 64 * kWaves, 0, stream>>>(a);
    });
  } else {
    const auto k = a.E <= 256 ? k_route_back<4> : k_route_back<16>;
    k<<<grid_of(a.T, kWaves), 64 * kWaves, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace fp8bs
