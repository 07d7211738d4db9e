// Residual addition, RMS norm and 1x128 quantization, and the norm's gradients
// (include/fp8bs_layer.h, fp8bs_rms_norm_quantize and fp8bs_rms_norm_backward).
//
// One workgroup per row at a time, the row in registers: sixteen lanes hold one
// 1x128 tile, eight values each, so the row's sum needs one pass through LDS and
// a tile's largest value four DPP steps.  y stays in FP32 between the norm and its
// codes (rounded to BF16 first, a code would be off by up to 2^-8 of the value more).
//
// HBM-bound.  8192 x 7168 with a residual: forward 70 us, 413 MB at 5.9 TB/s;
// backward 80 + 5 us (the sums over rows), 470 MB at 5.5 TB/s.  A plain copy of 2 GiB
// moves 4.9 TB/s; of these sizes a part is still in the last-level cache when the next
// call reads it, and nontemporal streams of 0.1 to 0.2 GB reach 6.1.  The forward pass
// keeps the vector unit busy 63 % of the time.  Narrow rows, forward, calls in a replayed
// graph: 8192 rows of 512, 1024 and 2048 take 8.5, 14.2 and 23.7 us (6.0, 12.0 and 23.9
// at the copy's rate), one, two and four waves per workgroup.
#include <algorithm>

#include "layer.h"
#include "quant_common.h"

namespace fp8bs {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The eight values of piece p (values 8 p .. 8 p + 7) of a BF16 row, still packed.
__device__ __forceinline__ u32x4 piece(const void* row, int p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row) + p);
}
// Stores past the caches in the forward pass, ordinary ones in the backward pass:
// 8192 x 7168, calls in a row on changing data, 69.8 against 76.2 us and 90.5
// against 85.9.  (Loads past the caches in both: 70 against 73, 84 against 91.)
template <bool NT>
__device__ __forceinline__ void put_piece(void* row, int p, u32x4 v) {
  u32x4* to = reinterpret_cast<u32x4*>(row) + p;
  if (NT) __builtin_nontemporal_store(v, to);
  else *to = v;
}
__device__ __forceinline__ void unpack8(float (&f)[8], u32x4 v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) f[2 * e] = bf16_lo(v[e]), f[2 * e + 1] = bf16_hi(v[e]);
}
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7])};
}
// Norm weights of a piece, BF16 or FP32.
__device__ __forceinline__ void weight8(float (&f)[8], const void* weight, bool f32, int p) {
  if (f32) {
    const float4* w = static_cast<const float4*>(weight) + 2 * p;
    const float4 a = w[0], b = w[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    unpack8(f, static_cast<const u32x4*>(weight)[p]);
  }
}

// Sum over a row's lanes (threadIdx.x; a workgroup has blockDim.y rows), the same
// order on every lane and call.  `red` has 16 floats of its own for each of two
// calls in a row: a wave may still read the last call's while another writes this
// one's.
__device__ __forceinline__ float group_sum(float v, float* red) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  const int waves = blockDim.x / 64;
  red += threadIdx.y * waves;
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
  __syncthreads();
  float t = 0.0f;
  for (int w = 0; w < waves; ++w) t += red[w];
  return t;
}

// V: pieces per lane.
template <int V, bool POW2>
__global__ __launch_bounds__(1024) void k_rms_norm(NormArgs a) {
  __shared__ float red[2][16];
  const int pieces = a.K / 8, threads = blockDim.x, tid = threadIdx.x;
  float w[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = v * threads + tid;
    if (p < pieces) weight8(w[v], a.weight, a.weight_f32, p);
  }
  int turn = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    const int64_t at = m * a.K;
    const uint16_t* xr = static_cast<const uint16_t*>(a.x) + at;
    const uint16_t* rr = static_cast<const uint16_t*>(a.residual) + at;
    u32x4 x[V], r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = v * threads + tid;
      x[v] = r[v] = u32x4{0u, 0u, 0u, 0u};
      if (p < pieces) {
        x[v] = piece(xr, p);
        if (a.residual) r[v] = piece(rr, p);
      }
    }
    float h[V][8], sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      unpack8(h[v], x[v]);
      if (a.residual) {
        // the stored sum is BF16, and the norm is that of the stored sum (what
        // the backward pass and the next layer see)
        float f[8];
        unpack8(f, r[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += h[v][e];
        const u32x4 b = pack8(f);
        unpack8(h[v], b);
        const int p = v * threads + tid;
        if (p < pieces) put_piece<true>(static_cast<uint16_t*>(a.h) + at, p, b);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(h[v][e], h[v][e], sum);
    }
    const float inv = 1.0f / sqrtf(group_sum(sum, red[turn]) / (float)a.K + a.eps);
    const uint32_t bits = __builtin_amdgcn_readfirstlane(__builtin_bit_cast(uint32_t, inv));
    const float rstd = __builtin_bit_cast(float, bits);
    if (a.rstd && tid == 0) a.rstd[m] = rstd;
    // rstd = up rest, up a power of two from 2^-16 to 2^63 and rest from 1 to 2 (below 1
    // only under 2^-16).  y = ((h up) weight) rest: the first product is exact (a BF16
    // number has no bit below 2^-133), so this rounds as (h weight) rstd does, but h
    // weight may leave FP32's normal range on its way to a y inside it.  (Choosing by the
    // weights' size where rstd < 2^-16, too: 8192 x 7168 73 us against 69.)
    const uint32_t power = max(bits & 0x7F800000u, 0x37800000u);
    const float up = __builtin_bit_cast(float, power);
    const float rest = rstd * __builtin_bit_cast(float, 0x7F000000u - power);   // (1 / up: 0 and NaN stay what they are)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = v * threads + tid;
      if (p >= pieces) break;                        // (all sixteen lanes of a tile or none)
      float amax = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[v][e] = h[v][e] * up * w[v][e] * rest;   // (exact up to rest for BF16 weights)
        amax = fmaxf(amax, __builtin_fabsf(h[v][e]));
      }
      if (a.y) put_piece<true>(static_cast<uint16_t*>(a.y) + at, p, pack8(h[v]));
      const TileScale t = tile_scale<POW2>(row16_max(amax));
      if (tid % 16 == 0) a.s[(int64_t)(p / 16) * a.M + m] = t.s;
      float c[8];
      if (__builtin_expect(__builtin_amdgcn_ballot_w64(t.sx != 1.0f) != 0, 0)) {
        // y is FP32, so a tile may lie below BF16's range: its scale is a few steps of
        // 2^-149 then, and quotients past 464 have to saturate (pack4_e4m3).  (Clamps
        // on every tile: 4096 x 16384 64.8 us against 63.1.)
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = clamp448(quot<POW2>(h[v][e] * t.sx, t));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = quot<POW2>(h[v][e], t);
      }
      // (ordinary stores: the product that reads the codes comes next)
      *reinterpret_cast<uint2*>(a.q + at + (int64_t)p * 8) =
          make_uint2(pack4_e4m3(c[0], c[1], c[2], c[3]), pack4_e4m3(c[4], c[5], c[6], c[7]));
    }
  }
}

// Row group g takes rows g, g + groups, ..., or with MANY blockDim.y rows of each
// such run at once (narrow rows: kBackLanes below); its sums for dweight stay in
// registers and leave as one partial row.  Two workgroups of seven waves per CU
// (7168 columns) cover each other's waits; the next row fetched ahead by one
// workgroup per CU (its registers leave no room for two) took 99 us against 84.
// Narrow rows, one at a time, leave a CU two to eight waves: 8192 rows of 512,
// 1024, 1536 and 2048 took 24.4, 28.7, 31.5 and 33.5 us, up to 512 lanes at work
// 12.7, 17.8, 25.5 and 28.5 (up to 1024: 14.6, 21.3, 24.1, 33.7; up to 256: 13.7,
// 21.1, 31.2, 33.2).
constexpr int kBackLanes = 512;
template <int V, bool MANY>
__global__ __launch_bounds__(MANY ? kBackLanes : 1024) void k_rms_norm_back(NormBackArgs a) {
  __shared__ float red[2][16];
  const int pieces = a.K / 8, threads = blockDim.x, tid = threadIdx.x;
  const int rows = MANY ? blockDim.y : 1, row = MANY ? threadIdx.y : 0;
  float w[V][8], dw[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = v * threads + tid;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[v][e] = dw[v][e] = 0.0f;
    if (p < pieces) weight8(w[v], a.weight, a.weight_f32, p);
  }
  int turn = 0;
  for (int64_t m0 = (int64_t)blockIdx.x * rows; m0 < a.M; m0 += (int64_t)a.groups * rows, turn ^= 1) {
    const int64_t m = m0 + row, at = m * a.K;
    const bool in = !MANY || m < a.M;                // (every wave takes part in the row sum's barrier)
    u32x4 dyp[V], hp[V], dhp[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = v * threads + tid;
      dyp[v] = hp[v] = dhp[v] = u32x4{0u, 0u, 0u, 0u};
      if (p < pieces && in) {
        dyp[v] = piece(static_cast<const uint16_t*>(a.dy) + at, p);
        hp[v] = piece(static_cast<const uint16_t*>(a.h) + at, p);
        if (a.dh) dhp[v] = piece(static_cast<const uint16_t*>(a.dh) + at, p);
      }
    }
    const float rstd = in ? a.rstd[m] : 0.0f;
    float g[V][8], n[V][8], dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      unpack8(g[v], dyp[v]);
      unpack8(n[v], hp[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[v][e] *= rstd;
        dw[v][e] = __builtin_fmaf(g[v][e], n[v][e], dw[v][e]);
        g[v][e] *= w[v][e];
        dot = __builtin_fmaf(g[v][e], n[v][e], dot);
      }
    }
    const float mean = group_sum(dot, red[turn]) / (float)a.K;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = v * threads + tid;
      if (p >= pieces || !in) break;
      float d[8];
      unpack8(d, dhp[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = __builtin_fmaf(rstd, __builtin_fmaf(-n[v][e], mean, g[v][e]), d[e]);
      put_piece<false>(static_cast<uint16_t*>(a.dx) + at, p, pack8(d));
    }
  }
  if (MANY) {                                        // the rows' sums, joined in their order
    __shared__ float join[8][kBackLanes];
    const int at = row * threads + tid;
#pragma unroll
    for (int e = 0; e < 8; ++e) join[e][at] = dw[0][e];
    __syncthreads();
    if (row) return;
    for (int o = 1; o < rows; ++o) {
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[0][e] += join[e][o * threads + tid];
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * a.K;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = v * threads + tid;
    if (p >= pieces) break;
    reinterpret_cast<float4*>(part)[2 * p] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
    reinterpret_cast<float4*>(part)[2 * p + 1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
  }
}

// dweight = the groups' partial rows added up: eight lanes of four columns (whole
// 128-byte lines), 64 runs of groups, joined in order.  8192 x 7168: 4.7 us, with
// four lanes (half lines) 6.5, with 16 lanes and 16 runs 11.9.
constexpr int kRuns = 64;
__global__ __launch_bounds__(8 * kRuns) void k_rms_norm_dweight(const float* part, int groups, int K, float* dweight,
                                                                bool accumulate) {
  __shared__ float4 red[kRuns][8];
  const int c = threadIdx.x % 8, r = threadIdx.x / 8;
  const int col = (blockIdx.x * 8 + c) * 4;          // (K is a multiple of 32)
  float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int g = r; g < groups; g += kRuns) {
    const float4 p = *reinterpret_cast<const float4*>(part + (int64_t)g * K + col);
    t.x += p.x, t.y += p.y, t.z += p.z, t.w += p.w;
  }
  for (int half = kRuns / 2; half >= 1; half /= 2) {
    red[r][c] = t;
    __syncthreads();
    if (r < half) {
      const float4 o = red[r + half][c];
      t.x += o.x, t.y += o.y, t.z += o.z, t.w += o.w;
    }
    __syncthreads();
  }
  if (r) return;
  float4* out = reinterpret_cast<float4*>(dweight + col);
  if (accumulate) t.x += out->x, t.y += out->y, t.z += out->z, t.w += out->w;
  *out = t;
}

// Pieces per lane, and the lanes, that hold a row.
struct Shape {
  int v, threads;
};
Shape shape_of(int K) {
  const int lanes = K / 8;
  const int v = lanes <= 256 ? 1 : 2;
  return {v, (lanes + 64 * v - 1) / (64 * v) * 64};
}

}  // namespace

int32_t norm_back_groups(int64_t M, int64_t) { return (int32_t)std::min<int64_t>(M, 512); }

hipError_t launch_rms_norm(const NormArgs& a, bool pow2, hipStream_t stream) {
  const Shape s = shape_of(a.K);
  const unsigned grid = (unsigned)std::min<int64_t>(a.M, 1 << 20);
  const auto k = pow2 ? (s.v == 1 ? k_rms_norm<1, true> : k_rms_norm<2, true>)
                      : (s.v == 1 ? k_rms_norm<1, false> : k_rms_norm<2, false>);
  k<<<grid, s.threads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_rms_norm_back(const NormBackArgs& a, hipStream_t stream) {
  if (a.groups) {
    const Shape s = shape_of(a.K);
    // rows at once: as many as the lanes allow and every group still has
    int rows = 1;
    while (s.v == 1 && 2 * rows * s.threads <= kBackLanes && 2 * rows * a.groups <= a.M) rows *= 2;
    const auto k = rows > 1 ? k_rms_norm_back<1, true> : s.v == 1 ? k_rms_norm_back<1, false> : k_rms_norm_back<2, false>;
    k<<<a.groups, dim3(s.threads, rows), 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  k_rms_norm_dweight<<<a.K / 32, 8 * kRuns, 0, stream>>>(a.part, a.groups, a.K, a.dweight, a.accumulate);
  return hipGetLastError();
}

}  // namespace fp8bs
