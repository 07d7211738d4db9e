// The experts of few tokens (include/fp8bs_layer.h, fp8bs_moe_experts):
//
//   k_moe_up    per expert, g and u = w13 x, then the weighted activations
//               weight g / (1 + exp(-g)) u, as two BF16 parts
//   k_moe_down  w2 times them, summed over the experts of a token
//   k_moe_join  adds the runs that k_moe_down was split over, if any
//
// Bound by HBM: every expert that has a token is read once, 3 H I codes for at
// most a few dozen rows of products.  So weights go from memory straight to the
// registers that the matrix core takes them from, each code to one wave, several
// loads ahead of their use; the tokens' rows come from L2.
//
// Rows.  A (token, expert) pair of the call is a row.  The rows of expert e lie
// one after the other from base(e), the number of places with a smaller id, in
// the order of their tokens; slot s is the s-th place of the call where E is
// larger than their number (the first place of each expert has the work), else
// expert s.
#include <algorithm>

#include "layer.h"
#include "quant_common.h"

namespace fp8bs {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxTokens = 128;
constexpr int kMaxPlaces = kMaxTokens * 16;
constexpr int kMaxChunks = 65536 / 128;

// A buffer of `bytes` (below 2^31) from `base`: reads past them give 0 without
// touching memory.  Offsets of chunks and rows that do not exist; either of them,
// and their sum with any offset that exists, is past every buffer of weights,
// and the sum of both past every buffer of rows (at most 2^24 bytes).
constexpr uint32_t kNoChunk = 0x80000000u, kNoRow = 0x90000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}
__device__ __forceinline__ float load4(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
}
__device__ __forceinline__ v8i join(u32x4 a, u32x4 b) {
  return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// This wave's number, on the scalar unit.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// ---- gate and up ----

// The rows of one slot, found by every workgroup of it.
struct Rows {
  int token[kMaxTokens];
  float weight[kMaxTokens];
};

// Fills `rows` and returns the slot; n = 0 where it has no work.  Every thread
// of the workgroup calls it.
__device__ __forceinline__ Slot find_rows(const ExpertArgs& a, int slot, Rows& rows) {
  __shared__ int below[kWaves], matches[kWaves], first[kWaves];
  const int places = a.T * a.topk, tid = threadIdx.x, wave = wave_id();
  const int e = __builtin_amdgcn_readfirstlane(a.slots < a.E ? a.ids[slot] : slot);
  // thread t looks through token t's places
  int lower = 0, hit = places;
  float w = 0.0f;
  if (tid < a.T) {
    for (int c = a.topk - 1; c >= 0; --c) {
      const int id = a.ids[tid * a.topk + c];
      lower += id >= 0 && id < e;
      if (id == e) {
        w += a.weights[tid * a.topk + c];
        hit = tid * a.topk + c;
      }
    }
  }
  const uint64_t mask = __builtin_amdgcn_ballot_w64(hit < places);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) lower += __shfl_xor(lower, d);
  int least = hit;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) least = min(least, __shfl_xor(least, d));
  if (tid % 64 == 0) below[wave] = lower, matches[wave] = __builtin_popcountll(mask), first[wave] = least;
  __syncthreads();
  Slot s{e, 0, 0, 0};
  int before = 0, lowest = places;
  for (int i = 0; i < kWaves; ++i) {
    s.base += below[i];
    s.n += matches[i];
    if (i < wave) before += matches[i];
    lowest = min(lowest, first[i]);
  }
  if (hit < places) {
    const int r = before + __builtin_popcountll(mask & ((1ull << (tid % 64)) - 1));
    rows.token[r] = tid;
    rows.weight[r] = w;
  }
  if ((uint32_t)e >= (uint32_t)a.E || (a.slots < a.E && lowest != slot)) s.n = 0;
  __syncthreads();
  return s;
}

// MF: 16-row fragments of this pass.  The waves take the 128-wide chunks of H in
// turn; U chunks are in flight.
template <int MF, int U>
__device__ __forceinline__ void up_rows(const ExpertArgs& a, const Slot& s, int row0, int col0, const Rows& rows,
                                        const float* scale_g, const float* scale_u, float* red) {
  const int lane = threadIdx.x % 64, wave = wave_id(), fr = lane % 16, fg = lane / 16;
  const int chunks = a.H / 128;
  const int64_t stride = a.H, panel = 2 * (int64_t)a.I * a.H;
  const auto wb = buffer(a.w13 + (int64_t)s.expert * panel, panel);
  const auto xb = buffer(a.x, (int64_t)a.T * a.H);
  const auto sb = buffer(a.sx, (int64_t)a.T * chunks * 4);
  const uint32_t gate = (uint32_t)((col0 + fr) * stride + fg * 16);
  const uint32_t up = gate + (uint32_t)(a.I * stride);
  uint32_t xrow[MF], srow[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int r = row0 + f * 16 + fr;
    const bool there = r < s.n;
    const int t = there ? rows.token[r] : 0;
    xrow[f] = there ? (uint32_t)(t * stride + fg * 16) : kNoRow;
    srow[f] = there ? (uint32_t)t * 4 : kNoRow;
  }

  struct Chunk {
    u32x4 g0, g1, u0, u1, x0[MF], x1[MF];
    float sx[MF];
  } c[U];
  auto fetch = [&](Chunk& k, int kb) {
    const uint32_t at = kb < chunks ? (uint32_t)kb * 128 : kNoChunk;
    const uint32_t sat = kb < chunks ? (uint32_t)(kb * a.T * 4) : kNoChunk;
    k.g0 = load16(wb, gate + at);
    k.g1 = load16(wb, gate + at + 64);
    k.u0 = load16(wb, up + at);
    k.u1 = load16(wb, up + at + 64);
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      k.x0[f] = load16(xb, xrow[f] + at);
      k.x1[f] = load16(xb, xrow[f] + at + 64);
      k.sx[f] = load4(sb, srow[f] + sat);
    }
  };
  v4f ag[MF], au[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) ag[f] = au[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < U; ++i) fetch(c[i], wave + i * kWaves);
  const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = wave; k0 < chunks; k0 += U * kWaves) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int kb = k0 + i * kWaves;
      const float sg = scale_g[min(kb, chunks - 1)], su = scale_u[min(kb, chunks - 1)];
      const v8i g = join(c[i].g0, c[i].g1), u = join(c[i].u0, c[i].u1);
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const v8i x = join(c[i].x0[f], c[i].x1[f]);
        const v4f pg = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(g, x, zero, 0, 0, 0, 0, 0, 0);
        const v4f pu = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(u, x, zero, 0, 0, 0, 0, 0, 0);
        const float wg = c[i].sx[f] * sg, wu = c[i].sx[f] * su;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ag[f][e] = __builtin_fmaf(pg[e], wg, ag[f][e]);
          au[f][e] = __builtin_fmaf(pu[e], wu, au[f][e]);
        }
      }
      fetch(c[i], kb + U * kWaves);
    }
  }
  // the waves' sums, [wave][fragment][gate, up][lane][4]
  v4f* mine = reinterpret_cast<v4f*>(red) + (wave * MF * 2) * 64 + lane;
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    mine[(f * 2) * 64] = ag[f];
    mine[(f * 2 + 1) * 64] = au[f];
  }
  __syncthreads();
  // thread -> row m, column n of a fragment: lane (n / 4) 16 + m has n % 4
  const int m = threadIdx.x / 16, n = threadIdx.x % 16, from = ((n / 4) * 16 + m) * 4 + n % 4;
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      g += red[((w * MF + f) * 2) * 256 + from];
      u += red[((w * MF + f) * 2 + 1) * 256 + from];
    }
    const int r = row0 + f * 16 + m;
    if (r < s.n) {
      const float v = rows.weight[r] * (g / (1.0f + expf(-g))) * u;
      const __bf16 hi = (__bf16)v, lo = (__bf16)(v - (float)hi);
      const int64_t at = (int64_t)(s.base + r) * a.I + col0 + n;
      a.hi[at] = __builtin_bit_cast(uint16_t, hi);
      a.lo[at] = __builtin_bit_cast(uint16_t, lo);
    }
  }
  __syncthreads();
}

// One workgroup per slot and 16 columns of I.
template <int MAXF>
__global__ __launch_bounds__(kThreads) void k_moe_up(ExpertArgs a) {
  __shared__ Rows rows;
  __shared__ float scale_g[kMaxChunks], scale_u[kMaxChunks];
  __shared__ __align__(16) float red[kWaves * MAXF * 2 * 256];
  const int tiles = a.I / 16, slot = blockIdx.x / tiles, col0 = (blockIdx.x % tiles) * 16;
  const Slot s = find_rows(a, slot, rows);
  if (blockIdx.x % tiles == 0) {                     // what k_moe_down needs to know
    if (threadIdx.x == 0) a.slot[slot] = s;
    for (int r = threadIdx.x; r < s.n; r += kThreads) a.token[s.base + r] = rows.token[r];
  }
  if (s.n == 0) return;
  const int chunks = a.H / 128;
  const float* sc = a.s13 + (int64_t)s.expert * (2 * a.I / 128) * chunks;
  for (int k = threadIdx.x; k < chunks; k += kThreads) {
    scale_g[k] = sc[(int64_t)(col0 / 128) * chunks + k];
    scale_u[k] = sc[(int64_t)((a.I + col0) / 128) * chunks + k];
  }
  __syncthreads();
  for (int row0 = 0; row0 < s.n; row0 += 16 * MAXF) {
    const int left = (s.n - row0 + 15) / 16;
    if (MAXF == 1 || left == 1) up_rows<1, 4>(a, s, row0, col0, rows, scale_g, scale_u, red);
    else if (MAXF == 2 || left == 2) up_rows<2 <= MAXF ? 2 : 1, 2>(a, s, row0, col0, rows, scale_g, scale_u, red);
    else up_rows<MAXF, 2>(a, s, row0, col0, rows, scale_g, scale_u, red);
  }
}

// ---- down ----

__device__ __forceinline__ v8bf to_bf16(uint32_t a, uint32_t b) {
  const v2bf p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const v2bf q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const v2bf r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const v2bf t = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return v8bf{p[0], p[1], q[0], q[1], r[0], r[1], t[0], t[1]};
}

// One wave, one slot: chunks first, first + step, ... of I; adds its products to
// the wave's own sums [token][16 columns].
template <int MF, int U>
__device__ __forceinline__ void down_rows(const ExpertArgs& a, const Slot& s, int row0, int col0, int first, int step,
                                          const uint8_t* tokens, float* sums) {
  const int lane = threadIdx.x % 64, fr = lane % 16, fg = lane / 16;
  const int chunks = a.I / 128;
  const int64_t panel = (int64_t)a.H * a.I;
  const auto wb = buffer(a.w2 + (int64_t)s.expert * panel, panel);
  const int64_t act = (int64_t)s.n * a.I * 2;        // rows of this slot (at most 2^24 bytes)
  const auto hb = buffer(a.hi + (int64_t)s.base * a.I, act), lb = buffer(a.lo + (int64_t)s.base * a.I, act);
  const float* sc = a.s2 + ((int64_t)s.expert * (a.H / 128) + col0 / 128) * chunks;
  const uint32_t wrow = (uint32_t)((col0 + fr) * (int64_t)a.I + fg * 32);
  uint32_t arow[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) arow[f] = (uint32_t)((row0 + f * 16 + fr) * (int64_t)a.I + fg * 32) * 2;  // past n: outside
  u32x4 w[U][2];
  float scale[U];
  auto fetch = [&](int i, int kb) {
    const uint32_t at = kb < chunks ? (uint32_t)kb * 128 : kNoChunk;
    w[i][0] = load16(wb, wrow + at);
    w[i][1] = load16(wb, wrow + at + 16);
    scale[i] = sc[min(kb, chunks - 1)];
  };
  v4f acc[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) acc[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < U; ++i) fetch(i, first + i * step);
  for (int k0 = first; k0 < chunks; k0 += U * step) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int kb = k0 + i * step;
      const uint32_t at = kb < chunks ? (uint32_t)kb * 256 : kNoRow;
      // 32 codes of a lane: four steps of eight
      const v8bf b[4] = {to_bf16(w[i][0].x, w[i][0].y), to_bf16(w[i][0].z, w[i][0].w), to_bf16(w[i][1].x, w[i][1].y),
                         to_bf16(w[i][1].z, w[i][1].w)};
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        v4f p{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t from = arow[f] + at + j * 16;
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], __builtin_bit_cast(v8bf, load16(hb, from)), p, 0, 0, 0);
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], __builtin_bit_cast(v8bf, load16(lb, from)), p, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[f][e] = __builtin_fmaf(p[e], scale[i], acc[f][e]);
      }
      fetch(i, kb + U * step);
    }
  }
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int r = row0 + f * 16 + fr;
    if (r < s.n) {                                   // (rows of a slot have different tokens)
      v4f* to = reinterpret_cast<v4f*>(sums + tokens[s.base + r] * 16 + fg * 4);
      *to += acc[f];
    }
  }
}

// One workgroup per 16 columns of H and run of slots.  Waves take (slot, part of
// I) items in turn, and add into sums of their own; those are added in order.
template <int MAXF>
__global__ __launch_bounds__(kThreads) void k_moe_down(ExpertArgs a, int parts) {
  extern __shared__ __align__(16) float sums[];      // [kWaves][T][16]
  __shared__ uint8_t tokens[kMaxPlaces];
  const int tiles = a.H / 16, col0 = (blockIdx.x % tiles) * 16, run = blockIdx.x / tiles;
  const int wave = wave_id();
  for (int i = threadIdx.x; i < kWaves * a.T * 16; i += kThreads) sums[i] = 0.0f;
  // (rows without a token are never read below)
  for (int i = threadIdx.x; i < a.T * a.topk; i += kThreads) tokens[i] = (uint8_t)a.token[i];
  __syncthreads();
  float* mine = sums + wave * a.T * 16;
  const int items = (a.slots - run + a.splits - 1) / a.splits * parts;
  for (int i = wave; i < items; i += kWaves) {
    Slot s = a.slot[run + i / parts * a.splits];
    s.expert = __builtin_amdgcn_readfirstlane(s.expert);
    s.base = __builtin_amdgcn_readfirstlane(s.base);
    s.n = __builtin_amdgcn_readfirstlane(s.n);
    for (int row0 = 0; row0 < s.n; row0 += 16 * MAXF) {
      const int left = (s.n - row0 + 15) / 16;
      if (MAXF == 1 || left == 1) down_rows<1, 4>(a, s, row0, col0, i % parts, parts, tokens, mine);
      else if (MAXF == 2 || left == 2) down_rows<2 <= MAXF ? 2 : 1, 4>(a, s, row0, col0, i % parts, parts, tokens, mine);
      else down_rows<MAXF, 4>(a, s, row0, col0, i % parts, parts, tokens, mine);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 16; i += kThreads) {
    float v = sums[i];
    for (int w = 1; w < kWaves; ++w) v += sums[w * a.T * 16 + i];
    const int64_t at = (int64_t)(i / 16) * a.H + col0 + i % 16;
    if (a.splits > 1) a.part[(int64_t)run * a.T * a.H + at] = v;
    else if (a.out_f32) static_cast<float*>(a.out)[at] = v;
    else static_cast<__bf16*>(a.out)[at] = (__bf16)v;
  }
}

__global__ __launch_bounds__(kThreads) void k_moe_join(ExpertArgs a) {
  const int64_t all = (int64_t)a.T * a.H, i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
  if (i >= all) return;                              // (all is a multiple of 128)
  v4f v = *reinterpret_cast<const v4f*>(a.part + i);
  for (int g = 1; g < a.splits; ++g) v += *reinterpret_cast<const v4f*>(a.part + g * all + i);
  if (a.out_f32) *reinterpret_cast<v4f*>(static_cast<float*>(a.out) + i) = v;
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + i) = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
}

int64_t aligned(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Parts of I that a slot's second product is cut into, so that the waves of a
// workgroup all have work where it has fewer slots than waves.
int parts_of(const ExpertArgs& a) {
  const int per = (a.slots + a.splits - 1) / a.splits;
  return std::max(1, std::min(kWaves / per, a.I / 128));
}

}  // namespace

void experts_plan(ExpertArgs& a) {
  a.slots = std::min(a.E, a.T * a.topk);
  // workgroups enough for four on each of 256 CUs
  const int tiles = a.H / 16;
  a.splits = std::max(1, std::min(a.slots, (1024 + tiles - 1) / tiles));
}

int64_t experts_workspace(ExpertArgs& a, void* base) {
  const int64_t places = (int64_t)a.T * a.topk;
  uint8_t* p = static_cast<uint8_t*>(base);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* here = p ? p + at : nullptr;
    at += aligned(bytes);
    return here;
  };
  a.hi = reinterpret_cast<uint16_t*>(take(places * a.I * 2));
  a.lo = reinterpret_cast<uint16_t*>(take(places * a.I * 2));
  a.slot = reinterpret_cast<Slot*>(take(a.slots * (int64_t)sizeof(Slot)));
  a.token = reinterpret_cast<int32_t*>(take(places * 4));
  a.part = reinterpret_cast<float*>(take(a.splits > 1 ? (int64_t)a.splits * a.T * a.H * 4 : 0));
  return at;
}

hipError_t launch_moe_experts(const ExpertArgs& a, hipStream_t stream) {
  const unsigned up = (unsigned)(a.I / 16 * a.slots), down = (unsigned)(a.H / 16 * a.splits);
  const size_t lds = (size_t)kWaves * a.T * 16 * 4;
  const int parts = parts_of(a);
  if (a.T <= 16) {
    k_moe_up<1><<<up, kThreads, 0, stream>>>(a);
    k_moe_down<1><<<down, kThreads, lds, stream>>>(a, parts);
  } else if (a.T <= 32) {
    k_moe_up<2><<<up, kThreads, 0, stream>>>(a);
    k_moe_down<2><<<down, kThreads, lds, stream>>>(a, parts);
  } else {
    k_moe_up<4><<<up, kThreads, 0, stream>>>(a);
    k_moe_down<4><<<down, kThreads, lds, stream>>>(a, parts);
  }
  if (a.splits > 1)
    k_moe_join<<<(unsigned)(((int64_t)a.T * a.H / 4 + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace fp8bs
