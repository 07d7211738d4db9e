// The experts of few tokens (include/fp8bs_layer.h, fp8bs_moe_experts):
//
//   k_moe_up    per expert, g and u = w13 x, then the weighted activations
//               weight g / (1 + exp(-g)) u, as two BF16 parts
//   k_moe_down  w2 times them
//   k_moe_join  the sums of each token's rows
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
  int token[kMaxTokens], place[kMaxTokens];
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
    rows.place[r] = hit;
    rows.weight[r] = w;
  }
  if ((uint32_t)e >= (uint32_t)a.E || (a.slots < a.E && lowest != slot)) s.n = 0;
  __syncthreads();
  return s;
}

// Column c of the activations is kept at place_of(c) of its row: the 16 codes
// that a lane of k_moe_down loads at once belong to two products, so the halves
// of 16 columns lie 32 apart, and the rows' 64-byte pieces of a product are whole.
__device__ __forceinline__ int place_of(int c) {
  return (c & ~63) + ((c >> 3) & 1) * 32 + ((c >> 4) & 3) * 8 + (c & 7);
}

// Adds up the waves' accumulators of MF x NC fragments and hands each sum to
// f(row, column, gate or only value, up), columns 16 per fragment.  `red` holds
// kWaves * MF * NC * 256 floats.
template <int MF, int NC>
__device__ __forceinline__ void leave(const v4f (&acc)[MF][NC], float* red) {
  v4f* mine = reinterpret_cast<v4f*>(red) + wave_id() * MF * NC * 64 + threadIdx.x % 64;
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int n = 0; n < NC; ++n) mine[(f * NC + n) * 64] = acc[f][n];
  __syncthreads();
}
// Row m, column c of fragment (f, n): lane (c / 4) 16 + m has c % 4.
template <int MF, int NC>
__device__ __forceinline__ float total(const float* red, int f, int n, int m, int c) {
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) t += red[((w * MF + f) * NC + n) * 256 + ((c / 4) * 16 + m) * 4 + c % 4];
  return t;
}

// MF: 16-row fragments of this pass; NG: 16-column fragments of gate and of up.
// The waves take the 128-wide chunks of H in turn; U chunks are in flight.
template <int MF, int NG, int U>
__device__ __forceinline__ void up_rows(const ExpertArgs& a, const Slot& s, int row0, int col0, const Rows& rows,
                                        const float* scale_g, const float* scale_u, float* red) {
  constexpr int NC = 2 * NG;
  const int lane = threadIdx.x % 64, wave = wave_id(), fr = lane % 16, fg = lane / 16;
  const int chunks = a.H / 128;
  const int64_t panel = 2 * (int64_t)a.I * a.H;
  const auto wb = buffer(a.w13 + (int64_t)s.expert * panel, panel);
  const auto xb = buffer(a.x, (int64_t)a.T * a.H);
  const auto sb = buffer(a.sx, (int64_t)a.T * chunks * 4);
  uint32_t wrow[NC], xrow[MF], srow[MF];
#pragma unroll
  for (int n = 0; n < NC; ++n) wrow[n] = (uint32_t)(((n / NG) * a.I + col0 + (n % NG) * 16 + fr) * (int64_t)a.H + fg * 16);
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int r = row0 + f * 16 + fr;
    const bool there = r < s.n;
    const int t = there ? rows.token[r] : 0;
    xrow[f] = there ? (uint32_t)(t * a.H + fg * 16) : kNoRow;
    srow[f] = there ? (uint32_t)t * 4 : kNoRow;
  }

  struct Chunk {
    u32x4 w0[NC], w1[NC], x0[MF], x1[MF];
    float sx[MF];
  } c[U];
  auto fetch = [&](Chunk& k, int kb) {
    const uint32_t at = kb < chunks ? (uint32_t)kb * 128 : kNoChunk;
    const uint32_t sat = kb < chunks ? (uint32_t)(kb * a.T * 4) : kNoChunk;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      k.w0[n] = load16(wb, wrow[n] + at);
      k.w1[n] = load16(wb, wrow[n] + at + 64);
    }
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      k.x0[f] = load16(xb, xrow[f] + at);
      k.x1[f] = load16(xb, xrow[f] + at + 64);
      k.sx[f] = load4(sb, srow[f] + sat);
    }
  };
  v4f acc[MF][NC];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int n = 0; n < NC; ++n) acc[f][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < U; ++i) fetch(c[i], wave + i * kWaves);
  const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = wave; k0 < chunks; k0 += U * kWaves) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int kb = k0 + i * kWaves;
      const float sg = scale_g[min(kb, chunks - 1)], su = scale_u[min(kb, chunks - 1)];
      v8i x[MF];
#pragma unroll
      for (int f = 0; f < MF; ++f) x[f] = join(c[i].x0[f], c[i].x1[f]);
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const v8i w = join(c[i].w0[n], c[i].w1[n]);
#pragma unroll
        for (int f = 0; f < MF; ++f) {
          const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x[f], zero, 0, 0, 0, 0, 0, 0);
          const float by = c[i].sx[f] * (n < NG ? sg : su);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[f][n][e] = __builtin_fmaf(p[e], by, acc[f][n][e]);
        }
      }
      fetch(c[i], kb + U * kWaves);
    }
  }
  leave(acc, red);
  const int m = threadIdx.x / 16, col = threadIdx.x % 16;
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int r = row0 + f * 16 + m;
    if (r >= s.n) continue;
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const float g = total<MF, NC>(red, f, n, m, col), u = total<MF, NC>(red, f, NG + n, m, col);
      const float v = rows.weight[r] * (g / (1.0f + expf(-g))) * u;
      const __bf16 hi = (__bf16)v, lo = (__bf16)(v - (float)hi);
      const int64_t at = (int64_t)(s.base + r) * a.I + place_of(col0 + n * 16 + col);
      a.hi[at] = __builtin_bit_cast(uint16_t, hi);
      a.lo[at] = __builtin_bit_cast(uint16_t, lo);
    }
  }
  __syncthreads();
}

// One workgroup per slot and 16 NG columns of I.
template <int MAXF, int NG>
__global__ __launch_bounds__(kThreads) void k_moe_up(ExpertArgs a) {
  __shared__ Rows rows;
  __shared__ float scale_g[kMaxChunks], scale_u[kMaxChunks];
  __shared__ __align__(16) float red[kWaves * MAXF * 2 * NG * 256];
  const int tiles = a.I / (16 * NG), slot = blockIdx.x / tiles, col0 = (blockIdx.x % tiles) * 16 * NG;
  const Slot s = find_rows(a, slot, rows);
  if (blockIdx.x % tiles == 0) {                     // what k_moe_down needs to know
    if (threadIdx.x == 0) a.slot[slot] = s;
    for (int r = threadIdx.x; r < s.n; r += kThreads) a.place[s.base + r] = rows.place[r];
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
    if (MAXF == 1 || left == 1) up_rows<1, NG, 3>(a, s, row0, col0, rows, scale_g, scale_u, red);
    else if (MAXF == 2 || left == 2) up_rows<2 <= MAXF ? 2 : 1, NG, 2>(a, s, row0, col0, rows, scale_g, scale_u, red);
    else up_rows<MAXF, NG, 2>(a, s, row0, col0, rows, scale_g, scale_u, red);
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

// MF row fragments, NC column fragments; the waves take the chunks of I in turn.
template <int MF, int NC, int U>
__device__ __forceinline__ void down_rows(const ExpertArgs& a, const Slot& s, int row0, int col0, float* red) {
  const int lane = threadIdx.x % 64, wave = wave_id(), fr = lane % 16, fg = lane / 16;
  const int chunks = a.I / 128;
  const int64_t panel = (int64_t)a.H * a.I;
  const auto wb = buffer(a.w2 + (int64_t)s.expert * panel, panel);
  const int64_t act = (int64_t)s.n * a.I * 2;        // rows of this slot (at most 2^24 bytes)
  const auto hb = buffer(a.hi + (int64_t)s.base * a.I, act), lb = buffer(a.lo + (int64_t)s.base * a.I, act);
  const float* sc = a.s2 + ((int64_t)s.expert * (a.H / 128) + col0 / 128) * chunks;
  uint32_t wrow[NC], arow[MF];
#pragma unroll
  for (int n = 0; n < NC; ++n) wrow[n] = (uint32_t)((col0 + n * 16 + fr) * (int64_t)a.I + fg * 16);
#pragma unroll
  for (int f = 0; f < MF; ++f) arow[f] = (uint32_t)((row0 + f * 16 + fr) * (int64_t)a.I + fg * 8) * 2;  // past n: outside
  struct Chunk {
    u32x4 w0[NC], w1[NC];
    float scale;
  } c[U];
  auto fetch = [&](Chunk& k, int kb) {
    const uint32_t at = kb < chunks ? (uint32_t)kb * 128 : kNoChunk;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      k.w0[n] = load16(wb, wrow[n] + at);
      k.w1[n] = load16(wb, wrow[n] + at + 64);
    }
    k.scale = sc[min(kb, chunks - 1)];
  };
  struct Acts {
    u32x4 hi[MF][4], lo[MF][4];
  };
  auto fetch_acts = [&](Acts& k, int kb) {
    const uint32_t at = kb < chunks ? (uint32_t)kb * 256 : kNoRow;
#pragma unroll
    for (int f = 0; f < MF; ++f)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        k.hi[f][j] = load16(hb, arow[f] + at + j * 64);
        k.lo[f][j] = load16(lb, arow[f] + at + j * 64);
      }
  };
  v4f acc[MF][NC];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int n = 0; n < NC; ++n) acc[f][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  // Loads return in the order they were issued, so the activations of a chunk
  // (from L2) go out ahead of weights (from memory) that are needed later.
  Acts x;
  fetch(c[0], wave);
  fetch_acts(x, wave);
#pragma unroll
  for (int i = 1; i < U; ++i) fetch(c[i], wave + i * kWaves);
  for (int k0 = wave; k0 < chunks; k0 += U * kWaves) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int kb = k0 + i * kWaves;
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const v8bf b[4] = {to_bf16(c[i].w0[n].x, c[i].w0[n].y), to_bf16(c[i].w0[n].z, c[i].w0[n].w),
                           to_bf16(c[i].w1[n].x, c[i].w1[n].y), to_bf16(c[i].w1[n].z, c[i].w1[n].w)};
#pragma unroll
        for (int f = 0; f < MF; ++f) {
          v4f p{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], __builtin_bit_cast(v8bf, x.hi[f][j]), p, 0, 0, 0);
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], __builtin_bit_cast(v8bf, x.lo[f][j]), p, 0, 0, 0);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[f][n][e] = __builtin_fmaf(p[e], c[i].scale, acc[f][n][e]);
        }
      }
      fetch_acts(x, kb + kWaves);
      fetch(c[i], kb + U * kWaves);
    }
  }
  leave(acc, red);
  const int m = threadIdx.x / 16, col = threadIdx.x % 16;
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int r = row0 + f * 16 + m;
    if (r >= s.n) continue;
    float* to = a.part + (int64_t)a.place[s.base + r] * a.H + col0 + col;
#pragma unroll
    for (int n = 0; n < NC; ++n) to[n * 16] = total<MF, NC>(red, f, n, m, col);
  }
  __syncthreads();
}

// One workgroup per slot and 16 NC columns of H.
template <int MAXF, int NC>
__global__ __launch_bounds__(kThreads) void k_moe_down(ExpertArgs a) {
  __shared__ __align__(16) float red[kWaves * MAXF * NC * 256];
  const int tiles = a.H / (16 * NC), slot = blockIdx.x / tiles, col0 = (blockIdx.x % tiles) * 16 * NC;
  Slot s = a.slot[slot];
  s.expert = __builtin_amdgcn_readfirstlane(s.expert);
  s.base = __builtin_amdgcn_readfirstlane(s.base);
  s.n = __builtin_amdgcn_readfirstlane(s.n);
  for (int row0 = 0; row0 < s.n; row0 += 16 * MAXF) {
    const int left = (s.n - row0 + 15) / 16;
    if (MAXF == 1 || left == 1) down_rows<1, NC, 2>(a, s, row0, col0, red);
    else if (MAXF == 2 || left == 2) down_rows<2 <= MAXF ? 2 : 1, NC, 2>(a, s, row0, col0, red);
    else down_rows<MAXF, NC, 2>(a, s, row0, col0, red);
  }
}

// out[t] = the rows of token t's places added up in turn.  Places without a row
// (an id outside, or one that stands further left too) are left out.
__global__ __launch_bounds__(kThreads) void k_moe_join(ExpertArgs a) {
  const int h = (blockIdx.x * kThreads + threadIdx.x) * 4, t = blockIdx.y;
  if (h >= a.H) return;
  const int32_t* ids = a.ids + t * a.topk;
  v4f v{0.0f, 0.0f, 0.0f, 0.0f};
  for (int c = 0; c < a.topk; ++c) {
    bool counts = (uint32_t)ids[c] < (uint32_t)a.E;
    for (int b = 0; b < c; ++b) counts = counts && ids[b] != ids[c];
    if (counts) v += *reinterpret_cast<const v4f*>(a.part + (int64_t)(t * a.topk + c) * a.H + h);
  }
  const int64_t at = (int64_t)t * a.H + h;
  if (a.out_f32) *reinterpret_cast<v4f*>(static_cast<float*>(a.out) + at) = v;
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
}

int64_t aligned(int64_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

void experts_plan(ExpertArgs& a) { a.slots = std::min(a.E, a.T * a.topk); }

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
  a.part = reinterpret_cast<float*>(take(places * a.H * 4));
  a.slot = reinterpret_cast<Slot*>(take(a.slots * (int64_t)sizeof(Slot)));
  a.place = reinterpret_cast<int32_t*>(take(places * 4));
  return at;
}

namespace {

template <int MAXF, int NG, int NC>
void launch(const ExpertArgs& a, hipStream_t stream) {
  k_moe_up<MAXF, NG><<<(unsigned)(a.I / (16 * NG) * a.slots), kThreads, 0, stream>>>(a);
  k_moe_down<MAXF, NC><<<(unsigned)(a.H / (16 * NC) * a.slots), kThreads, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_moe_experts(const ExpertArgs& a, hipStream_t stream) {
  if (a.T <= 16) launch<1, 2, 4>(a, stream);
  else launch<2, 2, 4>(a, stream);
  k_moe_join<<<dim3((unsigned)((a.H / 4 + kThreads - 1) / kThreads), (unsigned)a.T), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace fp8bs
