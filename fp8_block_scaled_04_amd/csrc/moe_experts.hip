// The experts of few tokens (include/fp8bs_layer.h, fp8bs_moe_experts):
//
//   k_moe_up    per expert, g and u = w13 x, then the weighted activations
//               weight g / (1 + exp(-g)) u, as two BF16 parts
//   k_moe_down  w2 times them
//   k_moe_join  the sums of each token's rows (not with one place per token; few
//               weights: k_moe_down_whole takes its place and that of k_moe_down)
//
// Bound by HBM: every expert that has a token is read once, 3 H I codes for at
// most a few dozen rows of products.  So weights go from memory straight to the
// registers that the matrix core takes them from, each code to one wave, several
// loads ahead of their use.  A CU has about 80 requests of 128 bytes under way at
// once, whatever its waves ask for, and the tokens' rows count among them.  Few
// rows per expert come from L2 beside the weights, K split over the waves of a
// workgroup; many rows go through LDS once per workgroup, its waves on different
// columns (k_moe_up_wide, k_moe_down_wide).
//
// H = 7168, I = 2048, 32 experts, 8 places: one token 46 + 25 + 5 us, 352 MB (5.1
// and 4.7 TB/s in the two products); 64 tokens 169 + 109 + 5 us, 1409 MB (5.6 and
// 4.3 TB/s: the second product's rows are four bytes a value).  A plain read moves
// 5.7 TB/s.
//
// A (token, expert) pair of the call is a row.  The rows of an expert lie one
// after the other in the order of their tokens, those of lower experts before.
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

// A buffer of `bytes` (below 2^31) from `base`: reads past them give 0 without
// touching memory.  Offsets of chunks and rows that do not exist; either of them,
// and their sum with any offset that exists, is past every buffer of weights,
// and the sum of both past every buffer of rows (at most 2^27 bytes).
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

// The bits of 16 lanes joined.
__device__ __forceinline__ uint32_t row16_or(uint32_t v) {
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);    // quad_perm [1, 0, 3, 2]
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);    // quad_perm [2, 3, 0, 1]
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true);   // row_half_mirror
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true);   // row_mirror
  return v;
}

// This wave's number, on the scalar unit.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

__device__ __forceinline__ float of_lane(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}

// ---- which rows each expert has ----

// One expert's rows, at most `block` of them, packed: expert (10 bits), first row
// (12), rows (8).
struct Job {
  int expert, start, n;
};
__device__ __forceinline__ uint32_t pack(int expert, int start, int n) { return expert | start << 10 | n << 22; }

// The call's rows and jobs.  k_moe_up works them out from ids, every workgroup in
// its own LDS: a bit per (expert, token), so that the order in which the bits are
// set does not matter; then sums over the experts.  The first workgroup leaves
// them in the workspace for k_moe_down.
struct Plan {
  uint32_t* job;    // [jobs]
  uint32_t* row;    // [rows] token << 16 | place
  float* weight;    // [rows]; k_moe_up only
  int jobs;

  __device__ __forceinline__ Job at(int j) const {
    const uint32_t p = __builtin_amdgcn_readfirstlane(job[j]);
    return {(int)(p & 1023), (int)(p >> 10 & 4095), (int)(p >> 22)};
  }
};
__host__ __device__ __forceinline__ int mask_words(int T) { return (T + 31) / 32; }
// (LDS of k_moe_up: jobs, rows, weights, the places' ids; bits and base of each expert)
int plan_bytes(const ExpertArgs& a) { return (a.T * a.topk * 4 + a.E * (mask_words(a.T) + 1)) * 4; }
int image_words(const ExpertArgs& a) { return 1 + 2 * a.T * a.topk; }

// `block`: rows that one pass over an expert's weights serves.  (About 3 us of a
// call; a kernel of its own costs more, 7 us.)
__device__ __forceinline__ Plan make_plan(const ExpertArgs& a, uint32_t* lds, int block) {
  __shared__ int waves[kWaves];
  const int tid = threadIdx.x, places = a.T * a.topk, words = mask_words(a.T);
  Plan p;
  p.job = lds;
  p.row = p.job + places;
  p.weight = reinterpret_cast<float*>(p.row + places);
  int* id = reinterpret_cast<int*>(p.weight + places);
  uint32_t* mask = reinterpret_cast<uint32_t*>(id + places);   // [E][words]
  int* base = reinterpret_cast<int*>(mask + a.E * words);      // rows of the experts before
  const float early = tid < places ? a.weights[tid] : 0.0f;    // (in flight with the ids)
  for (int i = tid; i < places; i += kThreads) id[i] = a.ids[i];
  for (int i = tid; i < a.E * words; i += kThreads) mask[i] = 0u;
  __syncthreads();
  for (int i = tid; i < places; i += kThreads) {
    const uint32_t e = (uint32_t)id[i];
    const int t = i / a.topk;
    if (e < (uint32_t)a.E) atomicOr(&mask[e * words + t / 32], 1u << (t % 32));
  }
  __syncthreads();
  // thread -> `each` experts in a row; rows and jobs before them, as one number
  const int each = (a.E + kThreads - 1) / kThreads;
  int mine = 0;
  auto rows_of = [&](int e) {
    int n = 0;
    for (int w = 0; w < words; ++w) n += __builtin_popcount(mask[e * words + w]);
    return n;
  };
  for (int e = tid * each; e < min(a.E, (tid + 1) * each); ++e) {
    const int n = rows_of(e);
    mine += n | ((n + block - 1) / block) << 16;
  }
  int before = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(before, d);
    if (tid % 64 >= d) before += o;
  }
  if (tid % 64 == 63) waves[tid / 64] = before;
  __syncthreads();
  before -= mine;
  int all = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < tid / 64) before += waves[w];
    all += waves[w];
  }
  p.jobs = __builtin_amdgcn_readfirstlane(all >> 16);
  for (int e = tid * each; e < min(a.E, (tid + 1) * each); ++e) {
    const int n = rows_of(e), start = before & 0xFFFF, job = before >> 16;
    base[e] = start;
    for (int r = 0; r < n; r += block) p.job[job + r / block] = pack(e, start + r, min(block, n - r));
    before += n | ((n + block - 1) / block) << 16;
  }
  __syncthreads();
  // a row per expert of a token: from the expert's first place there
  for (int i = tid; i < places; i += kThreads) {
    const int t = i / a.topk, e = id[i];
    bool first = (uint32_t)e < (uint32_t)a.E;
    for (int c = t * a.topk; c < i; ++c) first = first && id[c] != e;
    if (!first) continue;
    float w = i == tid ? early : a.weights[i];
    for (int c = i + 1; c < (t + 1) * a.topk; ++c)
      if (id[c] == e) w += a.weights[c];
    int r = base[e];
    for (int k = 0; k < t / 32; ++k) r += __builtin_popcount(mask[e * words + k]);
    r += __builtin_popcount(mask[e * words + t / 32] & ((1u << (t % 32)) - 1));
    p.row[r] = (uint32_t)t << 16 | (uint32_t)i;
    p.weight[r] = w;
  }
  __syncthreads();
  return p;
}

// (Places without a row hold what LDS held: never used.)
__device__ __forceinline__ void save_plan(const ExpertArgs& a, const Plan& p) {
  if (blockIdx.x != 0) return;
  for (int i = threadIdx.x; i < 2 * a.T * a.topk; i += kThreads) a.image[1 + i] = p.job[i];
  if (threadIdx.x == 0) a.image[0] = (uint32_t)p.jobs;
}

__device__ __forceinline__ Plan load_plan(const ExpertArgs& a, uint32_t* lds) {
  const int places = a.T * a.topk;
  Plan p{lds, lds + places, nullptr, __builtin_amdgcn_readfirstlane((int)a.image[0])};
  for (int i = threadIdx.x; i < 2 * places; i += blockDim.x) lds[i] = a.image[1 + i];
  __syncthreads();
  return p;
}

// ---- what both products share ----

// Column c of the activations is kept at place_of(c) of its row: the 16 codes
// that a lane of k_moe_down loads at once belong to two products, so the halves
// of 16 columns lie 32 apart, and the rows' 64-byte pieces of a product are whole.
__device__ __forceinline__ int place_of(int c) {
  return (c & ~63) + ((c >> 3) & 1) * 32 + ((c >> 4) & 3) * 8 + (c & 7);
}

// Columns h .. h + 3 of the call's result for token t.
__device__ __forceinline__ void put_out(const ExpertArgs& a, int t, int h, v4f v) {
  const int64_t at = (int64_t)t * a.H + h;
  if (a.out_f32) *reinterpret_cast<v4f*>(static_cast<float*>(a.out) + at) = v;
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
}

// A row of the second product, columns h .. h + 3: the result itself where a token
// has one place, else a part of it for k_moe_join.
__device__ __forceinline__ void put_row(const ExpertArgs& a, int place, int h, v4f v) {
  if (a.topk == 1) put_out(a, place, h, v);
  else *reinterpret_cast<v4f*>(a.part + (int64_t)place * a.H + h) = v;
}
// With one place per token: zeros for the tokens without an expert.
__device__ __forceinline__ void put_zeros(const ExpertArgs& a) {
  if (a.topk != 1) return;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    if ((uint32_t)a.ids[t] < (uint32_t)a.E) continue;
    for (int h = threadIdx.x * 4; h < a.H; h += kThreads * 4) put_out(a, t, h, v4f{0.0f, 0.0f, 0.0f, 0.0f});
  }
}

// The waves' accumulators of NC fragments, in LDS (kWaves * NC * 256 floats) for
// the sums over them.
template <int NC>
__device__ __forceinline__ void leave(const v4f (&acc)[NC], float* red) {
  v4f* mine = reinterpret_cast<v4f*>(red) + wave_id() * NC * 64 + threadIdx.x % 64;
#pragma unroll
  for (int n = 0; n < NC; ++n) mine[n * 64] = acc[n];
  __syncthreads();
}
// Row m of tokens, row c of the weights of fragment n: lane (c / 4) 16 + m has c % 4.
template <int NC>
__device__ __forceinline__ float total(const float* red, int n, int m, int c) {
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) t += red[(w * NC + n) * 256 + ((c / 4) * 16 + m) * 4 + c % 4];
  return t;
}

// The scales of one weight row block, chunk wave + kWaves l in lane l.
__device__ __forceinline__ float lane_scale(const float* block, int chunks) {
  const int kb = wave_id() + (threadIdx.x % 64) * kWaves;
  return kb < chunks ? block[kb] : 0.0f;
}
// Chunks of one of the `waves` that share an item, at least the U that it fetches
// ahead (those past the end are zeros): what is fetched is never more than one item
// ahead.
__device__ __forceinline__ int steps_of(int chunks, int waves, int U) {
  return max((chunks + waves - 1) / waves, U);
}

// ---- gate and up ----

// Items: one job (at most 16 rows) and COLS columns of I, so 2 COLS rows of w13 in
// fragments of 16: COLS / 16 of gate, then as many of up; with COLS = 8 one
// fragment of eight rows of each.  A workgroup walks its items; its waves take the
// 128-wide chunks of H in turn and keep U of them in flight, the first ones of the
// next item too.
template <int COLS>
__global__ __launch_bounds__(kThreads, 4) void k_moe_up(ExpertArgs a) {
  constexpr int NC = COLS / 8, U = 2, kHalf = COLS < 16 ? 8 : 16;
  extern __shared__ __align__(16) uint32_t lds[];
  __shared__ __align__(16) float red[kWaves * NC * 256];
  const Plan plan = make_plan(a, lds, 16);
  save_plan(a, plan);
  const int lane = threadIdx.x % 64, wave = wave_id(), fr = lane % 16, fg = lane / 16;
  const int chunks = a.H / 128, steps = steps_of(chunks, kWaves, U);
  const int tiles = a.I / COLS, items = plan.jobs * tiles;
  const int64_t panel = 2 * (int64_t)a.I * a.H;
  const auto xb = buffer(a.x, (int64_t)a.T * a.H);
  const auto sb = buffer(a.sx, (int64_t)a.T * chunks * 4);
  // whether fragment n, at this lane's row of it (r of a column, or of the result), is of gate
  auto is_gate = [&](int n, int r) { return COLS < 16 ? r < 8 : n < NC / 2; };

  // what is fetched next: chunk `step` (of this wave) of item `ahead`
  int ahead = blockIdx.x, step = 0;
  auto wb = buffer(a.w13, 0);
  uint32_t wrow[NC], xrow, srow;
  float next_g, next_u;                              // weight scales of item `ahead`
  auto aim = [&]() {
    const Job job = plan.at(min(ahead, items - 1) / tiles);
    const int col0 = min(ahead, items - 1) % tiles * COLS;
    wb = buffer(a.w13 + job.expert * panel, ahead < items ? panel : 0);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int col = col0 + (COLS < 16 ? fr % 8 : n % (COLS / kHalf) * 16 + fr);
      wrow[n] = (uint32_t)(((is_gate(n, fr) ? 0 : a.I) + col) * (int64_t)a.H + fg * 16);
    }
    const bool there = fr < job.n && ahead < items;
    const uint32_t t = there ? plan.row[job.start + fr] >> 16 : 0u;
    xrow = there ? t * (uint32_t)a.H + fg * 16 : kNoRow;
    srow = there ? t * 4 : kNoRow;
    const float* sc = a.s13 + (int64_t)job.expert * (2 * a.I / 128) * chunks;
    next_g = lane_scale(sc + (int64_t)(col0 / 128) * chunks, chunks);
    next_u = lane_scale(sc + (int64_t)((a.I + col0) / 128) * chunks, chunks);
  };
  struct Chunk {
    u32x4 w0[NC], w1[NC], x0, x1;
    float sx;
  } c[U];
  auto fetch = [&](Chunk& k) {
    const int kb = wave + step * kWaves;
    const uint32_t at = kb < chunks ? (uint32_t)kb * 128 : kNoChunk;
    const uint32_t sat = kb < chunks ? (uint32_t)(kb * a.T * 4) : kNoChunk;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      k.w0[n] = load16(wb, wrow[n] + at);
      k.w1[n] = load16(wb, wrow[n] + at + 64);
    }
    k.x0 = load16(xb, xrow + at);
    k.x1 = load16(xb, xrow + at + 64);
    k.sx = load4(sb, srow + sat);
    ++step;
  };
  if (ahead >= items) return;
  aim();
#pragma unroll
  for (int i = 0; i < U; ++i) fetch(c[i]);
  const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
  v4f acc[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) acc[n] = zero;
  int item = blockIdx.x, done = 0;
  float scale_g = next_g, scale_u = next_u;
  auto finish = [&]() {                              // item is whole: its activations
    const Job job = plan.at(item / tiles);
    const int col0 = item % tiles * COLS;
    leave(acc, red);
    for (int i = threadIdx.x; i < 16 * COLS; i += kThreads) {
      const int m = i / COLS, c = i % COLS;
      if (m >= job.n) break;
      const float g = total<NC>(red, c / 16, m, c % 16);
      const float u = COLS < 16 ? total<NC>(red, 0, m, 8 + c) : total<NC>(red, NC / 2 + c / 16, m, c % 16);
      const float v = plan.weight[job.start + m] * (g / (1.0f + expf(-g))) * u;
      const __bf16 hi = (__bf16)v, lo = (__bf16)(v - (float)hi);
      const int64_t at = (int64_t)(job.start + m) * a.I + place_of(col0 + c);
      a.hi[at] = __builtin_bit_cast(uint16_t, hi);
      a.lo[at] = __builtin_bit_cast(uint16_t, lo);
    }
    __syncthreads();
  };
  for (;;) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float sg = of_lane(scale_g, done), su = of_lane(scale_u, done);
      const v8i x = join(c[i].x0, c[i].x1);
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(c[i].w0[n], c[i].w1[n]), x, zero, 0, 0, 0, 0, 0,
                                                                      0);
        const float by = c[i].sx * (is_gate(n, fg * 4) ? sg : su);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = __builtin_fmaf(p[e], by, acc[n][e]);
      }
      if (step == steps) {
        ahead += gridDim.x;
        step = 0;
        aim();
      }
      fetch(c[i]);
      if (++done == steps) {
        finish();
        item += gridDim.x;
        if (item >= items) return;
        done = 0;
        scale_g = next_g;
        scale_u = next_u;
#pragma unroll
        for (int n = 0; n < NC; ++n) acc[n] = zero;
      }
    }
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

// Items: one job and COLS columns of H, walked like those of k_moe_up by KS waves
// that take the chunks of I in turn: one wave where there are items enough for all
// (nothing is shared but the plan then), else four.
template <int COLS, int KS>
__global__ __launch_bounds__(kThreads, 3) void k_moe_down(ExpertArgs a) {
  static_assert(KS == 1 || KS == kWaves, "the sums over waves and their barriers are the whole workgroup's");
  constexpr int NC = COLS / 16, U = 2;
  extern __shared__ __align__(16) uint32_t lds[];
  __shared__ __align__(16) float red[KS > 1 ? KS * NC * 256 : 1];
  const Plan plan = load_plan(a, lds);
  const int lane = threadIdx.x % 64, fr = lane % 16, fg = lane / 16;
  const int chunks = a.I / 128, steps = steps_of(chunks, KS, U), part = wave_id() % KS;
  const int tiles = a.H / COLS, items = plan.jobs * tiles, stride = gridDim.x * (kWaves / KS);
  const int64_t panel = (int64_t)a.H * a.I, acts = (int64_t)a.T * a.topk * a.I * 2;
  const auto hb = buffer(a.hi, acts), lb = buffer(a.lo, acts);
  put_zeros(a);

  // (the first item of every workgroup before the second of any)
  int item = wave_id() / KS * gridDim.x + blockIdx.x, ahead = item, step = 0;
  if (item >= items) return;
  auto wb = buffer(a.w2, 0);
  uint32_t wrow[NC], arow;
  const float *scale, *next_scale;
  auto aim = [&]() {
    const Job job = plan.at(min(ahead, items - 1) / tiles);
    const int col0 = min(ahead, items - 1) % tiles * COLS;
    wb = buffer(a.w2 + job.expert * panel, ahead < items ? panel : 0);
#pragma unroll
    for (int n = 0; n < NC; ++n) wrow[n] = (uint32_t)((col0 + n * 16 + fr) * (int64_t)a.I + fg * 16);
    next_scale = a.s2 + ((int64_t)job.expert * (a.H / 128) + col0 / 128) * chunks;
  };
  auto aim_acts = [&](int item) {
    const Job job = plan.at(min(item, items - 1) / tiles);
    arow = fr < job.n && item < items ? (uint32_t)((job.start + fr) * (int64_t)a.I + fg * 8) * 2 : kNoRow;
  };
  struct Chunk {
    u32x4 w0[NC], w1[NC];
  } c[U];
  auto fetch = [&](Chunk& k) {
    const int kb = part + step * KS;
    const uint32_t at = kb < chunks ? (uint32_t)kb * 128 : kNoChunk;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      k.w0[n] = load16(wb, wrow[n] + at);
      k.w1[n] = load16(wb, wrow[n] + at + 64);
    }
    ++step;
  };
  u32x4 hi[4], lo[4];
  auto fetch_acts = [&](int s) {
    const int kb = part + s * KS;
    const uint32_t at = kb < chunks ? (uint32_t)kb * 256 : kNoChunk;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = load16(hb, arow + at + j * 64);
      lo[j] = load16(lb, arow + at + j * 64);
    }
  };
  // Loads return in the order they were issued, so the activations of a chunk
  // (from L2) go out ahead of weights (from memory) that are needed later.
  aim();
  aim_acts(item);
  fetch(c[0]);
  fetch_acts(0);
#pragma unroll
  for (int i = 1; i < U; ++i) fetch(c[i]);
  const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
  v4f acc[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) acc[n] = zero;
  auto finish = [&]() {
    const Job job = plan.at(item / tiles);
    const int col0 = item % tiles * COLS;
    if (KS == 1) {
      if (fr >= job.n) return;                       // a lane has four columns of a row
      const int place = plan.row[job.start + fr] & 0xFFFF;
#pragma unroll
      for (int n = 0; n < NC; ++n) put_row(a, place, col0 + n * 16 + fg * 4, acc[n]);
    } else {
      leave(acc, red);
      const int m = threadIdx.x % 16, g = threadIdx.x / 16;
      if (m < job.n && g < COLS / 4) {
        const v4f* from = reinterpret_cast<const v4f*>(red) + threadIdx.x;   // fragment g / 4, its columns g % 4 * 4 ...
        v4f v = from[0];
#pragma unroll
        for (int w = 1; w < KS; ++w) v += from[w * NC * 64];
        put_row(a, plan.row[job.start + m] & 0xFFFF, col0 + g * 4, v);
      }
      __syncthreads();
    }
  };
  int done = 0;
  scale = next_scale;
  for (;;) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float s = scale[min(part + done * KS, chunks - 1)];
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const v8bf b[4] = {to_bf16(c[i].w0[n].x, c[i].w0[n].y), to_bf16(c[i].w0[n].z, c[i].w0[n].w),
                           to_bf16(c[i].w1[n].x, c[i].w1[n].y), to_bf16(c[i].w1[n].z, c[i].w1[n].w)};
        v4f p = zero;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], __builtin_bit_cast(v8bf, hi[j]), p, 0, 0, 0);
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], __builtin_bit_cast(v8bf, lo[j]), p, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = __builtin_fmaf(p[e], s, acc[n][e]);
      }
      const bool last = ++done == steps;
      if (last) aim_acts(item + stride);
      fetch_acts(last ? 0 : done);
      if (step == steps) {
        ahead += stride;
        step = 0;
        aim();
      }
      fetch(c[i]);
      if (last) {
        finish();
        item += stride;
        if (item >= items) return;
        done = 0;
        scale = next_scale;
#pragma unroll
        for (int n = 0; n < NC; ++n) acc[n] = zero;
      }
    }
  }
}

// Few tokens (at most 16): all experts of 16 columns of H in one workgroup, a row of
// the matrix core's result per token, so that the sums over experts stay in its
// accumulators and nothing is left to k_moe_join.  The waves take the chunks of all
// jobs in turn.
constexpr int kWholeWaves = 8;
__global__ __launch_bounds__(64 * kWholeWaves) void k_moe_down_whole(ExpertArgs a) {
  constexpr int U = 2;
  extern __shared__ __align__(16) uint32_t lds[];
  __shared__ __align__(16) v4f red[kWholeWaves * 64];
  const Plan plan = load_plan(a, lds);
  const int lane = threadIdx.x % 64, wave = wave_id(), fr = lane % 16, fg = lane / 16, col0 = blockIdx.x * 16;
  const int chunks = a.I / 128, units = plan.jobs * chunks;
  const int64_t panel = (int64_t)a.H * a.I, acts = (int64_t)a.T * a.topk * a.I * 2;
  const auto hb = buffer(a.hi, acts), lb = buffer(a.lo, acts);
  const uint32_t wrow = (uint32_t)((col0 + fr) * (int64_t)a.I + fg * 16);
  struct Chunk {
    u32x4 w0, w1;
  } c[U];
  auto fetch = [&](Chunk& k, int unit) {
    const int u = min(unit, units - 1), kb = u % chunks;
    const auto wb = buffer(a.w2 + plan.at(u / chunks).expert * panel, unit < units ? panel : 0);
    k.w0 = load16(wb, wrow + kb * 128);
    k.w1 = load16(wb, wrow + kb * 128 + 64);
  };
  u32x4 hi[4], lo[4];
  bool there;                                        // whether token fr has a row of the unit's job
  float scale;
  auto fetch_acts = [&](int unit) {
    const int u = min(unit, units - 1), kb = u % chunks;
    const Job job = plan.at(u / chunks);
    uint32_t tokens = fr < job.n ? 1u << (plan.row[job.start + fr] >> 16) : 0u;
    tokens = row16_or(tokens);
    there = unit < units && (tokens >> fr & 1);
    const int r = job.start + __builtin_popcount(tokens & ((1u << fr) - 1));
    const uint32_t at = there ? (uint32_t)(r * (int64_t)a.I + kb * 128 + fg * 8) * 2 : kNoRow;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = load16(hb, at + j * 64);
      lo[j] = load16(lb, at + j * 64);
    }
    scale = a.s2[((int64_t)job.expert * (a.H / 128) + col0 / 128) * chunks + kb];
  };
  const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
  v4f acc = zero;
  if (wave < units) {
    fetch(c[0], wave);
    fetch_acts(wave);
#pragma unroll
    for (int i = 1; i < U; ++i) fetch(c[i], wave + i * kWholeWaves);
    for (int unit = wave; unit < units; unit += U * kWholeWaves) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int u = unit + i * kWholeWaves;
        const v8bf b[4] = {to_bf16(c[i].w0.x, c[i].w0.y), to_bf16(c[i].w0.z, c[i].w0.w), to_bf16(c[i].w1.x, c[i].w1.y),
                           to_bf16(c[i].w1.z, c[i].w1.w)};
        v4f p = zero;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], __builtin_bit_cast(v8bf, hi[j]), p, 0, 0, 0);
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], __builtin_bit_cast(v8bf, lo[j]), p, 0, 0, 0);
        }
        // (a token without a row has zeros times whatever the codes and scales are)
        const float s = scale;
        const bool counts = there;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = counts ? __builtin_fmaf(p[e], s, acc[e]) : acc[e];
        fetch_acts(u + kWholeWaves);
        fetch(c[i], u + U * kWholeWaves);
      }
    }
  }
  red[wave * 64 + lane] = acc;
  __syncthreads();
  const int m = threadIdx.x / 4, g = threadIdx.x % 4;   // four columns of a token
  if (m >= a.T) return;
  v4f v = red[g * 16 + m];
#pragma unroll
  for (int w = 1; w < kWholeWaves; ++w) v += red[w * 64 + g * 16 + m];
  put_out(a, m, col0 + g * 4, v);
}

// ---- many rows per expert ----
//
// The tokens' rows of a job go through LDS, once per workgroup; its waves take
// different columns, all of K.  A piece of the rows is in flight while the one
// before is in use, in two buffers; one barrier per piece.

constexpr int kPiece = 4;   // chunks of H per piece in k_moe_up_wide

// Segment s (16 bytes) of a row of 8 (16) segments is kept at s ^ key: the 16
// rows that a wave reads at one segment fall on different banks.
__device__ __forceinline__ int swizzle8(int row, int s) { return s ^ ((row >> 1) & 7); }
__device__ __forceinline__ int swizzle16(int row, int s) { return s ^ (row & 15); }

// Work of one workgroup: a job and a unit of columns, or half of one.  Whole units
// read a job's rows half as often, halves leave less undone at the end: so as many
// whole units as fill the chip in rounds of two workgroups per CU come first, and
// the rest in halves (64 tokens of 32 experts of 7168 x 2048: 287 -> 279 us).  Two fit
// up to about 850 places; with more of them the plan's LDS leaves one per CU: 128 tokens
// of 8 of 32 experts of 7168 x 2048 take 424 us, 64 tokens of 16 of 32 take 460, where
// the weights alone are 248 at the read's rate.
struct Share {
  int unit, half;   // half: 0, 1, or -1 for both
};
__device__ __forceinline__ Share share_of(int block, int units) {
  const int whole = units & ~511;
  if (block < whole) return {block, -1};
  return {whole + (block - whole) / 2, (block - whole) % 2};
}

// One workgroup per job and 64 NG columns of I, 16 NG per wave.
template <int MF, int NG, int U>
__device__ __forceinline__ void up_wide(const ExpertArgs& a, const Plan& plan, const Job& job, int col0, uint8_t* stage) {
  // stage: [2][kPiece][16 MF rows][128], then scales [2][kPiece][16 MF + 2]
  constexpr int kRows = 16 * MF, kBuf = kPiece * kRows * 128, kPer = kRows * 8 * kPiece / kThreads, NC = 2 * NG;
  constexpr int kScales = kPiece * (kRows + 2);
  static_assert(kPiece % U == 0, "a chunk's place in the ring goes by its place in the piece");
  float* scales = reinterpret_cast<float*>(stage + 2 * kBuf);
  const int tid = threadIdx.x, lane = tid % 64, wave = wave_id(), fr = lane % 16, fg = lane / 16;
  const int chunks = a.H / 128, pieces = (chunks + kPiece - 1) / kPiece;
  const int64_t panel = 2 * (int64_t)a.I * a.H;
  const auto wb = buffer(a.w13 + job.expert * panel, panel);
  const auto xb = buffer(a.x, (int64_t)a.T * a.H);
  const int col = col0 + wave * 16 * NG;
  uint32_t wrow[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n)
    wrow[n] = (uint32_t)(((n / NG) * a.I + col + (n % NG) * 16 + fr) * (int64_t)a.H + fg * 16);

  // this thread's segments of a piece: row, chunk and place in the chunk
  u32x4 x[kPer];
  uint32_t from[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = i * kThreads + tid, r = p / (8 * kPiece), s = p % (8 * kPiece);
    from[i] = r < job.n ? (plan.row[job.start + min(r, job.n - 1)] >> 16) * (uint32_t)a.H + s * 16 : kNoRow;
  }
  // and its scales: of rows (one chunk each), of the weights
  constexpr int kPerScale = (kScales + kThreads - 1) / kThreads;
  float sc[kPerScale];
  auto fetch_piece = [&](int piece) {
    const uint32_t at = (uint32_t)piece * kPiece * 128;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = (i * kThreads + tid) % (8 * kPiece);
      x[i] = load16(xb, piece * kPiece + s / 8 < chunks ? from[i] + at : kNoRow);
    }
#pragma unroll
    for (int i = 0; i < kPerScale; ++i) {
      const int p = i * kThreads + tid, c = p / (kRows + 2), r = p % (kRows + 2), kb = piece * kPiece + c;
      sc[i] = 0.0f;
      if (p < kScales && kb < chunks) {
        const int64_t block = r == kRows ? col0 / 128 : (a.I + col0) / 128;
        if (r >= kRows) sc[i] = a.s13[((int64_t)job.expert * (2 * a.I / 128) + block) * chunks + kb];
        else if (r < job.n) sc[i] = a.sx[(int64_t)kb * a.T + (plan.row[job.start + r] >> 16)];
      }
    }
  };
  auto keep_piece = [&](int piece) {
    uint8_t* to = stage + (piece & 1) * kBuf;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = i * kThreads + tid, r = p / (8 * kPiece), s = p % (8 * kPiece);
      *reinterpret_cast<u32x4*>(to + ((s / 8) * kRows + r) * 128 + swizzle8(r, s % 8) * 16) = x[i];
    }
#pragma unroll
    for (int i = 0; i < kPerScale; ++i)
      if (i * kThreads + tid < kScales) scales[(piece & 1) * kScales + i * kThreads + tid] = sc[i];
  };
  u32x4 w[U][NC][2];
  auto fetch = [&](int i, int kb) {
    const uint32_t at = kb < chunks ? (uint32_t)kb * 128 : kNoChunk;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      w[i][n][0] = load16(wb, wrow[n] + at);
      w[i][n][1] = load16(wb, wrow[n] + at + 64);
    }
  };
  const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
  v4f acc[MF][NC];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int n = 0; n < NC; ++n) acc[f][n] = zero;
  fetch_piece(0);
#pragma unroll
  for (int i = 0; i < U; ++i) fetch(i, i);
  for (int piece = 0; piece < pieces; ++piece) {
    keep_piece(piece);
    __syncthreads();
    fetch_piece(piece + 1);
    const uint8_t* xs = stage + (piece & 1) * kBuf;
    const float* ss = scales + (piece & 1) * kScales;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const float sg = ss[i * (kRows + 2) + kRows], su = ss[i * (kRows + 2) + kRows + 1];
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const int r = f * 16 + fr;
        const uint8_t* row = xs + (i * kRows + r) * 128;
        const v8i xf = join(*reinterpret_cast<const u32x4*>(row + swizzle8(r, fg) * 16),
                            *reinterpret_cast<const u32x4*>(row + swizzle8(r, fg + 4) * 16));
        const float sx = ss[i * (kRows + 2) + r];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(w[i % U][n][0], w[i % U][n][1]), xf, zero, 0,
                                                                        0, 0, 0, 0, 0);
          const float by = sx * (n < NG ? sg : su);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[f][n][e] = __builtin_fmaf(p[e], by, acc[f][n][e]);
        }
      }
      fetch(i % U, piece * kPiece + i + U);
    }
  }
  // a lane has four columns of a row
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int r = f * 16 + fr;
    if (r >= job.n) continue;
    const float share = plan.weight[job.start + r];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      float hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float g = acc[f][n][e], v = share * (g / (1.0f + expf(-g))) * acc[f][NG + n][e];
        hi[e] = v;
        lo[e] = v - (float)(__bf16)v;
      }
      const int64_t at = (int64_t)(job.start + r) * a.I + place_of(col + n * 16 + fg * 4);
      *reinterpret_cast<uint2*>(a.hi + at) = make_uint2(pack2_bf16(hi[0], hi[1]), pack2_bf16(hi[2], hi[3]));
      *reinterpret_cast<uint2*>(a.lo + at) = make_uint2(pack2_bf16(lo[0], lo[1]), pack2_bf16(lo[2], lo[3]));
    }
  }
}

constexpr int kUpStage = 2 * kPiece * (64 * 128 + 66 * 4);   // bytes, for 64 rows

// A unit is 128 columns of I; with more than 32 rows its halves go one after the
// other, for their accumulators.
__global__ __launch_bounds__(kThreads, 2) void k_moe_up_wide(ExpertArgs a) {
  extern __shared__ __align__(16) uint32_t lds[];
  const Plan plan = make_plan(a, lds + kUpStage / 4, 64);
  save_plan(a, plan);
  const int tiles = a.I / 128, units = plan.jobs * tiles;
  const Share share = share_of(blockIdx.x, units);
  if (share.unit >= units) return;
  const Job job = plan.at(share.unit / tiles);
  const int col0 = share.unit % tiles * 128;
  uint8_t* stage = reinterpret_cast<uint8_t*>(lds);
  if (share.half < 0 && job.n <= 16) {
    up_wide<1, 2, 2>(a, plan, job, col0, stage);
  } else if (share.half < 0 && job.n <= 32) {
    up_wide<2, 2, 2>(a, plan, job, col0, stage);
  } else {
    for (int half = max(share.half, 0); half <= (share.half < 0 ? 1 : share.half); ++half) {
      __syncthreads();
      if (job.n <= 16) up_wide<1, 1, 4>(a, plan, job, col0 + half * 64, stage);
      else if (job.n <= 32) up_wide<2, 1, 4>(a, plan, job, col0 + half * 64, stage);
      else up_wide<4, 1, 4>(a, plan, job, col0 + half * 64, stage);
    }
  }
}

// One workgroup per job and 64 NC columns of H, 16 NC per wave; a piece is one
// chunk of I.
template <int MF, int NC, int U>
__device__ __forceinline__ void down_wide(const ExpertArgs& a, const Plan& plan, const Job& job, int col0,
                                          uint8_t* stage) {
  // stage: [2][hi, lo][16 MF rows][256]
  constexpr int kRows = 16 * MF, kBuf = 2 * kRows * 256, kPer = kBuf / 16 / kThreads;
  const int tid = threadIdx.x, lane = tid % 64, wave = wave_id(), fr = lane % 16, fg = lane / 16;
  const int chunks = a.I / 128;
  const int64_t panel = (int64_t)a.H * a.I, acts = (int64_t)a.T * a.topk * a.I * 2;
  const auto wb = buffer(a.w2 + job.expert * panel, panel);
  const auto hb = buffer(a.hi, acts), lb = buffer(a.lo, acts);
  const int col = col0 + wave * 16 * NC;             // (past H: nothing is read or written)
  const float* sc = a.s2 + ((int64_t)job.expert * (a.H / 128) + min(col, a.H - 1) / 128) * chunks;
  uint32_t wrow[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) wrow[n] = col < a.H ? (uint32_t)((col + n * 16 + fr) * (int64_t)a.I + fg * 16) : kNoRow;
  u32x4 x[kPer];
  uint32_t from[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = (i * kThreads + tid) / 16 % kRows, s = tid % 16;
    from[i] = r < job.n ? (uint32_t)((job.start + r) * (int64_t)a.I) * 2 + s * 16 : kNoRow;
  }
  auto fetch_piece = [&](int kb) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t at = kb < chunks ? from[i] + (uint32_t)kb * 256 : kNoRow;
      x[i] = i < kPer / 2 ? load16(hb, at) : load16(lb, at);
    }
  };
  auto keep_piece = [&](int kb) {
    uint8_t* to = stage + (kb & 1) * kBuf;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = i * kThreads + tid, r = p / 16;     // (rows of lo after those of hi)
      *reinterpret_cast<u32x4*>(to + r * 256 + swizzle16(r, tid % 16) * 16) = x[i];
    }
  };
  u32x4 w[U][NC][2];
  float scale[U];
  auto fetch = [&](int i, int kb) {
    const uint32_t at = kb < chunks ? (uint32_t)kb * 128 : kNoChunk;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      w[i][n][0] = load16(wb, wrow[n] + at);
      w[i][n][1] = load16(wb, wrow[n] + at + 64);
    }
    scale[i] = sc[min(kb, chunks - 1)];
  };
  const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
  v4f acc[MF][NC];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int n = 0; n < NC; ++n) acc[f][n] = zero;
  fetch_piece(0);
#pragma unroll
  for (int i = 0; i < U; ++i) fetch(i, i);
  for (int k0 = 0; k0 < chunks; k0 += U) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int kb = k0 + i;
      keep_piece(kb);
      __syncthreads();
      fetch_piece(kb + 1);
      const uint8_t* xs = stage + (kb & 1) * kBuf;
      v8bf b[NC][4];
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        b[n][0] = to_bf16(w[i][n][0].x, w[i][n][0].y);
        b[n][1] = to_bf16(w[i][n][0].z, w[i][n][0].w);
        b[n][2] = to_bf16(w[i][n][1].x, w[i][n][1].y);
        b[n][3] = to_bf16(w[i][n][1].z, w[i][n][1].w);
      }
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const int r = f * 16 + fr;
        v4f p[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) p[n] = zero;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v8bf hi = *reinterpret_cast<const v8bf*>(xs + r * 256 + swizzle16(r, j * 4 + fg) * 16);
          const v8bf lo = *reinterpret_cast<const v8bf*>(xs + (kRows + r) * 256 + swizzle16(r, j * 4 + fg) * 16);
#pragma unroll
          for (int n = 0; n < NC; ++n) p[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[n][j], hi, p[n], 0, 0, 0);
#pragma unroll
          for (int n = 0; n < NC; ++n) p[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[n][j], lo, p[n], 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[f][n][e] = __builtin_fmaf(p[n][e], scale[i], acc[f][n][e]);
      }
      fetch(i, kb + U);
    }
  }
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int r = f * 16 + fr;
    if (r >= job.n || col >= a.H) continue;
    const int place = plan.row[job.start + r] & 0xFFFF;
#pragma unroll
    for (int n = 0; n < NC; ++n) put_row(a, place, col + n * 16 + fg * 4, acc[f][n]);
  }
}

constexpr int kDownStage = 2 * 2 * 64 * 256;   // bytes, for 64 rows

// A unit is 256 columns of H (the last one may have 128).
__global__ __launch_bounds__(kThreads, 2) void k_moe_down_wide(ExpertArgs a) {
  extern __shared__ __align__(16) uint32_t lds[];
  const Plan plan = load_plan(a, lds + kDownStage / 4);
  put_zeros(a);
  const int tiles = (a.H + 255) / 256, units = plan.jobs * tiles;
  const Share share = share_of(blockIdx.x, units);
  if (share.unit >= units) return;
  const Job job = plan.at(share.unit / tiles);
  const int col0 = share.unit % tiles * 256;
  uint8_t* stage = reinterpret_cast<uint8_t*>(lds);
  if (share.half < 0 && job.n <= 16) {
    down_wide<1, 4, 2>(a, plan, job, col0, stage);
  } else if (share.half < 0 && job.n <= 32) {
    down_wide<2, 4, 2>(a, plan, job, col0, stage);
  } else {
    for (int half = max(share.half, 0); half <= (share.half < 0 ? 1 : share.half); ++half) {
      const int col = col0 + half * 128;
      if (col >= a.H) break;
      __syncthreads();
      if (job.n <= 16) down_wide<1, 2, 4>(a, plan, job, col, stage);
      else if (job.n <= 32) down_wide<2, 2, 4>(a, plan, job, col, stage);
      else down_wide<4, 2, 4>(a, plan, job, col, stage);
    }
  }
}

// ---- the sum over a token's experts ----

// out[t] = the rows of token t's places added up in turn.  A place has a row where
// its id is inside and stands no further left; the others are read too (inside the
// workspace; that way no read waits for the ids) and left out.
__global__ __launch_bounds__(kThreads) void k_moe_join(ExpertArgs a) {
  const int t = blockIdx.y, h0 = (blockIdx.x * kThreads + threadIdx.x) * 4, h = min(h0, a.H - 4), lane = threadIdx.x % 64;
  const int id = lane < a.topk ? a.ids[t * a.topk + lane] : -1;
  const v4f* from = reinterpret_cast<const v4f*>(a.part + (int64_t)t * a.topk * a.H + h);
  const int step = a.H / 4;
  v4f r[8];
  auto fetch = [&](int c0) {                         // eight in flight, of at most 16
#pragma unroll
    for (int c = 0; c < 8; ++c) r[c] = from[min(c0 + c, a.topk - 1) * step];
  };
  fetch(0);
  bool counts = (uint32_t)id < (uint32_t)a.E;
  for (int c = 0; c < a.topk; ++c) counts = counts && !(c < lane && __builtin_amdgcn_readlane(id, c) == id);
  const uint32_t there = (uint32_t)__builtin_amdgcn_ballot_w64(counts);
  v4f v{0.0f, 0.0f, 0.0f, 0.0f};
  for (int c0 = 0; c0 < a.topk; c0 += 8) {
    if (c0) fetch(c0);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (there >> (c0 + c) & 1) v += r[c];
  }
  if (h0 < a.H) put_out(a, t, h, v);
}

int64_t aligned(int64_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

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
  a.part = reinterpret_cast<float*>(take(a.topk == 1 ? 0 : places * a.H * 4));
  a.image = reinterpret_cast<uint32_t*>(take(image_words(a) * 4));
  return at;
}

namespace {

constexpr int kCus = 256;

// As many workgroups as run at once, or as may have an item.
unsigned grid_of(const ExpertArgs& a, int tiles, int per_cu) {
  const int64_t most = (int64_t)tiles * a.T * a.topk;
  return (unsigned)std::min<int64_t>(most, (int64_t)kCus * per_cu);
}

template <int COLS>
void launch_up(const ExpertArgs& a, hipStream_t stream) {
  k_moe_up<COLS><<<grid_of(a, a.I / COLS, 4), kThreads, plan_bytes(a), stream>>>(a);
}

template <int COLS, int KS>
void launch_down(const ExpertArgs& a, hipStream_t stream) {
  const int groups = (a.H / COLS + kWaves / KS - 1) / (kWaves / KS);
  k_moe_down<COLS, KS><<<grid_of(a, groups, 3), kThreads, a.T * a.topk * 8, stream>>>(a);
}

// Whether so little of w2 is read that the last sum, a kernel of its own with 2 us of
// its launch, costs more than 16 columns of H per workgroup do.  Calls in a row, in us,
// k_moe_down_whole against k_moe_down and k_moe_join, by (tokens, experts, topk, H, I):
// (1, 8, 2, 1024, 512) 16.7 / 18.7, (16, 4, 4, 512, 512) 16.7 / 19.8, (11, 4, 3, 3456, 128)
// 16.6 / 18.7, (16, 8, 4, 4096, 512) 24.0 / 26.6, (16, 16, 4, 2048, 256) 16.8 / 19.1; but
// (16, 4, 4, 1024, 1024) 20.2 / 19.2, (16, 16, 4, 1024, 512) 20.9 / 19.4, (1, 8, 8, 2048,
// 1024) 22.5 / 21.7, (16, 4, 4, 7168, 1024) 39.3 / 32.9, (1, 32, 8, 7168, 2048) 84.7 / 73.6.
// (Four or 16 waves, or four chunks in flight: none better over these.)
bool whole(const ExpertArgs& a, int experts) {
  const int chunks = experts * (a.I / 128) * ((a.H + 4095) / 4096);   // of a CU, with a workgroup on every one
  return a.T <= 16 && chunks <= (a.H < 2048 ? 16 : 32);
}

// Narrow items where there are few, so that more workgroups share the reading.
// Kernel times in us of both sides, by (tokens, experts, topk, H, I):
//   up, 8 columns against 16: (1, 2, 2, 6400, 256) 9.6 / 12.4, (1, 48, 5, 1792, 384)
//     7.6 / 8.4, (4, 64, 1, 2048, 768) 8.4 / 8.4, (3, 128, 5, 4224, 768) 25.3 / 24.0
//   down, 64 columns, one wave per item against four: (1, 32, 8, 7168, 2048) 25.0 /
//     26.6, (35, 32, 5, 4992, 256) 13.3 / 23.6, (39, 32, 5, 1408, 2048) 24.5 / 24.7; of
//     few items (2, 16, 4, 4096, 1024) 13.1 / 10.3, (1, 4, 2, 7168, 4096) 39.2 / 15.7
//   down, four waves, 64 columns against 32: (58, 32, 4, 1024, 1024) 12.1 / 14.4,
//     (4, 64, 1, 2048, 768) 6.6 / 5.8; 32 against 16: the same 5.2 / 6.0, (1, 4, 4,
//     1024, 1408) 5.6 / 5.2, (17, 1, 1, 512, 1024) 6.6 / 5.8, (20, 4, 1, 512, 2048) 8.0 / 6.9
ExpertTile narrow_tile(const ExpertArgs& a) {
  const int experts = std::min(a.E, a.T * a.topk);   // that may have rows
  const int up = experts * (a.I / 16) < 200 ? 8 : 16;
  if (whole(a, experts)) return {16, up, 16, kWholeWaves};
  const int items = experts * (a.H / 64);
  if (items >= 700) return {16, up, 64, 1};
  if (a.I <= 256) return {16, up, 32, 1};
  return {16, up, items >= 250 ? 64 : items > 64 ? 32 : 16, 4};
}

// Whether an expert has many rows, were they spread evenly, and the chip is full
// with fewer and larger shares.  Both products, wide against narrow: (32, 32, 8,
// 7168, 2048) 256 / 267 us, (24, 32, 8, 7168, 2048) 255 / 257, (64, 8, 4, 4096,
// 1536) 61 / 77, (32, 8, 8, 2048, 512) 26 / 24, (36, 4, 3, 2816, 256) 26 / 15.  With
// 64 rows and more the narrow kernels read an expert four times and more: (128, 2, 2,
// 7168, 2048) 82 / 169, (128, 1, 1, 7168, 2048) 76 / 98, (128, 2, 2, 4096, 512) 41 / 43,
// but (100, 1, 1, 512, 2048) 39 / 21.  One rule for both products, which sees neither the
// second one's units nor whether ids are outside [0, E) (places without rows count):
// few units leave most of the chip idle, (20, 4, 2, 512, 2048) 27 us, of 2.2 at the
// read's rate.
bool wide(const ExpertArgs& a) {
  const int experts = std::min(a.E, a.T * a.topk);
  const int places = a.T * a.topk;
  return (places >= 8 * experts && experts * (a.I / 128) >= 64) ||
         (places >= 64 * experts && (int64_t)experts * a.H * a.I >= 1 << 22);
}

}  // namespace

ExpertTile experts_tile(const ExpertArgs& a) { return wide(a) ? ExpertTile{64, 128, 256, 4} : narrow_tile(a); }

hipError_t launch_moe_experts(const ExpertArgs& a, hipStream_t stream) {
  const ExpertTile t = experts_tile(a);
  if (t.rows == 64) {
    // (jobs of up to 64 rows: at most one per expert with a row, and one more per 64 rows)
    const int64_t jobs = std::min(a.E, a.T * a.topk) + a.T * a.topk / 64;
    const size_t plan = plan_bytes(a);
    k_moe_up_wide<<<(unsigned)(jobs * (a.I / 64)), kThreads, kUpStage + plan, stream>>>(a);
    k_moe_down_wide<<<(unsigned)(jobs * ((a.H + 255) / 256) * 2), kThreads, kDownStage + plan, stream>>>(a);
  } else {
    if (t.up == 8) launch_up<8>(a, stream);
    else launch_up<16>(a, stream);
    if (t.waves == kWholeWaves) {
      k_moe_down_whole<<<a.H / 16, 64 * kWholeWaves, a.T * a.topk * 8, stream>>>(a);
      return hipGetLastError();
    }
    if (t.waves == 1 && t.down == 64) launch_down<64, 1>(a, stream);
    else if (t.waves == 1) launch_down<32, 1>(a, stream);
    else if (t.down == 64) launch_down<64, 4>(a, stream);
    else if (t.down == 32) launch_down<32, 4>(a, stream);
    else launch_down<16, 4>(a, stream);
  }
  // one place per token: nothing to add up, 3 us of a call (64 tokens, 16 experts of
  // 7168 x 2048: 139 -> 135 us; 32 tokens, 8 of 1024 x 512: 19 -> 16.5)
  if (a.topk == 1) return hipGetLastError();
  k_moe_join<<<dim3((unsigned)((a.H / 4 + kThreads - 1) / kThreads), (unsigned)a.T), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace fp8bs
