// Attention over the paged FP8 cache for many rows (prompts and chunks): the
// matrix-bound form of fp8bs_cache_attention.
//
// One workgroup per (sequence, head, 32 x waves rows, split of the cached
// tokens); a row is one (new token, query head of the group) pair.  It walks
// 64-token steps: the codes of a step are converted to BF16 once for all waves
// and staged in LDS, keys as [token][dim], values as [dim][token].  Each wave
// keeps 32 rows: Q in registers, S^T = K Q^T and O^T = V^T P^T by 32x32x16
// products.  S^T's result layout (lane = row, four consecutive tokens) is
// P^T's operand layout once the 16 tokens of a step are stored in LDS in the
// order 8 a + 4 half + i -> 8 half + 4 a + i.
//
// A wave alternates a matrix phase (scores of step t, outputs of step t - 1)
// with a softmax phase on the vector unit.  Of the two waves of a SIMD one
// meets the step's barrier before its matrix phase, the other after it, so
// that their phases interleave.  The staging rides in the matrix phase, whose
// vector slots are free: keys of step t + 1 and values of step t are converted
// and written there, the codes of the next ones requested.
//
// Two causal prompts of up to 6000 tokens (8 heads x 4, D = 128) take 460 us, 917
// TFLOP/s (450 to 473 us over several cards; a BF16 library product of 8192^3:
// 1207).  The matrix core is busy 41 % of the time and the vector unit 60 %:
// either alone would need about 180 and 270 us, so they hardly overlap in effect.
// D = 64 with capped scores (four 513-token chunks behind up to 9000) takes 190
// us: the vector unit is busy 60 % and waves wait 38 % of the time, beside 35
// spilled registers.
#include "cache_device.h"

namespace fp8bs {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kTok = 64;                             // tokens per step

template <int N>
struct Int {
  static constexpr int value = N;
};

// Whether any lane of the wave has it (wave-uniform).
__device__ __forceinline__ bool any_lane(bool x) { return __builtin_amdgcn_ballot_w64(x) != 0; }

// Keys: row = token, 16-byte chunks of 8 dims.  A wave's reads take one chunk
// of 32 rows: rows 16 bytes longer than D walk over all banks, and every read
// of a step is one lane address plus a constant.
template <int D>
constexpr int kPitch = D + 8;

template <int D>
__device__ __forceinline__ int k_at(int tok, int chunk) {
  return tok * kPitch<D> + chunk * 8;
}

// Values: row = dim, 16-byte chunks of 8 tokens.  Reads take one chunk of 32
// rows, writes half a chunk of every fourth row.
__device__ __forceinline__ int v_at(int dim, int chunk) {
  return dim * kTok + ((chunk ^ ((dim ^ (dim >> 2)) & 7)) * 8);
}

// Waves per SIMD.  D = 128: two; a wave's accumulators, queries and scores take
// 239 of 256 registers.  D = 64 is bound by the vector unit (a score costs the
// same there, its products half): three, as workgroups of their own, whose
// phases drift apart (513-token chunks 273 -> 213 us), though the 168 registers
// that leaves spill 35 (21 without a cap).  Second parts of the weights do not
// fit beside that: two.
template <int D, bool TWO>
constexpr int kPerSimd = D == 64 && !TWO ? 3 : 2;

// A weight meets the codes rounded to BF16 once: 2^-9 of it, about what the
// rounding of a BF16 output takes again.  TWO (FP32 outputs): as two BF16 parts,
// the second being what the first leaves, so that 2^-18 of it is lost; a step's
// outputs are then added before the scores of the next one.  The second products
// cost: prompts of up to 6000 tokens 603 us instead of 450, 25 tokens of each of 32
// sequences behind 4096 (D = 128, 128 rows) 162 instead of 86 (168 with one wave
// per SIMD and without the 38 spilled registers), the 513-token chunks (D = 64)
// 244 instead of 190.
template <int D, bool CAP, int WAVES, bool TWO>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(kPerSimd<D, TWO>, kPerSimd<D, TWO>)))
void k_attend_tiles(AttendArgs a, int row_tiles) {
  const CacheArgs& c = a.c;
  constexpr int T = 64 * WAVES, BM = 32 * WAVES;
  constexpr int KS = D / 16;                         // matrix steps of a score
  constexpr int DT = D / 32;                         // 32-dim tiles of the output
  constexpr int KP = kTok * (D / 8) / T;             // 8-byte key pieces per thread
  constexpr int VG = (kTok / 4) * (D / 4);           // 4 x 4 groups of values
  constexpr int VP = (VG + T - 1) / T;               // per thread
  __shared__ __attribute__((aligned(16))) uint16_t s_k[2][kTok * kPitch<D>];
  __shared__ __attribute__((aligned(16))) uint16_t s_v[2][kTok * D];

  // (sequence, head) pairs go round the XCDs, so that the row tiles of a pair
  // share one L2 and sequences of different lengths spread evenly; the last
  // row tiles (the most visible tokens) start first
  const int pairs = c.batch * c.heads;
  int pair, rt, split;
  {
    int id = blockIdx.x;
    const int per = row_tiles * a.splits;
    const int full = pairs & ~7;
    if (id < full * per) {
      pair = (id / (8 * per)) * 8 + id % 8;
      id = (id / 8) % per;
    } else {
      id -= full * per;
      const int left = pairs - full;
      pair = full + id % left;
      id /= left;
    }
    split = id % a.splits;
    rt = row_tiles - 1 - id / a.splits;
  }
  const int h = pair % c.heads, b = pair / c.heads;

  const Seq s = sequence(c, b);
  const int rows = s.n * a.group, row0 = rt * BM;
  if (row0 >= rows) return;
  const int begin = split * a.chunk;
  if (split > 0 && begin >= s.len) return;           // the join knows this from the length
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, r = lane & 31;
  const int last_row = min(row0 + BM - 1, rows - 1);
  const int seen_all = a.full ? s.len : min(s.len, s.base + last_row / a.group + 1);
  const int end = min(begin + a.chunk, seen_all);
  const int steps = end > begin ? (end - begin + kTok - 1) / kTok : 0;

  const int wrow0 = row0 + 32 * wave;
  const int row = min(wrow0 + r, rows - 1);          // rows past the end repeat the last one, not written
  const int tok = row / a.group, hq = h * a.group + row % a.group;
  const int seen = min(a.full ? s.len : min(s.len, s.base + tok + 1), end);
  // every row of the wave sees the tokens below this
  const int wave_seen = min(a.full ? s.len : min(s.len, s.base + min(wrow0, rows - 1) / a.group + 1), end);

  // a negative scale is moved into Q: the maximum of raw scores is then the
  // maximum of the scaled ones
  v8bf qf[KS];
  {
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)(s.row0 + tok) * a.ld_q + (int64_t)hq * D + half * 8;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint4 w = *reinterpret_cast<const uint4*>(q + 16 * k);
      w.x ^= flip; w.y ^= flip; w.z ^= flip; w.w ^= flip;
      qf[k] = __builtin_bit_cast(v8bf, w);
    }
  }
  const float fscale = __builtin_fabsf(a.scale);
  const float inv_cap = 1.0f / a.softcap;

  const int64_t page_bytes = ((int64_t)D) << c.lg_page;
  const int mask = (1 << c.lg_page) - 1;
  const int32_t* table = c.table + (int64_t)b * c.width;

  // Pages of a step's four 16-token groups: lane x holds group x % 4's, or -1
  // (absent, or past the end).  Looked up three steps ahead; group g's page
  // reaches the scalar unit by readlane.
  const int my_group = 16 * (lane & 3);
  auto lookup = [&](int t) { return table[min(t + my_group, s.len - 1) >> c.lg_page]; };
  auto check = [&](int raw, int t) {
    return t + my_group < s.len && (uint32_t)raw < (uint64_t)c.pages ? raw : -1;
  };
  const int64_t page_stride = page_bytes * c.heads;
  const uint8_t* const kpool = c.k + h * page_bytes;
  const uint8_t* const vpool = c.v + h * page_bytes;
  auto base_of = [&](const uint8_t* pool, int pages, int g) {
    return pool + max(__builtin_amdgcn_readlane(pages, g), 0) * page_stride;
  };

  // Staging: an absent group reads page 0 and is masked like one past the end.
  uint2 kraw[KP];
  uint32_t vraw[VP][4];
  auto load_k = [&](int pages, int t) {
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      const int piece = i * T + tid, kt = piece / (D / 8);
      const uint8_t* src = base_of(kpool, pages, __builtin_amdgcn_readfirstlane(kt >> 4)) + (t & mask) * D;
      kraw[i] = *reinterpret_cast<const uint2*>(src + (uint32_t)((kt & mask) * D + (piece % (D / 8)) * 8));
    }
  };
  auto load_v = [&](int pages, int t) {
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int grp = i * T + tid, t4 = grp / (D / 4) * 4;
      if (VG % T != 0 && grp >= VG) break;
      const uint8_t* src = base_of(vpool, pages, __builtin_amdgcn_readfirstlane(t4 >> 4)) + (t & mask) * D;
      const uint32_t at = (uint32_t)((t4 & mask) * D + (grp % (D / 4)) * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) vraw[i][j] = *reinterpret_cast<const uint32_t*>(src + (at + j * D));
    }
  };
  auto store_k = [&](int buf, int i) {
    const int piece = i * T + tid;
    v8bf f;
    unpack4(f, 0, kraw[i].x);
    unpack4(f, 4, kraw[i].y);
    *reinterpret_cast<v8bf*>(&s_k[buf][k_at<D>(piece / (D / 8), piece % (D / 8))]) = f;
  };
  // Values of some steps: tokens that are absent or past the end become zeros
  // (their rows may hold anything).
  auto clear_v = [&](int pages, int t) {
    if (t + kTok <= s.len && !any_lane(pages < 0)) return;
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int t4 = (i * T + tid) / (D / 4) * 4;
      if (VG % T != 0 && i * T + tid >= VG) break;
      const bool there = __builtin_amdgcn_readlane(pages, __builtin_amdgcn_readfirstlane(t4 >> 4)) >= 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) vraw[i][j] = there && t + t4 + j < s.len ? vraw[i][j] : 0u;
    }
  };
  auto store_v = [&](int buf, int i) {
    const int grp = i * T + tid, t4 = grp / (D / 4) * 4, d0 = (grp % (D / 4)) * 4;
    if (VG % T != 0 && grp >= VG) return;
    uint32_t o[4];
    transpose4(vraw[i], o);
    // tokens 16 u + 8 a + 4 half + i sit in chunk 2 u + half at 4 a + i
    const int chunk = 2 * (t4 / 16) + ((t4 >> 2) & 1), sub = ((t4 >> 3) & 1) * 4;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const v2bf lo = codes_to_bf16<false>(o[d]), hi = codes_to_bf16<true>(o[d]);
      uint2 w;
      w.x = __builtin_bit_cast(uint32_t, lo);
      w.y = __builtin_bit_cast(uint32_t, hi);
      *reinterpret_cast<uint2*>(&s_v[buf][v_at(d0 + d, chunk) + sub]) = w;
    }
  };
  // scales of a step's groups, in the lanes of their pages
  struct Scales { float k, v; };
  auto scales_of = [&](int pages) {
    const int64_t at = (int64_t)max(pages, 0) * c.heads + h;
    return Scales{c.ks[at], c.vs[at]};
  };
  auto lane_of = [](float x, int g) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), g));
  };

  constexpr int NS = D / 32;                         // products of a 16-token group, for scores and for outputs
  v16f o[DT], sc[2];                                 // outputs; scores: sc[u / 2][8 (u & 1) + i] is of group u
  v8bf pf[4], pl[4];                                 // weights of group u, times the value scale; (TWO) the second parts
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = v16f{};
  float m = -INFINITY, l = 0.0f;

  auto key = [&](int buf, int j) {                   // operand of score product j: token tile j / KS
    return *reinterpret_cast<const v8bf*>(&s_k[buf][k_at<D>(32 * (j / KS) + r, 2 * (j % KS) + half)]);
  };
  auto value = [&](int buf, int j) {                 // operand of output product j: group j / NS
    return *reinterpret_cast<const v8bf*>(&s_v[buf][v_at(32 * (j % NS) + r, 2 * (j / NS) + half)]);
  };
  constexpr int kAhead = 4;                          // LDS reads run this many products ahead
  auto add_outputs = [&](int buf) {
    v8bf ring[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) ring[j] = value(buf, j);
#pragma unroll
    for (int j = 0; j < 4 * NS; ++j) {
      o[j % NS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[j % kAhead], pf[j / NS], o[j % NS], 0, 0, 0);
      if (TWO) o[j % NS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[j % kAhead], pl[j / NS], o[j % NS], 0, 0, 0);
      if (j + kAhead < 4 * NS) ring[j % kAhead] = value(buf, j + kAhead);
    }
  };

  // Matrix phase: the scores of step t, then (not FIRST, which TWO always is) the
  // outputs of step t - 1, as one stream of products.  The sum so far is rescaled beside the
  // score products, every step: the vector unit is idle there, and no branch
  // surrounds the accumulators.  g0, g1, g2: pages of steps t, t + 1, t + 2.
  auto matrix = [&](auto first, int t, int it, int g0, int g1, int g2) {
    constexpr bool FIRST = decltype(first)::value != 0;
    constexpr int ALL = FIRST ? 4 * NS : 8 * NS;
    const int kb = it & 1, vb = kb ^ 1;              // keys t, values t - 1; keys t + 1 go to kb ^ 1, values t to kb
    auto operand = [&](int j) { return j < 4 * NS ? key(kb, j) : value(vb, j - 4 * NS); };
    __builtin_amdgcn_s_setprio(1);                   // ahead of the other wave's softmax: 504 -> 464 us on long prompts
    v8bf ring[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) ring[j] = operand(j);
    clear_v(g0, t);
#pragma unroll
    for (int j = 0; j < ALL; ++j) {
      if (j < 4 * NS) {
        const v16f zero = {};
        sc[j / KS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[j % kAhead], qf[j % KS], j % KS ? sc[j / KS] : zero, 0, 0, 0);
      } else {
        const int i = j - 4 * NS;
        o[i % NS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[j % kAhead], pf[i / NS], o[i % NS], 0, 0, 0);
      }
      if (j + kAhead < ALL) ring[j % kAhead] = operand(j + kAhead);
      // the staging, a piece every few products
      constexpr int kEvery = ALL / (KP + VP + 2);
      if (j % kEvery == kEvery - 1) {
        const int piece = j / kEvery;
        if (piece < VP) store_v(kb, piece);
        else if (piece < VP + KP) store_k(kb ^ 1, piece - VP);
        else if (piece == VP + KP) load_v(g1, t + kTok);
        else if (piece == VP + KP + 1) load_k(g2, t + 2 * kTok);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
  };

  // Softmax phase of step t.  `general`: some weights are masked, or some
  // capped scores are past the series; those steps form their scores twice
  // (maximum, weights), so that the common path keeps sc where the matrix core
  // left it.
  auto softmax = [&](int t, int g0, const Scales& sl) {
    float f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) f[u] = lane_of(sl.k * (fscale * (CAP ? 1.0f : kLog2e)), u);
    // an absent group's weights are 0, page 0's scale may be anything
    const float vscale = g0 >= 0 ? sl.v : 0.0f;
    // The common path takes the value scale into the exponent and out of the sum
    // again, once per group instead of once per weight; scales near the ends of
    // the FP32 range (zero among them) go the general way.
    const float vlog = __builtin_amdgcn_logf(vscale), vinv = __builtin_amdgcn_rcpf(vscale);
    bool general = t + kTok > wave_seen || any_lane(!(vscale >= 0x1p-60f && vscale <= 0x1p60f));
    auto masked = [&](int u, int i) {
      const int at = t + 16 * u + 8 * (i / 4) + 4 * half + (i & 3);
      float x = sc[u / 2][8 * (u & 1) + i] * f[u];
      if (CAP) x = capped(x, a.softcap, inv_cap) * kLog2e;
      return __builtin_amdgcn_readlane(g0, u) >= 0 && at < seen ? x : -INFINITY;
    };
    float top = -INFINITY;
    bool tiny = false;                               // all capped scores are within three terms of the series
    if (!general) {
      float low = INFINITY;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float x = sc[u / 2][8 * (u & 1)], y = x;
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          x = fmaxf(x, sc[u / 2][8 * (u & 1) + i]);
          if (CAP) y = fminf(y, sc[u / 2][8 * (u & 1) + i]);
        }
        top = fmaxf(top, x * f[u]);
        if (CAP) low = fminf(low, y * f[u]);
      }
      if (CAP) {
        const float big = fmaxf(top, -low) * inv_cap;
        general = any_lane(!(big < kCapSmall));
        tiny = !any_lane(!(big < kCapTiny));
        top *= kLog2e * tanh_ratio<5>(top * inv_cap);      // the cap keeps the order
      }
    }
    if (general) {
      top = -INFINITY;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, masked(u, i));
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    // The reference moves only when a weight would pass 2^8: the weights keep
    // their relative accuracy in BF16, and the sums theirs in FP32.
    if (any_lane(top > m + 8.0f)) {
      const float m2 = fmaxf(m, top);
      const float alpha = __builtin_amdgcn_exp2f(m - (m2 == -INFINITY ? 0.0f : m2));
      m = m2;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    auto weigh = [&](auto how) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        constexpr bool kGeneral = decltype(how)::value == 0;
        float sum = 0.0f;
        const float vs = lane_of(kGeneral ? vscale : vinv, u);
        const float to = kGeneral ? ref : ref - lane_of(vlog, u);
        const float fl = f[u] * kLog2e, fi = f[u] * inv_cap;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = sc[u / 2][8 * (u & 1) + e];
          float y;
          if (kGeneral) y = masked(u, e) - to;
          else if (CAP) y = __builtin_fmaf(x * fl, tanh_ratio<decltype(how)::value>(x * fi), -to);
          else y = __builtin_fmaf(x, f[u], -to);
          const float p = __builtin_amdgcn_exp2f(y);
          sum += p;
          const float w = kGeneral ? p * vs : p;
          pf[u][e] = (__bf16)w;
          if (TWO) pl[u][e] = (__bf16)(w - (float)pf[u][e]);
        }
        l = kGeneral ? l + sum : __builtin_fmaf(sum, vs, l);
        asm volatile("" : "+v"(l));                  // the sum stays here: sunk below, it would hold every weight
      }
    };
    if (general) weigh(Int<0>{});
    else if (CAP && !tiny) weigh(Int<5>{});
    else weigh(Int<3>{});
  };

  if (steps > 0) {
    const int group = WAVES == 8 ? wave / 4 : 0;     // the two waves of a SIMD
    int g0 = check(lookup(begin), begin), g1 = check(lookup(begin + kTok), begin + kTok);
    int g2 = check(lookup(begin + 2 * kTok), begin + 2 * kTok);
    load_k(g0, begin);
#pragma unroll
    for (int i = 0; i < KP; ++i) store_k(0, i);
    load_v(g0, begin);
    load_k(g1, begin + kTok);
    __syncthreads();
    Scales sl = scales_of(g0);
    int raw = lookup(begin + 3 * kTok);
    matrix(Int<1>{}, begin, 0, g0, g1, g2);
    int t = begin;
    for (int it = 1; it < steps; ++it, t += kTok) {
      // one barrier a step and wave, between its group's phases
      if (group == 1) __syncthreads();
      softmax(t, g0, sl);
      if (group == 0) __syncthreads();
      if (TWO) add_outputs((it - 1) & 1);
      g0 = g1;
      g1 = g2;
      g2 = check(raw, t + 3 * kTok);
      sl = scales_of(g0);
      raw = lookup(t + 4 * kTok);
      matrix(Int<TWO>{}, t + kTok, it, g0, g1, g2);
    }
    if (group == 1) __syncthreads();
    softmax(t, g0, sl);
    if (group == 0) __syncthreads();
    add_outputs((steps - 1) & 1);
  }
  l += __shfl_xor(l, 32);

  if (wrow0 + r >= rows) return;
  const int64_t at = (int64_t)(s.row0 + tok) * a.q_heads + hq;
  // o[d][4 a + i] is dim 32 d + 8 a + 4 half + i
  if (a.splits > 1) {
    float* part = a.part + ((int64_t)split * c.rows * a.q_heads + at) * D + 4 * half;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<v4f*>(part + 32 * d + 8 * i) = v4f{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
    if (half == 0) a.stat[(int64_t)split * c.rows * a.q_heads + at] = make_float2(m, l);
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y0 = o[d][4 * i] * inv, y1 = o[d][4 * i + 1] * inv, y2 = o[d][4 * i + 2] * inv, y3 = o[d][4 * i + 3] * inv;
      const int64_t e = at * D + 32 * d + 8 * i + 4 * half;
      if (a.out_f32) *reinterpret_cast<v4f*>(static_cast<float*>(a.out) + e) = v4f{y0, y1, y2, y3};
      else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + e) = make_uint2(pack2_bf16(y0, y1), pack2_bf16(y2, y3));
    }
  if (a.lse && half == 0) a.lse[at] = l == 0.0f ? -INFINITY : (m + __builtin_log2f(l)) * kLn2;
}

template <int D, bool CAP, bool TWO>
void launch(const AttendArgs& a, int row_tiles, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.c.batch * a.c.heads * row_tiles * a.splits));
  if constexpr (D == 128) {
    if (a.tile_rows == 256) {
      k_attend_tiles<D, CAP, 8, TWO><<<grid, 512, 0, stream>>>(a, row_tiles);
      return;
    }
  }
  k_attend_tiles<D, CAP, 4, TWO><<<grid, 256, 0, stream>>>(a, row_tiles);
}

template <int D, bool CAP>
void launch(const AttendArgs& a, int row_tiles, hipStream_t stream) {
  if (a.out_f32) launch<D, CAP, true>(a, row_tiles, stream);
  else launch<D, CAP, false>(a, row_tiles, stream);
}

}  // namespace

hipError_t launch_attend_tiles(const AttendArgs& a, int row_tiles, hipStream_t stream) {
  const bool cap = a.softcap > 0.0f;
  if (a.c.dim == 128) {
    if (cap) launch<128, true>(a, row_tiles, stream);
    else launch<128, false>(a, row_tiles, stream);
  } else {
    if (cap) launch<64, true>(a, row_tiles, stream);
    else launch<64, false>(a, row_tiles, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8bs
