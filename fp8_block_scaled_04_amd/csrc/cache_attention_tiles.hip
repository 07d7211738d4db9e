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
// Software pipeline: scores of step t + 1 (matrix core) are formed beside the
// softmax of step t (vector unit), so keys are staged two steps ahead, values
// one.  One barrier per step.
#include "cache_device.h"

namespace fp8bs {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kTok = 64;                             // tokens per step

template <int N>
struct Int {
  static constexpr int value = N;
};

// Keys: row = token, 16-byte chunks of 8 dims.  A wave's reads take one chunk
// of 32 rows, its writes whole rows: chunk ^ row spreads both over the banks.
template <int D>
__device__ __forceinline__ int k_at(int tok, int chunk) {
  return tok * D + ((chunk ^ (tok & (D / 8 - 1) & 15)) * 8);
}

// Values: row = dim, 16-byte chunks of 8 tokens.  Reads take one chunk of 32
// rows, writes half a chunk of every fourth row.
__device__ __forceinline__ int v_at(int dim, int chunk) {
  return dim * kTok + ((chunk ^ ((dim ^ (dim >> 2)) & 7)) * 8);
}

template <int D, bool CAP, int WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(2, 2)))
void k_attend_tiles(AttendArgs a, int row_tiles) {
  const CacheArgs& c = a.c;
  constexpr int T = 64 * WAVES, BM = 32 * WAVES;
  constexpr int KS = D / 16;                         // matrix steps of a score
  constexpr int DT = D / 32;                         // 32-dim tiles of the output
  constexpr int KP = kTok * (D / 8) / T;             // 8-byte key pieces per thread
  constexpr int VG = (kTok / 4) * (D / 4);           // 4 x 4 groups of values
  constexpr int VP = (VG + T - 1) / T;               // per thread
  __shared__ __attribute__((aligned(16))) uint16_t s_k[2][kTok * D];
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

  // Pages of a step's four 16-token groups (wave-uniform; -1: absent or past
  // the end), looked up three steps ahead.
  struct Pages { int p[4]; };
  auto lookup = [&](int t) {
    Pages g;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int tt = t + 16 * u;
      const int p = uniform_load(table + (min(tt, s.len - 1) >> c.lg_page));
      g.p[u] = (tt < s.len && (uint32_t)p < (uint64_t)c.pages) ? p : -1;
    }
    return g;
  };
  auto pick = [](const Pages& g, int u) { return u == 0 ? g.p[0] : u == 1 ? g.p[1] : u == 2 ? g.p[2] : g.p[3]; };
  auto base_of = [&](const uint8_t* pool, int p) { return pool + ((int64_t)max(p, 0) * c.heads + h) * page_bytes; };

  // Staging: an absent group reads page 0 and is masked like one past the end.
  uint2 kraw[KP];
  uint32_t vraw[VP][4];
  auto load_k = [&](const Pages& g, int t) {
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      const int piece = i * T + tid, kt = piece / (D / 8);
      const uint8_t* src = base_of(c.k, pick(g, __builtin_amdgcn_readfirstlane(kt >> 4))) + (t & mask) * D;
      kraw[i] = *reinterpret_cast<const uint2*>(src + (uint32_t)((kt & mask) * D + (piece % (D / 8)) * 8));
    }
  };
  auto store_k = [&](int buf) {
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      const int piece = i * T + tid;
      v8bf f;
      unpack4(f, 0, kraw[i].x);
      unpack4(f, 4, kraw[i].y);
      *reinterpret_cast<v8bf*>(&s_k[buf][k_at<D>(piece / (D / 8), piece % (D / 8))]) = f;
    }
  };
  auto load_v = [&](const Pages& g, int t) {
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int grp = i * T + tid, t4 = grp / (D / 4) * 4;
      if (VG % T != 0 && grp >= VG) break;
      const uint8_t* src = base_of(c.v, pick(g, __builtin_amdgcn_readfirstlane(t4 >> 4))) + (t & mask) * D;
      const uint32_t at = (uint32_t)((t4 & mask) * D + (grp % (D / 4)) * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) vraw[i][j] = *reinterpret_cast<const uint32_t*>(src + (at + j * D));
    }
  };
  // `clear`: some tokens of the step are absent or past the end, and their
  // rows may hold anything
  auto store_v = [&](int buf, const Pages& g, int t, bool clear) {
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int grp = i * T + tid, t4 = grp / (D / 4) * 4, d0 = (grp % (D / 4)) * 4;
      if (VG % T != 0 && grp >= VG) break;
      if (clear) {
        const bool there = pick(g, __builtin_amdgcn_readfirstlane(t4 >> 4)) >= 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) vraw[i][j] = there && t + t4 + j < s.len ? vraw[i][j] : 0u;
      }
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
    }
  };
  struct Scales { float k[4], v[4]; };
  auto scales_of = [&](const Pages& g) {
    Scales x;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t at = (int64_t)max(g.p[u], 0) * c.heads + h;
      x.k[u] = uniform_load(c.ks + at);
      const float v = uniform_load(c.vs + at);
      x.v[u] = g.p[u] >= 0 ? v : 0.0f;               // its weights are 0, page 0's scale may be anything
    }
    return x;
  };
  auto whole = [&](const Pages& g) { return (g.p[0] | g.p[1] | g.p[2] | g.p[3]) >= 0; };

  v16f o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = -INFINITY, l = 0.0f;

  // a quarter of a step's scores: token tile u / 2, half of the dims
  auto score = [&](v16f (&x)[2], int buf, int u) {
    if ((u & 1) == 0)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[u / 2][i] = 0.0f;
#pragma unroll
    for (int k = (u & 1) * (KS / 2); k < ((u & 1) + 1) * (KS / 2); ++k) {
      const v8bf kf = *reinterpret_cast<const v8bf*>(&s_k[buf][k_at<D>(32 * (u / 2) + r, 2 * k + half)]);
      x[u / 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[k], x[u / 2], 0, 0, 0);
    }
  };
  auto outputs = [&](const v8bf& pf, int buf, int u) {
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const v8bf vf = *reinterpret_cast<const v8bf*>(&s_v[buf][v_at(32 * d + r, 2 * u + half)]);
      o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf, o[d], 0, 0, 0);
    }
  };

  // One step: softmax of sc (step t) and the outputs it adds, beside the
  // scores nx of step t + 1.  Buffers: keys t + 1 in PAR ^ 1, values t in PAR.
  // g0, g1, g2: the pages of steps t, t + 1, t + 2.
  auto step = [&](v16f (&sc)[2], v16f (&nx)[2], auto par, int t, const Pages& g0, const Pages& g1, const Pages& g2,
                  const Scales& sl) {
    constexpr int PAR = decltype(par)::value;
    load_k(g2, t + 2 * kTok);
    load_v(g1, t + kTok);
    float f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) f[u] = sl.k[u] * fscale * (CAP ? 1.0f : kLog2e);
    // sc[u / 2][8 (u & 1) + i] belongs to the 16 tokens of group u
    if (CAP) {
      // caps well above the scores need only the series (capped_small)
      float big = 0.0f;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = sc[u / 2][8 * (u & 1) + i] * f[u];
          sc[u / 2][8 * (u & 1) + i] = x;
          big = fmaxf(big, __builtin_fabsf(x));
        }
      if (__any(!(big * inv_cap < kCapSmall))) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[u][i] = capped(sc[u][i], a.softcap, inv_cap) * kLog2e;
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[u][i] = capped_small(sc[u][i] * kLog2e, sc[u][i] * inv_cap);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) f[u] = 1.0f;
    }
    if (t + kTok > wave_seen || !whole(g0)) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = t + 16 * u + 8 * (i / 4) + 4 * half + (i & 3);
          sc[u / 2][8 * (u & 1) + i] = (g0.p[u] >= 0 && at < seen) ? sc[u / 2][8 * (u & 1) + i] * f[u] : -INFINITY;
        }
        f[u] = 1.0f;
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float x = sc[u / 2][8 * (u & 1)];
#pragma unroll
      for (int i = 1; i < 8; ++i) x = fmaxf(x, sc[u / 2][8 * (u & 1) + i]);
      top = fmaxf(top, x * f[u]);
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    // The reference moves only when a weight would pass 2^8: the weights keep
    // their relative accuracy in BF16, and the sums theirs in FP32.
    if (__any(top > m + 8.0f)) {
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
    v8bf pf[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      score(nx, PAR ^ 1, u);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[u / 2][8 * (u & 1) + i], f[u], -ref));
        sum += p;
        pf[u][i] = (__bf16)(p * sl.v[u]);
      }
      l += sum;
      asm volatile("" : "+v"(l));                    // the sum stays here: sunk below, it would hold 32 weights
      if (u > 0) outputs(pf[u - 1], PAR, u - 1);
    }
    outputs(pf[3], PAR, 3);
    store_k(PAR);
    store_v(PAR ^ 1, g1, t + kTok, t + 2 * kTok > s.len || !whole(g1));
    __syncthreads();
  };

  if (steps > 0) {
    v16f sa[2], sb[2];
    Pages g0 = lookup(begin), g1 = lookup(begin + kTok), g2 = lookup(begin + 2 * kTok);
    Scales sl = scales_of(g0);
    load_k(g0, begin);
    load_v(g0, begin);
    store_k(0);
    store_v(0, g0, begin, true);
    load_k(g1, begin + kTok);
    store_k(1);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) score(sa, 0, u);
    __syncthreads();
    for (int t = begin;;) {
      Pages g3 = lookup(t + 3 * kTok);
      Scales sn = scales_of(g1);
      step(sa, sb, Int<0>{}, t, g0, g1, g2, sl);
      t += kTok;
      if (t >= end) break;
      g0 = lookup(t + 3 * kTok);
      sl = scales_of(g2);
      step(sb, sa, Int<1>{}, t, g1, g2, g3, sn);
      t += kTok;
      if (t >= end) break;
      const Pages n1 = g3, n2 = g0;
      g0 = g2;
      g1 = n1;
      g2 = n2;
    }
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

template <int D, bool CAP>
void launch(const AttendArgs& a, int row_tiles, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.c.batch * a.c.heads * row_tiles * a.splits));
  if (a.tile_rows == 256) k_attend_tiles<D, CAP, 8><<<grid, 512, 0, stream>>>(a, row_tiles);
  else k_attend_tiles<D, CAP, 4><<<grid, 256, 0, stream>>>(a, row_tiles);
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
