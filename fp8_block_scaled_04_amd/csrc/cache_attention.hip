// Attention over the paged FP8 cache (include/fp8bs_cache.h,
// fp8bs_cache_attention).
//
// k_attend_rows: one workgroup per (sequence, head, 16 rows, split of the
// cached tokens).  A row is one (new token, query head of the group) pair, so
// the group's heads share every key and value read.  Each wave walks its own
// 32-token steps with a running maximum and sum per row; the four waves meet
// in LDS at the end, the splits in k_attend_join.
//
// Products are formed transposed, S^T = K Q^T and O^T = V^T P^T: the matrix
// core's result layout of S^T (lane = row, four consecutive tokens per lane)
// is then its operand layout of P^T, if the 32 tokens of a step are numbered
// 16 x tile + 4 x lane group + i, and no value moves between lanes.
//
// HBM bound: 2 D bytes of codes per cached token and head against 4 D flops
// per row.  Two waves' worth of steps in flight per wave and three workgroups
// per CU keep the reads coming: 446 MB of a 48-sequence step in 101 us, 444 MB
// of two 131,000-token contexts in 89 us (4.4 and 5.0 TB/s; a plain read of
// that size reaches 5.5).  Splits are joined by a kernel of its own (5 us).
#include "cache_device.h"

namespace fp8bs {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, kStep = 32;
constexpr int kMaxSplits = 64;                       // (with fewer than 12 pairs the chip is then not full)

template <int D, bool CAP>
__global__ __launch_bounds__(kThreads) void k_attend_rows(AttendArgs a, int row_tiles) {
  const CacheArgs& c = a.c;
  constexpr int DT = D / 16;                         // dims per lane of V, output tiles
  constexpr int KS = D / 32;                         // matrix steps of a score
  // several row tiles of a split run on one XCD, whose L2 then holds its codes
  int id = row_tiles > 1 ? xcd_remap(blockIdx.x, gridDim.x) : blockIdx.x;
  const int rt = id % row_tiles;
  id /= row_tiles;
  const int split = id % a.splits;
  id /= a.splits;
  const int h = id % c.heads, b = id / c.heads;
  const int begin = split * a.chunk;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Pages of this wave's steps: lane x holds that of 16-token group x % 2 of
  // step x / 2, 32 steps at a time.  The table is read before the lengths are
  // known (inside its row), so that one memory latency covers both.
  const int first = begin + wave * kStep;
  auto group_at = [&](int step) { return first + (step + lane / 2) * (kWaves * kStep) + (lane & 1) * 16; };
  auto entry = [&](int step) { return c.table[(int64_t)b * c.width + min(group_at(step) >> c.lg_page, c.width - 1)]; };
  int ahead = entry(0);

  const Seq s = sequence(c, b);
  const int rows = s.n * a.group, row0 = rt * 16;
  if (row0 >= rows) return;
  if (split > 0 && begin >= s.len) return;           // the join knows this from the length
  const int g = lane >> 4, r = lane & 15;
  const int last_row = min(row0 + 15, rows - 1);
  const int seen_all = a.full ? s.len : min(s.len, s.base + last_row / a.group + 1);
  const int end = min(begin + a.chunk, seen_all);

  // this lane's row (clamped: rows past the end repeat the last one and are
  // not written)
  const int row = min(row0 + r, rows - 1);
  const int tok = row / a.group, hq = h * a.group + row % a.group;
  const int seen = a.full ? s.len : min(s.len, s.base + tok + 1);
  const int all_see = a.full ? s.len : min(s.len, s.base + row0 / a.group + 1);   // slots every row sees

  v8bf qf[KS];
  {
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)(s.row0 + tok) * a.ld_q + (int64_t)hq * D + g * (D / 4);
#pragma unroll
    for (int k = 0; k < KS; ++k) qf[k] = *reinterpret_cast<const v8bf*>(q + 8 * k);
  }

  const float inv_cap = 1.0f / a.softcap;
  v4f o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;
  const int64_t page_bytes = ((int64_t)D) << c.lg_page;
  const int64_t page_stride = page_bytes * c.heads;
  const int mask = (1 << c.lg_page) - 1;
  const uint8_t* const kpool = c.k + h * page_bytes;
  const uint8_t* const vpool = c.v + h * page_bytes;

  int pg = -1;
  float ksc = 0.0f, vsc = 0.0f;
  auto lookup = [&](int step) {
    pg = group_at(step) < s.len && (uint32_t)ahead < (uint64_t)c.pages ? ahead : -1;
    const int64_t at = (int64_t)max(pg, 0) * c.heads + h;
    const float k = c.ks[at], v = c.vs[at];
    ksc = k * a.scale;                               // an absent group's scores are masked
    vsc = pg >= 0 ? v : 0.0f;
  };
  // Codes of one step.  An absent group reads page 0 and is masked.
  constexpr int KD = D / 16;                         // dwords of a key per lane
  typedef uint32_t Keys __attribute__((ext_vector_type(KD)));
  typedef uint32_t Vals __attribute__((ext_vector_type(DT / 4)));
  struct Raw {
    Keys k[2];
    Vals v[2][4];
  };
  const uint32_t k_off = (uint32_t)(r * D + g * (D / 4)), v_off = (uint32_t)(4 * g * D + r * DT);
  auto load = [&](Raw& x, int step, int t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t page = max(__builtin_amdgcn_readlane(pg, 2 * step + i), 0);
      const int row0 = (t + 16 * i) & mask;
      const uint8_t* kp = kpool + page * page_stride + row0 * D;
      const uint8_t* vp = vpool + page * page_stride + row0 * D;
      x.k[i] = *reinterpret_cast<const Keys*>(kp + k_off);
#pragma unroll
      for (int j = 0; j < 4; ++j) x.v[i][j] = *reinterpret_cast<const Vals*>(vp + (v_off + j * D));
    }
  };
  auto use = [&](Raw& y, int step, int t) {
    v4f x[2];
    float vscale[2];
    // all tokens of the step are there and every row sees them?
    const bool plain = t + kStep <= min(all_see, end) && __builtin_amdgcn_readlane(pg, 2 * step) >= 0 &&
                       __builtin_amdgcn_readlane(pg, 2 * step + 1) >= 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ksc), 2 * step + i));
      vscale[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, vsc), 2 * step + i));
      v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        v8bf kf;
        unpack4(kf, 0, y.k[i][2 * k]);
        unpack4(kf, 4, y.k[i][2 * k + 1]);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[k], acc, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float z = acc[j] * f;
        x[i][j] = (CAP ? capped(z, a.softcap, inv_cap) : z) * kLog2e;
      }
    }
    if (!plain) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool there = __builtin_amdgcn_readlane(pg, 2 * step + i) >= 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = t + 16 * i + 4 * g + j;
          x[i][j] = there && at < min(seen, end) ? x[i][j] : -INFINITY;
          const bool in = there && at < s.len;       // rows past the cached tokens hold anything
#pragma unroll
          for (int e = 0; e < DT / 4; ++e) y.v[i][j][e] = in ? y.v[i][j][e] : 0u;
        }
      }
    }
    float top = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                      fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float m2 = fmaxf(m, top);
    const float ref = m2 == -INFINITY ? 0.0f : m2;   // nothing seen yet: every weight is 0
    const float alpha = __builtin_amdgcn_exp2f(m - ref);
    m = m2;
    l *= alpha;
    // The weight meets the codes as two BF16 parts (2^-17 of it is lost): the
    // matrix core has time to spare here, and few rows leave no other error to
    // hide a single rounding behind.
    v8bf pf, pl;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = __builtin_amdgcn_exp2f(x[i][j] - ref);
        l += p;
        const float w = p * vscale[i];
        pf[4 * i + j] = (__bf16)w;
        pl[4 * i + j] = (__bf16)(w - (float)pf[4 * i + j]);
      }
#pragma unroll
    for (int e = 0; e < DT / 4; ++e) {
      uint32_t w[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t in[4] = {y.v[i][0][e], y.v[i][1][e], y.v[i][2][e], y.v[i][3][e]};
        transpose4(in, w[i]);
      }
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        v8bf vf;
        unpack4(vf, 0, w[0][d]);
        unpack4(vf, 4, w[1][d]);
        v4f& acc = o[4 * e + d];
        acc *= alpha;
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pl, acc, 0, 0, 0);
      }
    }
  };

  const int steps = first < end ? (end - first + kWaves * kStep - 1) / (kWaves * kStep) : 0;
  for (int s0 = 0; s0 < steps; s0 += 32) {
    if (s0 > 0) ahead = entry(s0);
    lookup(s0);
    const int n = min(32, steps - s0);
    const int t0 = first + s0 * (kWaves * kStep);
    // two sets of codes, the other one in flight (past the last step its codes
    // are asked for again: no branch around the loads)
    auto ask = [&](Raw& x, int i) {
      i = min(i, n - 1);
      load(x, i, t0 + i * (kWaves * kStep));
    };
    Raw even, odd;
    ask(even, 0);
    for (int i = 0; i < n; i += 2) {
      ask(odd, i + 1);
      use(even, i, t0 + i * (kWaves * kStep));
      ask(even, i + 2);
      if (i + 1 < n) use(odd, i + 1, t0 + (i + 1) * (kWaves * kStep));
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // the waves' maxima, sums and outputs meet in LDS; o[d][j] is dim
  // DT (4 g + j) + d of row r
  constexpr int kPitch = D + 4;
  __shared__ float s_o[kWaves][16][kPitch];
  __shared__ float2 s_ml[kWaves][16];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int d = 0; d < DT; d += 4)
      *reinterpret_cast<v4f*>(&s_o[wave][r][DT * (4 * g + j) + d]) = v4f{o[d][j], o[d + 1][j], o[d + 2][j], o[d + 3][j]};
  if (g == 0) s_ml[wave][r] = make_float2(m, l);
  __syncthreads();

  const int orow = tid / 16, d0 = (tid % 16) * DT;   // 16 threads per row, DT dims each
  if (row0 + orow >= rows) return;
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_ml[w][orow].x);
  const float ref = top == -INFINITY ? 0.0f : top;
  float total = 0.0f, y[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) y[d] = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float f = __builtin_amdgcn_exp2f(s_ml[w][orow].x - ref);
    total += f * s_ml[w][orow].y;
#pragma unroll
    for (int d = 0; d < DT; ++d) y[d] += f * s_o[w][orow][d0 + d];
  }
  const int otok = (row0 + orow) / a.group, ohq = h * a.group + (row0 + orow) % a.group;
  const int64_t at = (int64_t)(s.row0 + otok) * a.q_heads + ohq;
  if (a.splits > 1) {
    float* part = a.part + ((int64_t)split * c.rows * a.q_heads + at) * D + d0;
#pragma unroll
    for (int d = 0; d < DT; d += 4) *reinterpret_cast<v4f*>(part + d) = v4f{y[d], y[d + 1], y[d + 2], y[d + 3]};
    if (d0 == 0) a.stat[(int64_t)split * c.rows * a.q_heads + at] = make_float2(top, total);
    return;
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  if (a.out_f32) {
    float* out = static_cast<float*>(a.out) + at * D + d0;
#pragma unroll
    for (int d = 0; d < DT; d += 4)
      *reinterpret_cast<v4f*>(out + d) = v4f{y[d] * inv, y[d + 1] * inv, y[d + 2] * inv, y[d + 3] * inv};
  } else {
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at * D + d0);
#pragma unroll
    for (int d = 0; d < DT; d += 2) out[d / 2] = pack2_bf16(y[d] * inv, y[d + 1] * inv);
  }
  if (a.lse && d0 == 0) a.lse[at] = total == 0.0f ? -INFINITY : (top + __builtin_log2f(total)) * kLn2;
}

// Joins the splits: D / 4 lanes per (row, query head), four dims each.
template <int D>
__global__ __launch_bounds__(kThreads) void k_attend_join(AttendArgs a) {
  const CacheArgs& c = a.c;
  constexpr int L = D / 4, kRowsPerGroup = kThreads / L;
  const int64_t id = (int64_t)blockIdx.x * kRowsPerGroup + threadIdx.x / L;
  const int lane = threadIdx.x % L;
  const int hq = (int)(id % a.q_heads);
  const int64_t rest = id / a.q_heads;
  const int tok = (int)(rest % c.max_new), b = (int)(rest / c.max_new);
  if (b >= c.batch) return;
  const int lo = c.q_offsets[b], hi = c.q_offsets[b + 1];
  if (lo < 0 || hi < lo || hi > c.rows || tok >= hi - lo) return;
  const int64_t room = (int64_t)c.width << c.lg_page;
  const int len = (int)max((int64_t)0, min((int64_t)min(c.kv_lens[b], c.max_kv), room));
  const int parts = max(1, min(a.splits, (len + a.chunk - 1) / a.chunk));
  const int64_t at = (int64_t)(lo + tok) * a.q_heads + hq, stride = c.rows * a.q_heads;

  float top = -INFINITY;
  for (int p = lane; p < parts; p += L) top = fmaxf(top, a.stat[p * stride + at].x);
#pragma unroll
  for (int x = 1; x < L; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
  const float ref = top == -INFINITY ? 0.0f : top;
  float total = 0.0f;
  v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float2 st = a.stat[p * stride + at];
    const v4f part = *reinterpret_cast<const v4f*>(a.part + (p * stride + at) * D + 4 * lane);
    const float w = __builtin_amdgcn_exp2f(st.x - ref);
    total += w * st.y;
    y += w * part;
  }
  y *= total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t e = at * D + 4 * lane;
  if (a.out_f32) *reinterpret_cast<v4f*>(static_cast<float*>(a.out) + e) = y;
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + e) = make_uint2(pack2_bf16(y[0], y[1]), pack2_bf16(y[2], y[3]));
  if (a.lse && lane == 0) a.lse[at] = total == 0.0f ? -INFINITY : (top + __builtin_log2f(total)) * kLn2;
}

int row_tiles(const AttendArgs& a, int64_t new_tokens) {
  return (int)((new_tokens * a.group + a.tile_rows - 1) / a.tile_rows);
}

// max_new may be far above what the call's rows allow a sequence.
int launched_row_tiles(const AttendArgs& a) { return row_tiles(a, std::min<int64_t>(a.c.max_new, a.c.rows)); }

template <int D>
hipError_t launch(const AttendArgs& a, hipStream_t stream) {
  const int tiles = launched_row_tiles(a);
  const dim3 grid((unsigned)((int64_t)a.c.batch * a.c.heads * tiles * a.splits));
  if (a.tile_rows > 16) {
    if (hipError_t e = launch_attend_tiles(a, tiles, stream)) return e;
  } else if (a.softcap > 0.0f) k_attend_rows<D, true><<<grid, kThreads, 0, stream>>>(a, tiles);
  else k_attend_rows<D, false><<<grid, kThreads, 0, stream>>>(a, tiles);
  if (hipError_t e = hipGetLastError()) return e;
  if (a.splits == 1) return hipSuccess;
  const int64_t rows = (int64_t)a.c.batch * a.c.max_new * a.q_heads;
  constexpr int per = kThreads / (D / 4);
  k_attend_join<D><<<dim3((unsigned)((rows + per - 1) / per)), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

void attend_plan(AttendArgs& a) {
  const int64_t rows = (int64_t)a.c.max_new * a.group, pairs = (int64_t)a.c.batch * a.c.heads;
  // 16-row tiles read the codes once per 16 rows and bring the most workgroups;
  // the larger ones convert them once per tile.  Measured at 4096 cached
  // tokens, 8 heads: 64 rows of D = 128 in 86 us (16) or 63 us (128) for 16
  // sequences, 16 or 20 us for one; 256 rows 111 (128) or 104 us (256); 128
  // rows of D = 64 83 (16) or 64 us (128).
  // Little work in all stays on 16-row tiles, which fill the chip sooner and
  // round the weights to 2^-17 (the larger ones' single BF16 rounding for BF16
  // outputs puts them at 1.45 times the error of exact weights, over a few dozen
  // tokens at up to 1.67).  16 against larger, (row, head)
  // pairs / cached tokens, D = 128: 4096/128 in 6 or 13 us, 4096/1024 20 or 24,
  // 8192/256 20 or 17, 1024/32768 63 or 40; D = 64: 16384/512 11 or 20,
  // 8192/4096 37 or 44, 32768/1024 25 or 42, 65536/128 21 or 13, 1024/131072 125
  // or 93.
  const int64_t all = a.c.rows * a.q_heads, few = a.c.dim == 64 ? 1 << 15 : 1 << 12;
  if (all <= few && all * a.c.max_kv <= few * (a.c.dim == 64 ? 1024 : 2048)) a.tile_rows = 16;
  else if (a.c.dim == 64) a.tile_rows = rows <= 64 ? 16 : 128;
  else a.tile_rows = rows <= 32 || (rows <= 64 && pairs < 64) ? 16 : rows <= 128 ? 128 : 256;
  const int unit = a.tile_rows == 16 ? kWaves * kStep : 256;
  // Workgroups: what runs at once (three of 16 rows per CU), or twice that where
  // the causal rule leaves them unequal (one of 256 rows per CU, two
  // of 128).
  const int64_t target = a.tile_rows == 256 ? 512 : a.tile_rows == 128 ? 1024 : 768;
  const int64_t base = pairs * row_tiles(a, a.c.max_new);
  const int64_t units = ((int64_t)a.c.max_kv + unit - 1) / unit;
  int64_t want = base > 0 ? (target + base - 1) / base : 1;
  if (want > kMaxSplits) want = kMaxSplits;
  if (want > units) want = units;
  if (want < 1) want = 1;
  const int64_t per = units > 0 ? (units + want - 1) / want : 1;
  a.chunk = (int32_t)(per * unit);
  a.splits = units > 0 ? (int32_t)((units + per - 1) / per) : 1;
}

int64_t attend_workspace_bytes(const AttendArgs& a) {
  return a.splits > 1 ? (int64_t)a.splits * a.c.rows * a.q_heads * (a.c.dim + 2) * 4 : 0;
}

int64_t attend_items(const AttendArgs& a) {
  const int64_t tiles = (int64_t)a.c.heads * launched_row_tiles(a) * a.splits * (a.tile_rows == 256 ? 512 : kThreads);
  const int64_t join = a.splits > 1 ? (int64_t)a.c.max_new * a.q_heads * (a.c.dim / 4) + kThreads : 0;
  return std::max(tiles, join);
}

hipError_t launch_cache_attention(const AttendArgs& a, hipStream_t stream) {
  return launch_in_runs(a, attend_items(a), [&](const AttendArgs& run) {
    return run.c.dim == 128 ? launch<128>(run, stream) : launch<64>(run, stream);
  });
}

}  // namespace fp8bs
