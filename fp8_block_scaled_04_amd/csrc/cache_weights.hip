// The attention weight each cached token received (include/fp8bs_cache.h,
// fp8bs_cache_attention_weights): acc[j] (+)= sum over rows of exp(x_j - lse).
//
// Scores are formed as S = Q K^T: a lane then holds one token and several rows
// per matrix step, and the sum over rows stays in the lane.  A workgroup owns
// its slots (and its share of the rows): each sum has a fixed order.
//
// k_weights_rows (at most 16 rows, decoding): every key is read once and used
// once, 16x16x32 products.  k_weights_tiles (more rows): 32x32x16 products, 64
// tokens per wave with their keys in registers, Q walked through LDS 64 rows
// at a time.  Under the causal rule the first slots are seen by every row and
// the last ones by few, so the work of a (sequence, head) is cut into equal
// runs of (256-slot tile, 64-row step) pairs, one run per workgroup; the
// partial sums meet in k_weights_join, in order.
//
// k_weights_rows is HBM bound (D bytes of codes per cached token and head): 165
// MB of a 32-sequence step in 43 us, 3.8 TB/s; its workgroups live for one
// round of loads, whose latency the table entries and old sums no longer add
// to (56 us before).  k_weights_tiles takes the matrix core 2 D flops and the
// vector unit a multiply-add, an exponential and an addition per pair: 67
// GFLOP of a 3500-token prompt in 96 us with the join, 700 TFLOP/s; its capped
// form at D = 128 (168 us) spills 18 registers.
//
// Everything is FP32.  k_weights_tiles takes lse to base 2 once per row and keeps
// one running sum per slot over a run's rows, where an exact lse - x and a sum in
// parts would cost the loop another operation or register per score: sums of a
// 3500-token prompt are 2.0e-7 from exact, those of separate FP32 torch
// operations 6.4e-8.
#include "cache_device.h"

namespace fp8bs {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, kTiles = 4;
constexpr int kSlots = kWaves * kTiles * 16;         // per workgroup, both kernels

__device__ __forceinline__ float old_sum(const WeightArgs& a, const Seq& s, int64_t pair, int64_t slot) {
  return a.acc_in && slot < min(s.base, s.len) ? a.acc_in[pair * a.acc_slots + slot] : 0.0f;
}

template <int D, bool CAP>
__global__ __launch_bounds__(kThreads) void k_weights_rows(WeightArgs a, int tiles) {
  const CacheArgs& c = a.c;
  constexpr int KS = D / 32;
  const int tile = blockIdx.x % tiles, pair = blockIdx.x / tiles;
  const int h = pair % c.heads, b = pair / c.heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int64_t slot0 = (int64_t)tile * kSlots + wave * (kTiles * 16);
  if (slot0 >= a.acc_slots) return;
  // the table entries and the old sums are asked for before the lengths are
  // known (inside their rows): one memory latency covers all three
  int entry[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
    entry[i] = c.table[(int64_t)b * c.width + min(((int)slot0 + 16 * i) >> c.lg_page, c.width - 1)];
  const int64_t mine = slot0 + lane;                 // the slot this lane writes
  float old = 0.0f;
  if (a.acc_in && mine < a.acc_slots) old = a.acc_in[(int64_t)pair * a.acc_slots + mine];
  const Seq s = sequence(c, b);
  const int rows = s.n * a.group;
  const float inv_cap = 1.0f / a.softcap;
  float sum[kTiles] = {};
  bool there[kTiles] = {};

  if (slot0 < s.len && rows > 0) {
    const int64_t page_bytes = (int64_t)D << c.lg_page;
    uint2 raw[kTiles][KS];
    float f[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int tt = (int)slot0 + 16 * i;
      there[i] = tt < s.len && (uint32_t)entry[i] < (uint64_t)c.pages;
      const int page = __builtin_amdgcn_readfirstlane(there[i] ? entry[i] : 0);
      const int64_t at = (int64_t)page * c.heads + h;
      f[i] = c.ks[at];
      const uint8_t* kp = c.k + at * page_bytes + (int64_t)((tt & ((1 << c.lg_page) - 1)) + r) * D + g * (D / 4);
#pragma unroll
      for (int k = 0; k < KS; ++k) raw[i][k] = *reinterpret_cast<const uint2*>(kp + 8 * k);
    }
    const int qrow = min(r, rows - 1);
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)(s.row0 + qrow / a.group) * a.ld_q +
                        (int64_t)(h * a.group + qrow % a.group) * D + g * (D / 4);
    v8bf qf[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) qf[k] = *reinterpret_cast<const v8bf*>(q + 8 * k);
    float lse[4];
    int seen[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 4 * g + j, cl = min(row, rows - 1), tok = cl / a.group;
      lse[j] = a.lse[(int64_t)(s.row0 + tok) * a.q_heads + h * a.group + cl % a.group];
      seen[j] = (row < rows && lse[j] != -INFINITY) ? (a.full ? s.len : min(s.len, s.base + tok + 1)) : 0;
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      v4f x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        v8bf kf;
        unpack4(kf, 0, raw[i][k].x);
        unpack4(kf, 4, raw[i][k].y);
        x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[k], kf, x, 0, 0, 0);
      }
      const int slot = (int)slot0 + 16 * i + r;
      const float fs = f[i] * a.scale;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float y = x[j] * fs;
        if (CAP) y = capped(y, a.softcap, inv_cap);
        const float p = __builtin_amdgcn_exp2f((y - lse[j]) * kLog2e);
        sum[i] += slot < seen[j] ? p : 0.0f;
      }
    }
  }
  // lane 16 i + r keeps tile i's slot r
  float x = 0.0f;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    float y = there[i] ? sum[i] : 0.0f;
    y += __shfl_xor(y, 16);
    y += __shfl_xor(y, 32);
    if (g == i) x = y;
  }
  if (mine < a.acc_slots)
    a.acc_out[(int64_t)pair * a.acc_slots + mine] = (mine < min(s.base, s.len) ? old : 0.0f) + x;
}

typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 64;                            // Q rows per step

template <int N>
struct Int {
  static constexpr int value = N;
};

// Steps of tile t: 64 rows each, from the step of the first row that sees any of
// its slots.
struct Steps {
  int first, count;                                  // first row (a multiple of 64), steps
};
__device__ __forceinline__ Steps tile_steps(const WeightArgs& a, const Seq& s, int t) {
  const int rows = s.n * a.group;
  const int hidden = a.full ? 0 : min(s.n, max(0, t * kSlots - s.base)) * a.group;
  Steps x;
  x.first = hidden & ~(kRows - 1);
  x.count = (rows - x.first + kRows - 1) / kRows;    // (rows >= hidden)
  return x;
}

__device__ __forceinline__ int live_tiles(const Seq& s) { return (s.len + kSlots - 1) / kSlots; }

__device__ __forceinline__ int64_t all_steps(const WeightArgs& a, const Seq& s) {
  int64_t n = 0;
  for (int t = 0; t < live_tiles(s); ++t) n += tile_steps(a, s, t).count;
  return n;
}

// Run r of `all` steps cut into a.splits runs begins here.
__device__ __forceinline__ int64_t run_begin(const WeightArgs& a, int64_t all, int r) { return all * r / a.splits; }

// Where run r leaves its sums of tile t: r + t differs between any two of the
// (run, tile) pairs of one (sequence, head) that share work.
__device__ __forceinline__ float* partial(const WeightArgs& a, int tiles, int64_t pair, int r, int t) {
  return a.part + ((pair * (a.splits + tiles)) + r + t) * kSlots;
}

template <int D, bool CAP>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void k_weights_tiles(WeightArgs a, int tiles) {
  const CacheArgs& c = a.c;
  constexpr int KS = D / 16;                         // matrix steps of a score
  constexpr int CH = D / 8;                          // 16-byte chunks of a row
  constexpr int QP = kRows * CH / kThreads;          // per thread and step
  __shared__ __attribute__((aligned(16))) uint16_t s_q[2][kRows * D];
  __shared__ __attribute__((aligned(16))) float s_lse[2][kRows];     // log2 units; +inf: the row adds nothing
  __shared__ __attribute__((aligned(16))) int s_seen[2][kRows];

  // (sequence, head) pairs go round the XCDs, so that a pair's queries stay in
  // one L2
  const int pairs = c.batch * c.heads;
  int pair, run;
  {
    int id = blockIdx.x;
    const int full = pairs & ~7;
    if (id < full * a.splits) {
      pair = (id / (8 * a.splits)) * 8 + id % 8;
      run = (id / 8) % a.splits;
    } else {
      id -= full * a.splits;
      const int left = pairs - full;
      pair = full + id % left;
      run = id / left;
    }
  }
  const int h = pair % c.heads, b = pair / c.heads;
  const Seq s = sequence(c, b);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, r = lane & 31;
  const int rows = s.n * a.group;
  const float fscale = a.scale * (CAP ? 1.0f : kLog2e);
  const float inv_cap = 1.0f / a.softcap;
  const int64_t all = all_steps(a, s), from = run_begin(a, all, run), to = run_begin(a, all, run + 1);

  int64_t before = 0;                                // steps of the tiles so far
  for (int tile = 0; tile < live_tiles(s) && before < to; ++tile) {
    const Steps ts = tile_steps(a, s, tile);
    const int64_t lo = max(from - before, (int64_t)0), hi = min(to - before, (int64_t)ts.count);
    before += ts.count;
    if (lo >= hi) continue;
    const int begin = ts.first + (int)lo * kRows, end = min(rows, ts.first + (int)hi * kRows);
    const int64_t slot0 = (int64_t)tile * kSlots + wave * 64;
    float sum[2] = {0.0f, 0.0f};
    bool there[2] = {false, false};
    // this lane's keys: token slot0 + 32 u + r, dims D / 2 x half + 8 k ..
    v8bf kf[2][KS];
    float f[2];
    int mine[2];
    bool whole = slot0 + 64 <= s.len;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int tt = (int)min(slot0 + 32 * u + r, (int64_t)s.len - 1);
      int page = page_of(c, b, tt);
      there[u] = page >= 0 && slot0 + 32 * u + r < s.len;
      whole = whole && page >= 0;
      page = max(page, 0);
      const int64_t at = (int64_t)page * c.heads + h;
      f[u] = c.ks[at] * fscale;
      mine[u] = there[u] ? tt : 0x7FFFFFFF;
      const uint8_t* kp = c.k + (at << c.lg_page) * D + (int64_t)(tt & ((1 << c.lg_page) - 1)) * D + half * (D / 2);
#pragma unroll
      for (int k = 0; k < KS; k += 2) {
        const uint4 w = *reinterpret_cast<const uint4*>(kp + 8 * k);
        unpack4(kf[u][k], 0, w.x);
        unpack4(kf[u][k], 4, w.y);
        unpack4(kf[u][k + 1], 0, w.z);
        unpack4(kf[u][k + 1], 4, w.w);
      }
    }
    whole = __all(whole);

    // Where this thread's pieces of the next step's rows lie.  Row = token x
    // group + head: 64 rows on is 64 / group tokens and 64 % group heads on,
    // with a carry (no division in the loop).
    struct Place { const uint16_t* p; int g; };
    const int dtok = kRows / a.group, dhead = kRows % a.group;
    const int64_t ahead = (int64_t)dtok * a.ld_q + (int64_t)dhead * D, carry = a.ld_q - (int64_t)a.group * D;
    const uint16_t* qbase = static_cast<const uint16_t*>(a.q) + (int64_t)s.row0 * a.ld_q + (int64_t)h * a.group * D;
    Place at[QP];
#pragma unroll
    for (int i = 0; i < QP; ++i) {
      const int piece = i * kThreads + tid, row = begin + piece / CH, tok = row / a.group;
      at[i].g = row - tok * a.group;
      at[i].p = qbase + (int64_t)tok * a.ld_q + at[i].g * D + (piece % CH) * 8;
    }
    const float* lbase = a.lse + (int64_t)s.row0 * a.q_heads + h * a.group;
    int ltok = (begin + tid) / a.group, lhead = begin + tid - ltok * a.group;   // threads below kRows

    u32x4 qraw[QP];
    float lraw = 0.0f;
    int seen_at = 0;
    auto load = [&](int row0) {
#pragma unroll
      for (int i = 0; i < QP; ++i) {
        // rows past the end read the first one and add nothing
        const uint16_t* p = row0 + (i * kThreads + tid) / CH < rows ? at[i].p : qbase;
        qraw[i] = *reinterpret_cast<const u32x4*>(p);
        at[i].g += dhead;
        const bool over = at[i].g >= a.group;
        at[i].g -= over ? a.group : 0;
        at[i].p += ahead + (over ? carry : 0);
      }
      if (tid < kRows) {
        const bool in = row0 + tid < end;
        lraw = in ? lbase[(int64_t)ltok * a.q_heads + lhead] : -INFINITY;
        seen_at = a.full ? s.len : min(s.len, s.base + ltok + 1);
        lhead += dhead;
        const bool over = lhead >= a.group;
        lhead -= over ? a.group : 0;
        ltok += dtok + (over ? 1 : 0);
      }
    };
    auto store = [&](int buf) {
#pragma unroll
      for (int i = 0; i < QP; ++i) {
        const int piece = i * kThreads + tid, row = piece / CH;
        *reinterpret_cast<u32x4*>(&s_q[buf][row * D + (((piece % CH) ^ (row & (CH - 1))) * 8)]) = qraw[i];
      }
      if (tid < kRows) {
        s_lse[buf][tid] = lraw != -INFINITY ? lraw * kLog2e : INFINITY;
        s_seen[buf][tid] = seen_at;
      }
    };
    // Scores of the step's two 32-row tiles, as one stream of products; LDS
    // reads run kAhead operands (two products each) ahead.
    constexpr int kAhead = 4;
    auto scores = [&](v16f (&x0)[2], v16f (&x1)[2], int buf) {
      auto operand = [&](int j) {
        const int row = 32 * (j / KS) + r, chunk = half * KS + j % KS;
        return *reinterpret_cast<const v8bf*>(&s_q[buf][row * D + ((chunk ^ (row & (CH - 1))) * 8)]);
      };
      v8bf ring[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) ring[j] = operand(j);
#pragma unroll
      for (int j = 0; j < 2 * KS; ++j) {
        v16f(&x)[2] = j < KS ? x0 : x1;
        const v16f zero = {};
#pragma unroll
        for (int u = 0; u < 2; ++u)
          x[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[j % kAhead], kf[u][j % KS], j % KS ? x[u] : zero, 0, 0, 0);
        if (j + kAhead < 2 * KS) ring[j % kAhead] = operand(j + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // x[u][4 j + i] is row 32 t + 8 j + 4 half + i
    // SERIES (capped scores): every one is within the series of tanh.
    auto add_tile = [&](const v16f (&x)[2], int buf, int t, auto masked, auto series) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = 32 * t + 8 * j + 4 * half;
        const v4f lse = *reinterpret_cast<const v4f*>(&s_lse[buf][row]);
        int4 seen = {};
        if (decltype(masked)::value) seen = *reinterpret_cast<const int4*>(&s_seen[buf][row]);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y = x[u][4 * j + i];
            if (CAP && decltype(series)::value) y = __builtin_fmaf(y * (f[u] * kLog2e), tanh_ratio<5>(y * (f[u] * inv_cap)), -lse[i]);
            else if (CAP) y = __builtin_fmaf(capped(y * f[u], a.softcap, inv_cap), kLog2e, -lse[i]);
            else y = __builtin_fmaf(y, f[u], -lse[i]);
            float p = __builtin_amdgcn_exp2f(y);
            if (decltype(masked)::value) p = mine[u] < (i == 0 ? seen.x : i == 1 ? seen.y : i == 2 ? seen.z : seen.w) ? p : 0.0f;
            sum[u] += p;
          }
      }
      asm volatile("" : "+v"(sum[0]), "+v"(sum[1]));  // sums are taken here: sunk below, they would hold every score
    };
    auto add = [&](const v16f (&x)[2], int buf, int t, auto masked) {
      bool small = false;
      if (CAP) {
        float big = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float y = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) y = fmaxf(y, __builtin_fabsf(x[u][i]));
          big = fmaxf(big, y * __builtin_fabsf(f[u]));
        }
        small = __builtin_amdgcn_ballot_w64(!(big * inv_cap < kCapSmall)) == 0;
      }
      if (small) add_tile(x, buf, t, masked, Int<1>{});
      else add_tile(x, buf, t, masked, Int<0>{});
    };
    auto step = [&](int buf, auto masked) {
      v16f x0[2], x1[2];
      scores(x0, x1, buf);
      add(x0, buf, 0, masked);
      add(x1, buf, 1, masked);
    };
    load(begin);
    store(0);
    __syncthreads();
    int buf = 0;
    for (int row0 = begin; row0 < end; row0 += kRows, buf ^= 1) {
      const bool more = row0 + kRows < end;
      if (more) load(row0 + kRows);
      // does the step's first row see all of the wave's tokens?
      if (whole && __builtin_amdgcn_readfirstlane(s_seen[buf][0]) >= slot0 + 64) step(buf, Int<0>{});
      else step(buf, Int<1>{});
      if (more) store(buf ^ 1);
      __syncthreads();
    }
    float* part = partial(a, tiles, pair, run, tile) + wave * 64;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float x = there[u] ? sum[u] : 0.0f;
      x += __shfl_xor(x, 32);
      if (half == 0) part[32 * u + r] = x;
    }
  }
}

// One workgroup per (sequence, head, tile): every slot of acc_out is written.
__global__ __launch_bounds__(kSlots) void k_weights_join(WeightArgs a, int tiles) {
  const CacheArgs& c = a.c;
  const int64_t pair = blockIdx.x / tiles;
  const int tile = blockIdx.x % tiles;
  const int64_t slot = (int64_t)tile * kSlots + threadIdx.x;
  const Seq s = sequence(c, (int)(pair / c.heads));
  float x = 0.0f;
  if (slot < a.acc_slots) x = old_sum(a, s, pair, slot);
  // (no steps at all: no row sees a slot)
  const int64_t all = tile < live_tiles(s) && s.n > 0 ? all_steps(a, s) : 0;
  if (all > 0) {
    int64_t before = 0;
    for (int t = 0; t < tile; ++t) before += tile_steps(a, s, t).count;
    const int64_t after = before + tile_steps(a, s, tile).count;
    int run = (int)(before * a.splits / all);        // its end is past `before`, or the next one's is
    while (run > 0 && run_begin(a, all, run) > before) --run;
    for (; run < a.splits && run_begin(a, all, run) < after; ++run)
      if (max(run_begin(a, all, run), before) < min(run_begin(a, all, run + 1), after))
        x += partial(a, tiles, pair, run, tile)[threadIdx.x];
  }
  if (slot < a.acc_slots) a.acc_out[pair * a.acc_slots + slot] = x;
}

int slot_tiles(const WeightArgs& a) { return (int)((a.acc_slots + kSlots - 1) / kSlots); }

template <int D, bool CAP>
hipError_t launch(const WeightArgs& a, hipStream_t stream) {
  const int64_t pairs = (int64_t)a.c.batch * a.c.heads;
  const dim3 tiles((unsigned)(pairs * slot_tiles(a)));
  if (a.splits == 0) {
    k_weights_rows<D, CAP><<<tiles, kThreads, 0, stream>>>(a, slot_tiles(a));
    return hipGetLastError();
  }
  k_weights_tiles<D, CAP><<<dim3((unsigned)(pairs * a.splits)), kThreads, 0, stream>>>(a, slot_tiles(a));
  if (hipError_t e = hipGetLastError()) return e;
  k_weights_join<<<tiles, kSlots, 0, stream>>>(a, slot_tiles(a));
  return hipGetLastError();
}

}  // namespace

void weights_plan(WeightArgs& a) {
  const int64_t rows = (int64_t)a.c.max_new * a.group, pairs = (int64_t)a.c.batch * a.c.heads;
  a.splits = 0;
  if (rows <= 16) return;
  // What runs at once (two workgroups per CU) for one sequence, whose runs are
  // all alike; twice that for several, whose lengths differ.  At least eight
  // steps a run.
  int64_t want = pairs > 0 ? ((a.c.batch == 1 ? 512 : 1024) + pairs - 1) / pairs : 1;
  const int64_t most = (int64_t)slot_tiles(a) * ((rows + kRows - 1) / kRows) / 8;
  if (want > most) want = most;
  a.splits = want < 1 ? 1 : (int32_t)want;
}

int64_t weights_workspace_bytes(const WeightArgs& a) {
  return a.splits > 0 ? (int64_t)a.c.batch * a.c.heads * (a.splits + slot_tiles(a)) * kSlots * 4 : 0;
}

int64_t weights_items(const WeightArgs& a) {
  return (int64_t)a.c.heads * std::max(a.splits, slot_tiles(a)) * kThreads;   // (the join's among them)
}

hipError_t launch_cache_weights(const WeightArgs& a, hipStream_t stream) {
  const bool cap = a.softcap > 0.0f;
  return launch_in_runs(a, weights_items(a), [&](const WeightArgs& run) {
    if (run.c.dim == 128) return cap ? launch<128, true>(run, stream) : launch<128, false>(run, stream);
    return cap ? launch<64, true>(run, stream) : launch<64, false>(run, stream);
  });
}

}  // namespace fp8bs
