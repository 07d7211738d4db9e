// Eviction from the paged FP8 cache by accumulated attention weight
// (include/fp8bs_cache.h, fp8bs_cache_evict).
//
// k_evict_select picks the kept slots of one (sequence, head): a radix search
// over the sums' bits (11 + 11 + 10) finds the smallest kept value and how many
// slots of exactly that value fit; ballots and a prefix over them then place
// the kept slots in order.  The keys stay in registers where they fit.
// k_evict_move copies the codes, one workgroup per (destination page, head, K
// or V).
//
// The move is HBM bound: 16 sequences cut to 4096 tokens (8 heads of 128) in 59
// us, 262 MB at 4.4 TB/s; the search before it takes 20 us of latency (barriers
// of 16 waves, three rounds of LDS counts).
#include "cache_device.h"

namespace fp8bs {
namespace {

constexpr int kSelect = 1024, kMove = 256;

// Order-preserving map of a float to an unsigned key: larger value, larger
// key; -0 equals +0; NaN below every number.
__device__ __forceinline__ uint32_t rank_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kBins = 2048, kWavesSel = kSelect / 64;

// Exclusive prefix over n (a multiple of 64, at most 1024) counts in LDS, and
// their total in counts[n]; by the first wave, between two barriers.
template <int N>
__device__ __forceinline__ void scan_counts(int* counts) {
  constexpr int E = N / 64;
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int v[E], sum = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[e] = counts[lane * E + e];
      sum += v[e];
    }
    int up = sum;                                    // inclusive over the lanes
#pragma unroll
    for (int x = 1; x < 64; x *= 2) {
      const int y = __shfl_up(up, x);
      up += lane >= x ? y : 0;
    }
    int at = up - sum;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      counts[lane * E + e] = at;
      at += v[e];
    }
    if (lane == 63) counts[N] = up;
  }
  __syncthreads();
}

// NK: keys per thread that stay in registers.
template <int NK>
__global__ __launch_bounds__(kSelect) void k_evict_select(EvictArgs a) {
  const CacheArgs& c = a.c;
  const int h = blockIdx.x % c.heads, b = blockIdx.x / c.heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kBlock = NK * kSelect, kCounts = NK * kWavesSel;
  __shared__ __attribute__((aligned(16))) uint32_t hist[kBins];
  __shared__ int counts[kCounts + 1];
  __shared__ int s_digit, s_need, s_equal;

  const int len = cached_tokens(c, b);
  const int count = min(len, a.budget), recent = min(count, a.recent);
  const int others = len - recent;                   // candidates: slots [0, others)
  int need = count - recent;                         // of which this many stay
  const float* acc = a.acc + ((int64_t)b * c.heads + h) * a.acc_slots;
  float* acc_out = a.acc_out + ((int64_t)b * c.heads + h) * a.acc_slots;
  int32_t* kept = a.kept + ((int64_t)b * c.heads + h) * a.budget;

  // the last ones, and what lies past the count
  for (int i = tid; i < recent; i += kSelect) {
    kept[need + i] = others + i;
    acc_out[need + i] = acc[others + i];
  }
  for (int i = count + tid; i < a.budget; i += kSelect) kept[i] = -1;
  for (int64_t i = count + tid; i < a.acc_slots; i += kSelect) acc_out[i] = 0.0f;
  if (h == 0 && tid == 0) a.new_lens[b] = count;
  if (need == 0) return;
  if (need == others) {                              // nothing is evicted
    for (int i = tid; i < others; i += kSelect) {
      kept[i] = i;
      acc_out[i] = acc[i];
    }
    return;
  }

  float x[NK];
  auto load = [&](int base) {
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const int i = base + k * kSelect + tid;
      x[k] = i < others ? acc[i] : 0.0f;
    }
  };
  const bool resident = others <= kBlock;
  if (resident) load(0);

  // Smallest kept key, digit by digit: `wanted` of the `equal_all` keys that
  // agree with it in the known digits are kept, and all larger ones.  Done as
  // soon as all of them are (two digits usually tell real sums apart).
  uint32_t key = 0, known = 0;
  int wanted = need, equal_all = 0;
  for (int pass = 0; pass < 3 && wanted != equal_all; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    for (int i = tid; i < kBins; i += kSelect) hist[i] = 0;
    __syncthreads();
    for (int base = 0; base < others; base += kBlock) {
      if (!resident) load(base);
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const uint32_t u = rank_key(x[k]);
        if (base + k * kSelect + tid < others && (u & known) == key) atomicAdd(&hist[(u >> shift) & (bins - 1)], 1u);
      }
    }
    __syncthreads();
    if (wave == 0) {
      // lane x holds bins [32 x, 32 x + 32); counts of the larger keys come
      // from the lanes above
      int v[32], sum = 0;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        v[e] = (int)hist[lane * 32 + e];
        sum += v[e];
      }
      int up = sum;                                  // this lane's and all above
#pragma unroll
      for (int y = 1; y < 64; y *= 2) {
        const int z = __shfl_down(up, y);
        up += lane + y < 64 ? z : 0;
      }
      int above = up - sum;
      if (above < wanted && up >= wanted) {          // exactly one lane
        bool found = false;
#pragma unroll
        for (int e = 31; e >= 0; --e) {
          if (!found && above + v[e] >= wanted) {
            found = true;
            s_digit = lane * 32 + e;
            s_need = wanted - above;
            s_equal = v[e];
          }
          above += v[e];
        }
      }
    }
    __syncthreads();
    key |= (uint32_t)s_digit << shift;
    known |= (uint32_t)(bins - 1) << shift;
    wanted = s_need;
    equal_all = s_equal;
    __syncthreads();
  }

  // Kept candidates, in slot order.  Equal keys: the first `wanted` of them
  // (unless those are all there are, and no ranks are needed).
  int out = 0, met = 0;
  for (int base = 0; base < others; base += kBlock) {
    if (!resident) load(base);
    const int slot0 = base + tid;
    if (wanted < equal_all) {
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const uint64_t m = __ballot(slot0 + k * kSelect < others && (rank_key(x[k]) & known) == key);
        if (lane == 0) counts[k * kWavesSel + wave] = __popcll(m);
      }
      scan_counts<kCounts>(counts);
    }
    uint32_t take = 0;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const uint32_t u = rank_key(x[k]) & known;
      const bool in = slot0 + k * kSelect < others, tie = in && u == key;
      bool t = tie;
      if (wanted < equal_all) {
        const uint64_t m = __ballot(tie);
        t = tie && met + counts[k * kWavesSel + wave] + __popcll(m & ((1ull << lane) - 1ull)) < wanted;
      }
      if (t || (in && u > key)) take |= 1u << k;
    }
    if (wanted < equal_all) {
      met += counts[kCounts];
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const uint64_t m = __ballot((take >> k) & 1u);
      if (lane == 0) counts[k * kWavesSel + wave] = __popcll(m);
    }
    scan_counts<kCounts>(counts);
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const bool t = (take >> k) & 1u;
      const uint64_t m = __ballot(t);
      if (t) {
        const int at = out + counts[k * kWavesSel + wave] + __popcll(m & ((1ull << lane) - 1ull));
        kept[at] = slot0 + k * kSelect;
        acc_out[at] = x[k];
      }
    }
    out += counts[kCounts];
    __syncthreads();
  }
}

template <int D>
__global__ __launch_bounds__(kMove) void k_evict_move(EvictArgs a, int blocks) {
  const CacheArgs& c = a.c;
  int id = blockIdx.x;
  const int h = id % c.heads;
  id /= c.heads;
  const bool is_v = id & 1;
  id >>= 1;
  const int j = id % blocks, b = id / blocks;
  const int count = min(cached_tokens(c, b), a.budget);
  const int P = 1 << c.lg_page, start = j << c.lg_page;
  if (start >= count) return;
  const int to = a.dst_table[(int64_t)b * a.dst_width + j];
  if ((uint32_t)to >= (uint64_t)c.pages) return;
  const int32_t* kept = a.kept + ((int64_t)b * c.heads + h) * a.budget + start;
  const uint8_t* codes = is_v ? c.v : c.k;
  const float* scales = is_v ? c.vs : c.ks;
  const int n = min(P, count - start), tid = threadIdx.x;

  __shared__ int s_page[128];
  __shared__ int s_row[128];
  __shared__ float s_scale[128];
  __shared__ float red[kMove / 16];
  float top = 0.0f;
  if (tid < P) {
    int page = -1, row = 0;
    float s = 0.0f;
    if (tid < n) {
      const int slot = kept[tid];
      page = page_of(c, b, slot);
      row = slot & (P - 1);
      if (page >= 0) s = scales[(int64_t)page * c.heads + h];
    }
    s_page[tid] = page;
    s_row[tid] = row;
    s_scale[tid] = s;
    top = s;
  }
  top = row16_max(top);
  if (tid % 16 == 0) red[tid / 16] = top;
  __syncthreads();
  top = row16_max(red[tid % 16]);

  const int64_t dst = (int64_t)to * c.heads + h;
  if (tid == 0) (is_v ? c.vs : c.ks)[dst] = top;
  uint4* out = reinterpret_cast<uint4*>((is_v ? c.v : c.k) + dst * ((int64_t)P * D));
  const TileScale t = divide_by(top);
  constexpr int kPieces = D / 16;
  for (int i = tid; i < P * kPieces; i += kMove) {
    const int tok = i / kPieces, page = s_page[tok];
    uint4 x = {0u, 0u, 0u, 0u};
    if (page >= 0) {
      const float old = s_scale[tok];
      x = *reinterpret_cast<const uint4*>(codes + (((int64_t)page * c.heads + h) * P + s_row[tok]) * D +
                                          (i % kPieces) * 16);
      if (old != top) {
        x.x = reencode4(x.x, old, t);
        x.y = reencode4(x.y, old, t);
        x.z = reencode4(x.z, old, t);
        x.w = reencode4(x.w, old, t);
      }
    }
    out[i] = x;
  }
}

int dst_blocks(const EvictArgs& a) {
  const int most = a.budget < a.c.max_kv ? a.budget : a.c.max_kv;
  return (int)(((int64_t)most + (1 << a.c.lg_page) - 1) >> a.c.lg_page);
}

}  // namespace

int64_t evict_move_grid(const EvictArgs& a) { return 2 * (int64_t)a.c.batch * a.c.heads * dst_blocks(a); }

hipError_t launch_cache_evict(const EvictArgs& a, hipStream_t stream) {
  // up to 4096 or 16384 slots stay in registers; more are read again from
  // cache by each pass
  const dim3 pairs((unsigned)(a.c.batch * a.c.heads));
  if (a.c.max_kv <= 4 * kSelect) k_evict_select<4><<<pairs, kSelect, 0, stream>>>(a);
  else k_evict_select<16><<<pairs, kSelect, 0, stream>>>(a);
  if (hipError_t e = hipGetLastError()) return e;
  const dim3 grid((unsigned)evict_move_grid(a));
  if (grid.x == 0) return hipSuccess;
  if (a.c.dim == 128) k_evict_move<128><<<grid, kMove, 0, stream>>>(a, dst_blocks(a));
  else k_evict_move<64><<<grid, kMove, 0, stream>>>(a, dst_blocks(a));
  return hipGetLastError();
}

}  // namespace fp8bs
