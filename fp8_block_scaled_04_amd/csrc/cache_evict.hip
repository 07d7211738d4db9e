// Eviction from the paged FP8 cache by accumulated attention weight
// (include/fp8bs_cache.h, fp8bs_cache_evict).
//
// k_evict_select picks the kept slots of one (sequence, head): a radix search
// over the sums' bits (11 + 11 + 10) finds the smallest kept value and how many
// slots of exactly that value fit; ballots then place the kept slots in order, in
// LDS first, so that they are written (and their sums read) side by side.  The
// keys stay in registers where they fit.
// k_evict_move copies the codes, one workgroup per (destination page, head, K
// or V), and writes the new lengths.  Every search has read the old ones by
// then, and the copies take their counts from the kept slots, so both may be one
// array.
//
// The move is HBM bound: 16 sequences cut to 4096 tokens (8 heads of 128) in 60
// us, 262 MB at 4.4 TB/s (59 with counts from the lengths); the search before it
// takes 17.5 us of latency (its reads 2, each counted digit 3, ranks 4, what it
// writes 6), 7.5 us for 3 short ones.
#include "cache_device.h"

namespace fp8bs {
namespace {

constexpr int kSelect = 1024, kMove = 256;

// Order-preserving map of a float to an unsigned key: larger value, larger
// key; -0 equals +0; NaN below every number.
__device__ __forceinline__ uint32_t rank_key(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  const uint32_t key = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return x != x ? 0u : key;
}

constexpr int kBins = 2048, kWavesSel = kSelect / 64;

// Lanes below this one that are set in m.
__device__ __forceinline__ int lanes_below(uint64_t m) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// NK: keys per thread that stay in registers.
template <int NK>
__global__ __launch_bounds__(kSelect) void k_evict_select(EvictArgs a) {
  const CacheArgs& c = a.c;
  const int h = blockIdx.x % c.heads, b = blockIdx.x / c.heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int kBlock = NK * kSelect;
  __shared__ __attribute__((aligned(16))) uint32_t hist[kBins];
  __shared__ uint16_t picked[kBlock];                // kept slots of a block of keys, in order
  __shared__ int s_wave[kWavesSel], s_ties[kWavesSel];
  __shared__ int s_digit, s_need, s_equal;

  const int len = cached_tokens(c, b);
  const int count = min(len, a.budget), recent = min(count, a.recent);
  const int others = len - recent;                   // candidates: slots [0, others)
  const int need = count - recent;                   // of which this many stay
  const float* acc = a.acc + ((int64_t)b * c.heads + h) * a.acc_slots;
  float* acc_out = a.acc_out + ((int64_t)b * c.heads + h) * a.acc_slots;
  int32_t* kept = a.kept + ((int64_t)b * c.heads + h) * a.budget;

  // what lies past the count, here where the reads of the keys hide it
  for (int i = count + tid; i < a.budget; i += kSelect) kept[i] = -1;
  for (int64_t i = count + tid; i < a.acc_slots; i += kSelect) acc_out[i] = 0.0f;
  if (need == 0 || need == others) {                 // the last ones, or nothing is evicted
    for (int i = tid; i < count; i += kSelect) {
      kept[i] = len - count + i;
      acc_out[i] = acc[len - count + i];
    }
    return;
  }

  // A wave holds a run of slots, 64 per key: counts inside it stay in the scalar
  // unit, and slot order is (wave, key, lane).
  const int run = wave * (NK * 64) + lane;
  uint32_t u[NK];
  auto load = [&](int base) {
    float x[NK];                                     // all reads first, past the end the last one
#pragma unroll
    for (int k = 0; k < NK; ++k) x[k] = acc[min(base + run + 64 * k, others - 1)];
#pragma unroll
    for (int k = 0; k < NK; ++k) u[k] = rank_key(x[k]);
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
      const int left = others - base - run;
#pragma unroll
      for (int k = 0; k < NK; ++k)
        if (left > 64 * k && (u[k] & known) == key) atomicAdd(&hist[(u[k] >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // a thread holds two bins; counts of the larger keys come from the lanes and
    // waves above
    const int v0 = (int)hist[2 * tid], v1 = (int)hist[2 * tid + 1];
    int up = v0 + v1;                                // its own and all above
#pragma unroll
    for (int y = 1; y < 64; y *= 2) {
      const int z = __shfl_down(up, y);
      up += lane + y < 64 ? z : 0;
    }
    if (lane == 0) s_wave[wave] = up;
    __syncthreads();
#pragma unroll
    for (int w = 1; w < kWavesSel; ++w) up += w > wave ? s_wave[w] : 0;
    const int above = up - v0 - v1;
    if (above < wanted && up >= wanted) {            // exactly one thread
      const bool high = above + v1 >= wanted;
      s_digit = 2 * tid + high;
      s_need = wanted - above - (high ? 0 : v1);
      s_equal = high ? v1 : v0;
    }
    __syncthreads();
    key |= (uint32_t)s_digit << shift;
    known |= (uint32_t)(bins - 1) << shift;
    wanted = s_need;
    equal_all = s_equal;
  }

  // Kept candidates, in slot order.  Equal keys: the first `wanted` of them
  // (unless those are all there are, and no ranks are needed).
  int out = 0, met = 0;
  for (int base = 0; base < others; base += kBlock) {
    if (!resident) load(base);
    const int left = others - base - run;
    uint64_t take[NK];
    if (wanted < equal_all) {
      int ties = 0;
#pragma unroll
      for (int k = 0; k < NK; ++k) ties += __popcll(__ballot(left > 64 * k && (u[k] & known) == key));
      if (lane == 0) s_ties[wave] = ties;
      __syncthreads();
      int rank = met;
#pragma unroll
      for (int w = 0; w < kWavesSel; ++w) {
        rank += w < wave ? s_ties[w] : 0;
        met += s_ties[w];
      }
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const uint32_t x = u[k] & known;
        const bool in = left > 64 * k, tie = in && x == key;
        const uint64_t m = __ballot(tie);
        take[k] = __ballot((in && x > key) || (tie && rank + lanes_below(m) < wanted));
        rank += __popcll(m);
      }
    } else {
#pragma unroll
      for (int k = 0; k < NK; ++k) take[k] = __ballot(left > 64 * k && (u[k] & known) >= key);
    }
    int mine = 0;
#pragma unroll
    for (int k = 0; k < NK; ++k) mine += __popcll(take[k]);
    if (lane == 0) s_wave[wave] = mine;
    __syncthreads();
    int at = 0, n = 0;
#pragma unroll
    for (int w = 0; w < kWavesSel; ++w) {
      at += w < wave ? s_wave[w] : 0;
      n += s_wave[w];
    }
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      if ((take[k] >> lane) & 1u) picked[at + lanes_below(take[k])] = (uint16_t)(run + 64 * k);
      at += __popcll(take[k]);
    }
    __syncthreads();
    // the last block's are followed by the recent ones; four reads in flight
    const int all = n + (base + kBlock >= others ? recent : 0);
    for (int i = tid; i < all; i += 4 * kSelect) {
      int slot[4];
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int from = min(i + e * kSelect, all - 1);
        slot[e] = from < n ? base + picked[from] : others + from - n;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = acc[slot[e]];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int to = i + e * kSelect;
        if (to < all) {
          kept[out + to] = slot[e];
          acc_out[out + to] = x[e];
        }
      }
    }
    out += n;
  }
}

template <int D>
__global__ __launch_bounds__(kMove) void k_evict_move(EvictArgs a, int blocks, int copies) {
  const CacheArgs& c = a.c;
  const int tid = threadIdx.x;
  int id = blockIdx.x;
  if (id >= copies) {                                // the last workgroups: 256 lengths each
    const int b = (id - copies) * kMove + tid;
    if (b < c.batch) a.new_lens[b] = min(cached_tokens_of(c, b), a.budget);
    return;
  }
  const int h = id % c.heads;
  id /= c.heads;
  const bool is_v = id & 1;
  id >>= 1;
  const int j = id % blocks, b = id / blocks;
  const int P = 1 << c.lg_page, start = j << c.lg_page;
  const int32_t* kept = a.kept + ((int64_t)b * c.heads + h) * a.budget + start;
  // (asked for together)
  const int first = kept[0], slot = tid < min(P, a.budget - start) ? kept[tid] : -1;
  const int to = a.dst_table[(int64_t)b * a.dst_width + j];
  if (first < 0 || (uint32_t)to >= (uint64_t)c.pages) return;   // past the kept ones, or nowhere to go
  const uint8_t* codes = is_v ? c.v : c.k;
  const float* scales = is_v ? c.vs : c.ks;

  __shared__ int s_page[128];
  __shared__ int s_row[128];
  __shared__ float s_scale[128];
  __shared__ float red[kMove / 16];
  float top = 0.0f;
  if (tid < P) {
    int page = -1, row = 0;
    float s = 0.0f;
    if (slot >= 0) {
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

int64_t copies(const EvictArgs& a) { return 2 * (int64_t)a.c.batch * a.c.heads * dst_blocks(a); }

}  // namespace

int64_t evict_items(const EvictArgs& a) {
  return std::max<int64_t>((int64_t)a.c.heads * kSelect, (2 * (int64_t)a.c.heads * dst_blocks(a) + 1) * kMove);
}

hipError_t launch_cache_evict(const EvictArgs& call, hipStream_t stream) {
  return launch_in_runs(call, evict_items(call), [&](const EvictArgs& a) {
    // up to 4096 or 16384 slots stay in registers; more are read again from
    // cache by each pass
    const dim3 pairs((unsigned)(a.c.batch * a.c.heads));
    if (a.c.max_kv <= 4 * kSelect) k_evict_select<4><<<pairs, kSelect, 0, stream>>>(a);
    else k_evict_select<16><<<pairs, kSelect, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    const int n = (int)copies(a);
    const dim3 grid((unsigned)(n + (a.c.batch + kMove - 1) / kMove));
    if (a.c.dim == 128) k_evict_move<128><<<grid, kMove, 0, stream>>>(a, dst_blocks(a), n);
    else k_evict_move<64><<<grid, kMove, 0, stream>>>(a, dst_blocks(a), n);
    return hipGetLastError();
  });
}

}  // namespace fp8bs
