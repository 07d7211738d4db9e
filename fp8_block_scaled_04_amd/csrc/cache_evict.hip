// Eviction from the paged FP8 cache by accumulated attention weight
// (include/fp8bs_cache.h, fp8bs_cache_evict).
//
// k_evict_select picks the kept slots of one (sequence, head): a radix search
// over the sums' bits, eight at a time, finds the smallest kept value and how
// many slots of exactly that value fit; one pass in slot order then writes
// them.  k_evict_move copies the codes, one workgroup per (destination page,
// head, K or V).
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

// Exclusive prefix of a flag over the workgroup, and its total.  `scratch`
// holds one int per wave; two barriers.
__device__ __forceinline__ int prefix(bool flag, int* scratch, int& total) {
  const uint64_t m = __ballot(flag);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
  if (lane == 0) scratch[wave] = __popcll(m);
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSelect / 64; ++w) {
    const int x = scratch[w];
    before += w < wave ? x : 0;
    total += x;
  }
  return before + __popcll(m & ((1ull << lane) - 1ull));
}

__global__ __launch_bounds__(kSelect) void k_evict_select(EvictArgs a) {
  const CacheArgs& c = a.c;
  const int h = blockIdx.x % c.heads, b = blockIdx.x / c.heads;
  const int tid = threadIdx.x;
  __shared__ uint32_t hist[256];
  __shared__ int scratch[kSelect / 64];
  __shared__ uint32_t s_digit;
  __shared__ int s_need;

  const int len = cached_tokens(c, b);
  const int count = min(len, a.budget), recent = min(count, a.recent);
  const int others = len - recent;                   // candidates: slots [0, others)
  int need = count - recent;                         // of which this many stay
  const float* acc = a.acc + ((int64_t)b * c.heads + h) * a.acc_slots;
  float* acc_out = a.acc_out + ((int64_t)b * c.heads + h) * a.acc_slots;
  int32_t* kept = a.kept + ((int64_t)b * c.heads + h) * a.budget;

  // smallest kept key, digit by digit; `need` becomes the slots of exactly
  // that key to take
  uint32_t key = 0, known = 0;
  if (need > 0 && need < others) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelect) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < others; i += kSelect) {
        const uint32_t u = rank_key(acc[i]);
        if ((u & known) == key) atomicAdd(&hist[(u >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        int left = need, d = 255;
        while (d > 0 && (int)hist[d] < left) left -= (int)hist[d--];
        s_digit = (uint32_t)d;
        s_need = left;
      }
      __syncthreads();
      key |= s_digit << shift;
      known |= 255u << shift;
      need = s_need;
    }
  }
  const bool all = count - recent >= others;         // nothing is evicted
  const bool none = count == recent;

  int out = 0, equal = 0;                            // written, equal ones met so far
  for (int i0 = 0; i0 < len; i0 += kSelect) {
    const int i = i0 + tid;
    bool take = i < len && (i >= others || all);
    bool tie = false;
    float x = 0.0f;
    if (i < len) x = acc[i];
    if (!all && !none && i < others) {
      const uint32_t u = rank_key(x);
      take = u > key;
      tie = u == key;
    }
    int total;
    const int e = prefix(tie, scratch, total);
    if (tie && equal + e < need) take = true;
    equal += total;
    const int at = prefix(take, scratch, total);
    if (take) {
      kept[out + at] = i;
      acc_out[out + at] = x;
    }
    out += total;
  }
  for (int i = count + tid; i < a.budget; i += kSelect) kept[i] = -1;
  for (int64_t i = count + tid; i < a.acc_slots; i += kSelect) acc_out[i] = 0.0f;
  if (h == 0 && tid == 0) a.new_lens[b] = count;
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
  k_evict_select<<<dim3((unsigned)(a.c.batch * a.c.heads)), kSelect, 0, stream>>>(a);
  if (hipError_t e = hipGetLastError()) return e;
  const dim3 grid((unsigned)evict_move_grid(a));
  if (grid.x == 0) return hipSuccess;
  if (a.c.dim == 128) k_evict_move<128><<<grid, kMove, 0, stream>>>(a, dst_blocks(a));
  else k_evict_move<64><<<grid, kMove, 0, stream>>>(a, dst_blocks(a));
  return hipGetLastError();
}

}  // namespace fp8bs
