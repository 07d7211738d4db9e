// Quantized append to the paged FP8 cache (include/fp8bs_cache.h,
// fp8bs_cache_append).
//
// One workgroup per (sequence, touched page, head, K or V): it owns the page's
// scale and codes of that head, so the largest value, the new scale, the older
// codes' re-encoding and the new codes need no other workgroup.
//
// HBM bound: 3 bytes move per value.  The 13,600 new tokens of six prompts (8
// heads of 128, pages of 128) take 18.4 us a call, 87 MB at 4.7 TB/s; a plain
// copy moves 5.0.  (Reading the new values a second time instead of holding
// them: 24 us.)
#include "cache_device.h"

namespace fp8bs {
namespace {

constexpr int kThreads = 256;

int pages_touched(int max_new, int lg_page) {
  return (int)(((int64_t)max_new + (1 << lg_page) - 2) >> lg_page) + 1;  // any alignment of the first slot
}

// NP: 8-value pieces per thread of a whole page; the new values stay in
// registers between the maximum and the codes.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int D, int NP, bool POW2>
__global__ __launch_bounds__(kThreads) void k_cache_append(AppendArgs a, int blocks) {
  const CacheArgs& c = a.c;
  constexpr int kPieces = D / 8;                     // 8-value pieces of a token
  int id = blockIdx.x;
  const int h = id % c.heads;
  id /= c.heads;
  const bool is_v = id & 1;
  id >>= 1;
  const int j = id % blocks, b = id / blocks;

  const Seq s = sequence(c, b);
  const int first = max(s.base, 0);
  const int end = min(s.base + s.n, s.len);          // new slots [first, end); past the table there are none
  if (first >= end) return;
  const int blk = (first >> c.lg_page) + j;
  const int P = 1 << c.lg_page, start = blk << c.lg_page;
  const int lo = max(first, start), hi = min(end, start + P);
  if (lo >= hi) return;
  const int page = page_of(c, b, lo);
  if (page < 0) return;
  const int64_t at = (int64_t)page * c.heads + h;
  uint8_t* codes = (is_v ? c.v : c.k) + at * ((int64_t)P * D);
  float* scale = (is_v ? c.vs : c.ks) + at;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.v_new : a.k_new) +
                        (int64_t)(s.row0 + (lo - s.base)) * a.ld_new + (int64_t)h * D;

  const int items = (hi - lo) * kPieces;
  u32x4 x[NP];
  float amax = 0.0f;
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    const int i = n * kThreads + threadIdx.x;
    x[n] = u32x4{0u, 0u, 0u, 0u};
    if (i < items) x[n] = *reinterpret_cast<const u32x4*>(src + (int64_t)(i / kPieces) * a.ld_new + (i % kPieces) * 8);
  }
#pragma unroll
  for (int n = 0; n < NP; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      amax = fmaxf(amax, fmaxf(__builtin_fabsf(bf16_lo(x[n][e])), __builtin_fabsf(bf16_hi(x[n][e]))));
  __shared__ float red[kThreads / 16];
  amax = row16_max(amax);
  if (threadIdx.x % 16 == 0) red[threadIdx.x / 16] = amax;
  __syncthreads();
  amax = row16_max(red[threadIdx.x % 16]);

  const float old = lo > start ? *scale : 0.0f;
  const float now = fmaxf(old, amax > 0.0f ? tile_scale<POW2>(amax).s : 0.0f);
  const TileScale t = divide_by(now);
  __syncthreads();                                   // every thread has read the old scale
  if (threadIdx.x == 0) *scale = now;
  if (now != old) {                                  // older rows of the page, if any
    uint32_t* row = reinterpret_cast<uint32_t*>(codes);
    for (int i = threadIdx.x; i < (lo - start) * (D / 4); i += kThreads) row[i] = reencode4(row[i], old, t);
  }
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    const int i = n * kThreads + threadIdx.x;
    if (i >= items) break;
    uint2 q = {0u, 0u};
    if (now > 0.0f) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // (a division also with power-of-two scales: an older scale of the
        // page may be any number)
        y[2 * e] = div_rn(bf16_lo(x[n][e]) * t.sx, t.ss, t.r);
        y[2 * e + 1] = div_rn(bf16_hi(x[n][e]) * t.sx, t.ss, t.r);
      }
      q.x = pack4_e4m3_sat(y[0], y[1], y[2], y[3]);
      q.y = pack4_e4m3_sat(y[4], y[5], y[6], y[7]);
    }
    *reinterpret_cast<uint2*>(codes + (int64_t)(lo - start) * D + (int64_t)i * 8) = q;
  }
}

}  // namespace

namespace {

int64_t page_blocks(const CacheArgs& c) { return pages_touched((int)std::min<int64_t>(c.max_new, c.rows), c.lg_page); }

}  // namespace

int64_t append_items(const CacheArgs& c) { return 2 * (int64_t)c.heads * page_blocks(c) * kThreads; }

namespace {

template <int D, int NP>
void launch(const AppendArgs& a, bool pow2, hipStream_t stream) {
  const int blocks = (int)page_blocks(a.c);
  const dim3 grid((unsigned)(2 * (int64_t)a.c.batch * a.c.heads * blocks));
  if (pow2) k_cache_append<D, NP, true><<<grid, kThreads, 0, stream>>>(a, blocks);
  else k_cache_append<D, NP, false><<<grid, kThreads, 0, stream>>>(a, blocks);
}

template <int D>
void launch(const AppendArgs& a, bool pow2, hipStream_t stream) {
  // pieces of a page: P D / 8 (at most 2048); one decoded token needs only the
  // first
  const int pieces = (1 << a.c.lg_page) * D / 8;
  const int np = a.c.max_new == 1 || pieces <= kThreads ? 1 : pieces / kThreads;
  if (np == 1) launch<D, 1>(a, pow2, stream);
  else if (np == 2) launch<D, 2>(a, pow2, stream);
  else if (np == 4) launch<D, 4>(a, pow2, stream);
  else if constexpr (D == 128) launch<D, 8>(a, pow2, stream);
}

}  // namespace

hipError_t launch_cache_append(const AppendArgs& a, bool pow2, hipStream_t stream) {
  return launch_in_runs(a, append_items(a.c), [&](const AppendArgs& run) {
    if (run.c.dim == 128) launch<128>(run, pow2, stream);
    else launch<64>(run, pow2, stream);
    return hipGetLastError();
  });
}

}  // namespace fp8bs
