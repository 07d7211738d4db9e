// Device helpers of the cache kernels: one sequence's geometry, page lookup,
// code conversion, and re-encoding under another scale.
#pragma once

#include "cache.h"
#include "quant_common.h"

namespace fp8bs {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One sequence of a call.  Lengths come from device memory: `len` is clamped
// to what the launch and the table cover, so no value of them reads or writes
// out of range.  `base` is not: rows keep their slots whatever is left out, and
// every use of it takes the smaller of it and len.
struct Seq {
  int row0;   // first packed row
  int n;      // rows processed (at most max_new, all inside [0, rows))
  int len;    // cached tokens within the bounds
  int base;   // slot of the first row (negative: more rows than cached tokens; may pass len)
};

__device__ __forceinline__ int cached_tokens_of(const CacheArgs& c, int b) {
  const int64_t room = (int64_t)c.width << c.lg_page;
  return (int)max((int64_t)0, min((int64_t)min(c.kv_lens[b], c.max_kv), room));
}

// (b is the same for the whole wave; its numbers are kept on the scalar unit.)
__device__ __forceinline__ int cached_tokens(const CacheArgs& c, int b) {
  return __builtin_amdgcn_readfirstlane(cached_tokens_of(c, b));
}

__device__ __forceinline__ Seq sequence(const CacheArgs& c, int b) {
  Seq s;
  const int lo = __builtin_amdgcn_readfirstlane(c.q_offsets[b]);
  const int hi = __builtin_amdgcn_readfirstlane(c.q_offsets[b + 1]);
  s.row0 = lo;
  const bool fits = lo >= 0 && hi >= lo && hi <= c.rows;
  s.n = fits ? min(hi - lo, c.max_new) : 0;
  s.len = cached_tokens(c, b);
  const int all = __builtin_amdgcn_readfirstlane(c.kv_lens[b]);
  s.base = min(max(all, 0) - (fits ? hi - lo : 0), 1 << 30);   // (no slot lies past 2^30)
  return s;
}

// Page index of `slot` (below the cached tokens), or -1 for an entry outside
// the pool.
__device__ __forceinline__ int page_of(const CacheArgs& c, int b, int slot) {
  const int p = c.table[(int64_t)b * c.width + (slot >> c.lg_page)];
  return ((uint32_t)p < (uint64_t)c.pages) ? p : -1;
}

// Two E4M3 codes (the low or high half of w) as a BF16 pair: exact, every
// code is a BF16 value.
template <bool HI>
__device__ __forceinline__ v2bf codes_to_bf16(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI);
}

// Four codes -> four BF16 values at f[at .. at + 3].
__device__ __forceinline__ void unpack4(v8bf& f, int at, uint32_t w) {
  const v2bf a = codes_to_bf16<false>(w), b = codes_to_bf16<true>(w);
  f[at] = a[0];
  f[at + 1] = a[1];
  f[at + 2] = b[0];
  f[at + 3] = b[1];
}

// A scale prepared for fl32(x / s), |x| <= 448 s up to rounding (see
// TileScale: below s = 2^-69 both are taken times 2^64, which is exact).
// s = 0 gives quotients that are never used.
__device__ __forceinline__ TileScale divide_by(float s) {
#pragma clang fp contract(off)
  TileScale t;
  t.s = s;
  t.sx = (s < 0x1p-69f) ? 0x1p64f : 1.0f;
  t.ss = s * t.sx;
  t.r = 1.0f / t.ss;
  return t;
}

// Four codes of scale `old` encoded again under t.s: E4M3(fl32(fl32(c old) / s)).
__device__ __forceinline__ uint32_t reencode4(uint32_t w, float old, const TileScale& t) {
#pragma clang fp contract(off)
  const float a = __builtin_amdgcn_cvt_f32_fp8((int)w, 0) * old, b = __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * old;
  const float c = __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * old, d = __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * old;
  return pack4_e4m3_sat(div_rn(a * t.sx, t.ss, t.r), div_rn(b * t.sx, t.ss, t.r), div_rn(c * t.sx, t.ss, t.r),
                        div_rn(d * t.sx, t.ss, t.r));
}

// cap * tanh(x / cap), y = x / cap.  For |y| < kCapSmall by the odd series of
// tanh, so that small scores keep FP32 relative accuracy; above by
// 1 - 2 / (e^(2y) + 1).  tanh_ratio<TERMS>(y) is tanh(y) / y: three terms past
// the first serve |y| < kCapTiny, five |y| < kCapSmall (the next term is under
// 2^-26 there).
constexpr float kCapTiny = 0.16f, kCapSmall = 0.35f;

template <int TERMS>
__device__ __forceinline__ float tanh_ratio(float y) {
  const float z = y * y;
  float s = 0x1.ba1ba1ba1ba1cp-5f;                   // 17/315
  if (TERMS == 5) {
    s = 0x1.226e355e6c23dp-7f;                       // 1382/155925
    s = __builtin_fmaf(-s, z, 0x1.664f4882c10fap-6f);  // 62/2835
    s = __builtin_fmaf(-s, z, 0x1.ba1ba1ba1ba1cp-5f);
  }
  s = __builtin_fmaf(-s, z, 0x1.1111111111111p-3f);  // 2/15
  s = __builtin_fmaf(-s, z, 0x1.5555555555555p-2f);  // 1/3
  return __builtin_fmaf(-s, z, 1.0f);
}

__device__ __forceinline__ float capped(float x, float cap, float inv_cap) {
  const float y = x * inv_cap;
  const float e = __builtin_amdgcn_exp2f(y * (2.0f * kLog2e));
  const float large = __builtin_fmaf(-2.0f * cap, __builtin_amdgcn_rcpf(e + 1.0f), cap);
  return __builtin_fabsf(y) < kCapSmall ? x * tanh_ratio<5>(y) : large;
}

// Bytes of four tokens (a0..a3: the same four dims each) -> per dim the four
// tokens' bytes.
__device__ __forceinline__ void transpose4(const uint32_t a[4], uint32_t o[4]) {
  const uint32_t l0 = __builtin_amdgcn_perm(a[1], a[0], 0x05010400u), h0 = __builtin_amdgcn_perm(a[1], a[0], 0x07030602u);
  const uint32_t l1 = __builtin_amdgcn_perm(a[3], a[2], 0x05010400u), h1 = __builtin_amdgcn_perm(a[3], a[2], 0x07030602u);
  o[0] = __builtin_amdgcn_perm(l1, l0, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(l1, l0, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(h1, h0, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(h1, h0, 0x07060302u);
}

}  // namespace fp8bs
