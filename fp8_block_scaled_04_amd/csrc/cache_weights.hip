// The attention weight each cached token received (include/fp8bs_cache.h,
// fp8bs_cache_attention_weights): acc[j] (+)= sum over rows of exp(x_j - lse).
//
// One workgroup per (sequence, head, 256 slots) walks every row, so each
// slot's sum has one owner and a fixed order.  Scores are formed as S = Q K^T:
// a lane then holds one token and four rows per matrix step, and the sum over
// rows stays in the lane.
#include "cache_device.h"

namespace fp8bs {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, kTiles = 4;
constexpr int kSlots = kWaves * kTiles * 16;         // per workgroup

template <int D, bool CAP>
__global__ __launch_bounds__(kThreads) void k_cache_weights(WeightArgs a, int tiles) {
  const CacheArgs& c = a.c;
  constexpr int KS = D / 32;
  int id = blockIdx.x;
  const int tile = id % tiles;
  id /= tiles;
  const int h = id % c.heads, b = id / c.heads;
  const Seq s = sequence(c, b);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int64_t acc_at = ((int64_t)b * c.heads + h) * a.acc_slots;
  const int64_t slot0 = (int64_t)tile * kSlots + wave * (kTiles * 16);
  if (slot0 >= a.acc_slots) return;
  const int rows = s.n * a.group;
  const float inv_cap = 1.0f / a.softcap;
  float sum[kTiles] = {};

  if (slot0 < s.len && rows > 0) {
    v8bf kf[kTiles][KS];
    float f[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int tt = (int)slot0 + 16 * i;
      int page = page_of(c, b, min(tt, s.len - 1));
      const bool there = page >= 0;
      page = max(page, 0);
      const int64_t at = (int64_t)page * c.heads + h;
      f[i] = there ? c.ks[at] * a.scale : 0.0f;      // an absent page's tokens are dropped at the end
      const uint8_t* kp = c.k + (at << c.lg_page) * D + (int64_t)((tt & ((1 << c.lg_page) - 1)) + r) * D + g * (D / 4);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint2 w = *reinterpret_cast<const uint2*>(kp + 8 * k);
        unpack4(kf[i][k], 0, w.x);
        unpack4(kf[i][k], 4, w.y);
      }
    }
    // rows before the first that sees the wave's first slot add nothing
    const int skip = a.full ? 0 : max(0, (int)slot0 - s.base) * a.group;
    for (int row0 = skip & ~15; row0 < rows; row0 += 16) {
      const int qrow = min(row0 + r, rows - 1);
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)(s.row0 + qrow / a.group) * a.ld_q +
                          (int64_t)(h * a.group + qrow % a.group) * D + g * (D / 4);
      v8bf qf[KS];
#pragma unroll
      for (int k = 0; k < KS; ++k) qf[k] = *reinterpret_cast<const v8bf*>(q + 8 * k);
      float lse[4];
      int seen[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = row0 + 4 * g + j;
        const int cl = min(row, rows - 1), tok = cl / a.group;
        lse[j] = a.lse[(int64_t)(s.row0 + tok) * a.q_heads + h * a.group + cl % a.group];
        seen[j] = (row < rows && lse[j] != -INFINITY) ? (a.full ? s.len : min(s.len, s.base + tok + 1)) : 0;
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        v4f x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KS; ++k) x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[k], kf[i][k], x, 0, 0, 0);
        const int slot = (int)slot0 + 16 * i + r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float y = x[j] * f[i];
          if (CAP) y = capped(y, a.softcap, inv_cap);
          const float p = __builtin_amdgcn_exp2f((y - lse[j]) * kLog2e);
          sum[i] += slot < seen[j] ? p : 0.0f;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    float x = sum[i];
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    const int64_t slot = slot0 + 16 * i + r;
    if (g != 0 || slot >= a.acc_slots) continue;
    bool there = slot < s.len;
    if (there) there = page_of(c, b, (int)slot) >= 0;
    float old = 0.0f;
    if (a.acc_in && slot < min(s.base, s.len)) old = a.acc_in[acc_at + slot];
    a.acc_out[acc_at + slot] = there ? old + x : old;
  }
}

int slot_tiles(const WeightArgs& a) { return (int)((a.acc_slots + kSlots - 1) / kSlots); }

}  // namespace

int64_t weights_grid(const WeightArgs& a) { return (int64_t)a.c.batch * a.c.heads * slot_tiles(a); }

hipError_t launch_cache_weights(const WeightArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)weights_grid(a));
  const int t = slot_tiles(a);
  const bool cap = a.softcap > 0.0f;
  if (a.c.dim == 128) {
    if (cap) k_cache_weights<128, true><<<grid, kThreads, 0, stream>>>(a, t);
    else k_cache_weights<128, false><<<grid, kThreads, 0, stream>>>(a, t);
  } else {
    if (cap) k_cache_weights<64, true><<<grid, kThreads, 0, stream>>>(a, t);
    else k_cache_weights<64, false><<<grid, kThreads, 0, stream>>>(a, t);
  }
  return hipGetLastError();
}

}  // namespace fp8bs
