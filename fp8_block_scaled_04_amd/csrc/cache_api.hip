// C ABI of the paged FP8 cache (include/fp8bs_cache.h): argument checks and
// dispatch.
#include <cmath>

#include "abi_common.h"
#include "cache.h"
#include "fp8bs_cache.h"

namespace {

using fp8bs::aligned16;
using fp8bs::aligned4;
using fp8bs::CacheArgs;
using fp8bs::check_device;
using fp8bs::launched;

constexpr int64_t kMaxCount = int64_t(1) << 30;      // slots, rows: 32-bit indexes in the kernels
constexpr int64_t kMaxPairs = int64_t(1) << 40;      // (row, query head) pairs: bytes of 64 splits stay in 64 bits

bool sizes_fit(const fp8bs_cache& c, int64_t rows, int64_t max_new, int64_t max_kv) {
  if (c.batch < 0 || c.heads <= 0 || c.pages <= 0 || c.table_width <= 0) return false;
  if (c.page != 16 && c.page != 32 && c.page != 64 && c.page != 128) return false;
  if (c.dim != 64 && c.dim != 128) return false;
  if ((int64_t)c.table_width * c.page > kMaxCount || (int64_t)c.batch * c.heads > kMaxCount) return false;
  return rows >= 0 && rows <= kMaxCount && max_new >= 0 && max_new <= kMaxCount && max_kv >= 0 && max_kv <= kMaxCount;
}

bool query_sizes_fit(const fp8bs_cache& c, int64_t ld, int32_t q_heads, int64_t rows, int64_t max_new) {
  return q_heads > 0 && q_heads % c.heads == 0 && ld >= (int64_t)q_heads * c.dim && ld % 8 == 0 &&
         max_new * q_heads <= kMaxCount && rows * q_heads <= kMaxPairs;
}

CacheArgs args(const fp8bs_cache& c, const int32_t* q_offsets, int64_t rows, int32_t max_new, int32_t max_kv) {
  int32_t lg = 4;
  while ((1 << lg) < c.page) ++lg;
  return CacheArgs{c.k, c.ks, c.v, c.vs, c.table, c.kv_lens, q_offsets, c.pages, rows, c.batch, c.table_width,
                   c.heads, lg, c.dim, max_new, max_kv};
}

// keys (and values) of the cache, its table and lengths
fp8bs_status cache_pointers(const fp8bs_cache& c, bool values) {
  if (!c.k || !c.ks || (values && (!c.v || !c.vs)) || !c.table || !c.kv_lens) return FP8BS_ERR_NULL;
  if (!aligned16(c.k) || !aligned4(c.ks) || !aligned4(c.table) || !aligned4(c.kv_lens)) return FP8BS_ERR_ALIGN;
  if (values && (!aligned16(c.v) || !aligned4(c.vs))) return FP8BS_ERR_ALIGN;
  return FP8BS_OK;
}

// A cap's reciprocal and its double stay finite.
bool bad_scalars(float scale, float softcap) {
  return !std::isfinite(scale) || !(softcap == 0.0f || (softcap >= 0x1p-126f && softcap <= 0x1p126f));
}

// The plan of an attention call from its sizes; false for sizes it refuses.
bool attention_plan(const fp8bs_cache& c, int32_t q_heads, int64_t rows, int32_t max_new, int32_t max_kv,
                    fp8bs::AttendArgs& a) {
  if (!sizes_fit(c, rows, max_new, max_kv) || q_heads <= 0 ||
      !query_sizes_fit(c, (int64_t)q_heads * c.dim, q_heads, rows, max_new))
    return false;
  a.c = args(c, nullptr, rows, max_new, max_kv);
  a.q_heads = q_heads;
  a.group = q_heads / c.heads;
  attend_plan(a);
  return attend_items(a) <= fp8bs::kMaxItems;
}

}  // namespace

extern "C" {

fp8bs_status fp8bs_cache_append(const fp8bs_cache* cache, const void* k_new, const void* v_new, int64_t ld_new,
                                const int32_t* q_offsets, int64_t rows, int32_t max_new, uint32_t flags,
                                fp8bs_stream_t stream) {
  if (!cache) return FP8BS_ERR_NULL;
  const fp8bs_cache& c = *cache;
  if (!sizes_fit(c, rows, max_new, 0) || ld_new < (int64_t)c.heads * c.dim || ld_new % 8) return FP8BS_ERR_SHAPE;
  fp8bs::AppendArgs a{args(c, q_offsets, rows, max_new, (int32_t)kMaxCount), k_new, v_new, ld_new};
  if (append_items(a.c) > fp8bs::kMaxItems) return FP8BS_ERR_SHAPE;
  if (flags & ~(uint32_t)FP8BS_SCALE_POW2) return FP8BS_ERR_FLAGS;
  if (c.batch == 0 || rows == 0 || max_new == 0) return FP8BS_OK;
  if (!k_new || !v_new || !q_offsets) return FP8BS_ERR_NULL;
  if (fp8bs_status e = cache_pointers(c, true)) return e;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned4(q_offsets)) return FP8BS_ERR_ALIGN;
  if (fp8bs_status e = check_device()) return e;
  (void)hipGetLastError();
  return launched(fp8bs::launch_cache_append(a, (flags & FP8BS_SCALE_POW2) != 0, (hipStream_t)stream));
}

fp8bs_status fp8bs_cache_attention(const fp8bs_cache* cache, const void* q, int64_t ld_q, int32_t q_heads,
                                   const int32_t* q_offsets, int64_t rows, int32_t max_new, int32_t max_kv,
                                   float scale, float softcap, void* out, int32_t out_dtype, float* lse,
                                   uint32_t flags, void* workspace, int64_t workspace_bytes, fp8bs_stream_t stream) {
  if (!cache) return FP8BS_ERR_NULL;
  const fp8bs_cache& c = *cache;
  if (!sizes_fit(c, rows, max_new, max_kv) || !query_sizes_fit(c, ld_q, q_heads, rows, max_new)) return FP8BS_ERR_SHAPE;
  fp8bs::AttendArgs a{args(c, q_offsets, rows, max_new, max_kv), q, ld_q, q_heads, q_heads / c.heads, scale, softcap,
                      out, lse, out_dtype == FP8BS_OUT_FP32, (flags & FP8BS_MASK_FULL) != 0, 16, 0, 1, nullptr,
                      nullptr};
  attend_plan(a);
  const int64_t need = attend_workspace_bytes(a);
  if (attend_items(a) > fp8bs::kMaxItems || workspace_bytes < need) return FP8BS_ERR_SHAPE;
  if (out_dtype != FP8BS_OUT_BF16 && out_dtype != FP8BS_OUT_FP32) return FP8BS_ERR_FLAGS;
  if ((flags & ~(uint32_t)FP8BS_MASK_FULL) || bad_scalars(scale, softcap)) return FP8BS_ERR_FLAGS;
  if (c.batch == 0 || rows == 0 || max_new == 0) return FP8BS_OK;
  if (!q || !q_offsets || !out || (need > 0 && !workspace)) return FP8BS_ERR_NULL;
  if (fp8bs_status e = cache_pointers(c, true)) return e;
  if (!aligned16(q) || !aligned4(q_offsets) || !aligned16(out) || !aligned4(lse) || (need > 0 && !aligned16(workspace)))
    return FP8BS_ERR_ALIGN;
  if (fp8bs_status e = check_device()) return e;
  if (need > 0) {
    a.part = static_cast<float*>(workspace);
    a.stat = reinterpret_cast<float2*>(a.part + (int64_t)a.splits * rows * q_heads * c.dim);
  }
  (void)hipGetLastError();
  return launched(fp8bs::launch_cache_attention(a, (hipStream_t)stream));
}

fp8bs_status fp8bs_cache_attention_workspace(const fp8bs_cache* cache, int32_t q_heads, int64_t rows,
                                             int32_t max_new, int32_t max_kv, int64_t* bytes) {
  if (!cache) return FP8BS_ERR_NULL;
  fp8bs::AttendArgs a{};
  if (!attention_plan(*cache, q_heads, rows, max_new, max_kv, a)) return FP8BS_ERR_SHAPE;
  if (!bytes) return FP8BS_ERR_NULL;
  *bytes = attend_workspace_bytes(a);
  return FP8BS_OK;
}

int32_t fp8bs_cache_attention_tile(const fp8bs_cache* cache, int32_t q_heads, int64_t rows, int32_t max_new,
                                   int32_t max_kv) {
  fp8bs::AttendArgs a{};
  return cache && attention_plan(*cache, q_heads, rows, max_new, max_kv, a) ? a.tile_rows : 0;
}

fp8bs_status fp8bs_cache_attention_weights(const fp8bs_cache* cache, const void* q, int64_t ld_q, int32_t q_heads,
                                           const int32_t* q_offsets, int64_t rows, int32_t max_new, int32_t max_kv,
                                           float scale, float softcap, const float* lse, const float* acc_in,
                                           float* acc_out, int64_t acc_slots, uint32_t flags, void* workspace,
                                           int64_t workspace_bytes, fp8bs_stream_t stream) {
  if (!cache) return FP8BS_ERR_NULL;
  const fp8bs_cache& c = *cache;
  if (!sizes_fit(c, rows, max_new, max_kv) || !query_sizes_fit(c, ld_q, q_heads, rows, max_new)) return FP8BS_ERR_SHAPE;
  if (acc_slots < max_kv || acc_slots > kMaxCount) return FP8BS_ERR_SHAPE;
  fp8bs::WeightArgs a{args(c, q_offsets, rows, max_new, max_kv), q, ld_q, q_heads, q_heads / c.heads, scale, softcap,
                      lse, acc_in, acc_out, acc_slots, (flags & FP8BS_MASK_FULL) != 0, 0, nullptr};
  weights_plan(a);
  const int64_t need = weights_workspace_bytes(a);
  if (weights_items(a) > fp8bs::kMaxItems || workspace_bytes < need) return FP8BS_ERR_SHAPE;
  if ((flags & ~(uint32_t)FP8BS_MASK_FULL) || bad_scalars(scale, softcap)) return FP8BS_ERR_FLAGS;
  if (c.batch == 0 || acc_slots == 0) return FP8BS_OK;
  if ((rows > 0 && (!q || !lse)) || !q_offsets || !acc_out || (need > 0 && !workspace)) return FP8BS_ERR_NULL;
  if (fp8bs_status e = cache_pointers(c, false)) return e;
  if (!aligned16(q) || !aligned4(q_offsets) || !aligned4(lse) || !aligned4(acc_in) || !aligned4(acc_out) ||
      (need > 0 && !aligned16(workspace)))
    return FP8BS_ERR_ALIGN;
  if (fp8bs_status e = check_device()) return e;
  a.part = static_cast<float*>(workspace);
  (void)hipGetLastError();
  return launched(fp8bs::launch_cache_weights(a, (hipStream_t)stream));
}

fp8bs_status fp8bs_cache_attention_weights_workspace(const fp8bs_cache* cache, int32_t q_heads, int32_t max_new,
                                                     int64_t acc_slots, int64_t* bytes) {
  if (!cache) return FP8BS_ERR_NULL;
  const fp8bs_cache& c = *cache;
  if (!sizes_fit(c, 0, max_new, 0) || q_heads <= 0 || acc_slots < 0 || acc_slots > kMaxCount ||
      !query_sizes_fit(c, (int64_t)q_heads * c.dim, q_heads, 0, max_new))
    return FP8BS_ERR_SHAPE;
  if (!bytes) return FP8BS_ERR_NULL;
  fp8bs::WeightArgs a{};
  a.c = args(c, nullptr, 0, max_new, 0);
  a.q_heads = q_heads;
  a.group = q_heads / c.heads;
  a.acc_slots = acc_slots;
  weights_plan(a);
  *bytes = weights_workspace_bytes(a);
  return FP8BS_OK;
}

fp8bs_status fp8bs_cache_evict(const fp8bs_cache* cache, const float* acc, int64_t acc_slots,
                               const int32_t* dst_table, int32_t dst_width, int32_t max_kv, int32_t budget,
                               int32_t recent, int32_t* kept, int32_t* new_lens, float* acc_out,
                               fp8bs_stream_t stream) {
  if (!cache) return FP8BS_ERR_NULL;
  const fp8bs_cache& c = *cache;
  if (!sizes_fit(c, 0, 0, max_kv) || acc_slots < max_kv || acc_slots > kMaxCount) return FP8BS_ERR_SHAPE;
  if (budget <= 0 || budget > kMaxCount || recent < 0 || dst_width < 0) return FP8BS_ERR_SHAPE;
  if ((int64_t)dst_width * c.page < (budget < max_kv ? budget : max_kv)) return FP8BS_ERR_SHAPE;
  if (acc && acc == acc_out) return FP8BS_ERR_SHAPE;
  fp8bs::EvictArgs a{args(c, nullptr, 0, 0, max_kv), acc, acc_slots, dst_table, dst_width, budget, recent, kept,
                     new_lens, acc_out};
  if (evict_items(a) > fp8bs::kMaxItems) return FP8BS_ERR_SHAPE;
  if (c.batch == 0) return FP8BS_OK;
  if (!kept || !new_lens || (acc_slots > 0 && (!acc || !acc_out)) || (dst_width > 0 && !dst_table)) return FP8BS_ERR_NULL;
  if (fp8bs_status e = cache_pointers(c, true)) return e;
  if (!aligned4(acc) || !aligned4(dst_table) || !aligned4(kept) || !aligned4(new_lens) || !aligned4(acc_out))
    return FP8BS_ERR_ALIGN;
  if (fp8bs_status e = check_device()) return e;
  (void)hipGetLastError();
  return launched(fp8bs::launch_cache_evict(a, (hipStream_t)stream));
}

}  // extern "C"
