// Internal interface of the paged FP8 key/value cache kernels: launch
// arguments (host and device) and the launchers.  Arguments are checked by the
// C ABI layer; formats and rules are in include/fp8bs_cache.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace fp8bs {

// The cache and the sequences of one call, as the kernels take it.
struct CacheArgs {
  uint8_t* k;
  float* ks;
  uint8_t* v;
  float* vs;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* q_offsets;  // nullptr for the eviction
  int64_t pages;
  int64_t rows;              // packed rows of the call
  int32_t batch, width, heads;
  int32_t lg_page;           // P = 1 << lg_page
  int32_t dim;               // D
  int32_t max_new, max_kv;
};

struct AppendArgs {
  CacheArgs c;
  const void* k_new;
  const void* v_new;
  int64_t ld_new;
};

struct AttendArgs {
  CacheArgs c;
  const void* q;
  int64_t ld_q;
  int32_t q_heads, group;    // group = q_heads / heads
  float scale, softcap;
  void* out;
  float* lse;                // may be nullptr
  bool out_f32, full;
  int32_t tile_rows;         // rows per workgroup: 16 (k_attend_rows), 128 or 256 (k_attend_tiles)
  int32_t chunk, splits;     // cached tokens per split, splits
  float* part;               // [splits][rows][q_heads][D] when splits > 1
  float2* stat;              // [splits][rows][q_heads] (running max, log2 units; sum)
};

struct WeightArgs {
  CacheArgs c;
  const void* q;
  int64_t ld_q;
  int32_t q_heads, group;
  float scale, softcap;
  const float* lse;
  const float* acc_in;       // may be nullptr
  float* acc_out;
  int64_t acc_slots;
  bool full;
  int32_t splits;            // runs per (sequence, head); 0: k_weights_rows
  float* part;               // [batch][heads][splits + 256-slot tiles][256] when splits > 0
};

struct EvictArgs {
  CacheArgs c;
  const float* acc;
  int64_t acc_slots;
  const int32_t* dst_table;
  int32_t dst_width, budget, recent;
  int32_t* kept;
  int32_t* new_lens;
  float* acc_out;
};

// Work-items of the largest launch per sequence (at most kMaxItems; the ABI
// layer checks it).  Longer calls are launched in runs of sequences: a launch
// holds fewer than 2^32 work-items, and what passes that may be dropped without
// an error.
constexpr int64_t kMaxItems = ((int64_t)1 << 32) - 1;
int64_t append_items(const CacheArgs& c);
int64_t attend_items(const AttendArgs& a);
int64_t weights_items(const WeightArgs& a);
int64_t evict_items(const EvictArgs& a);

// Moves the arguments to sequences [first, first + n).
inline void take_run(CacheArgs& c, int first, int n) {
  c.table += (int64_t)first * c.width;
  c.kv_lens += first;
  if (c.q_offsets) c.q_offsets += first;
  c.batch = n;
}
inline void take_run(AppendArgs& a, int first, int n) { take_run(a.c, first, n); }
inline void take_run(AttendArgs& a, int first, int n) { take_run(a.c, first, n); }   // partial results go by row
inline void take_run(WeightArgs& a, int first, int n) {                             // each run uses the workspace anew
  take_run(a.c, first, n);
  const int64_t at = (int64_t)first * a.c.heads * a.acc_slots;
  if (a.acc_in) a.acc_in += at;
  a.acc_out += at;
}
inline void take_run(EvictArgs& a, int first, int n) {
  take_run(a.c, first, n);
  const int64_t pair = (int64_t)first * a.c.heads;
  a.acc += pair * a.acc_slots;
  a.acc_out += pair * a.acc_slots;
  a.kept += pair * a.budget;
  a.dst_table += (int64_t)first * a.dst_width;
  a.new_lens += first;
}

template <class Args, class Launch>
hipError_t launch_in_runs(const Args& a, int64_t items, Launch launch) {
  const int most = (int)std::min<int64_t>(a.c.batch, kMaxItems / std::max<int64_t>(items, 1));
  for (int first = 0; first < a.c.batch; first += most) {
    Args run = a;
    take_run(run, first, std::min(most, a.c.batch - first));
    if (hipError_t e = launch(run)) return e;
  }
  return hipSuccess;
}

// Sets tile_rows, chunk and splits from the sizes; the workspace is
// splits * rows * q_heads * (D + 2) floats when splits > 1, else none.
void attend_plan(AttendArgs& a);
int64_t attend_workspace_bytes(const AttendArgs& a);
// The same for the weights: splits, and the partial sums.
void weights_plan(WeightArgs& a);
int64_t weights_workspace_bytes(const WeightArgs& a);

hipError_t launch_cache_append(const AppendArgs& a, bool pow2, hipStream_t stream);
hipError_t launch_attend_tiles(const AttendArgs& a, int row_tiles, hipStream_t stream);
hipError_t launch_cache_attention(const AttendArgs& a, hipStream_t stream);
hipError_t launch_cache_weights(const WeightArgs& a, hipStream_t stream);
hipError_t launch_cache_evict(const EvictArgs& a, hipStream_t stream);

}  // namespace fp8bs
