// What the cache's append and attention kernels share (internal).
#pragma once
#include "common.cuh"

namespace moe {

// Workspace of both calls: the status block, the completion counters of the
// split attention items (three a CTA; of the tile kernel's one CTA an SM,
// eight), their partial results.
constexpr int KV_CTAS_PER_SM = 3;  // at most, of the streaming kernels
constexpr int KV_ROWS = 16;        // rows of a query tile, at most

inline int kv_grid_max() { return sm_count() * KV_CTAS_PER_SM; }
inline size_t kv_counter_off() { return sizeof(DeviceStatus); }
inline size_t kv_partial_off() { return align_up(kv_counter_off() + (size_t)kv_grid_max() * 3 * 4, 256); }
// A partial result: for each row its score maximum, its maximum of score less
// that + log2(value scale), its sum and d accumulators.
__host__ __device__ constexpr size_t kv_partial_floats(int d) { return (size_t)KV_ROWS * (d + 4); }
size_t kv_tile_partial_bytes(int d);  // kv_attention_tile.cu
inline size_t kv_ws_bytes(int d) {
  const size_t stream = (size_t)kv_grid_max() * 2 * kv_partial_floats(d) * 4, tile = kv_tile_partial_bytes(d);
  return kv_partial_off() + (stream > tile ? stream : tile);
}

// One sequence's part of a call, checked: n new rows from `row`, `len` tokens
// in all.  False (and a flag) when starts or lens are out of range.
__device__ __forceinline__ bool kv_sequence(const moe_kv_cache& c, const int32_t* starts, int t, int s, int& row,
                                            int& n, int& len) {
  const int a = starts[s], b = starts[s + 1];
  len = c.lens[s];
  row = a;
  n = b - a;
  return a >= 0 && b >= a && b <= t && len >= n && len <= (int64_t)c.max_blocks * c.block;
}

}  // namespace moe
