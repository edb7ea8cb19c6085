// What the two attention kernels over the 8-bit cache share (internal).
#pragma once
#include "kv_common.cuh"

namespace moe {

constexpr int UNIT = 128;  // tokens of a unit of work

struct AttnParams {
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* starts;
  int t, hq, G;       // G query heads read one key/value head
  float scale_log2;   // scale * log2(e)
  int block_log2;
  moe_kv_cache c;
  uint16_t* out;
  DeviceStatus* st;
  uint32_t* counters;
  float* partials;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct Seq {
  int row, n, len;
  bool ok;
};

__device__ __forceinline__ Seq load_seq(const AttnParams& p, int s) {
  Seq q;
  q.ok = kv_sequence(p.c, p.starts, p.t, s, q.row, q.n, q.len);
  if (!q.ok) q.n = 0;
  return q;
}
// Rows of a sequence's new tokens: below 2^32 (t <= 65536, hq < 65536).
__device__ __forceinline__ uint32_t seq_rows(const AttnParams& p, const Seq& q) { return (uint32_t)q.n * p.G; }

template <int ROWS>
__device__ __forceinline__ int q_tiles(const AttnParams& p, const Seq& q) {
  return (int)((seq_rows(p, q) + (uint64_t)(ROWS - 1)) / ROWS);
}
// Positions that the rows of query tile qt see, and its units.
template <int ROWS>
__device__ __forceinline__ int tile_seen(const AttnParams& p, const Seq& q, int qt) {
  const uint32_t rows = (uint32_t)min((uint64_t)seq_rows(p, q), (uint64_t)ROWS * (qt + 1));
  return q.len - q.n + (int)((rows - 1) / (uint32_t)p.G) + 1;
}
template <int ROWS>
__device__ __forceinline__ int tile_units(const AttnParams& p, const Seq& q, int qt) {
  return (tile_seen<ROWS>(p, q, qt) + UNIT - 1) / UNIT;
}
template <int ROWS, int EXTRA>
__device__ __forceinline__ int64_t seq_units(const AttnParams& p, const Seq& q) {
  int64_t w = 0;
  for (int qt = 0, m = q_tiles<ROWS>(p, q); qt < m; ++qt) w += EXTRA + tile_units<ROWS>(p, q, qt);
  return w * p.c.hkv;
}

// A CTA's run of units.  The work is the list of all (sequence, query tile of
// ROWS rows, key/value head) items in this order, each as many units of 128
// tokens as its rows see, after EXTRA units that stand for what an item costs
// whatever its length; CTA c of `ctas` takes units x0 .. x1 - 1 of the
// `total`, starting with unit u (EXTRA ones counted) of item (s, qt, h).
struct Work {
  int64_t total, ctas, x0, x1;
  int s, qt, h, u;
};

// a * b / c, in 32 bits where they hold the product: a 64-bit division takes
// some hundred instructions, and a CTA needs several before its first load.
__device__ __forceinline__ int64_t mul_div(int64_t a, int64_t b, int64_t c) {
  if (((a | b) >> 16) == 0 && (c >> 32) == 0) return (uint32_t)a * (uint32_t)b / (uint32_t)c;
  return a * b / c;
}

// The CTA that takes unit x: the last c with total * c / ctas <= x.
__device__ __forceinline__ int cta_of(const Work& w, int64_t x) {
  if (((x + 1) | w.total) >> 20 == 0 && w.ctas < 4096)
    return (int)(((uint32_t)(x + 1) * (uint32_t)w.ctas - 1) / (uint32_t)w.total);
  return (int)(((x + 1) * w.ctas - 1) / w.total);
}

// Called by all THREADS threads; scratch: THREADS / 32 + 2 values in shared
// memory.  False where the CTA has nothing to do.
template <int ROWS, int THREADS, int EXTRA = 0>
__device__ __forceinline__ bool find_work(const AttnParams& p, int64_t* scratch, Work& wk) {
  constexpr int WARPS = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t total = 0, w0 = 0;
  for (int s = tid; s < p.c.n_seq; s += THREADS) {
    const Seq q = load_seq(p, s);
    if (!q.ok && blockIdx.x == 0) raise_flag(p.st, FLAG_BAD_CACHE);
    const int64_t w = seq_units<ROWS, EXTRA>(p, q);
    if (s == tid) w0 = w;
    total += w;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
  if (lane == 0) scratch[warp] = total;
  __syncthreads();
  total = 0;
  for (int i = 0; i < WARPS; ++i) total += scratch[i];
  wk.total = total;
  wk.ctas = min((int64_t)gridDim.x, total);
  if (blockIdx.x >= wk.ctas) return false;
  wk.x0 = mul_div(total, blockIdx.x, wk.ctas);
  wk.x1 = mul_div(total, blockIdx.x + 1, wk.ctas);
  int64_t base = 0;
  for (int sb = 0; sb < p.c.n_seq; sb += THREADS) {
    int64_t w = w0;
    if (sb) w = sb + tid < p.c.n_seq ? seq_units<ROWS, EXTRA>(p, load_seq(p, sb + tid)) : 0;
    int64_t incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += u;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int64_t all = 0;
    for (int i = 0; i < WARPS; ++i) {
      if (i < warp) incl += scratch[i];
      all += scratch[i];
    }
    if (wk.x0 < base + all) {
      if (base + incl - w <= wk.x0 && wk.x0 < base + incl) {
        scratch[WARPS] = sb + tid;
        scratch[WARPS + 1] = base + incl - w;
      }
      break;
    }
    base += all;
  }
  __syncthreads();
  wk.s = (int)scratch[WARPS];
  const Seq q = load_seq(p, wk.s);
  int64_t off = wk.x0 - scratch[WARPS + 1];
  for (wk.qt = 0;; ++wk.qt) {
    const int units = EXTRA + tile_units<ROWS>(p, q, wk.qt);
    if (off < (int64_t)units * p.c.hkv) {
      if (off >> 31) {
        wk.h = (int)(off / units);
      } else {
        wk.h = (int)((uint32_t)off / (uint32_t)units);
      }
      wk.u = (int)(off - (int64_t)wk.h * units);
      return true;
    }
    off -= (int64_t)units * p.c.hkv;
  }
}

// Kernels for many rows a sequence (kv_attention_tile.cu).
cudaError_t launch_tile(const AttnParams& p, cudaStream_t s);

}  // namespace moe
