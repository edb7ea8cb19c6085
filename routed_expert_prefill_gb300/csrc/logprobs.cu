// Log probabilities of given tokens, entropy and top alternatives (moe_logprobs).
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include "api_checks.cuh"

namespace cg = cooperative_groups;

namespace moe {

namespace {

constexpr int LP_THREADS = 256;
constexpr int LP_ELEMS = 16;      // elements of a thread's part of a tile
constexpr int LP_RING = 12;       // 16-byte vectors of a thread on their way or in use
constexpr int LP_GROUP = 8;       // tiles between two rankings, at most
constexpr int LP_TOP = 32;        // alternatives, at most
constexpr int LP_CAND = 512;      // candidates that wait to be ranked
constexpr int LP_GROUPS = 64;     // of threads, whose largest values bound the alternatives
constexpr int LP_CLUSTER = 8;     // CTAs of a row, at most
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float FAR = -1e30f;     // stands for -inf where it is multiplied by zero
constexpr float NOT_A_NUMBER = __builtin_nanf("");

struct LogprobParams {
  const void* logits;
  int64_t stride;
  int t, n;
  const void* ids;
  int ids64, n_ids, top;
  float* logprob;
  float* entropy;
  float* lse;
  int32_t* top_ids;
  float* top_logprobs;
};

// What is known of a set of logits: m, the largest; s = sum p and u = sum p d,
// with d = (x - m) log2(e) and p = 2^d.
struct Stats {
  float m, s, u;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The same set's s and u with respect to the larger maximum m.
__device__ __forceinline__ void rebase(Stats& a, float m) {
  const float d = fmaxf((a.m - m) * LOG2E, FAR), f = ex2(d);
  a.u = f * fmaf(d, a.s, a.u);
  a.s *= f;
  a.m = m;
}

__device__ __forceinline__ Stats join(Stats a, Stats b) {
  const float m = fmaxf(a.m, b.m);
  rebase(a, m);
  rebase(b, m);
  return {m, a.s + b.s, a.u + b.u};
}

// Larger value first, then the lower index: whole numbers in that order.
__device__ __forceinline__ uint64_t key_of(float x, int i) {
  const int b = __float_as_int(x + 0.f);  // -0 counts as 0
  return ((uint64_t)(uint32_t)(b ^ ((b >> 31) | 0x80000000)) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t k = (uint32_t)(key >> 32);
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 v, float* e) {
    e[0] = __uint_as_float(v.x), e[1] = __uint_as_float(v.y), e[2] = __uint_as_float(v.z), e[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
};
template <>
struct Vec<uint16_t> {  // bf16
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 v, float* e) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) e[2 * i] = bf16lo(w[i]), e[2 * i + 1] = bf16hi(w[i]);
  }
  static __device__ __forceinline__ float load(const uint16_t* p) { return bf16f(*p); }
};

struct Shared {
  uint64_t cand[LP_CAND];
  uint64_t best[LP_TOP];
  Stats part[LP_THREADS / 32];
  Stats all;
  float largest[LP_THREADS];
  alignas(16) float group[LP_GROUPS];
  float bound;
  float thr;  // the top-th largest value so far, once there are as many; -inf before
  int count;
  int total;
};

// Each thread copies the vectors that it reads itself, so that its own copies
// are all that it waits for.
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
               : "memory");
}
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The `top` largest of the candidates to their first places and to best, in
// order; returns how many there are.  All threads call it after a barrier;
// what it leaves is visible to all.
__device__ int rank_candidates(Shared& sh, int top) {
  const int c = sh.count, quarter = threadIdx.x & 3;
  for (int i0 = 0; i0 < c; i0 += LP_THREADS / 4) {  // four threads a candidate
    const int i = i0 + (threadIdx.x >> 2);
    const uint64_t mine = i < c ? sh.cand[i] : ~0ull;
    int rank = 0;
#pragma unroll 4
    for (int j = quarter; j < c; j += 4) rank += sh.cand[j] > mine;
    rank += __shfl_xor_sync(~0u, rank, 1);
    rank += __shfl_xor_sync(~0u, rank, 2);
    if (quarter == 0 && i < c && rank < top) sh.best[rank] = mine;
  }
  __syncthreads();
  const int kept = min(c, top);
  if (threadIdx.x < kept) sh.cand[threadIdx.x] = sh.best[threadIdx.x];
  if (threadIdx.x == 0) {
    sh.count = kept;
    if (kept == top) sh.thr = value_of(sh.best[top - 1]);
  }
  __syncthreads();
  return kept;
}

// One row by a cluster of CTAs, each of which walks every csize-th tile of it:
// memory is read once, which is what bounds the kernel where there are many
// rows; where there are few, the CTAs of a cluster share one.
//
// Sums: a thread rebases its sums where its part of a tile has a new maximum,
// so that an element costs one exponential.  Alternatives: an element becomes
// a candidate if it is above the top-th largest value so far, which a thread
// first asks of its part's maximum; after 1, 2, 4, 8, 8, ... tiles the
// candidates are ranked, which gives the next bound.  A CTA's elements come in
// ascending order, tile by tile, so that an equal value of a later group takes
// no earlier one's place.  While there are too few candidates for a bound, the
// maxima of 64 groups of threads give one: the top-th largest of them is
// reached by as many elements.  -inf never becomes a candidate; a row that has
// too few other values is filled up at the end.
//
// 2048 rows of 131072 fp32 logits, 1074 MB: 152 us without alternatives (the
// copy rate), 159 with five, 170 with twenty.  A ranking after every tile took
// 280, after every fourth 197 (three CTAs an SM).  In bf16, 537 MB (79 us at the
// copy rate), 116 and, with twenty, 170 us: the instructions, 12.2 and 19.4 a
// value, which the bytes of fp32 hide.  One row by eight CTAs: 4.6 and 9.3 us,
// the latency of its barriers.
template <typename T, bool TOP>
__global__ void __launch_bounds__(LP_THREADS, 4) logprobs_kernel(LogprobParams p, int csize) {
  __shared__ Shared sh;
  extern __shared__ uint4 ring[];  // [stage][vector][thread]
  constexpr int N = Vec<T>::N, E = LP_ELEMS, VECS = E / N, TILE = LP_THREADS * VECS, STAGES = LP_RING / VECS;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / csize, rank = blockIdx.x % csize;
  const T* x = reinterpret_cast<const T*>(p.logits) + (size_t)row * p.stride;
  // elements before the first 16-byte boundary, whole vectors, the rest
  const int head = min(p.n, (int)((16 - (uintptr_t)x % 16) % 16 / sizeof(T)));
  const int nv = (p.n - head) / N, edge = p.n - nv * N;  // edge: head and rest together, fewer than 2 N
  const uint4* body = reinterpret_cast<const uint4*>(x + head);
  const auto fetch = [&](int v0, int stage) {
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int v = v0 + j * LP_THREADS + tid;
      if (v < nv) copy16(&ring[(stage * VECS + j) * LP_THREADS + tid], body + v);
    }
    copies_end_group();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch((rank + i * csize) * TILE, i);
  float given = NOT_A_NUMBER;
  if (rank == 0 && tid < p.n_ids) {
    const size_t at = (size_t)row * p.n_ids + tid;
    const int64_t id = p.ids64 ? reinterpret_cast<const int64_t*>(p.ids)[at] : reinterpret_cast<const int32_t*>(p.ids)[at];
    if (id >= 0 && id < p.n) given = Vec<T>::load(x + id);
  }
  Stats a{-FLT_MAX, 0.f, 0.f};
  int kept = 0;          // candidates as the last ranking left them
  bool fresh = false;    // this thread has added some since
  if (TOP) {
    if (tid == 0) sh.count = 0, sh.thr = -INFINITY;
    __syncthreads();
  }

  const auto sums = [&](const float* e) {  // and the largest of a thread's part
    float lm = -INFINITY;
#pragma unroll
    for (int i = 0; i < E; ++i) lm = fmaxf(lm, e[i]);
    if (lm > a.m) rebase(a, lm);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float d = (e[i] - a.m) * LOG2E, q = ex2(d);
      a.s += q;
      a.u = fmaf(q, fmaxf(d, FAR), a.u);
    }
    return lm;
  };
  // A bound from the largest values of groups of threads.  A group's threads
  // are LP_GROUPS apart, so that a short row has values in most of them (4096
  // bf16 rows of 1000, 20 alternatives: 39 us; with 32 groups of neighbours,
  // most of them empty, the bound was -inf and all values candidates: 785).
  const auto bound = [&](float lm) {
    sh.largest[tid] = lm;
    __syncthreads();
    if (tid < LP_GROUPS) {
      float g = lm;
#pragma unroll
      for (int i = LP_GROUPS; i < LP_THREADS; i += LP_GROUPS) g = fmaxf(g, sh.largest[tid + i]);
      sh.group[tid] = g;
    }
    __syncthreads();
    constexpr int SHARE = LP_THREADS / LP_GROUPS, OTHERS = LP_GROUPS / SHARE;  // threads of a value; what each compares it with
    const int mine = tid / SHARE, j0 = tid % SHARE * OTHERS;
    const float g = sh.group[mine];
    int above = 0;
#pragma unroll
    for (int j = j0; j < j0 + OTHERS; j += 4) {
      const float4 o = *reinterpret_cast<const float4*>(sh.group + j);
      above += (o.x > g) + (o.y > g) + (o.z > g) + (o.w > g) + (o.x == g & j < mine) + (o.y == g & j + 1 < mine) +
               (o.z == g & j + 2 < mine) + (o.w == g & j + 3 < mine);
    }
#pragma unroll
    for (int o = 1; o < SHARE; o <<= 1) above += __shfl_xor_sync(~0u, above, o);
    if (tid % SHARE == 0 && above == p.top - 1) sh.bound = g;
    __syncthreads();
    return sh.bound;
  };
  const auto add = [&](float f, int index) {  // past the list's end it is dropped, but counted
    const int at = atomicAdd(&sh.count, 1);
    if (at < LP_CAND) sh.cand[at] = key_of(f, index);
    fresh = true;
  };
  const auto index_at = [&](int v0) {
    const int first = head + (v0 + tid) * N;
    return [first](int i) { return first + i / N * (LP_THREADS * N) + i % N; };
  };
  // Ranks what has come since the last ranking, tiles v0, v0 + csize * TILE, ... before v1.
  const auto settle = [&](int v0, int v1) {
    if (!__syncthreads_or(fresh)) return;
    fresh = false;
    if (sh.count <= LP_CAND) {
      kept = rank_candidates(sh, p.top);
      return;
    }
    // More than the list holds.  The tiles are read again, one by one: a
    // tile's top-th largest key is found bit by bit, and those from it on are
    // candidates.
    for (int v = v0; v < v1; v += csize * TILE) {
      const auto index = index_at(v);
      const auto element = [&](int i) {
        const int at = v + i / N * LP_THREADS + tid;
        return at < nv ? Vec<T>::load(x + index(i)) : -INFINITY;
      };
      uint64_t low = 0;
      for (int bit = 63; bit >= 0; --bit) {
        __syncthreads();
        if (tid == 0) sh.total = 0, sh.count = kept;
        __syncthreads();
        const uint64_t key = low | (uint64_t)1 << bit;
        int c = 0;
#pragma unroll 1
        for (int i = 0; i < E; ++i) {
          const float f = element(i);
          c += f > -INFINITY && key_of(f, index(i)) >= key;
        }
        c = __reduce_add_sync(~0u, c);
        if (lane == 0 && c) atomicAdd(&sh.total, c);
        __syncthreads();
        if (sh.total >= p.top) low = key;
      }
#pragma unroll 1
      for (int i = 0; i < E; ++i) {
        const float f = element(i);
        if (f > -INFINITY && key_of(f, index(i)) >= low) sh.cand[atomicAdd(&sh.count, 1)] = key_of(f, index(i));
      }
      __syncthreads();
      kept = rank_candidates(sh, p.top);
    }
  };

  int stage = 0, group = 0, length = 1, first_v = rank * TILE;
  float thr = -INFINITY;
  for (int v0 = rank * TILE; v0 < nv; v0 += csize * TILE) {
    copies_wait<STAGES - 2>();
    float e[E];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      if (v0 + j * LP_THREADS + tid < nv) {
        Vec<T>::unpack(ring[(stage * VECS + j) * LP_THREADS + tid], e + j * N);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) e[j * N + i] = -INFINITY;
      }
    }
    const float lm = sums(e);
    const T* part = reinterpret_cast<const T*>(ring + stage * VECS * LP_THREADS);
    fetch(v0 + (STAGES - 1) * csize * TILE, (stage + STAGES - 1) % STAGES);
    stage = (stage + 1) % STAGES;
    if (!TOP) continue;
    if (group == 0) thr = sh.thr;
    const bool loose = thr == -INFINITY;  // the same for the whole CTA
    const float least = loose ? bound(lm) : thr;
    if (lm > -INFINITY && (lm > least || (loose && lm == least))) {
      const auto index = index_at(v0);
      uint32_t which = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) which |= (uint32_t)(e[i] > least || (loose && e[i] == least && e[i] > -INFINITY)) << i;
      for (; which; which &= which - 1) {  // one at a time, read again: few threads have any
        const int i = __ffs(which) - 1;
        add(Vec<T>::load(part + (i / N * LP_THREADS + tid) * N + i % N), index(i));
      }
    }
    if (loose || ++group == length || v0 + csize * TILE >= nv) {
      settle(first_v, v0 + 1);
      if (!loose && length < LP_GROUP) length *= 2;
      group = 0;
      first_v = v0 + csize * TILE;
    }
  }
  if (rank == 0 && edge) {
    const int at = tid < head ? tid : p.n - edge + tid;
    float e[E];
#pragma unroll
    for (int i = 0; i < E; ++i) e[i] = -INFINITY;
    if (tid < edge) e[0] = Vec<T>::load(x + at);
    sums(e);
    if (TOP) {
      if (e[0] > -INFINITY && e[0] >= sh.thr) add(e[0], at);  // too few to overflow the list
      settle(0, 0);
    }
  }

  // the CTA's sums, then the cluster's
#pragma unroll
  for (int o = 16; o; o >>= 1)
    a = join(a, {__shfl_xor_sync(~0u, a.m, o), __shfl_xor_sync(~0u, a.s, o), __shfl_xor_sync(~0u, a.u, o)});
  if (lane == 0) sh.part[warp] = a;
  __syncthreads();
  a = sh.part[0];
#pragma unroll
  for (int i = 1; i < LP_THREADS / 32; ++i) a = join(a, sh.part[i]);
  if (csize > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    if (tid == 0) sh.all = a;
    cluster.sync();
    uint64_t far = 0;
    if (rank == 0) {
      for (int i = 1; i < csize; ++i) a = join(a, *cluster.map_shared_rank(&sh.all, i));
      if (TOP && tid < csize * p.top) {
        const int who = tid / p.top, nth = tid % p.top;
        if (nth < *cluster.map_shared_rank(&sh.count, who)) far = cluster.map_shared_rank(sh.best, who)[nth];
      }
    }
    cluster.sync();
    if (rank != 0) return;
    if (TOP) {
      if (tid == 0) sh.count = 0;
      __syncthreads();
      if (far) sh.cand[atomicAdd(&sh.count, 1)] = far;
      __syncthreads();
      kept = rank_candidates(sh, p.top);
    }
  }
  const float ln_s = logf(a.s);
  const bool whole = a.s == a.s;  // false where the row holds +inf or NaN
  if (tid < p.n_ids) p.logprob[(size_t)row * p.n_ids + tid] = (given - a.m) - ln_s;
  if (tid == 0) {
    const float h = ln_s - LN2 * (a.u / a.s);
    if (p.lse) p.lse[row] = a.m + ln_s;
    if (p.entropy) p.entropy[row] = h < 0.f ? 0.f : h;
  }
  if (!TOP) return;
  const size_t to = (size_t)row * p.top;
  if (!whole) {
    if (tid < p.top) p.top_ids[to + tid] = -1, p.top_logprobs[to + tid] = NOT_A_NUMBER;
  } else if (tid < kept) {
    p.top_ids[to + tid] = ~(uint32_t)sh.best[tid];
    p.top_logprobs[to + tid] = (value_of(sh.best[tid]) - a.m) - ln_s;
  } else if (tid == kept) {  // -inf, the lowest indices first
    for (int i = kept, id = 0; i < p.top; ++id) {
      bool taken = false;
      for (int j = 0; j < kept; ++j) taken |= (uint32_t)id == ~(uint32_t)sh.best[j];
      if (taken) continue;
      p.top_ids[to + i] = id;
      p.top_logprobs[to + i++] = -INFINITY - ln_s;
    }
  }
}

constexpr int LP_RING_BYTES = LP_RING * LP_THREADS * 16;

template <typename T, bool TOP>
cudaError_t launch_logprobs(const LogprobParams& p, int csize, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.t * csize);
  cfg.blockDim = dim3(LP_THREADS);
  cfg.dynamicSmemBytes = LP_RING_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = csize;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = csize > 1 ? 2 : 1;
  cudaError_t e = set_smem_limit_once(logprobs_kernel<T, TOP>, LP_RING_BYTES);
  if (e != cudaSuccess) return e;
  MOE_LAUNCH("logprobs", s, { e = cudaLaunchKernelEx(&cfg, logprobs_kernel<T, TOP>, p, csize); });
  return e;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_logprobs(const void* logits, int64_t stride, int32_t logits_fp32, int32_t t, int32_t n, const void* ids,
                            int32_t ids_int64, int32_t n_ids, int32_t top, float* logprob, float* entropy, float* lse,
                            int32_t* top_ids, float* top_logprobs, void* stream) {
  if (t < 1 || t > 65536) return set_error(MOE_ESHAPE, "t=%d outside [1, 65536]", t);
  if (n < 1 || n > 1048576) return set_error(MOE_ESHAPE, "n=%d outside [1, 1048576]", n);
  if (stride < 0) return set_error(MOE_ESHAPE, "the row stride must not be negative");
  if (n_ids < 0 || n_ids > LP_THREADS) return set_error(MOE_ESHAPE, "n_ids=%d outside [0, %d]", n_ids, LP_THREADS);
  if (top < 0 || top > LP_TOP || top > n)
    return set_error(MOE_ESHAPE, "top=%d outside [0, %d]", top, n < LP_TOP ? n : LP_TOP);
  TRY(check_ptr(logits, "logits", logits_fp32 ? 4 : 2));
  TRY(check_ptr(ids, "ids", ids_int64 ? 8 : 4, n_ids == 0));
  TRY(check_ptr(logprob, "logprob", 4, n_ids == 0));
  TRY(check_ptr(entropy, "entropy", 4, true));
  TRY(check_ptr(lse, "lse", 4, true));
  TRY(check_ptr(top_ids, "top_ids", 4, top == 0));
  TRY(check_ptr(top_logprobs, "top_logprobs", 4, top == 0));
  const LogprobParams p{logits, stride, t, n, ids, ids_int64, n_ids, top, logprob, entropy, lse, top_ids, top_logprobs};
  // CTAs of a row: as many as leave every SM two, while each has a tile
  const int tile = LP_THREADS * LP_ELEMS;
  int csize = 1;
  while (csize < LP_CLUSTER && (int64_t)t * csize * 2 <= 2 * sm_count() && (int64_t)n >= 2 * csize * tile) csize *= 2;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = logits_fp32 ? (top ? launch_logprobs<float, true>(p, csize, s) : launch_logprobs<float, false>(p, csize, s))
                                    : (top ? launch_logprobs<uint16_t, true>(p, csize, s)
                                           : launch_logprobs<uint16_t, false>(p, csize, s));
  return cuda_status(e, "moe_logprobs launch");
}
