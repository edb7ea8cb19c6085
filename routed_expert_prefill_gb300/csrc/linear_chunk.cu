// Linear attention of many rows a sequence (moe_linear_attention) on the
// tensor cores' own path: chunks of 128 rows, accumulators in TMEM.
#include <math.h>

#include <initializer_list>

#include "linear_common.cuh"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr int CHUNK = 128;
// Warps: 0-7 compute, 8 issues the products, 9 works out the decays, 10 brings
// the tiles, 11 takes the results away.  Registers: 384 * 168 at launch, 256 *
// 208 + 128 * 88 after the split.
constexpr int LC_COMPUTE = 256, LC_THREADS = 384, W_ISSUE = 8, W_GAIN = 9, W_LOAD = 10, W_STORE = 11;
constexpr int LC_REGS = 208, LC_REGS_REST = 88;
constexpr uint64_t LC_WAIT_NS = 2000000000ull;
constexpr float LOG2E = 1.44269502f, LOG2E_REST = 1.92596299e-8f, LN2 = 0.693147181f;
constexpr float NOT_A_NUMBER = __builtin_nanf("");
// A row's log2 decay as it counts: below it the state of one row is 0 in the
// next whatever it was (2^-512 of an fp32 number).
constexpr float LEAST = -512.f;
// How far a key's factor may go above 1 (log2): beside scores and values, far
// from the end of fp32's range; what passes it all the same is worked out again.
constexpr float MILD = 40.f;

// What one CTA leaves for those that go on with its last chain: the state
// behind its part (or, if its part does not begin the chain, what the part
// adds) in the order in which its threads hold it, and the part's decay.
constexpr int PUB_EXTRA = 64;  // floats behind the state: the decay's factor, as Gains' keep and slow
__host__ __device__ constexpr size_t pub_floats(int d) { return (size_t)d * d + PUB_EXTRA; }

// Behind the status block of the workspace.
struct LinearSync {
  uint32_t done;  // CTAs that have finished; the last one clears all of this
  uint32_t pad[63];
};

struct ChunkParams {
  LinearParams p;
  LinearSync* sync;
  uint32_t* flags;  // [CTAs]: its part is published
  float* pub;       // [CTAs][pub_floats]
};

// Chunks c0 .. c1 - 1 of the nc of one sequence and head.  full: with its
// results, else only what it adds to a state of zero.
struct Part {
  int s, head, c0, c1, nc;
  int row, n, slot_in, slot_out;
  bool full;
};

// What the warps need to know of a chunk.
struct Ticket {
  int row, rows;          // its first row, how many it has
  int head;
  int slot_in, slot_out;  // of the part
  int before;             // chunks of the chain before the part
  bool full;
  bool begins, ends;      // the part
  int stage;              // of the walk: 0 the part is published, 1 a whole chain, 2 others began it
  bool closes;            // the part ends its chain
  bool on;                // there is a chunk
};

// Log2 decays as whole numbers of 2^-40: their sums and differences are exact.
constexpr float UNIT = 0x1p40f, PER_UNIT = 0x1p-40f;
// A part's decay as it counts: below it, it is 0.
constexpr long long PART_LEAST = -(1ll << 52);

// A state is multiplied by keep + slow = 2^g, slow 1 where the decay is slow:
// 2^g rounded to fp32 would be off by the same 2^-25 for every chunk.  (A
// function of its own: inlined at both places it made all chunks slower.)
__device__ __noinline__ void factor_of(float g, float& keep, float& slow) {
  const bool is_slow = g > -0.5f;
  keep = is_slow ? expm1f(g * LN2) : exp2f(g);
  slow = is_slow ? 1.f : 0.f;
}

// The decays of a chunk's rows: G_i is the log2 of the product of rows 0 .. i's.
struct alignas(16) Gains {  // read four at a time
  // with R_i = G_i less that of the first of its 32 rows: 2^-R_i where none of
  // the 32 is above 2^MILD (bit i / 32 of mild), else R_i
  float own[CHUNK];
  float last[CHUNK];   // 2^(G_127 - G_i)
  float first[CHUNK];  // 2^G_i
  float off[192];      // rows 32 q .. of q = 1, 2, 3, for i < 32 q: 2^(G_32q - G_i)
  long long end;       // G_127 in whole numbers of 2^-40
  uint32_t mild;
  float keep, slow;    // a state is multiplied by keep + slow = 2^G_127; slow is 1 for slow decays, else 0
};

struct LcShared {
  uint64_t t_full, qk_full[2], v_full, g_full, g_empty;
  uint64_t qk_done, sq_done, pv_done, ds_done;  // products
  uint64_t s_ready, p_ready, k_ready, o_ready;  // their operands, and the results
  uint64_t q_free;                              // the results have been read
  uint64_t met;                                 // the compute warps, all of them
  uint64_t drain;
  Gains g;
  Part first, last;  // the chains of the CTA's first and last chunk
  Ticket begin, next[2];  // for the compute warps: the first chunk, that behind the one at work
  int scan[LC_THREADS / 32];
  int total, longest;
  uint32_t tmem;
  int abort;  // 0, or the wait that gave up
};

template <int D>
struct Lc {
  static constexpr int TILE = CHUNK * D * 2;           // bytes of q, k or v of a chunk
  static constexpr int HALF = CHUNK * 128;             // a tile's 64 channels
  static constexpr int S_HALF = D * 128;               // the same of a state in bf16
  static constexpr int S_PART = D * D * 2;             // one part of a state in bf16
  static constexpr int Q0 = 0, K0 = 2 * TILE, V0 = 4 * TILE, X0 = 5 * TILE;
  static constexpr int TILES = 7 * TILE;
  static constexpr int TOTAL = TILES + (int)sizeof(LcShared);
  static constexpr int NC = D * D / LC_COMPUTE;        // values of the state a thread holds
  // TMEM columns: scores (then weights), state times queries, weights times values, what the chunk adds
  static constexpr int T_S = 0, T_SQ = 128, T_PV = 128 + D, T_DS = 128 + 2 * D;
};
static_assert(Lc<128>::TOTAL <= 227 * 1024, "shared memory of a CTA");
// CTAs wait for one another's states; two calls that run at once must not also
// wait for one another's tensor memory, so no SM has room for two CTAs.
static_assert(2 * (Lc<64>::TOTAL + 1024) > 228 * 1024, "one CTA an SM");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory descriptor of an operand whose rows are the product's inner
// dimension: 64 values of the outer one in 128 swizzled bytes, 8-row groups
// 1024 bytes apart, the next 64 values `outer` bytes on.
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t outer) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(outer >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor with either operand's rows as the inner dimension.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool a_rows, bool b_rows) {
  return idesc_bf16(M, N) | ((uint32_t)a_rows << 15) | ((uint32_t)b_rows << 16);
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* tm, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(tm), "r"(x), "r"(y),
               "r"(smem_u32(src))
               : "memory");
}

// One column of the warp's lanes, waited for.
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\ntcgen05.wait::ld.sync.aligned;" : "=r"(r) : "r"(taddr) : "memory");
}

__device__ __forceinline__ float2 pair(const uint32_t* r) { return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1])); }

// Two values as a bf16 pair, rounded; what is left of them takes their place.
__device__ __forceinline__ uint32_t take_rounded(float2& v) {
  const uint32_t w = pack_bf16x2(v.x, v.y);
  v = fma2(make_float2(bf16lo(w), bf16hi(w)), both(-1.f), v);
  return w;
}
// The same, cut to 8 bits: after two of these 8 are left, so that three parts are the value.
__device__ __forceinline__ uint32_t cut(float2 v) { return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632); }
__device__ __forceinline__ uint32_t take_cut(float2& v) {
  const uint32_t w = cut(v);
  v = fma2(make_float2(__uint_as_float(__float_as_uint(v.x) & 0xFFFF0000u), __uint_as_float(__float_as_uint(v.y) & 0xFFFF0000u)),
           both(-1.f), v);
  return w;
}

// A thread's values of a state, 32 bytes at a time (where they begin at a
// multiple of that): a warp's lanes hold different rows, and with 16 each
// sector would be asked for twice, with more of them on their way than L1 holds.
template <int N>
__device__ __forceinline__ void load_state(float (&S)[N], const float* from) {
  if ((uintptr_t)from % 32 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(S[i]), "=f"(S[i + 1]), "=f"(S[i + 2]), "=f"(S[i + 3]), "=f"(S[i + 4]), "=f"(S[i + 5]), "=f"(S[i + 6]),
                     "=f"(S[i + 7])
                   : "l"(from + i)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(from + i);
      S[i] = v.x, S[i + 1] = v.y, S[i + 2] = v.z, S[i + 3] = v.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void store_state(float* to, const float (&S)[N]) {
  if ((uintptr_t)to % 32 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + i), "f"(S[i]), "f"(S[i + 1]),
                   "f"(S[i + 2]), "f"(S[i + 3]), "f"(S[i + 4]), "f"(S[i + 5]), "f"(S[i + 6]), "f"(S[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
  }
}

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Chunks of one head of a sequence; one without rows has one, if its state
// moves to another slot.  0 (and a flag) where starts or slots are out of range.
__device__ __forceinline__ int chunks_of(const LinearParams& p, int s, bool report) {
  int row, n, in, out;
  if (!linear_sequence(p, s, row, n, in, out)) {
    if (report) raise_flag(p.st, FLAG_BAD_STATE);
    return 0;
  }
  return n ? (n + CHUNK - 1) / CHUNK : in != out && out >= 0;
}

__device__ __forceinline__ Part part_of(const LinearParams& p, int s, int head) {
  Part t;
  t.s = s;
  t.head = head;
  linear_sequence(p, s, t.row, t.n, t.slot_in, t.slot_out);
  t.c0 = 0;
  t.c1 = t.nc = t.n ? (t.n + CHUNK - 1) / CHUNK : 1;  // of a sequence that has any
  t.full = true;
  return t;
}

// Another head's whole chain of the same sequence.
__device__ __forceinline__ Part chain_of(Part t, int head) {
  t.head = head;
  t.c0 = 0;
  t.c1 = t.nc;
  t.full = true;
  return t;
}

// A walk over the chunks of a CTA's run, part by part: first the part that
// other CTAs go on with, so that they need not wait long (inside a chain: what
// it adds); then whole chains; last the part that others began.
struct Walk {
  Part t;
  int c;      // the chunk, if any is left
  int stage;  // of t; 3: none left
  int s, head;
  bool left;  // (s, head) has not been looked at

  __device__ __forceinline__ void begin(const LinearParams& p, const LcShared& sh) {
    s = sh.first.s;
    head = sh.first.head;
    left = true;
    stage = 0;
    if (sh.last.c1 < sh.last.nc) {
      t = sh.last;
      t.full = t.c0 == 0;
      c = t.c0;
    } else {
      next_part(p, sh);
    }
  }
  __device__ __forceinline__ void next_part(const LinearParams& p, const LcShared& sh) {
    while (stage < 2 && left) {
      const bool is_last = s == sh.last.s && head == sh.last.head;
      bool whole;
      if (s == sh.first.s && head == sh.first.head) {
        t = sh.first;
        whole = t.c0 == 0 && t.c1 == t.nc;
      } else {
        if (is_last)
          t = sh.last;
        else if (s == sh.first.s || s == sh.last.s)
          t = chain_of(s == sh.first.s ? sh.first : sh.last, head);
        else
          t = part_of(p, s, head);
        whole = t.c1 == t.nc;
      }
      if (is_last) {
        left = false;
      } else if (++head == p.hv) {
        head = 0;
        do ++s;
        while (s != sh.last.s && chunks_of(p, s, false) == 0);
      }
      if (whole) {
        stage = 1;
        c = t.c0;
        return;
      }
    }
    if (stage < 2 && sh.first.c0 > 0) {
      t = sh.first;
      stage = 2;
      c = t.c0;
    } else {
      stage = 3;
    }
  }
  __device__ __forceinline__ void next(const LinearParams& p, const LcShared& sh) {
    if (++c == t.c1) next_part(p, sh);
  }
  __device__ __forceinline__ bool more() const { return stage < 3; }
  __device__ __forceinline__ Ticket ticket() const {
    return {t.row + c * CHUNK, min(CHUNK, t.n - c * CHUNK), t.head, t.slot_in, t.slot_out, t.c0, t.full, c == t.c0, c + 1 == t.c1,
            stage, t.c1 == t.nc, stage < 3};
  }
};

// sum_(j <= i) w_ij (q_i . k_j) v_j of one row and channel, for those whose
// products over the chunk met a value that is not finite.
__device__ __noinline__ float weighted_values(const LinearParams& p, int d, int row0, int i, int head, int channel) {
  const int hk = head / (p.hv / p.hk);
  const uint16_t* q = p.q + (size_t)(row0 + i) * p.q_stride + hk * d;
  float sum = 0.f, w = 1.f;
  for (int j = i; j >= 0; --j) {
    const uint16_t* k = p.k + (size_t)(row0 + j) * p.k_stride + hk * d;
    float z = 0.f;
    for (int c = 0; c < d; ++c) z = fmaf(bf16f(q[c]), bf16f(k[c]), z);
    sum = fmaf(z * w, bf16f(p.v[(size_t)(row0 + j) * p.v_stride + head * d + channel]), sum);
    if (!isfinite(sum)) break;
    w *= expf(decay_of(p.log_decay[(size_t)(row0 + j) * p.decay_stride + head]));
  }
  return sum;
}

// The list of all chunks (sequence by sequence, head by head) is cut into
// equal runs, one a CTA.  Over a chunk of 128 rows, with G_i as in Gains,
//
//   out_i = scale * (2^G_i q_i S + sum_(j <= i) 2^(G_i - G_j) (q_i . k_j) v_j)
//   S <- 2^G_127 S + sum_j 2^(G_127 - G_j) k_j v_j^T,
//
// four products of 128 rows.  Operands that are not bf16 to begin with are
// taken in parts: the weights and the state, for results that are rounded to
// bf16, in two (2^-17 of each); the keys times their decays, which enter the
// state, in three (2^-25).  The state stays in fp32 registers and is added to
// there, since the tensor cores' sums may cut where fp32 rounds.
//
// A chain that is cut is joined through L2: each CTA works out the part that
// others go on with first, and the part that others began last.  Where a
// whole run lies inside a chain, what it adds is worked out first, without
// results.
//
// What bounds it (D = 128): a chunk takes some 9000 clocks.  Its 64 products
// of 128 x 128 x 16 take 6500 (100 each beside the conversions' traffic, 66
// alone) and shared memory moves 800 KB, 6300 clocks' worth, more than half of
// it the products' operands; the conversions (weights, keys in three parts, the
// state in two) are as long as the products and overlap with them in part:
// queries times state beside the weights, weights times values beside the
// keys, keys times values beside the results.  A chunk's code is run once a
// chunk and fetched as often, so that short loops beat unrolled ones.  Six
// prompts of 13355 rows and 32 heads, 355 MB: 127 us, 0.41 of the copy rate; of
// heads of 64, 93 us.  Slower: 16 compute warps of 96 registers, the keys' parts
// in bf16 arithmetic, keys converted in halves with the first one's products
// beside the second, queries in TMEM for both of their products, loops over 32
// keys and results instead of 16 (138; heads of 64: 107), a chunk's code
// unrolled (180 KB; 208).
template <int D>
__global__ void __launch_bounds__(LC_THREADS, 1)
    linear_chunk_kernel(const __grid_constant__ ChunkParams cp, const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_o) {
  using L = Lc<D>;
  constexpr int NC = L::NC;
  extern __shared__ __align__(1024) unsigned char smem[];
  LcShared& sh = *reinterpret_cast<LcShared*>(smem + L::TILES);
  const LinearParams& p = cp.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();

  if (warp == W_ISSUE) {
    tmem_alloc(&sh.tmem, 512);
    if (lane == 0) {
      for (uint64_t* b : {&sh.t_full, &sh.qk_full[0], &sh.qk_full[1], &sh.v_full, &sh.g_full, &sh.qk_done, &sh.sq_done, &sh.pv_done,
                          &sh.ds_done, &sh.drain, &sh.q_free})
        mbar_init(b, 1);
      for (uint64_t* b : {&sh.g_empty, &sh.s_ready, &sh.p_ready, &sh.k_ready, &sh.o_ready, &sh.met}) mbar_init(b, LC_COMPUTE / 32);
      fence_mbar_init();
      sh.abort = 0;
    }
  }

  // ---- the CTA's run
  int own_chunks = 0;  // of the thread's first sequence
  {
    int total = 0, longest = 0;
    for (int s = tid; s < p.n_seq; s += LC_THREADS) {
      const int c = chunks_of(p, s, blockIdx.x == 0);
      if (s == tid) own_chunks = c;
      total += c;
      longest = max(longest, c);
    }
    total = __reduce_add_sync(~0u, total);
    longest = __reduce_max_sync(~0u, longest);
    if (tid == 0) sh.total = sh.longest = 0;
    __syncthreads();
    if (lane == 0) {
      atomicAdd(&sh.total, total);
      atomicMax(&sh.longest, longest);
    }
    __syncthreads();
  }
  const int64_t all = (int64_t)sh.total * p.hv;
  // Equal runs, but none so short that joining a chain's runs (a state from L2
  // each) takes longer than the runs do (a twentieth against a twelfth, caches
  // cold: 2000 rows of a head of 128 in 38 us against 41, 8191 rows of four such
  // heads in 65 against 59, of heads of 64 in 43 against 42).
  // A chain little longer than a run is not worth a cut, since a run inside it
  // is passed twice (seven prompts of 5741, 16 heads of 64: 203 us with 34 chunks
  // a run, 159 with a chain's 45; of heads of 128 259 and 207; but two prompts of
  // 3108, 32 heads, 25 chunks a chain: 110 with 11 a run, 122 uncut).
  int64_t run = max((all + gridDim.x - 1) / gridDim.x, (int64_t)ceilf(sqrtf(sh.longest / 20.f)));
  if (sh.longest <= 1.6f * run) run = max(run, (int64_t)sh.longest);
  const int64_t a = run * blockIdx.x, b = min(a + run, all);
  const uint32_t tmem = sh.tmem;
  if (a < b) {
    int before = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += LC_THREADS) {
      const int s = s0 + tid, c = s0 == 0 ? own_chunks : s < p.n_seq ? chunks_of(p, s, false) : 0;
      int in = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(~0u, in, o);
        if (lane >= o) in += u;
      }
      __syncthreads();
      if (lane == 31) sh.scan[warp] = in;
      __syncthreads();
      int base = before;
      for (int i = 0; i < LC_THREADS / 32; ++i) {
        if (i < warp) base += sh.scan[i];
        before += sh.scan[i];
      }
      const int64_t lo = (int64_t)(base + in - c) * p.hv, hi = lo + (int64_t)c * p.hv;
      if (lo <= a && a < hi) {
        const int off = (int)(a - lo);
        Part t = part_of(p, s, off / c);
        t.c0 = off % c;
        t.c1 = (int)min((int64_t)c, t.c0 + (b - a));
        sh.first = t;
      }
      if (lo < b && b <= hi) {
        const int off = (int)(b - 1 - lo);
        Part t = part_of(p, s, off / c);
        t.c0 = (int)max((int64_t)0, a - lo - (int64_t)t.head * c);
        t.c1 = off % c + 1;
        sh.last = t;
      }
    }
  }
  __syncthreads();
  tc_fence_after();

  volatile int* abort = &sh.abort;
  // A bounded wait, for whole warps: one goes on or gives up as one.  `site` is reported at the end.
  const auto wait = [&](uint64_t* bar, uint32_t& phase, int site) {
    bool ok = __all_sync(~0u, mbar_try_wait(bar, phase));
    if (!ok) {
      const uint64_t t0 = globaltimer();
      do ok = __all_sync(~0u, mbar_try_wait_sleep(bar, phase, 200000u));
      while (!ok && !__any_sync(~0u, *abort || globaltimer() - t0 > LC_WAIT_NS));
      if (!ok && !*abort) *abort = site;
    }
    phase ^= 1;
    return ok;
  };

  if (warp >= W_ISSUE) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LC_REGS_REST));
    if (warp == W_ISSUE && a < b) {
      // ---- products
      const uint32_t sb = smem_u32(smem);
      // descriptors: tiles of queries and keys with channels as the inner dimension, of keys, values and states with rows
      constexpr uint32_t BUF = L::TILE >> 4, ROWS16 = 2048 >> 4;
      const uint64_t qd = desc_sw128(sb + L::Q0), kd = desc_sw128(sb + L::K0);
      // with D = 64 the keys' 64 channels count twice, as the product's 128 rows
      const uint64_t kr = desc_rows(sb + L::K0, D == 128 ? L::HALF : 0), xr = desc_rows(sb + L::X0, D == 128 ? L::HALF : 0);
      const uint64_t vr = desc_rows(sb + L::V0, L::HALF), sr = desc_rows(sb + L::X0, L::S_HALF);
      const auto step = [](int k) { return (uint32_t)((k >> 2) * L::HALF + (k & 3) * 32) >> 4; };
      uint32_t f_qk[2] = {}, f_v = 0, f_s = 0, f_p = 0, f_k = 0;
      const auto scores = [&](int buf) {
        tc_fence_after();
        if (elect_one()) {
          const uint64_t qb = qd + buf * BUF, kb = kd + buf * BUF;
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k)
            mma_bf16(tmem + L::T_S, qb + step(k), kb + step(k), idesc(128, 128, false, false), k > 0);
          mma_commit(&sh.qk_done);
        }
        __syncwarp();
      };
      Walk w;  // a chunk ahead of the products
      w.begin(p, sh);
      Ticket now = w.ticket();
      bool ok = wait(&sh.qk_full[0], f_qk[0], 60);
      if (ok && now.full) scores(0);
      for (int buf = 0; ok && now.on; buf ^= 1) {
        const bool full = now.full;
        w.next(p, sh);
        const Ticket next = w.ticket();
        if (!(ok = wait(&sh.s_ready, f_s, 61))) break;
        tc_fence_after();
        if (full) {
          if (elect_one()) {
            const uint64_t qb = qd + buf * BUF;
#pragma unroll 1
            for (int part = 0; part < 2; ++part)
#pragma unroll 1
              for (int k = 0; k < D / 16; ++k)
                mma_bf16(tmem + L::T_SQ, qb + step(k), sr + (part * (L::S_PART >> 4) + k * ROWS16), idesc(128, D, false, true),
                         part + k > 0);
            mma_commit(&sh.sq_done);
          }
          __syncwarp();
        }
        if (!(ok = wait(&sh.v_full, f_v, 62))) break;
        if (full) {
          if (!(ok = wait(&sh.p_ready, f_p, 63))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll 1
            for (int part = 0; part < 2; ++part)
#pragma unroll 1
              for (int k = 0; k < CHUNK / 16; ++k)
                mma_bf16_ta(tmem + L::T_PV, tmem + L::T_S + 16 * k + 8 * part, vr + k * ROWS16,
                            idesc(128, D, false, true), part + k > 0);
            mma_commit(&sh.pv_done);
          }
          __syncwarp();
        }
        if (!(ok = wait(&sh.k_ready, f_k, 64))) break;
        if (elect_one()) {
          const uint64_t kb = kr + buf * BUF;
#pragma unroll 1
          for (int part = 0; part < 3; ++part)
#pragma unroll 1
            for (int k = 0; k < CHUNK / 16; ++k)
              mma_bf16(tmem + L::T_DS, (part == 0 ? kb : xr + (part - 1) * BUF) + k * ROWS16, vr + k * ROWS16,
                       idesc(128, D, true, true), part + k > 0);
          mma_commit(&sh.ds_done);
        }
        __syncwarp();
        if (next.on) {  // its scores take the weights' place: products run in order
          if (!(ok = wait(&sh.qk_full[buf ^ 1], f_qk[buf ^ 1], 60))) break;
          if (next.full) scores(buf ^ 1);
        }
        now = next;
      }
      if (!ok) {  // what is in flight ends before its memory goes
        const int never = 0;
        if (elect_one()) mma_commit(&sh.drain);
        __syncwarp();
        mbar_wait(&sh.drain, 0, &never, LC_WAIT_NS);
      }
    } else if (warp == W_LOAD && a < b) {
      // ---- queries and keys two chunks ahead, values one
      uint32_t f_ds = 0, f_q = 0;
      const auto load = [&](const CUtensorMap* tm, int col, int row, int at, uint64_t* bar) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) tma_load_2d(smem + at + h * L::HALF, tm, col + 64 * h, row, bar);
      };
      const int heads = p.hv / p.hk;
      uint32_t n_qk = 0, n_v = 0;
      const auto load_qk = [&](const Ticket& c) {
        const int buf = n_qk++ & 1;
        if (elect_one()) {
          const int col = c.head / heads * D;
          mbar_arrive_expect_tx(&sh.qk_full[buf], c.full ? 2 * L::TILE : L::TILE);
          load(&tm_k, col, c.row, L::K0 + buf * L::TILE, &sh.qk_full[buf]);
          if (c.full) load(&tm_q, col, c.row, L::Q0 + buf * L::TILE, &sh.qk_full[buf]);
        }
        __syncwarp();
      };
      const auto load_v = [&](const Ticket& c) {
        ++n_v;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sh.v_full, L::TILE);
          load(&tm_v, c.head * D, c.row, L::V0, &sh.v_full);
        }
        __syncwarp();
      };
      Walk w;
      w.begin(p, sh);
      const auto advance = [&]() {
        if (w.more()) w.next(p, sh);
        return w.ticket();
      };
      Ticket now = w.ticket();
      load_qk(now);
      // all CTAs begin at once: what the first chunk needs first goes ahead of the rest
      uint32_t f_first = 0;
      bool ok = wait(&sh.qk_full[0], f_first, 79);
      load_v(now);
      Ticket next = advance();
      if (next.on) load_qk(next);
      while (ok && now.on) {
        const Ticket ahead = advance();
        if (!(ok = wait(&sh.ds_done, f_ds, 66))) break;
        if (next.on) load_v(next);
        if (now.full && !(ok = wait(&sh.q_free, f_q, 69))) break;
        if (ahead.on) load_qk(ahead);
        now = next;
        next = ahead;
      }
      if (!ok) {  // what is in flight ends before its memory goes: the last tiles asked for
        const int never = 0;
        for (int i = 0; i < 2; ++i)
          if (n_qk > (uint32_t)i) mbar_wait(&sh.qk_full[i], ((n_qk - 1 - i) / 2) & 1, &never, LC_WAIT_NS);
        mbar_wait(&sh.v_full, (n_v - 1) & 1, &never, LC_WAIT_NS);
      }
    } else if (warp == W_STORE && a < b) {
      // ---- results, from the queries' place
      Walk w;
      w.begin(p, sh);
      uint32_t f_o = 0;
      for (int buf = 0; w.more(); buf ^= 1) {
        const Ticket c = w.ticket();
        if (c.full) {
          if (!wait(&sh.o_ready, f_o, 65)) break;
          if (elect_one()) {
            if (c.rows == CHUNK) {
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_store_2d(&tm_o, c.head * D + 64 * h, c.row, smem + L::Q0 + buf * L::TILE + h * L::HALF);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
              asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
            mbar_arrive(&sh.q_free);
          }
          __syncwarp();
        }
        w.next(p, sh);
      }
      if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      __syncwarp();
    } else if (warp == W_GAIN && a < b) {
      // ---- decays: four rows a lane, a chunk ahead in registers, their values another one ahead.
      // (In fp64 their sums took 6000 clocks a chunk.)
      const auto load = [&](const Ticket& c, float (&g)[4]) {
        if (!c.on) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * lane + i;
          g[i] = r < c.rows ? p.log_decay[(size_t)(c.row + r) * p.decay_stride + c.head] : 0.f;
        }
      };
      Walk w;
      w.begin(p, sh);
      uint32_t f_empty = 1;
      Ticket c = w.ticket();
      if (lane == 0) {
        sh.begin = c;
        mbar_arrive(&sh.t_full);
      }
      float g[4];
      load(c, g);
      for (int buf = 0; c.on; buf ^= 1) {
        long long v[4], at = 0;
        bool bad[4], nan = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // log2(e) in two parts, the product's rounding kept
          const float x = decay_of(g[i]), l = x * LOG2E, rest = fmaf(x, LOG2E_REST, fmaf(x, LOG2E, -l));
          bad[i] = nan |= x != x;
          at += l < LEAST ? (long long)LEAST * (1ll << 40) : __float2ll_rn(l * UNIT) + __float2ll_rn(rest * UNIT);
          v[i] = at;
        }
        w.next(p, sh);
        const Ticket ahead = w.ticket();
        load(ahead, g);  // their values come while this chunk's are worked out
        if (ahead.on && ahead.begins && ahead.full && ahead.stage < 2 && ahead.slot_in >= 0) {  // the state that a part begins from
          const float* from = p.states + ((size_t)ahead.slot_in * p.hv + ahead.head) * D * D;
          for (int i = lane; i < D * D / 32; i += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + 32 * i));
        }
        long long in = at;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long u = __shfl_up_sync(~0u, in, o);
          if (lane >= o) in += u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += in - at;
        const auto value = [&](long long x) { return __ll2float_rn(x) * PER_UNIT; };
        const long long end = __shfl_sync(~0u, v[3], 31);
        const long long ref0 = __shfl_sync(~0u, v[0], lane & 24);
        // a row whose decay is NaN, and those behind it
        const uint32_t nans = __ballot_sync(~0u, nan);
#pragma unroll
        for (int i = 0; i < 4; ++i) bad[i] |= (nans & ((1u << lane) - 1)) != 0;
        float own[4], last[4], first[4], off[3][4];
        const bool mild = value(__shfl_sync(~0u, v[3], lane | 7) - ref0) >= -MILD;
        const uint32_t milds = __ballot_sync(~0u, mild);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float rel = value(v[i] - ref0);
          own[i] = mild ? ex2(-rel) : rel;
          last[i] = nans ? NOT_A_NUMBER : ex2(value(end - v[i]));
          first[i] = bad[i] ? NOT_A_NUMBER : ex2(value(v[i]));
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const long long ref = __shfl_sync(~0u, v[0], 8 * q + 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) off[q][i] = ex2(value(ref - v[i]));
        }
        float keep, slow;
        factor_of(value(end), keep, slow);
        if (nans) keep = NOT_A_NUMBER;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // worked out before the wait, not behind it
          asm volatile("" : "+f"(own[i]), "+f"(last[i]), "+f"(first[i]), "+f"(off[0][i]), "+f"(off[1][i]), "+f"(off[2][i]), "+f"(keep));
        if (!wait(&sh.g_empty, f_empty, 67)) break;
        Gains& to = sh.g;
        const int r = 4 * lane;
        *reinterpret_cast<float4*>(&to.own[r]) = make_float4(own[0], own[1], own[2], own[3]);
        *reinterpret_cast<float4*>(&to.last[r]) = make_float4(last[0], last[1], last[2], last[3]);
        *reinterpret_cast<float4*>(&to.first[r]) = make_float4(first[0], first[1], first[2], first[3]);
#pragma unroll
        for (int q = 0; q < 3; ++q)
          if (lane < 8 * q + 8)
            *reinterpret_cast<float4*>(&to.off[16 * q * (q + 1) + r]) = make_float4(off[q][0], off[q][1], off[q][2], off[q][3]);
        if (lane == 31) {
          to.mild = (milds & 1) | (milds >> 8 & 1) << 1 | (milds >> 16 & 1) << 2 | (milds >> 24 & 1) << 3;
          to.keep = keep;
          to.slow = slow;
          to.end = end;
        }
        if (lane == 30) sh.next[buf] = ahead;  // the compute warps have read the one of two chunks ago
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.g_full);
        c = ahead;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LC_REGS));
    const int quarter = warp & 3, group = warp >> 2;
    const int row = 32 * quarter + lane;  // of the chunk, in the products whose rows are the queries'
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    uint32_t f_qk[2] = {}, f_v = 0, f_g = 0, f_sc = 0, f_sq = 0, f_pv = 0, f_ds = 0, f_met = 0, f_t = 0;
    float S[NC];
    // rows of the state in TMEM: lanes, the upper 64 a copy of the lower with D = 64
    const int s_row = row % D;
    const int s_col = D == 128 ? 64 * group : 16 * ((quarter >> 1) + 2 * group);

    const auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // All compute warps; bounded like every wait, since a warp that gave up does not come.
    const auto meet = [&]() {
      arrive(&sh.met);
      return wait(&sh.met, f_met, 77);
    };
    const auto write_state = [&]() {  // both bf16 parts, as the operand of the products with the queries
#pragma unroll
      for (int c = 0; c < NC; c += 8) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 v = make_float2(S[c + 2 * i], S[c + 2 * i + 1]);
          hi[i] = take_rounded(v);
          lo[i] = pack_bf16x2(v.x, v.y);
        }
        const int col = s_col + c;
        unsigned char* to = smem + L::X0 + (col >> 6) * L::S_HALF + sw128_off(s_row, (col & 63) >> 3);
        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(to + L::S_PART) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_async_smem();
    };
    const auto state_at = [&](int slot, int head) {
      return p.states + ((size_t)slot * p.hv + head) * D * D + s_row * D + s_col;
    };
    // The state that the CTA's first part goes on from, from the CTAs before it.
    const auto join = [&](int chunks) {
      const int from = blockIdx.x - (int)((chunks + run - 1) / run);  // the CTA that begins the chain
      if (tid < (int)blockIdx.x - from) {
        const uint64_t t0 = globaltimer();
        while (!load_acquire(&cp.flags[from + tid])) {
          __nanosleep(64);
          if (*abort) break;
          if (globaltimer() - t0 > LC_WAIT_NS) {
            *abort = 68;
            break;
          }
        }
      }
      if (!meet() || __any_sync(~0u, *abort)) return false;
#pragma unroll 1
      for (int b = from; b < (int)blockIdx.x; ++b) {
        const float* at = cp.pub + b * pub_floats(D);
        const float keep = __ldcg(at + D * D), slow = __ldcg(at + D * D + 1);
#pragma unroll
        for (int i = 0; i < NC; i += 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(at + i * LC_COMPUTE + 4 * tid));
          if (b == from) {
            S[i] = v.x, S[i + 1] = v.y, S[i + 2] = v.z, S[i + 3] = v.w;
          } else {
            S[i] = fmaf(S[i], slow, fmaf(S[i], keep, v.x)), S[i + 1] = fmaf(S[i + 1], slow, fmaf(S[i + 1], keep, v.y));
            S[i + 2] = fmaf(S[i + 2], slow, fmaf(S[i + 2], keep, v.z)), S[i + 3] = fmaf(S[i + 3], slow, fmaf(S[i + 3], keep, v.w));
          }
        }
      }
      return true;
    };

    long long decay = 0;  // of the part, exact (one that is NaN shows in its state)
    Ticket t;
    t.on = a < b && wait(&sh.t_full, f_t, 78);
    if (t.on) t = sh.begin;
    for (int buf = 0; t.on; t = sh.next[buf], buf ^= 1) {
      const bool full = t.full;
      const int rows = t.rows;
      if (t.begins) {
        decay = 0;
        if (t.stage == 2) {
          if (!join(t.before)) break;
        } else {
#pragma unroll
          for (int i = 0; i < NC; ++i) S[i] = 0.f;
          if (full && t.slot_in >= 0) load_state(S, state_at(t.slot_in, t.head));
        }
      }
      if (full) write_state();
      tc_fence_before();
      arrive(&sh.s_ready);
      if (!wait(&sh.g_full, f_g, 70)) break;
      const float keep = sh.g.keep, slow = sh.g.slow;
      const bool mild = sh.g.mild >> quarter & 1;
      decay = max(decay + sh.g.end, PART_LEAST);
      if (full) {
        // weights: scores times the decays between key and query, in two bf16
        // parts over the scores' own columns.  The decay is a row's factor
        // times a key's, both relative to the first of the warp's rows; the
        // row's waits for the results, unless that would make the keys' of the
        // warp's own rows too large.
        if (!wait(&sh.qk_done, f_sc, 71)) break;
        tc_fence_after();
        const float own = sh.g.own[row], mine = mild ? 1.f : ex2(own);
        // The loops over blocks stay loops: unrolled, a chunk is some 80 KB of
        // code, and fetching it takes longer than running it.
#pragma unroll 1
        for (int j0 = 64 * group; j0 < 64 * group + 64; j0 += 16) {
          const int j32 = j0 & ~31;
          if (j32 > 32 * quarter) {
            const uint32_t none[16] = {};
            tmem_st<16>(lanes + L::T_S + j0, none);
            continue;
          }
          uint32_t z[16];
          tmem_ld16(lanes + L::T_S + j0, z);
          tmem_ld_wait();
          tmem_ld_fence(z);
          const bool all = j32 < 32 * quarter;
          if (!all) {  // a score counts only where its key is seen, whatever it is
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = i + (j0 & 16) <= lane ? z[i] : 0;
          }
          const float* by = all ? &sh.g.off[16 * quarter * (quarter - 1) + j0] : &sh.g.own[j0];
          uint32_t w[16];  // of 16 keys each: eight columns of first parts, eight of second ones
          float4 by4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) by4[i] = *reinterpret_cast<const float4*>(by + 4 * i);
          if (!mild) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float4& f = by4[i];
              if (all)
                f = make_float4(f.x * mine, f.y * mine, f.z * mine, f.w * mine);
              else  // (of keys behind the row, not above 1)
                f = make_float4(ex2(fminf(own - f.x, 0.f)), ex2(fminf(own - f.y, 0.f)), ex2(fminf(own - f.z, 0.f)),
                                ex2(fminf(own - f.w, 0.f)));
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 f = by4[i];
            const uint32_t* s = &z[4 * i];
            float2 u = mul2(pair(s), make_float2(f.x, f.y)), v = mul2(pair(s + 2), make_float2(f.z, f.w));
            uint32_t* o = w + 2 * i;
            o[0] = take_rounded(u);
            o[8] = pack_bf16x2(u.x, u.y);
            o[1] = take_rounded(v);
            o[9] = pack_bf16x2(v.x, v.y);
          }
          tmem_st<16>(lanes + L::T_S + j0, w);
        }
        tmem_st_wait();
      }
      if (!wait(&sh.qk_full[buf], f_qk[buf], 72)) break;
      if (rows < CHUNK) {  // rows of no sequence or of another
        if (!wait(&sh.v_full, f_v, 73)) break;
        f_v ^= 1;  // taken back below
        for (int e = tid; e < (CHUNK - max(rows, 0)) * (D / 8); e += LC_COMPUTE) {
          const int r = CHUNK - 1 - e / (D / 8), ch = e % (D / 8);
          const int to = (ch >> 3) * L::HALF + sw128_off(r, ch & 7);
          *reinterpret_cast<uint4*>(smem + L::V0 + to) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        if (!meet()) break;
      }
      f_v ^= 1;  // this chunk's
      if (full) {
        tc_fence_before();
        arrive(&sh.p_ready);
        if (!wait(&sh.sq_done, f_sq, 74)) break;  // the state's operand is free
      }
      // keys times the decays behind them, in three parts of 8 bits: one in the
      // keys' place, two in that of the state's
      {
        const int r = tid % CHUNK, half = tid / CHUNK;  // neighbours hold neighbouring rows: no bank twice
        const float f = sh.g.last[r];
        unsigned char* kp = smem + L::K0 + buf * L::TILE;
        const auto off = [&](int i) {
          const int ch = half * (D / 16) + i;
          return (ch >> 3) * L::HALF + sw128_off(r, ch & 7);
        };
#pragma unroll 2
        for (int i = 0; i < D / 16; ++i) {
          uint4 v = *reinterpret_cast<const uint4*>(kp + off(i));
          if (r >= rows) v = make_uint4(0, 0, 0, 0);
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[3][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2 x = mul2(make_float2(bf16lo(in[j]), bf16hi(in[j])), both(f));
            o[0][j] = take_cut(x);
            o[1][j] = take_cut(x);
            o[2][j] = cut(x);
          }
          *reinterpret_cast<uint4*>(kp + off(i)) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
          *reinterpret_cast<uint4*>(smem + L::X0 + off(i)) = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
          *reinterpret_cast<uint4*>(smem + L::X0 + L::TILE + off(i)) = make_uint4(o[2][0], o[2][1], o[2][2], o[2][3]);
        }
      }
      fence_async_smem();
      arrive(&sh.k_ready);
      if (full) {
        const float first = sh.g.first[row], mine = mild ? __frcp_rn(sh.g.own[row]) : 1.f;
        arrive(&sh.g_empty);  // all of the chunk's decays have been read
        if (!wait(&sh.pv_done, f_pv, 75)) break;
        tc_fence_after();
        uint16_t* out = p.out + ((size_t)(t.row + row) * p.hv + t.head) * D;
        unsigned char* stage = smem + L::Q0 + buf * L::TILE;  // the queries' place: no product reads them any more
        const auto put = [&](int col, auto v) {  // to the row's channels col, ...
          if (rows == CHUNK)
            *reinterpret_cast<decltype(v)*>(stage + (col >> 6) * L::HALF + sw128_off(row, (col & 63) >> 3) + (col & 7) * 2) = v;
          else if (row < rows)
            *reinterpret_cast<decltype(v)*>(out + col) = v;
        };
        float2 finite = both(0.f);  // NaN: a value that is not finite has met the rows before its own
#pragma unroll 1
        for (int col = group * (D / 2); col < (group + 1) * (D / 2); col += 16) {
          uint32_t x[16], y[16], o[8];
          tmem_ld16(lanes + L::T_SQ + col, x);
          tmem_ld16(lanes + L::T_PV + col, y);
          tmem_ld_wait();
          tmem_ld_fence(x);
          tmem_ld_fence(y);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            finite = fma2(pair(y + i), both(0.f), finite);
            const float2 v = fma2(pair(x + i), both(p.scale * first), mul2(pair(y + i), both(p.scale * mine)));
            o[i / 2] = pack_bf16x2(v.x, v.y);
          }
          put(col, make_uint4(o[0], o[1], o[2], o[3]));
          put(col + 8, make_uint4(o[4], o[5], o[6], o[7]));
        }
        if (__any_sync(~0u, finite.x + finite.y != 0.f && row < rows)) {
#pragma unroll 1
          for (int col = group * (D / 2); col < (group + 1) * (D / 2); ++col) {
            uint32_t x, y;
            tmem_ld1(lanes + L::T_SQ + col, x);
            tmem_ld1(lanes + L::T_PV + col, y);
            if (!isfinite(__uint_as_float(y)) && row < rows)
              put(col, f2bf(p.scale * fmaf(first, __uint_as_float(x), weighted_values(p, D, t.row, row, t.head, col))));
            __syncwarp();
          }
        }
        fence_async_smem();
        arrive(&sh.o_ready);
      } else {
        arrive(&sh.g_empty);
      }
      if (!wait(&sh.ds_done, f_ds, 76)) break;
      tc_fence_after();
      // a slow decay as in the recurrent kernel
      constexpr int AT_ONCE = NC < 32 ? 1 : 2;
      if (rows > 0)  // else the state is carried over as it is
#pragma unroll
      for (int j = 0; j < NC / 16; j += AT_ONCE) {
        uint32_t x[AT_ONCE][16];
#pragma unroll
        for (int h = 0; h < AT_ONCE; ++h) tmem_ld16(lanes + L::T_DS + s_col + 16 * (j + h), x[h]);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < AT_ONCE; ++h) {
          tmem_ld_fence(x[h]);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float* s = S + 16 * (j + h) + i;
            const float2 v = make_float2(s[0], s[1]), w = fma2(v, both(slow), fma2(v, both(keep), pair(x[h] + i)));
            s[0] = w.x, s[1] = w.y;
          }
        }
      }
      if (!t.ends) continue;
      if (t.stage == 0) {  // others go on from here
        float* to = cp.pub + blockIdx.x * pub_floats(D);
#pragma unroll
        for (int i = 0; i < NC; i += 4)
          *reinterpret_cast<float4*>(to + i * LC_COMPUTE + 4 * tid) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
        if (tid == 0) factor_of((float)decay * PER_UNIT, to[D * D], to[D * D + 1]);
        __threadfence();
        if (!meet()) break;
        if (tid == 0 && !((p.st->stall & MOE_STALL_GRID_BARRIER) && blockIdx.x == 0))
          store_release(&cp.flags[blockIdx.x], 1u);
      } else if (t.closes && t.slot_out >= 0) {
        store_state(state_at(t.slot_out, t.head), S);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_ISSUE) tmem_dealloc(tmem, 512);
  if (tid == 0 && sh.abort && atomicOr(&p.st->flags, FLAG_TIMEOUT) == 0) p.st->timeout_site = sh.abort;
  // the last CTA clears what the next call counts on
  if (tid == 0) {
    __threadfence();
    sh.total = atomicAdd(&cp.sync->done, 1u) + 1 == gridDim.x;
  }
  __syncthreads();
  if (sh.total) {
    for (int i = tid; i < (int)gridDim.x; i += LC_THREADS) cp.flags[i] = 0;
    if (tid == 0) cp.sync->done = 0;
  }
}

template <int D>
cudaError_t launch(const ChunkParams& c, int grid, cudaStream_t s) {
  auto* kern = linear_chunk_kernel<D>;
  cudaError_t e = set_smem_limit_once(kern, Lc<D>::TOTAL);
  const LinearParams& p = c.p;
  CUtensorMap q, k, v, o;
  const auto map = [&](CUtensorMap* m, const void* base, int heads, int64_t stride) {
    if (e == cudaSuccess)
      e = tmap_2d(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)heads * D, p.t, (uint64_t)stride * 2, 64, CHUNK,
                  CU_TENSOR_MAP_SWIZZLE_128B);
  };
  map(&q, p.q, p.hk, p.q_stride);
  map(&k, p.k, p.hk, p.k_stride);
  map(&v, p.v, p.hv, p.v_stride);
  map(&o, p.out, p.hv, (int64_t)p.hv * D);
  if (e != cudaSuccess) return e;
  MOE_LAUNCH("linear_chunk", s,
             { e = launch_k(kern, dim3(grid), dim3(LC_THREADS), (size_t)Lc<D>::TOTAL, s, c, q, k, v, o); });
  return e;
}

}  // namespace

size_t linear_chunk_ws_bytes(int d) {
  return sizeof(LinearSync) + align_up((size_t)sm_count() * 4, 256) + (size_t)sm_count() * pub_floats(d) * 4;
}

cudaError_t launch_linear_chunk(const LinearParams& p, int d, unsigned char* ws, cudaStream_t s) {
  const ChunkParams c{p, (LinearSync*)ws, (uint32_t*)(ws + sizeof(LinearSync)),
                      (float*)(ws + sizeof(LinearSync) + align_up((size_t)sm_count() * 4, 256))};
  const int64_t most = (int64_t)p.hv * (p.t / CHUNK + p.n_seq);  // chunks of all heads, at most
  const int grid = (int)(most < sm_count() ? most : sm_count());
  return d == 128 ? launch<128>(c, grid, s) : launch<64>(c, grid, s);
}

}  // namespace moe
