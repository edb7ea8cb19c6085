// Linear attention of many rows a sequence (moe_linear_attention) on the
// tensor cores' own path: chunks of 128 rows, accumulators in TMEM.
#include <math.h>

#include "linear_common.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr int CHUNK = 128;
constexpr int LC_THREADS = 256;
constexpr uint64_t LC_WAIT_NS = 2000000000ull;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// A row's log2 decay as it counts: below it the state of one row is 0 in the
// next whatever it was (2^-512 of an fp32 number), and sums over a chunk stay
// exact whole numbers and fractions.
constexpr float LEAST = -512.f;
constexpr float NOT_A_NUMBER = __builtin_nanf("");

// log2 of a product of decays, n + f with a whole number n: differences of two
// keep the fraction's 24 bits however large both are.
struct Gain {
  float n, f;
};

// What one CTA leaves for those that go on with its last chain: the state
// behind its part (or, if its part does not begin the chain, what the part
// adds) and the part's decay.
constexpr int PUB_EXTRA = 64;  // floats behind the state: the decay
constexpr size_t pub_floats(int d) { return (size_t)d * d + PUB_EXTRA; }

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

// Chunks c0 .. c1 - 1 of the nc of one sequence and head.
struct Part {
  int s, head, c0, c1, nc;
  int row, n, slot_in, slot_out;
};

struct LcShared {
  uint64_t bar[4];  // scores, state times queries, weights times values, state: done
  Gain gain[2][CHUNK];
  int poison[128];  // first row whose value of a channel is not finite; CHUNK: none
  int scan[8];
  int total, longest;
  int at[2][2];  // where the CTA's first and last chunk are: sequence, chunks before it
  uint32_t tmem;
  int abort;
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
  static constexpr int NC = D * D / LC_THREADS;        // values of the state a thread holds
  // TMEM columns: scores (then weights), state times queries, weights times values, what the chunk adds
  static constexpr int T_S = 0, T_SQ = 128, T_PV = 128 + D, T_DS = 128 + 2 * D;
};

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

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  const int bytes = on ? 16 : 0;  // 0: sixteen zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two fp32 values as bf16 pairs whose sum is them up to 2^-17: v becomes what is left.
__device__ __forceinline__ uint32_t take_bf16(float& a, float& b) {
  const uint32_t w = pack_bf16x2(a, b);
  a -= bf16lo(w);
  b -= bf16hi(w);
  return w;
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

template <int D>
__global__ void __launch_bounds__(LC_THREADS, 1) linear_chunk_kernel(ChunkParams cp) {
  using L = Lc<D>;
  constexpr int NC = L::NC;
  extern __shared__ __align__(1024) unsigned char smem[];
  LcShared& sh = *reinterpret_cast<LcShared*>(smem + L::TILES);
  const LinearParams& p = cp.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quarter = warp & 3, group = warp >> 2;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    tmem_alloc(&sh.tmem, 512);
    if (lane == 0) {
      for (int i = 0; i < 4; ++i) mbar_init(&sh.bar[i], 1);
      fence_mbar_init();
      sh.abort = 0;
    }
  }
  if (tid < 128) sh.poison[tid] = CHUNK;

  // ---- the CTA's run of the list of all chunks: sequences, their heads, their chunks
  int total = 0, longest = 0;
  for (int s = tid; s < p.n_seq; s += LC_THREADS) {
    const int c = chunks_of(p, s, blockIdx.x == 0);
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
  const int64_t all = (int64_t)sh.total * p.hv;
  longest = sh.longest;
  // Equal runs, but none so short that joining a chain's runs (a state from L2
  // each) takes longer than the runs do.
  const int64_t run = max((all + gridDim.x - 1) / gridDim.x, (int64_t)ceilf(sqrtf(longest / 12.f)));
  const int64_t a = run * blockIdx.x, b = min(a + run, all);
  const uint32_t tmem = sh.tmem;
  uint32_t phase[4] = {};
  const int never = 0;

  const auto wait_bar = [&](int i) {
    if (!mbar_wait(&sh.bar[i], phase[i], (volatile int*)&sh.abort, LC_WAIT_NS) && !sh.abort) {
      if (atomicOr(&p.st->flags, FLAG_TIMEOUT) == 0) p.st->timeout_site = 60 + i;
      sh.abort = 1;
    }
    phase[i] ^= 1;
  };

  float S[NC];
  // rows of the state in TMEM: lanes, the upper 64 a copy of the lower with D = 64
  const int s_row = (32 * quarter + lane) % D;
  const int s_col = D == 128 ? 64 * group : 16 * ((quarter >> 1) + 2 * group);

  // ---- one part; full: with its results, else only what it adds to a state of zero
  const auto load_tile = [&](const uint16_t* x, int64_t stride, size_t row0, int col, int rows, int at) {
    const uint32_t base = smem_u32(smem) + at;
#pragma unroll
    for (int i = 0; i < CHUNK * D / 8 / LC_THREADS; ++i) {
      const int e = tid + i * LC_THREADS, r = e / (D / 8), c = e % (D / 8);
      const bool on = r < rows;
      cp16(base + (c >> 3) * L::HALF + sw128_off(r, c & 7), on ? x + (row0 + r) * stride + col + c * 8 : x, on);
    }
  };
  const auto write_state = [&]() {  // both bf16 parts, as the operand of the products with the queries
#pragma unroll
    for (int c = 0; c < NC; c += 8) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float u = S[c + 2 * i], v = S[c + 2 * i + 1];
        hi[i] = take_bf16(u, v);
        lo[i] = pack_bf16x2(u, v);
      }
      const int col = s_col + c;
      unsigned char* to = smem + L::X0 + (col >> 6) * L::S_HALF + sw128_off(s_row, (col & 63) >> 3);
      *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(to + L::S_PART) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  };

  // Runs the part's chunks on S; returns the log2 of its decays' product.
  const auto run_part = [&](const Part& t, bool full) -> double {
    const int hk = t.head / (p.hv / p.hk);
    const int rows_all = t.n;
    const auto rows_of = [&](int c) { return min(CHUNK, rows_all - c * CHUNK); };
    const auto row_of = [&](int c) { return (size_t)(t.row + c * CHUNK); };
    float g[4] = {};
    const auto load_gains = [&](int c) {  // warp 7: four rows a lane
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * lane + i;
        g[i] = r < rows_of(c) ? p.log_decay[(row_of(c) + r) * p.decay_stride + t.head] : 0.f;
      }
    };
    double decay = 0.0;
    const auto scan_gains = [&](int to) {
      double sum[4], at = 0.0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float l = decay_of(g[i]) * LOG2E;
        at += l < LEAST ? (double)LEAST : (double)decay_of(g[i]) * 1.4426950408889634;
        sum[i] = at;
      }
      double in = at;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double u = __shfl_up_sync(~0u, in, o);
        if (lane >= o) in += u;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double v = in - at + sum[i], n = rint(v);
        sh.gain[to][4 * lane + i] = Gain{(float)n, (float)(v - n)};
      }
    };
    const auto load_qk = [&](int c) {
      if (full) load_tile(p.q, p.q_stride, row_of(c), hk * D, rows_of(c), L::Q0 + (c & 1) * L::TILE);
      load_tile(p.k, p.k_stride, row_of(c), hk * D, rows_of(c), L::K0 + (c & 1) * L::TILE);
      cp_commit();
    };
    const auto load_v = [&](int c) {
      load_tile(p.v, p.v_stride, row_of(c), t.head * D, rows_of(c), L::V0);
      cp_commit();
    };
    __syncthreads();  // the decays of the part before are still read
    load_qk(t.c0);
    load_v(t.c0);
    if (warp == 7) {
      load_gains(t.c0);
      scan_gains(t.c0 & 1);
    }
    if (full) write_state();

    for (int c = t.c0; c < t.c1; ++c) {
      const bool more = c + 1 < t.c1;
      const uint32_t sb = smem_u32(smem), q0 = sb + L::Q0 + (c & 1) * L::TILE, k0 = sb + L::K0 + (c & 1) * L::TILE,
                     v0 = sb + L::V0, x0 = sb + L::X0;
      const Gain* gain = sh.gain[c & 1];
      cp_wait<1>();  // queries and keys
      fence_async_smem();
      tc_fence_before();
      __syncthreads();
      if (sh.abort) break;
      if (full && warp == 0) {
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = (k >> 2) * L::HALF + (k & 3) * 32;
            mma_bf16(tmem + L::T_S, desc_sw128(q0 + o), desc_sw128(k0 + o), idesc(128, 128, false, false), k > 0);
          }
          mma_commit(&sh.bar[0]);
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_bf16(tmem + L::T_SQ, desc_sw128(q0 + (k >> 2) * L::HALF + (k & 3) * 32),
                       desc_rows(x0 + part * L::S_PART + k * 2048, L::S_HALF), idesc(128, D, false, true), part + k > 0);
          mma_commit(&sh.bar[1]);
        }
        __syncwarp();
      }
      if (more)
        load_qk(c + 1);
      else
        cp_commit();  // an empty group keeps the count
      if (warp == 7 && more) load_gains(c + 1);
      const Gain end = gain[CHUNK - 1];
      const int row = 32 * quarter + lane;  // of the chunk, in the products whose rows are the queries'
      if (full) {
        // weights: scores times the decays between key and query, in two bf16 parts over the scores' own columns
        wait_bar(0);
        tc_fence_after();
        const Gain mine = gain[row];
        const uint32_t at = tmem + ((uint32_t)(32 * quarter) << 16) + L::T_S + 64 * group;
        uint32_t hi[32], lo[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int j0 = 64 * group + 16 * j;
          if (j0 > 32 * quarter + 31) {  // behind all of the warp's rows
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[8 * j + i] = lo[8 * j + i] = 0;
            continue;
          }
          uint32_t r[16];
          tmem_ld16(at + 16 * j, r);
          tmem_ld_wait();
          tmem_ld_fence(r);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 two = *reinterpret_cast<const float4*>(&gain[j0 + 2 * i]);
            float u = __uint_as_float(r[2 * i]) * ex2((mine.n - two.x) + (mine.f - two.y));
            float v = __uint_as_float(r[2 * i + 1]) * ex2((mine.n - two.z) + (mine.f - two.w));
            u = j0 + 2 * i <= row ? u : 0.f;
            v = j0 + 2 * i + 1 <= row ? v : 0.f;
            hi[8 * j + i] = take_bf16(u, v);
            lo[8 * j + i] = pack_bf16x2(u, v);
          }
        }
        tmem_st<32>(at, hi);
        tmem_st<32>(at + 32, lo);
        tmem_st_wait();
      }
      // values: one that is not finite would reach the rows before it (0 times
      // it is NaN), so it is taken out and its channel's rows are marked
      cp_wait<1>();
      bool odd = false;
#pragma unroll
      for (int i = 0; i < CHUNK * D / 8 / LC_THREADS; ++i) {
        const int e = tid + i * LC_THREADS, r = e / (D / 8), ch = e % (D / 8);
        uint4* at = reinterpret_cast<uint4*>(smem + L::V0 + (ch >> 3) * L::HALF + sw128_off(r, ch & 7));
        const uint4 v = *at;
        const uint32_t any = ((v.x & 0x7F807F80u) + 0x00800080u) | ((v.y & 0x7F807F80u) + 0x00800080u) |
                             ((v.z & 0x7F807F80u) + 0x00800080u) | ((v.w & 0x7F807F80u) + 0x00800080u);
        if (any & 0x80008000u) {
          odd = true;
          uint16_t* el = reinterpret_cast<uint16_t*>(at);
          for (int j = 0; j < 8; ++j)
            if ((el[j] & 0x7F80) == 0x7F80) {
              el[j] = 0;
              atomicMin(&sh.poison[8 * ch + j], r);
            }
        }
      }
      fence_async_smem();
      tc_fence_before();
      const bool poisoned = __syncthreads_or(odd);
      if (sh.abort) {  // the products in flight end before their memory goes
        if (full) mbar_wait(&sh.bar[1], phase[1], &never, LC_WAIT_NS);
        break;
      }
      if (full) {
        if (warp == 0) {
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int k = 0; k < CHUNK / 16; ++k)
                mma_bf16_ta(tmem + L::T_PV, tmem + L::T_S + 64 * (k >> 2) + 32 * part + 8 * (k & 3),
                            desc_rows(v0 + k * 2048, L::HALF), idesc(128, D, false, true), part + k > 0);
            mma_commit(&sh.bar[2]);
          }
          __syncwarp();
        }
        wait_bar(1);  // the state's operand is free
      }
      // keys times the decays behind them, in three bf16 parts (2^-25): one in
      // the keys' place, two in that of the state's
      {
        const int r = tid >> 1, half = tid & 1;
        const float w = ex2((end.n - gain[r].n) + (end.f - gain[r].f));
        unsigned char* kp = smem + L::K0 + (c & 1) * L::TILE;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int ch = half * (D / 16) + i;
          const uint32_t off = (ch >> 3) * L::HALF + sw128_off(r, ch & 7);
          const uint4 v = *reinterpret_cast<const uint4*>(kp + off);
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[3][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x = bf16lo(in[j]) * w, y = bf16hi(in[j]) * w;
            o[0][j] = take_bf16(x, y);
            o[1][j] = take_bf16(x, y);
            o[2][j] = pack_bf16x2(x, y);
          }
          *reinterpret_cast<uint4*>(kp + off) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
          *reinterpret_cast<uint4*>(smem + L::X0 + off) = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
          *reinterpret_cast<uint4*>(smem + L::X0 + L::TILE + off) = make_uint4(o[2][0], o[2][1], o[2][2], o[2][3]);
        }
      }
      fence_async_smem();
      __syncthreads();
      if (warp == 0) {
        if (elect_one()) {
          // with D = 64 the keys' 64 channels count twice, as the product's 128 rows
          constexpr uint32_t outer = D == 128 ? L::HALF : 0;
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            const uint32_t from = part == 0 ? k0 : x0 + (part - 1) * L::TILE;
#pragma unroll
            for (int k = 0; k < CHUNK / 16; ++k)
              mma_bf16(tmem + L::T_DS, desc_rows(from + k * 2048, outer), desc_rows(v0 + k * 2048, L::HALF),
                       idesc(128, D, true, true), part + k > 0);
          }
          mma_commit(&sh.bar[3]);
        }
        __syncwarp();
      }
      if (full) {
        wait_bar(2);
        tc_fence_after();
        const float before = ex2(gain[row].n + gain[row].f);
        const uint32_t at = tmem + ((uint32_t)(32 * quarter) << 16) + group * (D / 2);
        uint16_t* out = p.out + ((row_of(c) + row) * p.hv + t.head) * D + group * (D / 2);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          uint32_t x[16], y[16];
          tmem_ld16(at + L::T_SQ + 16 * j, x);
          tmem_ld16(at + L::T_PV + 16 * j, y);
          tmem_ld_wait();
          tmem_ld_fence(x);
          tmem_ld_fence(y);
          float o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[i] = p.scale * fmaf(before, __uint_as_float(x[i]), __uint_as_float(y[i]));
            if (poisoned && sh.poison[group * (D / 2) + 16 * j + i] <= row) o[i] = NOT_A_NUMBER;
          }
          if (row < rows_of(c)) {
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              *reinterpret_cast<uint4*>(out + 16 * j + i) =
                  make_uint4(pack_bf16x2(o[i], o[i + 1]), pack_bf16x2(o[i + 2], o[i + 3]), pack_bf16x2(o[i + 4], o[i + 5]),
                             pack_bf16x2(o[i + 6], o[i + 7]));
          }
        }
      }
      wait_bar(3);
      tc_fence_after();
      if (more)
        load_v(c + 1);
      else
        cp_commit();
      if (warp == 7 && more) scan_gains((c + 1) & 1);
      // S times the chunk's decay, plus what it adds; a slow decay as in the recurrent kernel
      const float whole = end.n + end.f;
      const bool slow = whole > -0.5f;
      const float f = slow ? expm1f(whole * LN2) : exp2f(whole);
      decay += (double)end.n + (double)end.f;
#pragma unroll
      for (int j = 0; j < NC / 16; ++j) {
        uint32_t x[16];
        tmem_ld16(tmem + ((uint32_t)(32 * quarter) << 16) + L::T_DS + s_col + 16 * j, x);
        tmem_ld_wait();
        tmem_ld_fence(x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float& s = S[16 * j + i];
          s = fmaf(s, f, slow ? s + __uint_as_float(x[i]) : __uint_as_float(x[i]));
          if (poisoned && sh.poison[s_col + 16 * j + i] < CHUNK) s = NOT_A_NUMBER;
        }
      }
      if (poisoned) {
        __syncthreads();
        if (tid < 128) sh.poison[tid] = CHUNK;
      }
      if (full && more) write_state();
    }
    cp_wait<0>();
    return decay;
  };

  const auto state_at = [&](int slot, int head) { return p.states + ((size_t)slot * p.hv + head) * D * D + s_row * D + s_col; };
  const auto begin_chain = [&](const Part& t, bool full) {
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (full && t.slot_in >= 0) v = *reinterpret_cast<const float4*>(state_at(t.slot_in, t.head) + i);
      S[i] = v.x, S[i + 1] = v.y, S[i + 2] = v.z, S[i + 3] = v.w;
    }
  };
  const auto end_chain = [&](const Part& t) {
    if (t.slot_out < 0 || sh.abort) return;
#pragma unroll
    for (int i = 0; i < NC; i += 4)
      *reinterpret_cast<float4*>(state_at(t.slot_out, t.head) + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
  };
  const auto publish = [&](double decay) {
    float* to = cp.pub + blockIdx.x * pub_floats(D);
#pragma unroll
    for (int i = 0; i < NC; i += 4)
      *reinterpret_cast<float4*>(to + s_row * D + s_col + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
    if (tid == 0) to[D * D] = (float)decay;
    __threadfence();
    __syncthreads();
    if (tid == 0 && !sh.abort && !((p.st->stall & MOE_STALL_GRID_BARRIER) && blockIdx.x == 0))
      store_release(&cp.flags[blockIdx.x], 1u);
  };
  // The state that this CTA's first part goes on from, from the CTAs before it.
  const auto join = [&](const Part& t) {
    const int from = blockIdx.x - (int)((t.c0 + run - 1) / run);  // the CTA that begins the chain
    if (tid < blockIdx.x - from) {
      const uint64_t t0 = globaltimer();
      while (!load_acquire(&cp.flags[from + tid])) {
        __nanosleep(64);
        if (globaltimer() - t0 > LC_WAIT_NS) {
          if (atomicOr(&p.st->flags, FLAG_TIMEOUT) == 0) p.st->timeout_site = 64;
          sh.abort = 1;
          break;
        }
      }
    }
    __syncthreads();
    if (sh.abort) return;
    for (int b = from; b < (int)blockIdx.x; ++b) {
      const float* at = cp.pub + b * pub_floats(D);
      const float f = b == from ? 0.f : exp2f(__ldcg(at + D * D));
#pragma unroll
      for (int i = 0; i < NC; i += 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(at + s_row * D + s_col + i));
        if (b == from) {
          S[i] = v.x, S[i + 1] = v.y, S[i + 2] = v.z, S[i + 3] = v.w;
        } else {
          S[i] = fmaf(S[i], f, v.x), S[i + 1] = fmaf(S[i + 1], f, v.y), S[i + 2] = fmaf(S[i + 2], f, v.z),
          S[i + 3] = fmaf(S[i + 3], f, v.w);
        }
      }
    }
  };

  if (a < b) {
    // where the first and the last chunk are
    int before = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += LC_THREADS) {
      const int s = s0 + tid, c = s < p.n_seq ? chunks_of(p, s, false) : 0;
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
      for (int i = 0; i < 8; ++i) {
        if (i < warp) base += sh.scan[i];
        before += sh.scan[i];
      }
      const int64_t lo = (int64_t)(base + in - c) * p.hv, hi = lo + (int64_t)c * p.hv;
      if (lo <= a && a < hi) sh.at[0][0] = s, sh.at[0][1] = base + in - c;
      if (lo < b && b <= hi) sh.at[1][0] = s, sh.at[1][1] = base + in - c;
    }
    __syncthreads();
    const auto part_of = [&](int s, int head) {
      Part t;
      t.s = s;
      t.head = head;
      linear_sequence(p, s, t.row, t.n, t.slot_in, t.slot_out);
      t.c0 = 0;
      t.c1 = t.nc = chunks_of(p, s, false);
      return t;
    };
    Part first, last;
    {
      const int s = sh.at[0][0], nc = chunks_of(p, s, false);
      const int64_t off = a - (int64_t)sh.at[0][1] * p.hv;
      first = part_of(s, (int)(off / nc));
      first.c0 = (int)(off % nc);
      first.c1 = (int)min((int64_t)nc, first.c0 + (b - a));
    }
    {
      const int s = sh.at[1][0], nc = chunks_of(p, s, false);
      const int64_t off = b - 1 - (int64_t)sh.at[1][1] * p.hv;
      last = part_of(s, (int)(off / nc));
      last.c1 = (int)(off % nc) + 1;
    }
    const auto same = [](const Part& x, const Part& y) { return x.s == y.s && x.head == y.head; };
    if (same(first, last)) last.c0 = first.c0, first.c1 = last.c1;
    // 0: the part that other CTAs go on with, so that they need not wait long;
    // inside a chain, what it adds.  1: whole chains.  2: the part that others began.
    int stage = last.c1 < last.nc ? 0 : 1;
    Part next = first;
    bool left = true;  // next has not been looked at
    while (!sh.abort) {
      Part t;
      bool full = true;
      if (stage == 0) {
        t = last;
        full = t.c0 == 0;
      } else if (stage == 1) {
        bool found = false;
        while (left && !found) {
          t = next;
          found = t.c0 == 0 && t.c1 == t.nc;
          if (same(next, last)) {
            left = false;
          } else {
            int s = next.s, head = next.head + 1;
            if (head == p.hv) {
              head = 0;
              do ++s;
              while (chunks_of(p, s, false) == 0);  // the last part's sequence has some
            }
            next = part_of(s, head);
            if (same(next, last)) next = last;
          }
        }
        if (!found) {
          if (first.c0 == 0) break;
          stage = 2;
        }
      }
      if (stage == 2) {
        t = first;
        join(t);
        if (sh.abort) break;
      } else {
        begin_chain(t, full);
      }
      const double decay = run_part(t, full);
      if (stage == 0)
        publish(decay);
      else if (t.c1 == t.nc)
        end_chain(t);
      if (stage == 2) break;
      stage = 1;
    }
  }
  cp_wait<0>();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
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
cudaError_t launch(const ChunkParams& p, int grid, cudaStream_t s) {
  auto* kern = linear_chunk_kernel<D>;
  cudaError_t e = set_smem_limit_once(kern, Lc<D>::TOTAL);
  if (e != cudaSuccess) return e;
  MOE_LAUNCH("linear_chunk", s, { e = launch_k(kern, dim3(grid), dim3(LC_THREADS), (size_t)Lc<D>::TOTAL, s, p); });
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
