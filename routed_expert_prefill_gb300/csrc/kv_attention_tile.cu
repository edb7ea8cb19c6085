// Causal attention over the paged 8-bit cache on the tensor cores' own path
// (tcgen05, accumulators in TMEM): sequences with many new rows.
#include <limits.h>
#include <math.h>

#include "kv_attention.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr int T_ROWS = 256;  // query rows of an item: two tiles of 128
// Warps: 0-3 softmax and products of tile 0, 4-7 of tile 1, 8-11 bring the
// keys and values.  Twelve, so that a thread may hold 168 registers.
constexpr int T_WARPS = 12, W_KEYS = 8;
constexpr int T_THREADS = T_WARPS * 32;
// Units that an item counts for beside its own, when the work is cut: its
// query rows, first scales and results are worth about four (one prompt of
// 4096 tokens, 32 heads on 8: 433 us with none, 252 with two, 202 with five;
// two prompts behind contexts 335, 324, 315, and 327 with eight).
constexpr int ITEM_COST = 4;
constexpr int SC_RING = 4;   // tiles whose scales are kept
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr float GROWTH = 8.f;  // how far (log2) a row's weights may outgrow 1 before its sums are rescaled

// One CTA's part of an item: units u0 .. u1 - 1 of it.
struct Piece {
  int row, new_rows, len;  // of the sequence
  int s, qt, h, u0, u1;
  int n[2];                // units that the rows of either tile see
  int seen;                // positions that the item's rows see
  int64_t first;           // where the item's unit 0 stands in the work
};

// A warp's walk over the CTA's pieces.  It lives in shared memory and one lane
// advances it, which leaves the unit loops their registers (no spills).
struct Walk {
  int64_t x;
  int s, qt, h, u;
  Piece P;
  int more;
};

struct TileShared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], o_full[2], drain[2];
  uint64_t sc_full[SC_RING];
  float sc_k[SC_RING][8], sc_log[SC_RING][8], sc_inv[SC_RING][8], sc_ref[SC_RING];
  float red[4];
  uint32_t arrived[2];
  uint32_t tmem;
  int abort;
  int issuing;  // 1 while one tile's thread hands its products over
  int64_t scratch[T_WARPS + 2];
  Work work;
  Walk walk[T_WARPS];
};


// The next piece of the warp's walk into W.P; false at the end.
__device__ __forceinline__ bool next_piece(const AttnParams& p, const Work& w, Walk& W) {
  __syncwarp();  // every lane is done with the last piece
  if ((threadIdx.x & 31) == 0) {
    Piece& P = W.P;
    W.more = 0;
    while (W.x < w.x1 && !W.more) {
      const Seq q = load_seq(p, W.s);
      P.row = q.row, P.new_rows = q.n, P.len = q.len;
      P.s = W.s, P.qt = W.qt, P.h = W.h;
      P.seen = tile_seen<T_ROWS>(p, q, W.qt);
      const int units = (P.seen + UNIT - 1) / UNIT;
      const int end = (int)min((int64_t)(ITEM_COST + units), W.u + (w.x1 - W.x));
      P.u0 = max(W.u - ITEM_COST, 0);
      P.u1 = end - ITEM_COST;
      P.first = W.x - W.u + ITEM_COST;
      P.n[0] = tile_units<128>(p, q, 2 * W.qt);
      P.n[1] = seq_rows(p, q) > (uint32_t)T_ROWS * W.qt + 128 ? units : 0;
      W.more = P.u1 > P.u0;  // not if the run ends among the units that stand for the item's cost
      W.x += end - W.u;
      W.u = 0;
      if (W.x < w.x1 && ++W.h == p.c.hkv) {
        W.h = 0;
        if (++W.qt == q_tiles<T_ROWS>(p, q)) {
          W.qt = 0;
          do ++W.s;
          while (load_seq(p, W.s).n == 0);  // x < x1 <= total: a later sequence has rows
        }
      }
    }
  }
  __syncwarp();
  return W.more != 0;
}

template <int D>
struct Smem {
  static constexpr int Q = 128 * D * 2, K = UNIT * D * 2, V = D * UNIT * 2;
  static constexpr int RAW = 2 * UNIT * D;  // codes of a unit as they come
  static constexpr int TOTAL = 2 * Q + 2 * K + 2 * V + RAW + (int)sizeof(TileShared);
  static_assert(TOTAL <= 227 * 1024, "shared memory of a CTA");
};
template <int D>
constexpr size_t partial_floats() { return (size_t)128 * (D + 2); }  // accumulators, maximum, sum of a tile's rows

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Ties the registers of a load to this point, after tmem_ld_wait.
__device__ __forceinline__ void ld32_fence(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// Instruction descriptor, kind::f16: D fp32, A and B fp16, both K-major.
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Codes c of bytes 0 and 2, and of bytes 1 and 3, as the fp16 numbers
// (c + 128) * 2^-24: below fp16's normal range the bits are the value.
__device__ __forceinline__ uint32_t codes_even(uint32_t w) { return (w ^ 0x80808080u) & 0x00FF00FFu; }
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) { return ((w >> 8) ^ 0x00808080u) & 0x00FF00FFu; }
// Byte B of two words as exact fp16 numbers: under the exponent of 1024 the
// byte c ^ 0x80 is 1024 + 128 + c.
template <int B>
__device__ __forceinline__ uint32_t f16_pair(uint32_t a, uint32_t b) {
  const uint32_t v = (__byte_perm(a, b, B | (4 + B) << 8) & 0x00FF00FFu) ^ 0x64806480u;
  return half2_bits(__hsub2(*reinterpret_cast<const __half2*>(&v), __floats2half2_rn(1152.f, 1152.f)));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 x, y, z, r;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 r, x, y, z;\nmov.b64 {%0, %1}, r;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 x, y, r;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 r, x, y;\nmov.b64 {%0, %1}, r;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ void named_barrier(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// The work is cut as in the streaming kernel, over items of 256 query rows
// (a position's heads next to each other) and units of 128 tokens.
//
// Four warps bring the keys and values of each unit, copied one unit ahead,
// and store them as fp16 numbers in the swizzled operand layout: the
// keys' codes raw, as (c + 128) 2^-24 (128 2^-24 times the query row's sum
// comes off the score), the values' as c itself, transposed.  Two groups of
// four warps own a tile of 128 rows each: one thread issues S = Q K^T and
// O += P V, and while one tile's weights are being taken the tensor cores
// work for the other.  A thread owns a row: S comes from TMEM and P goes back
// over it as fp16, the second product's A operand, while O stays in TMEM for
// all units.  Weights are taken against the maximum so far, in one pass over
// S; only if one would outgrow 2^8 are O and the sums rescaled and the pass
// repeated.
//
// Scales: the key scale of a run of 16 tokens multiplies the fp32 scores.  The
// value scale vs, relative to the item's largest, enters the weights through
// its logarithm: P = 2^(s + log2 vs - M), at most 2^8 whatever the scales
// are, and the softmax's sum takes each run's sum of P back by 1 / vs.
template <int D>
__global__ void __launch_bounds__(T_THREADS, 1) kv_attention_tile_kernel(AttnParams p) {
  extern __shared__ __align__(1024) unsigned char smem_tile[];  // operand tiles: 1024-byte aligned
  unsigned char* sq = smem_tile;
  unsigned char* sk = sq + 2 * Smem<D>::Q;
  unsigned char* sv = sk + 2 * Smem<D>::K;
  unsigned char* raw = sv + 2 * Smem<D>::V;
  TileShared& S = *reinterpret_cast<TileShared*>(raw + Smem<D>::RAW);
  constexpr uint32_t S_COL = 0, O_COL = 256;  // tile x: S at 128 x, O at 256 + D x
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hkv = p.c.hkv;
  {
    Work found;
    if (!find_work<T_ROWS, T_THREADS, ITEM_COST>(p, S.scratch, found)) return;
    if (tid == 0) S.work = found;
    if (lane == 0) {
      Walk& W = S.walk[warp];
      W.x = found.x0, W.s = found.s, W.qt = found.qt, W.h = found.h, W.u = found.u;
    }
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], 4);  // one arrival a warp
      mbar_init(&S.k_empty[i], 2);  // released for either tile
      mbar_init(&S.v_full[i], 4);
      mbar_init(&S.v_empty[i], 2);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.o_full[i], 1);
      mbar_init(&S.drain[i], 1);
    }
    for (int i = 0; i < SC_RING; ++i) mbar_init(&S.sc_full[i], 1);
    S.abort = 0;
    S.issuing = 0;
    fence_mbar_init();
  }
  if (warp == W_KEYS) tmem_alloc(&S.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;

  volatile int* abort = &S.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
    if (mbar_wait(bar, parity, abort, WAIT_NS)) return true;
    if (!*abort) {
      if (atomicOr(&p.st->flags, FLAG_TIMEOUT) == 0) p.st->timeout_site = site;
      *abort = 1;
    }
    return false;
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
    return __all_sync(~0u, wait(bar, parity, site)) != 0;
  };

  const Piece& P = S.walk[warp].P;
  if (warp < W_KEYS) {
    // ------------------------------------------------- softmax and products
    const int X = warp >> 2, r = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's quarter of the lanes
    const uint32_t s_addr = lanes + S_COL + 128 * X, o_addr = lanes + O_COL + D * X;
    unsigned char* q_tile = sq + X * Smem<D>::Q;
    uint32_t units_done = 0, tiles = 0, pieces = 0;  // of the CTA; of this tile
    bool ok = true;
    constexpr uint32_t ID_S = idesc_f16(128, UNIT), ID_O = idesc_f16(128, D);
    // The products, by one thread a tile, elected in its first warp.  A tile hands over all it has at
    // once, O += P V of its unit and S of the next, and the other waits: taken
    // in turns product by product, both tiles' would end at the same time, and
    // both softmaxes run while the tensor cores idle.
    auto lock = [&]() {
      uint64_t t0 = 0;
      for (uint32_t i = 1; atomicCAS(&S.issuing, 0, 1) != 0; ++i) {
        if (i & 63) continue;
        const uint64_t now = globaltimer();
        if (t0 == 0) t0 = now;
        if (*abort || now - t0 > WAIT_NS) return false;
      }
      return true;
    };
    auto unlock = [&]() { atomicExch(&S.issuing, 0); };
    auto issue_scores = [&](uint32_t it) {
      const uint32_t q0 = smem_u32(q_tile), k0 = smem_u32(sk + (it & 1) * Smem<D>::K);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (k >> 2) * (128 * 128) + (k & 3) * 32;
        mma_bf16(tmem + S_COL + 128 * X, desc_sw128(q0 + off), desc_sw128(k0 + off), ID_S, k > 0);
      }
      mma_commit(&S.s_full[X]);
      mma_commit(&S.k_empty[it & 1]);
    };
    auto issue_outputs = [&](uint32_t it, bool first) {
      const uint32_t v0 = smem_u32(sv + (it & 1) * Smem<D>::V);
#pragma unroll
      for (int k = 0; k < UNIT / 16; ++k)
        mma_bf16_ta(tmem + O_COL + D * X, tmem + S_COL + 128 * X + 8 * k, desc_sw128(v0 + (k >> 2) * (D * 128) + (k & 3) * 32),
                    ID_O, !first || k > 0);
      mma_commit(&S.v_empty[it & 1]);
    };
    // units that this tile's rows do not see are given back as they come
    auto release = [&](uint32_t it) {
      if (wait(&S.k_full[it & 1], (it >> 1) & 1, 59)) mbar_arrive(&S.k_empty[it & 1]);
      if (wait(&S.v_full[it & 1], (it >> 1) & 1, 60)) mbar_arrive(&S.v_empty[it & 1]);
    };
    while (ok && next_piece(p, S.work, S.walk[warp])) {
      const int last = min(P.u1, P.n[X]);
      if (P.u0 >= last) {
        if (r == 0)
          for (int u = P.u0; u < P.u1; ++u) release(units_done + u - P.u0);
        units_done += P.u1 - P.u0;
        continue;
      }
      const int64_t rr = (int64_t)T_ROWS * P.qt + 128 * X + r, rows = (int64_t)P.new_rows * p.G;
      const bool live_row = rr < rows;
      const int qi = live_row ? (int)(rr / p.G) : 0, head = live_row ? P.h * p.G + (int)(rr % p.G) : 0;
      const int before = P.len - P.new_rows;
      // rows past the last store nothing, so they may see all
      const int limit = live_row ? before + qi : INT_MAX;
      const int first_limit = before + (int)(((int64_t)T_ROWS * P.qt + 128 * X) / p.G);
      // ---- the warp's 32 query rows, scaled by a power of two into fp16: a
      // row's D / 8 pieces in neighbouring lanes, so that all loads of eight
      // are in flight together
      float f, off;  // score per product; what the keys' 128s add to a product
      {
        constexpr int LPR = D / 8, RPL = 32 / LPR;  // lanes of a row, rows of a load
        const int c = lane % LPR;
        f = off = 0.f;
#pragma unroll
        for (int b = 0; b < 32; b += 8 * RPL) {
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t rr = (uint32_t)T_ROWS * P.qt + 128 * X + 32 * (warp & 3) + b + i * RPL + lane / LPR;
            v[i] = make_uint4(0, 0, 0, 0);
            if (rr < (uint32_t)rows)
              v[i] = *reinterpret_cast<const uint4*>(p.q + (int64_t)(P.row + (int)(rr / (uint32_t)p.G)) * p.q_stride +
                                                     (size_t)(P.h * p.G + (int)(rr % (uint32_t)p.G)) * D + 8 * c);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            float m = 0.f, sum = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(fabsf(bf16lo(x[e])), fabsf(bf16hi(x[e]))));
#pragma unroll
            for (int o = 1; o < LPR; o *= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            // its largest magnitude goes to [2^14, 2^15); a negative scale goes
            // into the row, so that f is not
            const int ex = min(max((int)(__float_as_uint(m) >> 23) - 127, -100), 127);
            const float up = copysignf(__uint_as_float((uint32_t)(127 + 14 - ex) << 23), p.scale_log2);
            auto two = [&](uint32_t a, uint32_t b, bool hi) {
              const __half2 h = __floats2half2_rn((hi ? bf16hi(a) : bf16lo(a)) * up, (hi ? bf16hi(b) : bf16lo(b)) * up);
              sum += __low2float(h) + __high2float(h);
              return half2_bits(h);
            };
            // channels in the keys' order: 0 2 1 3 of every four
            const int row = 32 * (warp & 3) + b + i * RPL + lane / LPR;
            *reinterpret_cast<uint4*>(q_tile + (c >> 3) * (128 * 128) + sw128_off(row, c & 7)) =
                make_uint4(two(x[0], x[1], false), two(x[0], x[1], true), two(x[2], x[3], false), two(x[2], x[3], true));
#pragma unroll
            for (int o = 1; o < LPR; o *= 2) sum += __shfl_xor_sync(~0u, sum, o);
            // to the lanes that own the rows
            const int ex_of = __shfl_sync(~0u, ex, (lane % RPL) * LPR);
            const float sum_of = __shfl_sync(~0u, sum, (lane % RPL) * LPR);
            if (lane / RPL == b / RPL + i) {
              f = __uint_as_float((uint32_t)(127 - 14 + ex_of) << 23) * fabsf(p.scale_log2) * 0x1p24f;
              off = sum_of * 0x1p-17f;  // 128 * 2^-24
            }
          }
        }
        fence_async_smem();
        named_barrier(2 + X);
        if ((warp & 3) == 0) {
          if (!(ok = wait_warp(&S.k_full[units_done & 1], (units_done >> 1) & 1, 57))) break;
          tc_fence_after();
          if (elect_one() && lock()) {
            issue_scores(units_done);
            unlock();
          }
          __syncwarp();
        }
      }
      float M = -INFINITY, l = 0.f, ref = 1.f;
      for (int u = P.u0; u < last; ++u) {
        const uint32_t it = units_done + u - P.u0, slot = it % SC_RING;
        // the scales' barrier second: scores imply that its phase is this
        // unit's, not one of an earlier turn
        if (!(ok = wait_warp(&S.s_full[X], tiles & 1, 51))) break;
        if (!(ok = wait_warp(&S.sc_full[slot], (it / SC_RING) & 1, 52))) break;
        ++tiles;
        tc_fence_after();
        const bool masked = u * UNIT + UNIT - 1 > first_limit;
        const int see = limit - u * UNIT;  // the last token of the unit that this row sees
        ref = S.sc_ref[slot];
        if (masked) {  // the causal edge: what a row does not see becomes -inf in place
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(s_addr + 32 * c, v);
            tmem_ld_wait();
            ld32_fence(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 32 * c + i <= see ? v[i] : 0xFF800000u;
            tmem_st<32>(s_addr + 32 * c, v);
          }
          tmem_st_wait();
        }
        // Scores are S a + log2 vs - off a, a >= 1e-30 so that -inf stays what
        // it is.
        if (__any_sync(~0u, M == -INFINITY)) {  // a first unit: the row's maximum
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(s_addr + 32 * c, v);
            tmem_ld_wait();
            ld32_fence(v);
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              float mx = -INFINITY;
#pragma unroll
              for (int i = 16 * h2; i < 16 * h2 + 16; ++i) mx = fmaxf(mx, __uint_as_float(v[i]));
              const float a = fmaxf(f * S.sc_k[slot][2 * c + h2], 1e-30f);
              top = fmaxf(top, fmaf(mx, a, fmaf(-off, a, S.sc_log[slot][2 * c + h2])));
            }
          }
          if (M == -INFINITY) M = top;  // nothing summed yet: nothing to rescale
        }
        // ---- the weights against the maximum so far; again, with the sums
        // rescaled, if a row's outgrow 2^GROWTH (twice at most: scores beyond
        // 2^24, whose units are above 1, may leave more than that)
        uint32_t w[4][16];
        float add;
        for (int again = 0;; ++again) {
          const float at = M == -INFINITY ? 0.f : M;
          float most = -INFINITY;
          add = 0.f;
          uint32_t vb[2][32];
          tmem_ld32(s_addr, vb[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t(&v)[32] = vb[c & 1];
            tmem_ld_wait();
            ld32_fence(v);
            if (c < 3) tmem_ld32(s_addr + 32 * (c + 1), vb[(c + 1) & 1]);
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              const float a = fmaxf(f * S.sc_k[slot][2 * c + h2], 1e-30f);
              const float b = fmaf(-off, a, S.sc_log[slot][2 * c + h2] - at);
              float2 sum = make_float2(0.f, 0.f);
#pragma unroll
              for (int i = 16 * h2; i < 16 * h2 + 16; i += 2) {
                float2 z = fma2(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), make_float2(a, a),
                                make_float2(b, b));
                most = fmaxf(fmaxf(most, z.x), z.y);
                z = make_float2(ex2(z.x), ex2(z.y));
                sum = add2(sum, z);
                w[c][i >> 1] = half2_bits(__float22half2_rn(z));
              }
              add = fmaf(sum.x + sum.y, S.sc_inv[slot][2 * c + h2], add);
            }
          }
          if (again == 2 || !__any_sync(~0u, most > GROWTH)) break;
          const float by = fmaxf(most, 0.f), drop = ex2(-by);
          M += by;
          l *= drop;
          if (u > P.u0) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(o_addr + 32 * c, v);
              tmem_ld_wait();
              ld32_fence(v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * drop);
              tmem_st<32>(o_addr + 32 * c, v);
            }
          }
        }
        l += add;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st<16>(s_addr + 16 * c, w[c]);
        tmem_st_wait();
        tc_fence_before();
        named_barrier(2 + X);  // every row's weights are there
        if ((warp & 3) == 0) {
          const bool more = u + 1 < last;
          if (!(ok = wait_warp(&S.v_full[it & 1], (it >> 1) & 1, 58))) break;
          if (more && !(ok = wait_warp(&S.k_full[(it + 1) & 1], ((it + 1) >> 1) & 1, 57))) break;
          tc_fence_after();
          if (elect_one() && lock()) {
            issue_outputs(it, u == P.u0);
            if (more)
              issue_scores(it + 1);
            else
              mma_commit(&S.o_full[X]);
            unlock();
          }
          __syncwarp();
        }
      }
      if (ok && r == 0)
        for (int u = last; u < P.u1; ++u) release(units_done + u - P.u0);
      if (!ok) break;
      units_done += P.u1 - P.u0;
      // ---- the piece's sums
      if (!(ok = wait_warp(&S.o_full[X], pieces & 1, 53))) break;
      ++pieces;
      tc_fence_after();
      const int c0 = cta_of(S.work, P.first), c1 = cta_of(S.work, P.first + P.n[X] - 1);
      const int cta = blockIdx.x;
      uint16_t* dst = p.out + ((size_t)(P.row + qi) * p.hq + head) * D;
      if (c0 == c1) {
        const float k = l == 0.f ? 0.f : ref / l;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(o_addr + 32 * c, v);
          tmem_ld_wait();
          ld32_fence(v);
          if (live_row)
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(v[i + 2 * e]) * k, __uint_as_float(v[i + 2 * e + 1]) * k);
              *reinterpret_cast<uint4*>(dst + 32 * c + i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        tc_fence_before();
      } else {
        // a tile that spans CTAs: the last one to finish joins the parts in order
        auto part = [&](int c) { return p.partials + (size_t)((2 * c + (c == c0)) * 2 + X) * partial_floats<D>(); };
        float* mine = part(cta);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(o_addr + 32 * c, v);
          tmem_ld_wait();
          ld32_fence(v);
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(mine + ((8 * c + i / 4) * 128 + r) * 4) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
        tc_fence_before();
        mine[128 * D + r] = M;
        mine[128 * D + 128 + r] = l;
        __threadfence();
        named_barrier(2 + X);
        if (r == 0) S.arrived[X] = atomicAdd(p.counters + 2 * c0 + X, 1u);
        named_barrier(2 + X);
        if (S.arrived[X] == (uint32_t)(c1 - c0)) {
          __threadfence();
          if (r == 0) p.counters[2 * c0 + X] = 0;
          float top = -INFINITY, sum = 0.f;
          for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(part(c) + 128 * D + r));
          if (top == -INFINITY) top = 0.f;
          for (int c = c0; c <= c1; ++c) sum += __ldcg(part(c) + 128 * D + 128 + r) * ex2(__ldcg(part(c) + 128 * D + r) - top);
          const float k = sum == 0.f ? 0.f : ref / sum;
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            float acc[32] = {};
            for (int c = c0; c <= c1; ++c) {
              const float drop = ex2(__ldcg(part(c) + 128 * D + r) - top) * k;
              float4 v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = __ldcg(reinterpret_cast<const float4*>(part(c) + ((d / 4 + i) * 128 + r) * 4));
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                acc[4 * i] = fmaf(v[i].x, drop, acc[4 * i]), acc[4 * i + 1] = fmaf(v[i].y, drop, acc[4 * i + 1]);
                acc[4 * i + 2] = fmaf(v[i].z, drop, acc[4 * i + 2]), acc[4 * i + 3] = fmaf(v[i].w, drop, acc[4 * i + 3]);
              }
            }
            if (live_row)
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                *reinterpret_cast<uint4*>(dst + d + i) =
                    make_uint4(pack_bf16x2(acc[i], acc[i + 1]), pack_bf16x2(acc[i + 2], acc[i + 3]),
                               pack_bf16x2(acc[i + 4], acc[i + 5]), pack_bf16x2(acc[i + 6], acc[i + 7]));
          }
        }
      }
    }
    // after a wait that gave up: the products in flight end before TMEM goes
    if (*abort && r == 0) {
      int never = 0;
      mma_commit(&S.drain[X]);
      mbar_wait(&S.drain[X], 0, &never, WAIT_NS);
    }
  } else {
    // ------------------------------------------------------ keys and values
    // A thread copies and converts the same pieces of 16 codes, one unit
    // ahead, through its own places in `raw`.
    const int w = warp & 3, ct = tid & 127;
    // keys: tokens 32 w + 8 (i & 3) + lane % 8, piece lane / 8 + 4 (i >> 2);
    // values: tokens 8 vo + i, piece vc
    constexpr int NK = D / 16;
    const int vo = D == 128 ? (lane & 7) + 8 * (w >> 1) : (lane & 7) + 8 * (w & 1);
    const int vc = D == 128 ? (lane >> 3) + 4 * (w & 1) : lane >> 3;
    const bool has_v = D == 128 || w < 2;
    const int64_t page_bytes = (int64_t)hkv * p.c.block * D, vstep = p.c.n_pages * page_bytes;
    unsigned char* raw_k = raw + ct * 16;
    unsigned char* raw_v = raw + UNIT * D + (D == 128 ? ct : ct & 63) * 16;
    constexpr int K_STEP = 2048, V_STEP = D == 128 ? 2048 : 1024;
    const int k_lane = (lane & 7) * D + 16 * (lane >> 3), v_lane = (vo & 1) * 8 * D + 16 * vc;
    // where the pieces go: keys in row lane % 8 of an 8-row group, 16-byte
    // chunks 2 c and 2 c + 1; values, transposed, in chunk vo % 8 of 16 rows
    const uint32_t k_to[2] = {sw128_off(lane & 7, 2 * (lane >> 3)), sw128_off(lane & 7, 2 * (lane >> 3) + 1)};
    uint32_t it = 0;
    bool ok = true;
    while (ok && next_piece(p, S.work, S.walk[warp])) {
      const int32_t* table = p.c.table + (size_t)P.s * p.c.max_blocks;
      const int8_t* codes = p.c.codes + (int64_t)P.h * p.c.block * D;
      const float* scales = p.c.scales + P.h;
      const int seen = P.seen, end = P.u1;
      auto page_at = [&](int pos) {
        const int page = __ldg(table + (pos >> p.block_log2));
        if (page >= 0 && page < p.c.n_pages) return page;
        raise_flag(p.st, FLAG_BAD_CACHE);
        return -1;
      };
      // page of run lane % 8 of unit u; -1: no token of it is seen
      auto pages_of = [&](int u) {
        const int pos = u * UNIT + 16 * (lane & 7);
        return u < end && pos < seen ? page_at(pos) : -1;
      };
      auto scale_of = [&](int page, int64_t isv) {
        return page < 0 ? 0.f : __ldg(scales + (isv * p.c.n_pages + page) * hkv);
      };
      // a run without a page is read from page 0: its weights are 0
      auto load_k = [&](int u, int pages) {
        if (u < end)
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // the warp's two runs
            const int page = max(__shfl_sync(~0u, pages, 2 * w + e), 0);
            const int8_t* src = codes + page * page_bytes + ((u * UNIT + 16 * (2 * w + e)) & (p.c.block - 1)) * D + k_lane;
#pragma unroll
            for (int c = 0; c < NK / 4; ++c)
#pragma unroll
              for (int o = 0; o < 2; ++o) cp_async16(raw_k + (4 * c + 2 * e + o) * K_STEP, src + 8 * o * D + 64 * c);
          }
        cp_async_commit();
      };
      auto load_v = [&](int u, int pages) {
        if (u < end) {
          const int page = max(__shfl_sync(~0u, pages, vo >> 1), 0);
          const int8_t* src = codes + vstep + page * page_bytes + ((u * UNIT + 16 * (vo >> 1)) & (p.c.block - 1)) * D + v_lane;
          if (has_v)
#pragma unroll
            for (int i = 0; i < 8; ++i) cp_async16(raw_v + i * V_STEP, src + i * D);
        }
        cp_async_commit();
      };
      // pages come two units ahead, codes and scales one
      int pages = pages_of(P.u0), next_pages = pages_of(P.u0 + 1);
      load_k(P.u0, pages);
      load_v(P.u0, pages);
      float ks = scale_of(pages, 0), vs = scale_of(pages, 1);
      // the item's largest value scale; 0 if every value is, and then so is the
      // result
      float vref = 0.f;
      for (int b = ct; b << p.block_log2 < seen; b += 128) vref = fmaxf(vref, scale_of(page_at(b << p.block_log2), 1));
#pragma unroll
      for (int o = 16; o; o >>= 1) vref = fmaxf(vref, __shfl_xor_sync(~0u, vref, o));
      named_barrier(1);  // the last item's values are read
      if (lane == 0) S.red[w] = vref;
      named_barrier(1);
      vref = fmaxf(fmaxf(S.red[0], S.red[1]), fmaxf(S.red[2], S.red[3]));
      const float vref_log = vref > 0.f ? __log2f(vref) : 0.f;
      for (int u = P.u0; u < end; ++u, ++it) {
        const uint32_t st = it & 1, par = ((it >> 1) & 1) ^ 1;
        if (!(ok = wait_warp(&S.k_empty[st], par, 54))) break;
        // the slot's last unit, SC_RING back, is past every softmax thread: the
        // products that freed this K stage came after its weights
        if (w == 0 && lane < 8) {
          const uint32_t slot = it % SC_RING;
          const float lg = pages < 0 ? -INFINITY : fmaxf(__log2f(vs) - vref_log, -60.f);
          S.sc_k[slot][lane] = ks;
          S.sc_log[slot][lane] = lg;
          S.sc_inv[slot][lane] = pages < 0 ? 0.f : ex2(-lg);
          if (lane == 0) S.sc_ref[slot] = vref;
          __syncwarp(0xFF);
          if (lane == 0) mbar_arrive(&S.sc_full[slot]);
        }
        cp_async_wait<1>();
        {
          unsigned char* dst = sk + st * Smem<D>::K + 4 * w * 1024;
#pragma unroll 4
          for (int i = 0; i < NK; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(raw_k + i * K_STEP);
            unsigned char* rows = dst + (i & 3) * 1024 + (i >> 2) * (128 * 128);
            *reinterpret_cast<uint4*>(rows + k_to[0]) =
                make_uint4(codes_even(v.x), codes_odd(v.x), codes_even(v.y), codes_odd(v.y));
            *reinterpret_cast<uint4*>(rows + k_to[1]) =
                make_uint4(codes_even(v.z), codes_odd(v.z), codes_even(v.w), codes_odd(v.w));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.k_full[st]);
        load_k(u + 1, next_pages);
        const int after_pages = pages_of(u + 2);
        if (w == 0) {
          ks = scale_of(next_pages, 0);
          vs = scale_of(next_pages, 1);
        }
        if (!(ok = wait_warp(&S.v_empty[st], par, 55))) break;
        cp_async_wait<1>();
        if (has_v) {
          unsigned char* dst = sv + st * Smem<D>::V + (vo >> 3) * (D * 128) + 2 * vc * 1024;
#pragma unroll 2
          for (int q = 0; q < 4; ++q) {
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const uint32_t*>(raw_v + i * V_STEP + 4 * q);
            // channel 4 q + ch of the piece; its 8-row group and its row there
            unsigned char* rows = dst + (q >> 1) * 1024 + (q & 1) * 512;
            auto put = [&](int ch, uint4 v) {
              *reinterpret_cast<uint4*>(rows + ch * 128 + (((vo & 7) ^ (4 * (q & 1) + ch)) << 4)) = v;
            };
            put(0, make_uint4(f16_pair<0>(x[0], x[1]), f16_pair<0>(x[2], x[3]), f16_pair<0>(x[4], x[5]), f16_pair<0>(x[6], x[7])));
            put(1, make_uint4(f16_pair<1>(x[0], x[1]), f16_pair<1>(x[2], x[3]), f16_pair<1>(x[4], x[5]), f16_pair<1>(x[6], x[7])));
            put(2, make_uint4(f16_pair<2>(x[0], x[1]), f16_pair<2>(x[2], x[3]), f16_pair<2>(x[4], x[5]), f16_pair<2>(x[6], x[7])));
            put(3, make_uint4(f16_pair<3>(x[0], x[1]), f16_pair<3>(x[2], x[3]), f16_pair<3>(x[4], x[5]), f16_pair<3>(x[6], x[7])));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.v_full[st]);
        load_v(u + 1, next_pages);
        pages = next_pages;
        next_pages = after_pages;
      }
    }
    cp_async_wait<0>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_KEYS) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const AttnParams& p, cudaStream_t s) {
  auto* kern = kv_attention_tile_kernel<D>;
  cudaError_t e = set_smem_limit_once(kern, Smem<D>::TOTAL);
  if (e != cudaSuccess) return e;
  MOE_LAUNCH("kv_attention_tile", s,
             { e = launch_k(kern, dim3(sm_count()), dim3(T_THREADS), (size_t)Smem<D>::TOTAL, s, p); });
  return e;
}

}  // namespace

size_t kv_tile_partial_bytes(int d) {
  return (size_t)sm_count() * 4 * (d == 64 ? partial_floats<64>() : partial_floats<128>()) * 4;
}

cudaError_t launch_tile(const AttnParams& p, cudaStream_t s) { return p.c.d == 64 ? launch<64>(p, s) : launch<128>(p, s); }

}  // namespace moe
