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
// Warps: 0-3 softmax of tile 0, 4-7 of tile 1, 8-10 bring the keys, 11 issues
// the products, 12-15 bring the values.
constexpr int T_WARPS = 16, W_KEYS = 8, W_MMA = 11, W_VALUES = 12;
constexpr int KEY_WARPS = W_MMA - W_KEYS;
constexpr int T_THREADS = T_WARPS * 32;
// Units that an item counts for beside its own, when the work is cut: its
// query rows, first scales and results take as long as about three (two
// prompts behind contexts, the kernel alone: 292 us with two, 285 with three,
// 288 with four, 294 with five; one prompt of 4096 tokens, 32 heads on 8: 205,
// 189, 187, 189).
constexpr int ITEM_COST = 3;
constexpr int SC_RING = 4;   // tiles whose scales are kept
constexpr int RED_RING = 4;  // pieces whose largest value scales are kept
constexpr uint64_t WAIT_NS = 2000000000ull;
// A row's weights are taken against a reference 2^ABOVE below its largest, so
// that those fp16 rounds to nothing are below 2^-32 of that: taken against the
// largest itself, a long context's small weights were lost from 2^-25 on, and
// with them what they add up to.  LIMIT: what the weights of 64 tokens may add
// up to before the row's sums are rescaled; none is then above it, which fp16
// holds, and if they exceed it the largest is above 4 * 2^ABOVE.
constexpr float ABOVE = 7.f, LIMIT = 32768.f;

// One CTA's part of an item: units u0 .. u1 - 1 of it.
struct Piece {
  int row, new_rows, len;  // of the sequence
  int s, qt, h, u0, u1;
  int n[2];                // units that the rows of either tile see
  int seen;                // positions that the item's rows see
  int64_t first;           // where the item's unit 0 stands in the work
};

// A warp's walk over the CTA's pieces.  It lives in shared memory and one lane
// advances it, which leaves the unit loops their registers (some 20 bytes are
// spilt outside of them).
struct Walk {
  int64_t x;
  int s, qt, h, u;
  Seq q;           // sequence s
  uint32_t piece;  // number of P among the walk's
  Piece P;
  int more;
};

struct TileShared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], q_full[2], drain;  // of a tile
  uint64_t p_full[2][2], o_step[2][2];         // of its halves
  uint64_t sc_full[SC_RING], raw_full[2][UNIT / 16];
  float sc_k[SC_RING][8], sc_log[SC_RING][8], sc_inv[SC_RING][8], sc_ref[SC_RING];
  uint64_t red_full[RED_RING];
  float red[RED_RING][KEY_WARPS];  // largest value scales of a piece, by warp
  uint32_t tmem;
  int abort;
  int64_t scratch[T_WARPS + 2];
  Work work;
  Walk walk[T_WARPS];
};


// The next piece of the warp's walk into W.P; false at the end.
// ALONE: called by one thread of a warp.
template <bool ALONE = false>
__device__ __forceinline__ bool next_piece(const AttnParams& p, const Work& w, Walk& W) {
  if (!ALONE) __syncwarp();  // every lane is done with the last piece
  if (ALONE || (threadIdx.x & 31) == 0) {
    Piece& P = W.P;
    W.more = 0;
    while (W.x < w.x1 && !W.more) {
      const Seq q = W.q;
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
      W.piece += W.more;
      W.x += end - W.u;
      W.u = 0;
      if (W.x < w.x1 && ++W.h == p.c.hkv) {
        W.h = 0;
        if (++W.qt == q_tiles<T_ROWS>(p, q)) {
          W.qt = 0;
          do W.q = load_seq(p, ++W.s);
          while (W.q.n == 0);  // x < x1 <= total: a later sequence has rows
        }
      }
    }
  }
  if (!ALONE) __syncwarp();
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

template <class T>
__device__ __forceinline__ T* shfl_ptr(T* x, int lane) {
  return reinterpret_cast<T*>(__shfl_sync(~0u, (unsigned long long)x, lane));
}

// The work is cut as in the streaming kernel, over items of 256 query rows
// (a position's heads next to each other) and units of 128 tokens.
//
// Three warps bring the keys and four the values of each unit, copied one unit
// ahead by bulk copies, and store them as fp16 numbers in the swizzled operand
// layout: the keys' codes raw, as (c + 128) 2^-24 (128 2^-24 times the query
// row's sum comes off the score), the values' as c itself, transposed.  One
// thread issues S = Q K^T and O += P V for two tiles of 128 rows.  The weights
// come in halves of 64 tokens, so that a half's O += P V runs beside the
// softmax of the next and a softmax thread needs few registers; S is asked for
// whole, since with 64 columns Q would be read twice as often as the tensor
// cores allow (342 us against 305).  A softmax thread owns a row: S comes from
// TMEM and P goes back over it as fp16, the second product's A operand, while
// O stays in TMEM for all units.  Weights are taken against the maximum so
// far, in one pass over S; only if a half's add up to more than LIMIT are O and
// the sums rescaled and the pass repeated.
//
// Two prompts of 2600 tokens behind contexts of up to 3000, 32 heads on 8:
// 282 us, 266 GFLOP, 0.48 of the measured bf16 rate; one prompt of 4096 tokens:
// 189 us.  No unit is full: a unit takes some 4000 clocks, of which the tensor
// cores work 2050; the rest is the softmax's chain and the conversion of the
// codes, which run beside each other.
//
// Scales: the key scale of a run of 16 tokens multiplies the fp32 scores.  The
// value scale vs, relative to the item's largest, enters the weights through
// its logarithm: P = 2^(s + log2 vs - M), at most LIMIT whatever the scales
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
      W.q = load_seq(p, found.s);
      W.piece = ~0u;
    }
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], KEY_WARPS);  // one arrival a warp
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.v_full[i], 4);
      mbar_init(&S.v_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i][0], 4);
      mbar_init(&S.p_full[i][1], 4);
      mbar_init(&S.q_full[i], 4);
      mbar_init(&S.o_step[i][0], 1);
      mbar_init(&S.o_step[i][1], 1);
    }
    for (int i = 0; i < SC_RING; ++i) mbar_init(&S.sc_full[i], 1);
    for (int i = 0; i < 2 * UNIT / 16; ++i) mbar_init(&S.raw_full[0][i], 1);
    for (int i = 0; i < RED_RING; ++i) mbar_init(&S.red_full[i], KEY_WARPS - 1);
    mbar_init(&S.drain, 1);
    S.abort = 0;
    fence_mbar_init();
  }
  if (warp == W_MMA) tmem_alloc(&S.tmem, 512);
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
    // ------------------------------------------------------------- softmax
    const int X = warp >> 2, r = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's quarter of the lanes
    const uint32_t s_addr = lanes + S_COL + 128 * X, o_addr = lanes + O_COL + D * X;
    unsigned char* q_tile = sq + X * Smem<D>::Q;
    uint32_t units_done = 0, tiles = 0;  // of the CTA; of this tile
    bool ok = true;
    // A tile that spans CTAs: the parts are counted for each warp's rows (no
    // warp waits for another here), a part that was given up with its bit in
    // the upper half, and the last one sets the count to zero again, whatever
    // became of the others: so the next call finds it as this one did.  True
    // in the warp that comes last, if every part is there.
    auto first_cta = [&]() { return cta_of(S.work, P.first); };
    auto last_cta = [&]() { return cta_of(S.work, P.first + P.n[X] - 1); };
    auto count_part = [&](uint32_t add) {
      static_assert(W_KEYS <= 3 * KV_CTAS_PER_SM, "counters of an SM");
      const int c0 = first_cta();
      uint32_t* counter = p.counters + W_KEYS * c0 + warp;
      uint32_t others = 0;
      if (lane == 0) others = atomicAdd(counter, add);
      others = __shfl_sync(~0u, others, 0);
      if ((others & 0xFFFFu) != (uint32_t)(last_cta() - c0)) return false;
      __threadfence();
      if (lane == 0) *counter = 0;
      return (others + add) >> 16 == 0;
    };
    while (ok && next_piece(p, S.work, S.walk[warp])) {
      const int last = min(P.u1, P.n[X]);
      if (P.u0 >= last) {
        units_done += P.u1 - P.u0;
        continue;
      }
      // The thread's row is a token and a head.
      const uint32_t first_row = (uint32_t)T_ROWS * P.qt + 128 * X, G = p.G;
      const int token0 = first_row / G, token = (first_row + r) / G, head = P.h * (int)G + (first_row + r) % G;
      const bool live_row = token < P.new_rows;
      const int before = P.len - P.new_rows;
      // rows past the last store nothing, so they may see all
      const int limit = live_row ? before + token : INT_MAX;
      const int first_limit = before + token0;
      // ---- the warp's 32 query rows, scaled by a power of two into fp16, in
      // their places in the tile; D / 8 neighbouring lanes take a row, whose
      // address its own thread has.
      constexpr int LPR = D / 8, RPL = 32 / LPR;  // lanes of a row, rows of a turn
      const int c8 = lane % LPR, k8 = 32 * (warp & 3) + lane / LPR;
      auto q_place = [&](int k) { return q_tile + (c8 >> 3) * (128 * 128) + sw128_off(k, c8 & 7); };
      float f = 0.f, off = 0.f;  // score per product; what the keys' 128s add to a product
      {
        const uint16_t* row = live_row ? p.q + (int64_t)(P.row + token) * p.q_stride + head * D : nullptr;
#pragma unroll 1
        for (int b = 0; b < 32; b += 8 * RPL) {
          const uint16_t* src[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) src[i] = shfl_ptr(row, b + i * RPL + lane / LPR);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (src[i])
              cp_async16(q_place(k8 + b + i * RPL), src[i] + 8 * c8);
            else
              *reinterpret_cast<uint4*>(q_place(k8 + b + i * RPL)) = make_uint4(0, 0, 0, 0);
          }
        }
        cp_async_commit();
        cp_async_wait<0>();  // a lane converts what it copied
#pragma unroll 1
        for (int b = 0; b < 32; b += 8 * RPL) {
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const uint4*>(q_place(k8 + b + i * RPL));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t m = 0;  // magnitudes, as whole numbers
#pragma unroll
            for (int e = 0; e < 4; ++e) m = __vmaxu2(m, x[e] & 0x7FFF7FFFu);
#pragma unroll
            for (int o = 1; o < LPR; o *= 2) m = __vmaxu2(m, __shfl_xor_sync(~0u, m, o));
            // the largest goes to [2^14, 2^15); a negative scale goes into the
            // row, so that f is not
            const int ex = min(max((int)(max(m >> 16, m & 0xFFFF) >> 7) - 127, -100), 127);
            const float up = copysignf(__uint_as_float((uint32_t)(127 + 14 - ex) << 23), p.scale_log2);
            // the sum is that of the rows before they are rounded: only what
            // is 2^-29 of the largest and less is
            float2 part = make_float2(0.f, 0.f);
            auto two = [&](float a, float b) {
              const float2 y = make_float2(a * up, b * up);
              part = add2(part, y);
              return half2_bits(__float22half2_rn(y));
            };
            // channels in the keys' order: 0 2 1 3 of every four
            *reinterpret_cast<uint4*>(q_place(k8 + b + i * RPL)) =
                make_uint4(two(bf16lo(x[0]), bf16lo(x[1])), two(bf16hi(x[0]), bf16hi(x[1])), two(bf16lo(x[2]), bf16lo(x[3])),
                           two(bf16hi(x[2]), bf16hi(x[3])));
            float sum = part.x + part.y;
#pragma unroll
            for (int o = 1; o < LPR; o *= 2) sum += __shfl_xor_sync(~0u, sum, o);
            // to the lanes that own the rows
            const int ex_of = __shfl_sync(~0u, ex, (lane % RPL) * LPR);
            const float sum_of = __shfl_sync(~0u, sum, (lane % RPL) * LPR);
            if (lane / RPL == b / RPL + i) {
              f = __uint_as_float((uint32_t)(127 - 14 + ex_of) << 23) * fabsf(p.scale_log2) * 0x1p12f;
              off = sum_of * 0x1p-17f;  // 128 * 2^-24
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.q_full[X]);
      }
      float M = -INFINITY, l = 0.f, ref = 1.f;
      for (int u = P.u0; u < last && ok; ++u, ++tiles) {
        const uint32_t it = units_done + u - P.u0, slot = it % SC_RING;
        if (!(ok = wait_warp(&S.s_full[X], tiles & 1, 51))) break;
        // the scales' barrier second: scores imply that its phase is this
        // unit's, not one of an earlier turn
        if (!(ok = wait_warp(&S.sc_full[slot], (it / SC_RING) & 1, 52))) break;
        tc_fence_after();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint32_t sh = s_addr + 64 * half;
          const float *sck = S.sc_k[slot] + 4 * half, *scl = S.sc_log[slot] + 4 * half, *sci = S.sc_inv[slot] + 4 * half;
          const int pos0 = u * UNIT + 64 * half;
          const int see = limit - pos0;  // the last token of the half that this row sees
          ref = S.sc_ref[slot];
          if (pos0 + 63 > first_limit) {  // the causal edge: what a row does not see becomes -inf in place
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t v[32];
              tmem_ld32(sh + 32 * c, v);
              tmem_ld_wait();
              ld32_fence(v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 32 * c + i <= see ? v[i] : 0xFF800000u;
              tmem_st<32>(sh + 32 * c, v);
            }
            tmem_st_wait();
          }
          // Scores are S a + log2 vs - off a, a >= 1e-30 so that -inf stays
          // what it is.
          auto largest = [&]() {
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t v[32];
              tmem_ld32(sh + 32 * c, v);
              tmem_ld_wait();
              ld32_fence(v);
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2) {
                float mx = -INFINITY;
#pragma unroll
                for (int i = 16 * h2; i < 16 * h2 + 16; ++i) mx = fmaxf(mx, __uint_as_float(v[i]));
                const float a = fmaxf(f * sck[2 * c + h2], 1e-30f);
                top = fmaxf(top, fmaf(mx, a, fmaf(-off, a, scl[2 * c + h2])));
              }
            }
            return top;
          };
          if (__any_sync(~0u, M == -INFINITY)) {  // nothing seen so far: the row's maximum
            const float top = largest();
            if (M == -INFINITY) M = top - ABOVE;  // nothing summed yet: nothing to rescale
          }
          // ---- the weights against the maximum so far; again, with the sums
          // rescaled, if a row's outgrow LIMIT.  Scores and their maximum are
          // rounded alike before M comes off, so that the largest weight is
          // 2^ABOVE but for the rounding of M, 4 times at most, however large
          // the scores are
          uint32_t w[2][16];
          float add;
          for (int again = 0;; ++again) {
            const float at = M == -INFINITY ? 0.f : M;
            add = 0.f;
            float all = 0.f;
            uint32_t vb[2][32];
            tmem_ld32(sh, vb[0]);
            tmem_ld32(sh + 32, vb[1]);
            tmem_ld_wait();
            ld32_fence(vb[0]);
            ld32_fence(vb[1]);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2) {
                const float a = fmaxf(f * sck[2 * c + h2], 1e-30f);
                const float b = fmaf(-off, a, scl[2 * c + h2]);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 16 * h2; i < 16 * h2 + 16; i += 2) {
                  // rounded as `largest` rounds, and only then taken off M
                  float2 z = fma2(make_float2(__uint_as_float(vb[c][i]), __uint_as_float(vb[c][i + 1])),
                                  make_float2(a, a), make_float2(b, b));
                  z = add2(z, make_float2(-at, -at));
                  z = make_float2(ex2(z.x), ex2(z.y));
                  sum = add2(sum, z);
                  w[c][i >> 1] = half2_bits(__float22half2_rn(z));
                }
                add = fmaf(sum.x + sum.y, sci[2 * c + h2], add);
                all += sum.x + sum.y;
              }
            // no weight above the limit if their sum is not
            if (again || !__any_sync(~0u, all > LIMIT)) break;
            const float top = largest();  // by the whole warp
            const float to = all > LIMIT ? fmaxf(top - ABOVE, at) : at, drop = ex2(at - to);
            if (all > LIMIT) M = to;
            l *= drop;
            if (u > P.u0 || half) {
              // O is the first half's until its product has ended (the products
              // before have: the unit's scores came after them)
              if (half && !(ok = wait_warp(&S.o_step[X][0], tiles & 1, 53))) break;
              tc_fence_after();
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
          if (!ok) break;
          l += add;
          tmem_st<16>(sh, w[0]);
          tmem_st<16>(sh + 16, w[1]);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.p_full[X][half]);
        }
      }
      if (!ok) break;
      units_done += P.u1 - P.u0;
      // ---- the piece's sums
      if (!(ok = wait_warp(&S.o_step[X][1], (tiles - 1) & 1, 53))) break;
      tc_fence_after();
      // Results go out through the rows' places in the query tile, which no
      // product reads any more: whole rows a store instead of 32 pieces of 16
      // bytes.
      auto put = [&](int chunk, uint4 v) {
        *reinterpret_cast<uint4*>(q_tile + (chunk >> 3) * (128 * 128) + sw128_off(r, chunk & 7)) = v;
      };
      auto write_out = [&]() {
        __syncwarp();
        uint16_t* row = live_row ? p.out + ((size_t)(P.row + token) * p.hq + head) * D : nullptr;
#pragma unroll 1
        for (int b = 0; b < 32; b += 8 * RPL) {
          uint16_t* dst[8];
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dst[i] = shfl_ptr(row, b + i * RPL + lane / LPR);
            v[i] = *reinterpret_cast<const uint4*>(q_place(k8 + b + i * RPL));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (dst[i]) *reinterpret_cast<uint4*>(dst[i] + 8 * c8) = v[i];
        }
        __syncwarp();
      };
      if (P.u0 == 0 && last == P.n[X]) {  // all of the tile's units
        const float k = l == 0.f ? 0.f : ref / l;
#pragma unroll 2
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(o_addr + 32 * c, v);
          tmem_ld_wait();
          ld32_fence(v);
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(v[i + 2 * e]) * k, __uint_as_float(v[i + 2 * e + 1]) * k);
            put(4 * c + i / 8, make_uint4(w[0], w[1], w[2], w[3]));
          }
        }
        tc_fence_before();
        write_out();
      } else {
        // a tile that spans CTAs: the last one to finish joins the parts in order
        const int c0 = first_cta(), c1 = last_cta();
        auto part = [&](int c) { return p.partials + (size_t)((2 * c + (c == c0)) * 2 + X) * partial_floats<D>(); };
        float* mine = part(blockIdx.x);
#pragma unroll 1
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
        __syncwarp();
        if (count_part(1)) {
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
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              put((d + i) / 8, make_uint4(pack_bf16x2(acc[i], acc[i + 1]), pack_bf16x2(acc[i + 2], acc[i + 3]),
                                          pack_bf16x2(acc[i + 4], acc[i + 5]), pack_bf16x2(acc[i + 6], acc[i + 7])));
          }
          write_out();
        }
      }
    }
    if (!ok) {  // a wait gave up: this piece and those that would have come
      do {
        const int last = min(P.u1, P.n[X]);
        if (P.u0 < last && !(P.u0 == 0 && last == P.n[X])) count_part(0x10001u);
      } while (next_piece(p, S.work, S.walk[warp]));
    }
  } else if (warp == W_MMA) {
    // ------------------------------------------------------------ products
    if (elect_one()) {
      constexpr uint32_t ID_S = idesc_f16(128, UNIT), ID_O = idesc_f16(128, D);
      uint32_t it = 0, q_turn[2] = {0, 0}, p_turn[2] = {0, 0};
      bool ok = true;
      auto scores = [&](int X, uint32_t unit) {
        const uint32_t q0 = smem_u32(sq + X * Smem<D>::Q), k0 = smem_u32(sk + (unit & 1) * Smem<D>::K);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t o = (k >> 2) * (128 * 128) + (k & 3) * 32;
          mma_bf16(tmem + S_COL + 128 * X, desc_sw128(q0 + o), desc_sw128(k0 + o), ID_S, k > 0);
        }
        mma_commit(&S.s_full[X]);
      };
      auto outputs = [&](int X, uint32_t unit, int half, bool first) {
        const uint32_t v0 = smem_u32(sv + (unit & 1) * Smem<D>::V) + half * (D * 128);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16_ta(tmem + O_COL + D * X, tmem + S_COL + 128 * X + 64 * half + 8 * k, desc_sw128(v0 + k * 32), ID_O,
                      !first || k > 0);
        mma_commit(&S.o_step[X][half]);
      };
      while (ok && next_piece<true>(p, S.work, S.walk[warp])) {
        const int last[2] = {min(P.u1, P.n[0]), min(P.u1, P.n[1])};
        // unit `it` is the piece's first
#pragma unroll
        for (int X = 0; X < 2; ++X)
          if (ok && P.u0 < last[X]) ok = wait(&S.q_full[X], q_turn[X]++ & 1, 56);
        if (!ok || !(ok = wait(&S.k_full[it & 1], (it >> 1) & 1, 57))) break;
        tc_fence_after();
#pragma unroll
        for (int X = 0; X < 2; ++X)
          if (P.u0 < last[X]) scores(X, it);
        mma_commit(&S.k_empty[it & 1]);
        for (int u = P.u0; u < P.u1 && ok; ++u, ++it) {
          if (!(ok = wait(&S.v_full[it & 1], (it >> 1) & 1, 58))) break;
          const bool more = u + 1 < P.u1;
          bool have_k = false;
#pragma unroll
          for (int X = 0; X < 2; ++X)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (!ok || u >= last[X]) continue;
              // one barrier a half: the softmax may be a half ahead
              if (!(ok = wait(&S.p_full[X][half], p_turn[X] & 1, 59))) continue;
              p_turn[X] += half;
              tc_fence_after();
              outputs(X, it, half, u == P.u0 && half == 0);
              if (half && u + 1 < last[X]) {
                if (!have_k && !(ok = wait(&S.k_full[(it + 1) & 1], ((it + 1) >> 1) & 1, 60))) continue;
                have_k = true;
                tc_fence_after();
                scores(X, it + 1);
              }
            }
          mma_commit(&S.v_empty[it & 1]);
          if (more) {
            if (!have_k && ok) ok = wait(&S.k_full[(it + 1) & 1], ((it + 1) >> 1) & 1, 60);
            mma_commit(&S.k_empty[(it + 1) & 1]);
          }
        }
      }
      if (!ok) {  // after a wait that gave up: the products in flight end before TMEM goes
        int never = 0;
        mma_commit(&S.drain);
        mbar_wait(&S.drain, 0, &never, WAIT_NS);
      }
    }
  } else {
    // ------------------------------------------------------- keys or values
    // The codes come in runs of 16 tokens, one bulk copy each, a unit ahead:
    // a warp waits for its own runs, converts them and asks for the next
    // unit's into the same places.
    // The first CTA asks for none under the MOE_STALL_WEIGHT_COPIES test hook:
    // its waits run out.
    const bool keys = warp < W_VALUES;
    const bool stalled = blockIdx.x == 0 && (p.st->stall & MOE_STALL_WEIGHT_COPIES);
    const int w = keys ? warp - W_KEYS : warp - W_VALUES;
    // keys: runs w, w + KEY_WARPS, ..; values: runs 2 w and 2 w + 1
    constexpr int RUN = 16 * D, RUNS = UNIT / 16;
    const int run0 = keys ? w : 2 * w, run_step = keys ? KEY_WARPS : 1, run1 = keys ? RUNS : 2 * w + 2;
    const int64_t page_bytes = (int64_t)hkv * p.c.block * D;
    unsigned char* mine = raw + (keys ? 0 : UNIT * D);
    uint64_t* came = S.raw_full[keys ? 0 : 1];
    // keys: D / 16 neighbouring lanes take a token's pieces of 16 codes, one
    // half (k_flip) before the other, which keeps loads and stores of eight
    // lanes in different banks
    constexpr int PIECES = D / 16, ROWS = 32 / PIECES;
    const int kc = lane % PIECES, kr = lane / PIECES;
    const int k_flip = D == 128 ? ((kc >> 2) ^ kr) & 1 : (kr >> 1) & 1;
    // values: 8 tokens vo of the warp's 32, piece vc; words (q + v_turn) % 4 of
    // it, again for the banks
    const int vo = 4 * w + (lane & 3), vc = (lane >> 2) % PIECES;
    const int v_turn = (lane & 3) + vc + (D == 128 ? 0 : 2 * (lane >> 4));
    // Where the pieces come from and go to, worked out once: a key half of the
    // first rows of a run (an odd turn's rows lie 4 or 8 on), a value word.
    uint32_t k_to[2][2], v_to[D / 32], v_ch[4];
    int k_from[2], v_from[D / 32];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      k_from[e] = kr * D + 16 * kc + 8 * (k_flip ^ e);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        k_to[i][e] = (kc >> 2) * (128 * 128) + sw128_off(ROWS * i + kr, 2 * (kc & 3) + (k_flip ^ e));
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int q = (i + v_turn) & 3;
      v_from[i] = 8 * vo * D + 16 * vc + 4 * q;
      v_to[i] = (vo >> 3) * (D * 128) + (2 * vc + (q >> 1)) * 1024 + (q & 1) * 512 + (((vo >> 2) ^ q) & 1) * 64;
    }
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) v_ch[ch] = ch * 128 + (((vo & 3) ^ ch) << 4);
    uint32_t it = 0;
    bool ok = true;
    while (ok && next_piece(p, S.work, S.walk[warp])) {
      const int32_t* table = p.c.table + (size_t)P.s * p.c.max_blocks;
      const int8_t* codes = p.c.codes + (keys ? 0 : p.c.n_pages * page_bytes) + (int64_t)P.h * p.c.block * D;
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
      // one run of unit u < end, by one lane; a run without a page is read from
      // page 0: its weights are 0
      auto fetch = [&](int u, int run, int page) {
        if (stalled) return;
        mbar_arrive_expect_tx(&came[run], RUN);
        bulk_copy_g2s(mine + run * RUN, codes + max(page, 0) * page_bytes + ((u * UNIT + 16 * run) & (p.c.block - 1)) * D, RUN,
                      &came[run]);
      };
      // pages come two units ahead, codes and scales one
      int pages = pages_of(P.u0), next_pages = pages_of(P.u0 + 1);
      if (lane >= run0 && lane < run1 && (lane - run0) % run_step == 0) fetch(P.u0, lane, pages);
      float ks = 0.f, vs = 0.f, vref = 0.f, vref_log = 0.f;
      if (keys) {
        ks = scale_of(pages, 0);
        vs = scale_of(pages, 1);
        // the item's largest value scale; 0 if every value is, and then so is
        // the result
        for (int b = 32 * w + lane; b << p.block_log2 < seen; b += 32 * KEY_WARPS)
          vref = fmaxf(vref, scale_of(page_at(b << p.block_log2), 1));
#pragma unroll
        for (int o = 16; o; o >>= 1) vref = fmaxf(vref, __shfl_xor_sync(~0u, vref, o));
        // the first warp, which writes the scales, has the others'; a warp is two
        // pieces ahead of it at most, as the stages hold two units
        const uint32_t piece = S.walk[warp].piece, slot = piece % RED_RING;
        if (w && lane == 0) {
          S.red[slot][w] = vref;
          mbar_arrive(&S.red_full[slot]);
        }
        if (w == 0) {
          if (!(ok = wait_warp(&S.red_full[slot], (piece / RED_RING) & 1, 61))) {
            for (int run = run0; run < run1 && !stalled; run += run_step) {
              int never = 0;
              mbar_wait(&came[run], it & 1, &never, WAIT_NS);
            }
            break;
          }
          for (int i = 1; i < KEY_WARPS; ++i) vref = fmaxf(vref, S.red[slot][i]);
        }
        vref_log = vref > 0.f ? __log2f(vref) : 0.f;
      }
      for (int u = P.u0; u < end; ++u, ++it) {
        const uint32_t st = it & 1, par = ((it >> 1) & 1) ^ 1;
        int run = run0;
        ok = wait_warp(keys ? &S.k_empty[st] : &S.v_empty[st], par, 54);
        if (ok && keys && w == 0 && lane < 8) {
          // the slot's last unit, SC_RING back, is past every softmax thread:
          // the products that freed this K stage came after its weights
          const uint32_t slot = it % SC_RING;
          const float lg = pages < 0 ? -INFINITY : fmaxf(__log2f(vs) - vref_log, -60.f);
          S.sc_k[slot][lane] = ks * 0x1p12f;  // half of the codes' 2^24; the row's factor has the other half
          S.sc_log[slot][lane] = lg;
          S.sc_inv[slot][lane] = pages < 0 ? 0.f : ex2(-lg);
          if (lane == 0) S.sc_ref[slot] = vref;
          __syncwarp(0xFF);
          if (lane == 0) mbar_arrive(&S.sc_full[slot]);
        }
        for (; ok && run < run1; run += run_step) {
          if (!(ok = wait_warp(&came[run], it & 1, 55))) break;
          if (keys) {
            unsigned char* dst = sk + st * Smem<D>::K + 2048 * run;
            const unsigned char* src = mine + run * RUN;
            // all loads of the run first: with each before its store the run
            // took three times as long
            uint2 v[16 / ROWS][2];
#pragma unroll
            for (int i = 0; i < 16 / ROWS; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                v[i][e] = *reinterpret_cast<const uint2*>(src + k_from[e] + ROWS * i * D);
#pragma unroll
            for (int i = 0; i < 16 / ROWS; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                *reinterpret_cast<uint4*>(dst + k_to[i & 1][e] + 1024 * (i >> 1)) =
                    make_uint4(codes_even(v[i][e].x), codes_odd(v[i][e].x), codes_even(v[i][e].y), codes_odd(v[i][e].y));
          } else if (run & 1) {  // both of the warp's runs are there
            unsigned char* dst = sv + st * Smem<D>::V;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              uint32_t x[8];
#pragma unroll
              for (int t = 0; t < 8; ++t) x[t] = *reinterpret_cast<const uint32_t*>(mine + v_from[i] + t * D);
              // channel 4 q + ch of the piece: row 4 (q & 1) + ch of an 8-row group
              auto put = [&](int ch, uint4 v) { *reinterpret_cast<uint4*>(dst + (v_to[i] + v_ch[ch])) = v; };
              put(0, make_uint4(f16_pair<0>(x[0], x[1]), f16_pair<0>(x[2], x[3]), f16_pair<0>(x[4], x[5]), f16_pair<0>(x[6], x[7])));
              put(1, make_uint4(f16_pair<1>(x[0], x[1]), f16_pair<1>(x[2], x[3]), f16_pair<1>(x[4], x[5]), f16_pair<1>(x[6], x[7])));
              put(2, make_uint4(f16_pair<2>(x[0], x[1]), f16_pair<2>(x[2], x[3]), f16_pair<2>(x[4], x[5]), f16_pair<2>(x[6], x[7])));
              put(3, make_uint4(f16_pair<3>(x[0], x[1]), f16_pair<3>(x[2], x[3]), f16_pair<3>(x[4], x[5]), f16_pair<3>(x[6], x[7])));
            }
          }
          if (u + 1 < end && (keys || (run & 1))) {
            const int page = __shfl_sync(~0u, next_pages, run), page0 = __shfl_sync(~0u, next_pages, run & ~1);
            __syncwarp();  // every lane has read the run
            if (lane == 0) {
              if (!keys) fetch(u + 1, run - 1, page0);
              fetch(u + 1, run, page);
            }
          }
        }
        if (!ok) {  // after a wait that gave up: the copies in flight end before the block's memory goes
          int never = 0;
          for (int r = run0; r < run1 && !stalled; r += run_step) {
            const bool ahead = keys ? r < run : false;  // asked for unit u + 1 already
            if (!ahead || u + 1 < end) mbar_wait(&came[r], (it + ahead) & 1, &never, WAIT_NS);
          }
          break;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(keys ? &S.k_full[st] : &S.v_full[st]);
        pages = next_pages;
        next_pages = pages_of(u + 2);
        if (keys && w == 0) {
          ks = scale_of(pages, 0);
          vs = scale_of(pages, 1);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_MMA) tmem_dealloc(tmem, 512);
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
