// Causal attention over the paged 8-bit key/value cache (moe_kv_attention).
#include <limits.h>
#include <math.h>

#include "kv_attention.cuh"

namespace moe {

namespace {

constexpr int AT_WARPS = 4;
constexpr int AT_THREADS = AT_WARPS * 32;
constexpr float ABOVE = 14.f;                        // the largest fp16 weight is 2^ABOVE
constexpr int WARP_TOKENS = 32;                      // tokens of one warp step
static_assert(UNIT == AT_WARPS * WARP_TOKENS, "a CTA step is a unit");

// Variants by the rows of a query tile, 8 NT: how many CTAs an SM holds and
// how many steps a warp's ring.
template <int NT>
struct Shape {
  static constexpr int ROWS = 8 * NT, CTAS = NT == 1 ? 3 : 2, STAGES = NT == 1 ? 2 : 3;
};

template <int D, int NT>
constexpr int at_smem() {
  const int ring = AT_WARPS * Shape<NT>::STAGES * 2 * WARP_TOKENS * D, sums = AT_WARPS * 8 * NT * (D + 4) * 4;
  return ring > sums ? ring : sums;
}

// Where the 16-byte piece c of token t's key or value goes among a step's 32,
// so that the lanes of one shared-memory pass read different banks: pieces
// j of two tokens for the keys, piece g of four tokens 2 j apart by two for
// the values.
template <int D>
__device__ __forceinline__ int k_at(int t, int c) {
  return D == 128 ? t * 128 + ((c ^ (t & 1) << 2) << 4) : t * 64 + (c << 4);
}
template <int D>
__device__ __forceinline__ int v_at(int t, int c) {
  if (D == 128) return t * 128 + ((c ^ (t & 7)) << 4);
  const int r = (t >> 1 & 15) | (t & 1) << 4;
  return r * 64 + ((c ^ (r & 2)) << 4);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Codes c of bytes 0 and 2, and of bytes 1 and 3, as the fp16 numbers
// (c + 128) * 2^-24: below fp16's normal range the bits are the value.
__device__ __forceinline__ uint32_t codes_even(uint32_t w) { return (w ^ 0x80808080u) & 0x00FF00FFu; }
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) { return ((w >> 8) ^ 0x00808080u) & 0x00FF00FFu; }

// Byte B of two words as exact fp16 numbers: under the exponent of 1024 the
// byte c ^ 0x80 is 1024 + 128 + c.
template <int B>
__device__ __forceinline__ uint32_t codes_pair(uint32_t a, uint32_t b) {
  const uint32_t v = (__byte_perm(a, b, B | (4 + B) << 8) & 0x00FF00FFu) ^ 0x64806480u;
  return half2_bits(__hsub2(*reinterpret_cast<const __half2*>(&v), __floats2half2_rn(1152.f, 1152.f)));
}

// The work is the list of all (sequence, query tile, key/value head) items,
// each as many 128-token steps as its rows see, cut into equal runs of steps,
// one a CTA: long and short sequences load the SMs alike.  An item that
// spans several CTAs leaves a partial result per CTA; the last CTA to finish
// joins them in CTA order.
//
// Within an item the CTA's four warps take 32 tokens each per step and hold
// all 8 NT query rows.  Each warp keeps its next step or two in flight by
// asynchronous copies into a ring of its own.  The products are taken
// transposed, S^T = K Q^T and O^T = V^T P^T in m16n8k16, so that tokens and
// channels fill the 16 rows and eight query rows, a common group of heads,
// the eight columns; S^T's fragments become P^T's by 8 x 8 transposes.  The
// order of the channels inside a product of q and k is free (both operands
// use the same), and so is the order of the output channels, so a lane reads
// 16 bytes in a row of a key and of a value as its part of the fragments.
//
// Codes enter exactly.  A key's code is read as (c + 128) 2^-24, and 128 2^-24
// times the query row's sum is taken off the score (8 products deep, so the
// difference loses nothing that matters); values, summed over all tokens, are
// converted to c itself.  The key scale multiplies the fp32 scores; the value
// scale enters the weights, p_j = exp2(s_j - m) vs_j, through its logarithm
// with a running maximum of its own, so that the fp16 weights are at most
// 2^ABOVE whatever the scales are; that far up, those that fp16 rounds to
// nothing are below 2^-39 of the largest (2^-25 without it: what the small
// weights of a long context add up to was lost).  That maximum, V, is of
// s_j - m + log2 vs_j: beside large scores the logarithm would lose its bits
// (a value 4% off at scores of 2^20, in powers of two).
//
// 48 sequences of up to 20000 tokens, 32 heads on 4, one new token each: 108 us
// for 626 MB, 0.86 of the copy rate; the unpacking (ALU pipe 0.6 full) is next.
template <int D, int NT>
__global__ void __launch_bounds__(AT_THREADS, Shape<NT>::CTAS) kv_attention_kernel(AttnParams p) {
  constexpr int ROWS = Shape<NT>::ROWS, STAGES = Shape<NT>::STAGES;
  constexpr int KL = D / 64;   // 16-byte loads of a key per lane
  constexpr int VW = D / 32;   // 4-byte words of a value per lane
  constexpr int NO = D / 16;   // output tiles of 16 channels
  constexpr int STAGE = 2 * WARP_TOKENS * D;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* ring = smem + (threadIdx.x >> 5) * STAGES * STAGE;
  float(*osum)[ROWS][D + 4] = reinterpret_cast<float(*)[ROWS][D + 4]>(smem);  // after an item's steps
  __shared__ float sm[AT_WARPS][ROWS], sV[AT_WARPS][ROWS], sl[AT_WARPS][ROWS];
  __shared__ int64_t scan[AT_WARPS + 2];
  __shared__ uint32_t arrived;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, j = lane & 3;
  const int hkv = p.c.hkv;

  Work wk;
  if (!find_work<ROWS, AT_THREADS>(p, scan, wk)) return;
  const int64_t x1 = wk.x1;
  const int cta = blockIdx.x;
  int s = wk.s, qt = wk.qt, h = wk.h, u0 = wk.u;
  Seq q = load_seq(p, s);

  int64_t x = wk.x0;
  while (x < x1) {
    const int units = tile_units<ROWS>(p, q, qt), seen = tile_seen<ROWS>(p, q, qt);
    const int u1 = (int)min((int64_t)units, u0 + (x1 - x));
    const int rows = (int)min(seq_rows(p, q) - (uint32_t)qt * ROWS, (uint32_t)ROWS);
    // The loads that wait for one another come first: the rows of q beside the
    // pages, then codes and scales by the pages, and the arithmetic on q last.
    uint2 q_raw[NT][KL * 4];
    int q_token[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t rr = (uint32_t)qt * ROWS + 8 * t + g;
      const int i = (int)(rr / (uint32_t)p.G), head = h * p.G + (int)(rr % (uint32_t)p.G);
      q_token[t] = i;
#pragma unroll
      for (int w = 0; w < KL * 4; ++w) {
        q_raw[t][w] = make_uint2(0, 0);
        if (8 * t + g < rows)
          q_raw[t][w] = *reinterpret_cast<const uint2*>(p.q + (int64_t)(q.row + i) * p.q_stride + (size_t)head * D +
                                                        64 * (w >> 2) + 16 * j + 4 * (w & 3));
      }
    }
    float m[NT][2], V[NT][2], l[NT][2], o[NT][NO][4];  // o: in units of 2^(m + V - ABOVE)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = V[t][0] = V[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int i = 0; i < NO; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
    }

    // a lane copies 16 bytes, piece lane_c of every (512 / D)-th token from lane_tok on
    const int lane_c = lane % (D / 16), lane_tok = lane / (D / 16);
    const int64_t page_bytes = (int64_t)hkv * p.c.block * D, vstep = p.c.n_pages * page_bytes;
    const int8_t* lane_k = p.c.codes + (int64_t)h * p.c.block * D + lane_tok * D + 16 * lane_c;
    // this warp's steps: 32 tokens each, UNIT apart
    const int first = u0 * UNIT + warp * WARP_TOKENS, stop = min(u1 * UNIT, seen);
    const int steps = first < stop ? (stop - first + UNIT - 1) / UNIT : 0;
    // Page and scales of the runs of 16 tokens, two a step, run r in lane
    // r % 32, fetched a chunk of 16 steps ahead.
    auto page_of = [&](int chunk) {
      const int step = chunk * 16 + (lane >> 1), pos = first + step * UNIT + 16 * (lane & 1);
      if (step >= steps || pos >= seen) return -1;
      const int page = __ldg(p.c.table + (size_t)s * p.c.max_blocks + (pos >> p.block_log2));
      if (page >= 0 && page < p.c.n_pages) return page;
      raise_flag(p.st, FLAG_BAD_CACHE);
      return -1;
    };
    auto scale_of = [&](int page, int isv) {
      return page < 0 ? 1.f : __ldg(p.c.scales + ((size_t)isv * p.c.n_pages + page) * hkv + h);
    };
    int chunk_now = 0;
    int page = page_of(0), next_page = page_of(1);
    float kscale, vscale, next_k = 0.f, next_v = 0.f;
    auto issue = [&](int step) {
      if (step < steps) {
        unsigned char* dst = ring + (step % STAGES) * STAGE;
        const int pg_lane = (step >> 4) != chunk_now ? next_page : page;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int pg = __shfl_sync(~0u, pg_lane, (2 * step + r) & 31);
          if (pg < 0) continue;
          const int8_t* k = lane_k + pg * page_bytes + ((first + step * UNIT + 16 * r) & (p.c.block - 1)) * D;
          const int8_t* v = k + vstep;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            cp_async16(dst + k_at<D>(16 * r + lane_tok + i * (512 / D), lane_c), k + 512 * i);
            cp_async16(dst + 32 * D + v_at<D>(16 * r + lane_tok + i * (512 / D), lane_c), v + 512 * i);
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < (STAGES > 2 ? STAGES - 1 : 2); ++i) issue(i);
    kscale = scale_of(page, 0), vscale = scale_of(page, 1);

    // ---- query fragments, each row scaled by a power of two into fp16
    uint32_t qb[NT][KL * 4][2];
    float F[NT][2], off_q[NT][2];  // of rows 2 j, 2 j + 1: score per product, 128 2^-24 times the row's sum
    int limit[NT][2];              // last position seen
    int all_see = INT_MAX;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + g;
      const int i = q_token[t];
      const uint2(&raw)[KL * 4] = q_raw[t];
      float m = 0.f, sum = 0.f;
#pragma unroll
      for (int w = 0; w < KL * 4; ++w) {
        m = fmaxf(m, fmaxf(fmaxf(fabsf(bf16lo(raw[w].x)), fabsf(bf16hi(raw[w].x))),
                           fmaxf(fabsf(bf16lo(raw[w].y)), fabsf(bf16hi(raw[w].y)))));
      }
      m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
      m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
      // the row's largest magnitude goes to [2^14, 2^15)
      const int ex = min(max((int)(__float_as_uint(m) >> 23) - 127, -100), 127);
      const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
#pragma unroll
      for (int w = 0; w < KL * 4; ++w) {
        // with the keys' bytes 0 and 2, then 1 and 3
        const __half2 a = __floats2half2_rn(bf16lo(raw[w].x) * up, bf16lo(raw[w].y) * up);
        const __half2 b = __floats2half2_rn(bf16hi(raw[w].x) * up, bf16hi(raw[w].y) * up);
        qb[t][w][0] = half2_bits(a);
        qb[t][w][1] = half2_bits(b);
        sum += (__low2float(a) + __high2float(a)) + (__low2float(b) + __high2float(b));
      }
      sum += __shfl_xor_sync(~0u, sum, 1);
      sum += __shfl_xor_sync(~0u, sum, 2);
      // 2^24 of the codes, half here and half with the key scale: neither then
      // passes fp32's range before their product does
      const float f = __uint_as_float((uint32_t)(127 - 14 + ex) << 23) * p.scale_log2 * 0x1p12f;
      // rows past the last: nothing of theirs is stored, so they may see all
      const int lim = r < rows ? q.len - q.n + i : INT_MAX;
      all_see = min(all_see, lim);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        F[t][c] = __shfl_sync(~0u, f, 4 * (2 * j + c));
        off_q[t][c] = __shfl_sync(~0u, sum, 4 * (2 * j + c)) * 0x1p-17f;
        limit[t][c] = __shfl_sync(~0u, lim, 4 * (2 * j + c));
      }
    }
    all_see = __reduce_min_sync(~0u, all_see);

    for (int i = 0; i < steps; ++i) {
      if ((i & 15) == 0 && i) {  // the next chunk's runs
        page = next_page;
        kscale = next_k;
        vscale = next_v;
        ++chunk_now;
        next_page = page_of(chunk_now + 1);
      }
      if ((i & 15) == 8) {
        next_k = scale_of(next_page, 0);
        next_v = scale_of(next_page, 1);
      }
      cp_async_wait<(STAGES > 2 ? STAGES - 2 : 1)>();
      __syncwarp();  // this step's codes are there, and the last step's are read by every lane
      if (STAGES > 2) issue(i + STAGES - 1);
      const unsigned char* src = ring + (i % STAGES) * STAGE;
      const int pos0 = first + i * UNIT;
      float ksc[2], vlog[2];
      bool live[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int run = (2 * i + r) & 31;
        live[r] = __shfl_sync(~0u, page, run) >= 0;
        ksc[r] = __shfl_sync(~0u, kscale, run) * 0x1p12f;
        vlog[r] = __log2f(__shfl_sync(~0u, vscale, run));
      }
      // ---- scores: row g of tile a is token 16 a + g, column c query row c
      float sc[NT][2][4] = {};
#pragma unroll
      for (int e = 0; e < KL; ++e) {
        uint32_t kw[2][2][4];  // of either run, tokens g and g + 8
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + k_at<D>(16 * a + 8 * o + g, 4 * e + j));
            kw[a][o][0] = v.x, kw[a][o][1] = v.y, kw[a][o][2] = v.z, kw[a][o][3] = v.w;
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int a = 0; a < 2; ++a) {  // the runs' chains side by side
            const uint32_t k[4] = {codes_even(kw[a][0][i]), codes_even(kw[a][1][i]), codes_odd(kw[a][0][i]),
                                   codes_odd(kw[a][1][i])};
#pragma unroll
            for (int t = 0; t < NT; ++t) mma_f16(sc[t][a], k, qb[t][4 * e + i][0], qb[t][4 * e + i][1]);
          }
      }
      const bool whole = live[0] && live[1] && pos0 + WARP_TOKENS - 1 <= all_see;
      uint32_t pb[NT][2][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float f = F[t][c] * ksc[a], d = -off_q[t][c] * f;
            sc[t][a][c] = fmaf(sc[t][a][c], f, d);
            sc[t][a][2 + c] = fmaf(sc[t][a][2 + c], f, d);
          }
        if (!whole) {
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!live[a] || pos0 + 16 * a + 8 * (e >> 1) + g > limit[t][e & 1]) sc[t][a][e] = -INFINITY;
        }
        // ---- the running maxima; V at first against the old m, so that both
        // go through the lanes side by side
        float um[2], uV[2], nV[2], down[2];
        bool far = false;
        auto top_V = [&](int c, float ref) {
          return fmaxf(fmaxf(sc[t][0][c], sc[t][0][2 + c]) - ref + vlog[0],
                       fmaxf(sc[t][1][c], sc[t][1][2 + c]) - ref + vlog[1]);
        };
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float old = m[t][c];
          float nm = fmaxf(fmaxf(sc[t][0][c], sc[t][0][2 + c]), fmaxf(sc[t][1][c], sc[t][1][2 + c]));
          nV[c] = top_V(c, old);
#pragma unroll
          for (int s = 4; s < 32; s *= 2) {
            nm = fmaxf(nm, __shfl_xor_sync(~0u, nm, s));
            nV[c] = fmaxf(nV[c], __shfl_xor_sync(~0u, nV[c], s));
          }
          m[t][c] = nm = fmaxf(nm, old);
          // rows that have seen nothing yet: any finite reference does
          um[c] = nm == -INFINITY ? 0.f : nm;
          down[c] = old - um[c];
          nV[c] += down[c];
          l[t][c] *= ex2(down[c]);
          far |= nm != old && !(down[c] > -1024.f);
        }
        if (__any_sync(~0u, far)) {  // an old maximum far off, or none
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            nV[c] = top_V(c, um[c]);
#pragma unroll
            for (int s = 4; s < 32; s *= 2) nV[c] = fmaxf(nV[c], __shfl_xor_sync(~0u, nV[c], s));
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float was = V[t][c] + down[c];  // what was, against the new m
          V[t][c] = nV[c] = fmaxf(nV[c], was);  // (-inf in all places gives no number: then that of `was`)
          uV[c] = nV[c] == -INFINITY ? 0.f : nV[c];
          if (__any_sync(~0u, nV[c] != was)) {
            const float drop = ex2(was - uV[c]);
#pragma unroll
            for (int i = 0; i < NO; ++i) {
              o[t][i][c] *= drop;
              o[t][i][2 + c] *= drop;
            }
          }
        }
        // ---- weights, transposed into the second product's operand
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const float v0 = vlog[a] + ABOVE - uV[0], v1 = vlog[a] + ABOVE - uV[1];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float z0 = sc[t][a][2 * e] - um[0], z1 = sc[t][a][2 * e + 1] - um[1];
            l[t][0] += ex2(z0);
            l[t][1] += ex2(z1);
            pb[t][a][e] = transpose8x8(half2_bits(__floats2half2_rn(ex2(z0 + v0), ex2(z1 + v1))));
          }
        }
      }
      // ---- values: tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9 of run a, channels
      // (D / 8) g on; row g of output tile i is channel (D / 8) g + 2 i, row
      // g + 8 the next one
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        uint32_t vv[4][VW];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const unsigned char* vp = src + 32 * D + v_at<D>(16 * a + (e >> 1) * 8 + 2 * j + (e & 1), (D / 8) * g >> 4);
          if (VW == 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(vp);
            vv[e][0] = w.x, vv[e][1] = w.y, vv[e][VW - 2] = w.z, vv[e][VW - 1] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(vp + 8 * (g & 1));
            vv[e][0] = w.x, vv[e][1] = w.y;
          }
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t c0[4] = {codes_pair<0>(vv[0][w], vv[1][w]), codes_pair<1>(vv[0][w], vv[1][w]),
                                  codes_pair<0>(vv[2][w], vv[3][w]), codes_pair<1>(vv[2][w], vv[3][w])};
          const uint32_t c1[4] = {codes_pair<2>(vv[0][w], vv[1][w]), codes_pair<3>(vv[0][w], vv[1][w]),
                                  codes_pair<2>(vv[2][w], vv[3][w]), codes_pair<3>(vv[2][w], vv[3][w])};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_f16(o[t][2 * w], c0, pb[t][a][0], pb[t][a][1]);
            mma_f16(o[t][2 * w + 1], c1, pb[t][a][0], pb[t][a][1]);
          }
        }
      }
      if (STAGES == 2) {
        __syncwarp();
        issue(i + 2);
      }
    }
    cp_async_wait<0>();

    // ---- the four warps' results
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int s = 4; s < 32; s *= 2) l[t][c] += __shfl_xor_sync(~0u, l[t][c], s);
        if (g == 0) {
          const int r = 8 * t + 2 * j + c;
          sm[warp][r] = m[t][c];
          sV[warp][r] = V[t][c];
          sl[warp][r] = l[t][c];
        }
      }
    __syncthreads();  // also: every warp is done with its ring
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * t + 2 * j + c;
        float um = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r])), top = -INFINITY;
        if (um == -INFINITY) um = 0.f;
#pragma unroll
        for (int w = 0; w < AT_WARPS; ++w) top = fmaxf(top, sV[w][r] + (sm[w][r] - um));
        if (top == -INFINITY) top = 0.f;
        const float drop = ex2(V[t][c] + (m[t][c] - um) - top);
#pragma unroll
        for (int i = 0; i < NO; ++i)
          *reinterpret_cast<float2*>(&osum[warp][r][(D / 8) * g + 2 * i]) =
              make_float2(o[t][i][c] * drop, o[t][i][2 + c] * drop);
      }
    __syncthreads();
    constexpr int TPR = AT_THREADS / ROWS, DPT = D / TPR;  // threads of a row, channels of a thread
    const int r = tid / TPR, d0 = (tid % TPR) * DPT;
    float cm = -INFINITY, cV = -INFINITY, cl = 0.f, acc[DPT];
#pragma unroll
    for (int w = 0; w < AT_WARPS; ++w) cm = fmaxf(cm, sm[w][r]);
#pragma unroll
    for (int w = 0; w < AT_WARPS; ++w) {
      const float down = sm[w][r] - (cm == -INFINITY ? 0.f : cm);
      cV = fmaxf(cV, sV[w][r] + down);
      cl += sl[w][r] * ex2(down);
    }
#pragma unroll
    for (int i = 0; i < DPT; ++i)
      acc[i] = osum[0][r][d0 + i] + osum[1][r][d0 + i] + osum[2][r][d0 + i] + osum[3][r][d0 + i];

    const int64_t item = x - u0;  // the item's first step
    const int c0 = cta_of(wk, item), c1 = cta_of(wk, item + units - 1);
    bool write = true;
    if (c0 != c1) {
      // A part per CTA, joined JOIN at a time: the last CTA of a group to
      // finish joins its parts into the group's first, the last group the
      // item.  (By one CTA at once, an item cut into 256 parts took 55 us of
      // 64 for that.)  The order of the sums is that of the CTAs.
      constexpr int JOIN = 16;
      const size_t pf = kv_partial_floats(D);
      auto part_of = [&](int c) { return p.partials + (size_t)(2 * c + (c == c0)) * pf; };
      auto put = [&](float* to) {
        if (r < rows) {
#pragma unroll
          for (int i = 0; i < DPT; i += 4)
            *reinterpret_cast<float4*>(to + r * D + d0 + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
          if (tid % TPR == 0) *reinterpret_cast<float4*>(to + ROWS * D + 4 * r) = make_float4(cm, cV, cl, 0.f);
        }
      };
      // true in the CTA that comes last of `all`
      auto last_of = [&](uint32_t* counter, int all) {
        __threadfence();
        __syncthreads();
        if (tid == 0) arrived = atomicAdd(counter, 1u);
        __syncthreads();
        if (arrived != (uint32_t)(all - 1)) return false;
        if (tid == 0) *counter = 0;
        __threadfence();
        return true;
      };
      // parts from, from + step, ... up to `to` into acc, cm, cV, cl
      auto join = [&](int from, int to, int step) {
        cm = cV = -INFINITY;
        cl = 0.f;
#pragma unroll
        for (int i = 0; i < DPT; ++i) acc[i] = 0.f;
        if (r >= rows) return;
        float4 st[JOIN];
#pragma unroll
        for (int i = 0; i < JOIN; ++i) {
          const int c = from + i * step;
          st[i] = c <= to ? __ldcg(reinterpret_cast<const float4*>(part_of(c) + ROWS * D + 4 * r))
                          : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
          cm = fmaxf(cm, st[i].x);
        }
        const float um = cm == -INFINITY ? 0.f : cm;
#pragma unroll
        for (int i = 0; i < JOIN; ++i) {
          st[i].x -= um;
          st[i].y += st[i].x;
          cV = fmaxf(cV, st[i].y);
        }
        const float uV = cV == -INFINITY ? 0.f : cV;
#pragma unroll
        for (int i = 0; i < JOIN; ++i) {
          const int c = from + i * step;
          if (c > to) break;
          cl += st[i].z * ex2(st[i].x);
          const float drop = ex2(st[i].y - uV);
#pragma unroll
          for (int e = 0; e < DPT; e += 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(part_of(c) + r * D + d0 + e));
            acc[e] = fmaf(v.x, drop, acc[e]);
            acc[e + 1] = fmaf(v.y, drop, acc[e + 1]);
            acc[e + 2] = fmaf(v.z, drop, acc[e + 2]);
            acc[e + 3] = fmaf(v.w, drop, acc[e + 3]);
          }
        }
      };
      const int parts = c1 - c0 + 1, group = c0 + (cta - c0) / JOIN * JOIN, end = min(group + JOIN - 1, c1);
      put(part_of(cta));
      // Counters of a CTA: of the item that starts in it and its first group,
      // and of the group that it leads in an item from before.
      write = last_of(p.counters + 3 * group + (group == c0 ? 1 : 2), end - group + 1);
      if (write) {
        join(group, end, 1);
        if (parts > JOIN) {
          __syncthreads();  // every thread has read the group's first part
          put(part_of(group));
          const int groups = (parts + JOIN - 1) / JOIN;
          write = last_of(p.counters + 3 * c0, groups);
          if (write) {
            float gm = -INFINITY, gV = -INFINITY, gl = 0.f, ga[DPT] = {};
            // more than JOIN groups (over 256 parts): in turns
            for (int i = 0; i < groups; i += JOIN) {
              join(c0 + i * JOIN, min(c1, c0 + (i + JOIN) * JOIN - 1), JOIN);
              const float nm = fmaxf(gm, cm), um = nm == -INFINITY ? 0.f : nm;
              gl = gl * ex2(gm - um) + cl * ex2(cm - um);
              gV += gm - um;
              cV += cm - um;
              const float nV = fmaxf(gV, cV), uV = nV == -INFINITY ? 0.f : nV;
              const float f0 = ex2(gV - uV), f1 = ex2(cV - uV);
#pragma unroll
              for (int e = 0; e < DPT; ++e) ga[e] = ga[e] * f0 + acc[e] * f1;
              gm = nm, gV = nV;
            }
            cm = gm, cV = gV, cl = gl;
#pragma unroll
            for (int e = 0; e < DPT; ++e) acc[e] = ga[e];
          }
        }
      }
    }
    if (write && r < rows) {
      // sum p vs v = 2^(V - ABOVE) of what was accumulated; nothing seen, or all
      // values zero: 0
      const float k = cl == 0.f ? 0.f : (cV == -INFINITY ? 0.f : exp2f(cV)) / cl;
      const uint32_t rr = (uint32_t)qt * ROWS + r;
      uint16_t* dst = p.out + ((size_t)(q.row + rr / (uint32_t)p.G) * p.hq + (size_t)h * p.G + rr % (uint32_t)p.G) * D + d0;
#pragma unroll
      for (int i = 0; i < DPT; ++i) acc[i] *= 1.f / (1 << (int)ABOVE);
#pragma unroll
      for (int i = 0; i < DPT; i += 4)
        *reinterpret_cast<uint2*>(dst + i) = make_uint2(pack_bf16x2(acc[i] * k, acc[i + 1] * k),
                                                        pack_bf16x2(acc[i + 2] * k, acc[i + 3] * k));
    }
    __syncthreads();  // the shared sums are free again
    // ---- next item
    x += u1 - u0;
    u0 = 0;
    if (x < x1 && ++h == hkv) {
      h = 0;
      if (++qt == q_tiles<ROWS>(p, q)) {
        qt = 0;
        do q = load_seq(p, ++s);
        while (q.n == 0);  // x < x1 <= total: a later sequence has rows
      }
    }
  }
}

// More query rows a sequence and key head than this, on average: the tile
// kernel.  Sixteen sequences of 8000 tokens, 32 heads on 8: 16 rows 73 us
// streaming, 131 in tiles; 32 rows 123 and 132; 40 rows 178 and 132.  An average
// is all the host knows, and it is poor where sequences differ: a prompt of 2048
// tokens among 31 single tokens behind 8000 takes 300 us, the two parts apart
// 75 and 94; 512 new tokens behind 7488 in one of 64 slots 430 us, alone 87.
constexpr int TILE_ROWS = 32;

template <int D, int NT>
cudaError_t launch_stream(const AttnParams& p, cudaStream_t s) {
  auto* kern = kv_attention_kernel<D, NT>;
  cudaError_t e = set_smem_limit_once(kern, at_smem<D, NT>());
  if (e != cudaSuccess) return e;
  const dim3 grid(sm_count() * Shape<NT>::CTAS), block(AT_THREADS);
  MOE_LAUNCH("kv_attention", s, { e = launch_k(kern, grid, block, at_smem<D, NT>(), s, p); });
  return e;
}

}  // namespace

cudaError_t launch_kv_attention(const uint16_t* q, int64_t q_stride, const int32_t* starts, int t, int hq,
                                float scale, const moe_kv_cache& c, uint16_t* out, unsigned char* ws,
                                cudaStream_t s) {
  AttnParams p;
  p.q = q;
  p.q_stride = q_stride;
  p.starts = starts;
  p.t = t;
  p.hq = hq;
  p.G = hq / c.hkv;
  p.scale_log2 = scale * 1.44269504088896340736f;
  p.block_log2 = c.block == 16 ? 4 : c.block == 32 ? 5 : c.block == 64 ? 6 : 7;
  p.c = c;
  p.out = out;
  p.st = reinterpret_cast<DeviceStatus*>(ws);
  p.counters = reinterpret_cast<uint32_t*>(ws + kv_counter_off());
  p.partials = reinterpret_cast<float*>(ws + kv_partial_off());
  if ((int64_t)t * p.G > (int64_t)TILE_ROWS * c.n_seq) return launch_tile(p, s);
  // Eight rows a tile where they hold a token's group of heads and no
  // sequence has more than one token on average, else sixteen.
  const bool small = p.G <= 8 && t <= c.n_seq;
  return c.d == 64 ? (small ? launch_stream<64, 1>(p, s) : launch_stream<64, 2>(p, s))
                   : (small ? launch_stream<128, 1>(p, s) : launch_stream<128, 2>(p, s));
}

}  // namespace moe
