// Causal attention over the paged 8-bit key/value cache (moe_kv_attention).
#include <math.h>

#include "kv_common.cuh"

namespace moe {

namespace {

constexpr int AT_WARPS = 4;
constexpr int AT_THREADS = AT_WARPS * 32;
constexpr int WARP_TOKENS = 32;                      // tokens of one warp step
constexpr int UNIT = AT_WARPS * WARP_TOKENS;         // tokens of one CTA step
constexpr int STAGES = 3;                            // steps of a warp in its ring

__host__ __device__ constexpr int at_smem(int d) {
  const int ring = AT_WARPS * STAGES * 2 * WARP_TOKENS * d, sums = AT_WARPS * KV_ROWS * (d + 4) * 4;
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

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct AttnParams {
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* starts;
  int t, hq, G;       // G query heads read one key/value head
  float scale_log2;   // scale * log2(e)
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

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two biased codes (code + 128, in bytes SEL selects) as exact fp16 numbers:
// under the exponent of 1024 a byte b is 1024 + b.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
  uint32_t v;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(v) : "r"(w), "r"(0x64646464u), "n"(SEL));
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), __floats2half2_rn(1152.f, 1152.f));
  return *reinterpret_cast<const uint32_t*>(&r);
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
__device__ __forceinline__ int q_tiles(const AttnParams& p, const Seq& q) {
  return (int)(((int64_t)q.n * p.G + KV_ROWS - 1) / KV_ROWS);
}
// CTA steps of query tile qt: up to the last position its last row sees.
__device__ __forceinline__ int tile_seen(const AttnParams& p, const Seq& q, int qt) {
  const int64_t rows = min((int64_t)q.n * p.G, (int64_t)KV_ROWS * (qt + 1));
  return q.len - q.n + (int)((rows - 1) / p.G) + 1;
}
__device__ __forceinline__ int tile_units(const AttnParams& p, const Seq& q, int qt) {
  return (tile_seen(p, q, qt) + UNIT - 1) / UNIT;
}
__device__ __forceinline__ int64_t seq_units(const AttnParams& p, const Seq& q) {
  int64_t w = 0;
  for (int qt = 0, m = q_tiles(p, q); qt < m; ++qt) w += tile_units(p, q, qt);
  return w * p.c.hkv;
}

// The work is the list of all (sequence, query tile, key/value head) items,
// each as many 128-token steps as its rows see, cut into equal runs of steps,
// one a CTA: long and short sequences load the SMs alike.  An item that
// spans several CTAs leaves a partial result per CTA; the last CTA to finish
// joins them in CTA order.
//
// Within an item the CTA's four warps take 32 tokens each per step and hold
// all 16 query rows.  Each warp keeps two steps in flight by asynchronous
// copies into a ring of its own.  The order of the channels inside a product
// of q and k is free (both operands use the same), and so is the order of the
// output channels, so a lane reads 16 bytes in a row of a key and of a value
// as its part of the m16n8k16 fragments.  Codes become exact fp16 numbers; the key scale multiplies the fp32 scores and the value scale
// enters the weights, p_j = exp2(s_j - m) vs_j, through its logarithm with a
// running maximum M of its own, so that the fp16 weights are at most 1
// whatever the scales are.
template <int D>
__global__ void __launch_bounds__(AT_THREADS, KV_CTAS_PER_SM) kv_attention_kernel(AttnParams p) {
  constexpr int KL = D / 64;   // 16-byte loads of a key per lane
  constexpr int VW = D / 32;   // 4-byte words of a value per lane
  constexpr int NO = D / 8;    // output tiles of 8 channels
  constexpr int STAGE = 2 * WARP_TOKENS * D;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* ring = smem + (threadIdx.x >> 5) * STAGES * STAGE;
  float(*osum)[KV_ROWS][D + 4] = reinterpret_cast<float(*)[KV_ROWS][D + 4]>(smem);  // after an item's steps
  __shared__ float sm[AT_WARPS][KV_ROWS], sM[AT_WARPS][KV_ROWS], sl[AT_WARPS][KV_ROWS];
  __shared__ int64_t scan[AT_WARPS];
  __shared__ int64_t found_at;
  __shared__ int found_s;
  __shared__ uint32_t arrived;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, j = lane & 3;
  const int hkv = p.c.hkv;

  // total steps, then the sequence that holds this CTA's first step
  int64_t total = 0;
  for (int s = tid; s < p.c.n_seq; s += AT_THREADS) {
    const Seq q = load_seq(p, s);
    if (!q.ok && blockIdx.x == 0) raise_flag(p.st, FLAG_BAD_CACHE);
    total += seq_units(p, q);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
  if (lane == 0) scan[warp] = total;
  __syncthreads();
  total = scan[0] + scan[1] + scan[2] + scan[3];
  const int64_t ctas = min((int64_t)gridDim.x, total);
  const int cta = blockIdx.x;
  if (cta >= ctas) return;
  const int64_t x0 = total * cta / ctas, x1 = total * (cta + 1) / ctas;
  int64_t base = 0;
  for (int sb = 0; sb < p.c.n_seq; sb += AT_THREADS) {
    const int64_t w = sb + tid < p.c.n_seq ? seq_units(p, load_seq(p, sb + tid)) : 0;
    int64_t incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += u;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    for (int i = 0; i < warp; ++i) incl += scan[i];
    const int64_t all = scan[0] + scan[1] + scan[2] + scan[3];
    if (x0 < base + all) {
      if (base + incl - w <= x0 && x0 < base + incl) {
        found_s = sb + tid;
        found_at = base + incl - w;
      }
      break;
    }
    base += all;
  }
  __syncthreads();
  int s = found_s;
  Seq q = load_seq(p, s);
  int qt = 0, h = 0, u0 = 0;
  int64_t off = x0 - found_at;
  for (;; ++qt) {
    const int units = tile_units(p, q, qt);
    if (off < (int64_t)units * hkv) {
      h = (int)(off / units);
      u0 = (int)(off % units);
      break;
    }
    off -= (int64_t)units * hkv;
  }

  int64_t x = x0;
  while (x < x1) {
    const int units = tile_units(p, q, qt), seen = tile_seen(p, q, qt);
    const int u1 = (int)min((int64_t)units, u0 + (x1 - x));
    const int rows = (int)min((int64_t)q.n * p.G - (int64_t)qt * KV_ROWS, (int64_t)KV_ROWS);
    // ---- query fragments, each row scaled by a power of two into fp16
    uint32_t qa[KL * 4][4];
    float f[2];
    int limit[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g + 8 * e;
      uint2 raw[KL * 4];
      float m = 0.f;
      const int64_t rr = (int64_t)qt * KV_ROWS + r;
      const int i = (int)(rr / p.G), head = h * p.G + (int)(rr % p.G);
      limit[e] = r < rows ? q.len - q.n + i : -1;
#pragma unroll
      for (int w = 0; w < KL * 4; ++w) {
        raw[w] = make_uint2(0, 0);
        if (r < rows)
          raw[w] = *reinterpret_cast<const uint2*>(p.q + (int64_t)(q.row + i) * p.q_stride + (size_t)head * D +
                                                   64 * (w >> 2) + 16 * j + 4 * (w & 3));
        m = fmaxf(m, fmaxf(fmaxf(fabsf(bf16lo(raw[w].x)), fabsf(bf16hi(raw[w].x))),
                           fmaxf(fabsf(bf16lo(raw[w].y)), fabsf(bf16hi(raw[w].y)))));
      }
      m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
      m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
      // the row's largest magnitude goes to [256, 512)
      const int ex = min(max((int)(__float_as_uint(m) >> 23) - 127, -100), 127);
      const float up = __uint_as_float((uint32_t)(127 + 8 - ex) << 23);
      f[e] = __uint_as_float((uint32_t)(max(127 - 8 + ex, 1)) << 23) * p.scale_log2;
#pragma unroll
      for (int w = 0; w < KL * 4; ++w) {
        const __half2 a = __floats2half2_rn(bf16lo(raw[w].x) * up, bf16hi(raw[w].x) * up);
        const __half2 b = __floats2half2_rn(bf16lo(raw[w].y) * up, bf16hi(raw[w].y) * up);
        qa[w][e] = *reinterpret_cast<const uint32_t*>(&a);
        qa[w][2 + e] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    float m[2] = {-INFINITY, -INFINITY}, M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[NO][4] = {};

    const int64_t vstep = (int64_t)p.c.n_pages * hkv * p.c.block * D;
    // this warp's steps: 32 tokens each, UNIT apart
    const int first = u0 * UNIT + warp * WARP_TOKENS, stop = min(u1 * UNIT, seen);
    const int steps = first < stop ? (stop - first + UNIT - 1) / UNIT : 0;
    // Page and scales of the runs of 16 tokens, two a step, run r in lane
    // r % 32, fetched a chunk of 16 steps ahead.
    auto page_of = [&](int chunk) {
      const int step = chunk * 16 + (lane >> 1), pos = first + step * UNIT + 16 * (lane & 1);
      if (step >= steps || pos >= seen) return -1;
      const int page = __ldg(p.c.table + (size_t)s * p.c.max_blocks + pos / p.c.block);
      if (page >= 0 && page < p.c.n_pages) return page;
      raise_flag(p.st, FLAG_BAD_CACHE);
      return -1;
    };
    auto scale_of = [&](int page, int isv) {
      return page < 0 ? 1.f : __ldg(p.c.scales + ((size_t)isv * p.c.n_pages + page) * hkv + h);
    };
    int chunk_now = 0;
    int page = page_of(0), next_page = page_of(1);
    float kscale = scale_of(page, 0), vscale = scale_of(page, 1), next_k = 0.f, next_v = 0.f;
    auto issue = [&](int step) {
      if (step < steps) {
        unsigned char* dst = ring + (step % STAGES) * STAGE;
        const int ahead = (step >> 4) != chunk_now;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int src_lane = (2 * step + r) & 31;
          const int pg = __shfl_sync(~0u, ahead ? next_page : page, src_lane);
          if (pg < 0) continue;
          const int pos = first + step * UNIT + 16 * r;
          const int8_t* src = p.c.codes + (((size_t)pg * hkv + h) * p.c.block + pos % p.c.block) * D;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const int c = lane % (D / 16), tok = lane / (D / 16) + i * (512 / D);
            const int8_t* from = src + tok * D + 16 * c;
            cp_async16(dst + k_at<D>(16 * r + tok, c), from);
            cp_async16(dst + 32 * D + v_at<D>(16 * r + tok, c), from + vstep);
          }
        }
      }
      cp_async_commit();
    };
    issue(0);
    issue(1);

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
      cp_async_wait<STAGES - 2>();
      __syncwarp();  // this step's codes are there, and the last step's are read by every lane
      issue(i + STAGES - 1);
      const unsigned char* src = ring + (i % STAGES) * STAGE;
      const int pos0 = first + i * UNIT;
      float ksc[2], vlog[2];
      bool live[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int run = (2 * i + r) & 31;
        live[r] = __shfl_sync(~0u, page, run) >= 0;
        ksc[r] = __shfl_sync(~0u, kscale, run);
        vlog[r] = __log2f(__shfl_sync(~0u, vscale, run));
      }
      // ---- scores
      float sc[4][4] = {};
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int e = 0; e < KL; ++e) {
          const uint4 c = *reinterpret_cast<const uint4*>(src + k_at<D>(8 * a + g, 4 * e + j));
          const uint32_t w[4] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u, c.z ^ 0x80808080u, c.w ^ 0x80808080u};
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_f16(sc[a], qa[4 * e + i], codes_f16<0x4140>(w[i]), codes_f16<0x4342>(w[i]));
        }
      float nm[2] = {m[0], m[1]}, nM[2] = {M[0], M[1]};
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = a >> 1, pos = pos0 + 8 * a + 2 * j + (e & 1);
          sc[a][e] = live[r] && pos <= limit[e >> 1] ? sc[a][e] * (ksc[r] * f[e >> 1]) : -INFINITY;
          nm[e >> 1] = fmaxf(nm[e >> 1], sc[a][e]);
          nM[e >> 1] = fmaxf(nM[e >> 1], sc[a][e] + vlog[r]);
        }
      float um[2], uM[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        nm[e] = fmaxf(nm[e], __shfl_xor_sync(~0u, nm[e], 1));
        nm[e] = fmaxf(nm[e], __shfl_xor_sync(~0u, nm[e], 2));
        nM[e] = fmaxf(nM[e], __shfl_xor_sync(~0u, nM[e], 1));
        nM[e] = fmaxf(nM[e], __shfl_xor_sync(~0u, nM[e], 2));
        // rows that have seen nothing yet: any finite reference does
        um[e] = nm[e] == -INFINITY ? 0.f : nm[e];
        uM[e] = nM[e] == -INFINITY ? 0.f : nM[e];
        l[e] *= ex2(m[e] - um[e]);
        const float drop = ex2(M[e] - uM[e]);
        m[e] = nm[e];
        M[e] = nM[e];
        if (__any_sync(~0u, drop != 1.f))
#pragma unroll
          for (int t = 0; t < NO; ++t) {
            o[t][2 * e] *= drop;
            o[t][2 * e + 1] *= drop;
          }
      }
      // ---- weights, and their products with the values
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t pa[4];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float z0 = sc[2 * r + a][2 * e], z1 = sc[2 * r + a][2 * e + 1];
            l[e] += ex2(z0 - um[e]) + ex2(z1 - um[e]);
            const __half2 w = __floats2half2_rn(ex2(z0 + vlog[r] - uM[e]), ex2(z1 + vlog[r] - uM[e]));
            pa[2 * a + e] = *reinterpret_cast<const uint32_t*>(&w);
          }
        // values of tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9 of the run, D / 8 channels from (D / 8) g on
        uint32_t vv[4][VW];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const unsigned char* vp = src + 32 * D + v_at<D>(16 * r + (e >> 1) * 8 + 2 * j + (e & 1), (D / 8) * g >> 4);
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
          uint32_t lo[2], hi[2];  // bytes of two tokens side by side
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            lo[e] = __byte_perm(vv[2 * e][w], vv[2 * e + 1][w], 0x5140) ^ 0x80808080u;
            hi[e] = __byte_perm(vv[2 * e][w], vv[2 * e + 1][w], 0x7362) ^ 0x80808080u;
          }
          mma_f16(o[4 * w + 0], pa, codes_f16<0x4140>(lo[0]), codes_f16<0x4140>(lo[1]));
          mma_f16(o[4 * w + 1], pa, codes_f16<0x4342>(lo[0]), codes_f16<0x4342>(lo[1]));
          mma_f16(o[4 * w + 2], pa, codes_f16<0x4140>(hi[0]), codes_f16<0x4140>(hi[1]));
          mma_f16(o[4 * w + 3], pa, codes_f16<0x4342>(hi[0]), codes_f16<0x4342>(hi[1]));
        }
      }
    }

    cp_async_wait<0>();

    // ---- the four warps' results
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(~0u, l[e], 1);
      l[e] += __shfl_xor_sync(~0u, l[e], 2);
      if (j == 0) {
        sm[warp][g + 8 * e] = m[e];
        sM[warp][g + 8 * e] = M[e];
        sl[warp][g + 8 * e] = l[e];
      }
    }
    __syncthreads();  // also: every warp is done with its ring
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g + 8 * e;
      float top = fmaxf(fmaxf(sM[0][r], sM[1][r]), fmaxf(sM[2][r], sM[3][r]));
      if (top == -INFINITY) top = 0.f;
      const float drop = ex2(M[e] - top);
      // output tile i, column c stands for channel (D / 8) c + i
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < NO; ++i) osum[warp][r][(D / 8) * (2 * j + c) + i] = o[i][2 * e + c] * drop;
    }
    __syncthreads();
    const int r = tid >> 3, d0 = (tid & 7) * (D / 8);  // 8 threads a row
    float cm = -INFINITY, cM = -INFINITY, cl = 0.f, acc[D / 8];
#pragma unroll
    for (int w = 0; w < AT_WARPS; ++w) {
      cm = fmaxf(cm, sm[w][r]);
      cM = fmaxf(cM, sM[w][r]);
    }
#pragma unroll
    for (int w = 0; w < AT_WARPS; ++w) cl += sl[w][r] * ex2(sm[w][r] - (cm == -INFINITY ? 0.f : cm));
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      acc[i] = osum[0][r][d0 + i] + osum[1][r][d0 + i] + osum[2][r][d0 + i] + osum[3][r][d0 + i];

    const int64_t item = x - u0;  // the item's first step
    const int c0 = (int)(((item + 1) * ctas - 1) / total), c1 = (int)(((item + units) * ctas - 1) / total);
    bool write = true;
    if (c0 != c1) {
      const size_t pf = kv_partial_floats(D);
      float* mine = p.partials + (size_t)(2 * cta + (cta == c0)) * pf;
      if (r < rows) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) mine[r * D + d0 + i] = acc[i];
        if ((tid & 7) == 0) {
          float* sp = mine + KV_ROWS * D + 4 * r;
          sp[0] = cm, sp[1] = cM, sp[2] = cl;
        }
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) arrived = atomicAdd(p.counters + c0, 1u);
      __syncthreads();
      write = arrived == (uint32_t)(c1 - c0);
      if (write) {
        __threadfence();
        if (tid == 0) p.counters[c0] = 0;
        cm = cM = -INFINITY;
        cl = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) acc[i] = 0.f;
        if (r < rows) {
          for (int c = c0; c <= c1; ++c) {
            const float* sp = p.partials + (size_t)(2 * c + (c == c0)) * pf + KV_ROWS * D + 4 * r;
            cm = fmaxf(cm, __ldcg(sp));
            cM = fmaxf(cM, __ldcg(sp + 1));
          }
          for (int c = c0; c <= c1; ++c) {
            const float* part = p.partials + (size_t)(2 * c + (c == c0)) * pf;
            const float* sp = part + KV_ROWS * D + 4 * r;
            cl += __ldcg(sp + 2) * ex2(__ldcg(sp) - (cm == -INFINITY ? 0.f : cm));
            const float drop = ex2(__ldcg(sp + 1) - (cM == -INFINITY ? 0.f : cM));
#pragma unroll
            for (int i = 0; i < D / 8; i += 4) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(part + r * D + d0 + i));
              acc[i] = fmaf(v.x, drop, acc[i]);
              acc[i + 1] = fmaf(v.y, drop, acc[i + 1]);
              acc[i + 2] = fmaf(v.z, drop, acc[i + 2]);
              acc[i + 3] = fmaf(v.w, drop, acc[i + 3]);
            }
          }
        }
      }
    }
    if (write && r < rows) {
      // sum p vs v = 2^(M - m) of what was accumulated; nothing seen, or all
      // values zero: 0
      const float k = cl == 0.f ? 0.f : (cM == -INFINITY ? 0.f : exp2f(cM - cm)) / cl;
      const int64_t rr = (int64_t)qt * KV_ROWS + r;
      uint16_t* dst = p.out + ((size_t)(q.row + rr / p.G) * p.hq + (size_t)h * p.G + rr % p.G) * D + d0;
#pragma unroll
      for (int i = 0; i < D / 8; i += 8)
        *reinterpret_cast<uint4*>(dst + i) =
            make_uint4(pack_bf16x2(acc[i] * k, acc[i + 1] * k), pack_bf16x2(acc[i + 2] * k, acc[i + 3] * k),
                       pack_bf16x2(acc[i + 4] * k, acc[i + 5] * k), pack_bf16x2(acc[i + 6] * k, acc[i + 7] * k));
    }
    __syncthreads();  // the shared sums are free again
    // ---- next item
    x += u1 - u0;
    u0 = 0;
    if (x < x1 && ++h == hkv) {
      h = 0;
      if (++qt == q_tiles(p, q)) {
        qt = 0;
        do q = load_seq(p, ++s);
        while (q.n == 0);  // x < x1 <= total: a later sequence has rows
      }
    }
  }
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
  p.c = c;
  p.out = out;
  p.st = reinterpret_cast<DeviceStatus*>(ws);
  p.counters = reinterpret_cast<uint32_t*>(ws + kv_counter_off());
  p.partials = reinterpret_cast<float*>(ws + kv_partial_off());
  const dim3 grid(kv_grid_max()), block(AT_THREADS);
  auto* kern = c.d == 64 ? kv_attention_kernel<64> : kv_attention_kernel<128>;
  cudaError_t e = set_smem_limit_once(kern, at_smem(c.d));
  if (e != cudaSuccess) return e;
  MOE_LAUNCH("kv_attention", s, { e = launch_k(kern, grid, block, at_smem(c.d), s, p); });
  return e;
}

}  // namespace moe
