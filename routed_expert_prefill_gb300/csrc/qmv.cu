// Product of rows with 4-bit weights and group scales (moe_qmv).
#include "api_checks.cuh"

namespace moe {

namespace {

struct QmvParams {
  const uint16_t* x;
  int64_t x_stride;
  const int8_t* xc;
  const float* xs;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* biases;
  int t, n, k;
  void* y;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool f16) {
  if (f16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The pairs of codes (i, i + 4) of a word as the numbers 1 + q / 16, exact in
// bf16 (4 of its 7 mantissa bits) and in fp16 (4 of 10): the code's bits are
// shifted under a fixed exponent.
template <bool F16>
__device__ __forceinline__ void codes_to_pairs(uint32_t w, uint32_t (&o)[4]) {
  constexpr uint32_t MASK = F16 ? 0x03C003C0u : 0x00780078u, ONE = F16 ? 0x3C003C00u : 0x3F803F80u;
  if (F16) {
    o[0] = ((w << 6) & MASK) | ONE;
    o[1] = ((w << 2) & MASK) | ONE;
    o[2] = ((w >> 2) & MASK) | ONE;
    o[3] = ((w >> 6) & MASK) | ONE;
  } else {
    o[0] = ((w << 3) & MASK) | ONE;
    o[1] = ((w >> 1) & MASK) | ONE;
    o[2] = ((w >> 5) & MASK) | ONE;
    o[3] = ((w >> 9) & MASK) | ONE;
  }
}

constexpr int QMV_WARPS = 8;

// ---------------------------------------------------------------------------
// Few rows: weights streamed through shared memory.
// ---------------------------------------------------------------------------

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int QS_ROW = 160;  // bytes of a weight row's 4 groups in shared memory: 128 and a shift of 8 banks
constexpr int QS_STAGE = 16 * QS_ROW;  // a unit's codes
constexpr int QS_CHUNKS = 4;            // 16-byte pieces of a tile's scales and biases that a thread carries
constexpr int QS_MAX_K = 64 * 64 * QS_CHUNKS;

// Bytes between rows of a tile's scales in shared memory: eight rows read
// together, 8 bytes each, fall on different banks.
__host__ __device__ constexpr int qs_s_pitch(int groups) { return ((2 * groups + 15) & ~15) + 16; }

// Bytes between rows of x in shared memory, 2 bytes a value: lanes of two rows
// read together, 16 bytes each at steps of 32; the pad puts the second row's
// reads on the other banks.
__host__ __device__ constexpr int qs_x_pitch(int k) { return 2 * k + 16; }

// Codes as operands without arithmetic: the bits of a code, masked in place,
// read as a number.  Below the smallest normal exponent, and in the first
// binade above it, the value is linear in the bits: bits * 2^-133 in bf16 (up
// to 255), bits * 2^-24 in fp16 (up to 2047).  A code 4 bits up weighs 16
// times as much, which the staged x makes up for; one shift brings the upper
// two codes of a half down.
__device__ __forceinline__ void codes_raw(uint32_t w, uint32_t (&o)[4]) {
  const uint32_t h = w >> 8;
  o[0] = w & 0x000F000Fu;
  o[1] = w & 0x00F000F0u;
  o[2] = h & 0x000F000Fu;
  o[3] = h & 0x00F000F0u;
}

template <bool F16>
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// v * 2^e for any e in [-252, 254], as two exact powers of two.
__device__ __forceinline__ float times_pow2(float v, int e) {
  const int a = e / 2, b = e - a;
  return v * __uint_as_float((uint32_t)(127 + a) << 23) * __uint_as_float((uint32_t)(127 + b) << 23);
}

size_t qs_smem(const QmvParams& p, int nt, int teams, int stages) {
  return (size_t)teams * QMV_WARPS * stages * QS_STAGE            // rings
         + (size_t)teams * 2 * QMV_WARPS * 16 * 8 * nt * 4         // sums
         + (size_t)teams * 2 * 2 * 16 * qs_s_pitch(p.k >> 6)       // scales and biases of two tiles
         + (size_t)(p.k >> 6) * 8 * nt * (p.xc ? 8 : 4)            // group sums of x, scales of 8-bit rows
         + (size_t)p.t * qs_x_pitch(p.k);                          // x
}

// y for t <= 8 NT rows, when what counts is how fast the weights come.  The CTA stages x once; then each of its TEAMS teams
// of eight warps walks tiles of 16 weight rows.  A team's warps split k in
// units of 4 groups (128 bytes of a weight row), the same units in every
// tile, and each warp keeps S - 1 units in flight by asynchronous copies into
// a ring of its own, across tiles: only the sums at a tile's end make a
// team's warps wait for one another.  A tile's scales and biases, contiguous
// in memory, pass through the team's registers one tile ahead: fetched row by
// row with the codes they cost a shared-memory pass a row and unit, as much
// as all reads of the codes (62.5 us a call of 4 rows of 4096 with 131072
// weight rows that way).  VEC: 16-byte pieces of the scales lie within rows
// (k a multiple of 512).
//
// The kernel is bound by instructions before it is by memory unless a code
// costs little, so codes enter as they are (codes_raw) and x carries the
// rest: bf16 rows are scaled by a power of two that takes the row's largest
// magnitude to [2^120, 2^121), where products with code * 2^-133 are ordinary
// fp32 numbers, and the result is scaled back; 8-bit rows need no scaling.
// The pairs that meet codes 4 bits up are divided by 16.  All of it is exact
// but for values more than 2^240 below their row's largest.
template <int NT, int TEAMS, int S, bool F16, bool VEC>
__global__ void __launch_bounds__(TEAMS * QMV_WARPS * 32, 1) qmv_stream_kernel(QmvParams p, bool out32) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int rowmax[8 * NT];
  constexpr int THREADS = TEAMS * QMV_WARPS * 32;
  const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
  const int team = threadIdx.x / (QMV_WARPS * 32), warp = (threadIdx.x >> 5) % QMV_WARPS;
  const int groups = p.k >> 6, units = (groups + 3) >> 2, x_pitch = qs_x_pitch(p.k);
  unsigned char* ring = smem + (size_t)(threadIdx.x >> 5) * S * QS_STAGE;
  float* red = reinterpret_cast<float*>(smem + (size_t)TEAMS * QMV_WARPS * S * QS_STAGE) +
               (size_t)team * 2 * QMV_WARPS * 8 * NT * 16;  // [2][warp][8 NT][16]
  const int s_pitch = qs_s_pitch(groups);
  unsigned char* scb = smem + (size_t)TEAMS * QMV_WARPS * (S * QS_STAGE + 2 * 8 * NT * 16 * 4);
  float* xsum = reinterpret_cast<float*>(scb + (size_t)TEAMS * 2 * 2 * 16 * s_pitch);
  scb += (size_t)team * 2 * 2 * 16 * s_pitch;  // [2][scales, biases][16] rows of s_pitch bytes
  unsigned char* xsm = reinterpret_cast<unsigned char*>(xsum + groups * 8 * NT * (F16 ? 2 : 1));
  const int ub = units * warp / QMV_WARPS, ue = units * (warp + 1) / QMV_WARPS;
  const int tiles = (p.n + 15) >> 4, step = gridDim.x * TEAMS, tile0 = blockIdx.x * TEAMS + team;
  const size_t row_bytes = (size_t)p.k >> 1;
  pdl_wait();
  pdl_trigger();

  int it = tile0, iu = ub;  // the next unit to copy
  auto issue = [&](int stage) {
    if (it < tiles && iu < ue) {
      unsigned char* dst = ring + stage * QS_STAGE;
      const int g0 = iu * 4, row0 = it * 16, c = lane & 7;
      const uint8_t* src = p.codes + ((size_t)row0 + (lane >> 3)) * row_bytes + g0 * 32 + 16 * c;
      dst += (lane >> 3) * QS_ROW + 16 * c;
      if (VEC || g0 + (c >> 1) < groups) {
        if (row0 + 16 <= p.n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) cp_async16(dst + 4 * i * QS_ROW, src + i * 4 * row_bytes);
        } else {  // rows past the end stay as they are; their results are not stored
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (row0 + 4 * i + (lane >> 3) < p.n) cp_async16(dst + 4 * i * QS_ROW, src + i * 4 * row_bytes);
        }
      }
      if (++iu == ue) {
        iu = ub;
        it += step;
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);

  // a tile's scales and biases: 2 * groups pieces of 16 bytes each
  const int tt = threadIdx.x % (QMV_WARPS * 32);
  const size_t s_end = (size_t)p.n * groups * 2;  // bytes of either array
  uint4 sc[QS_CHUNKS];
  int s_off[QS_CHUNKS];  // where a piece goes (VEC)
#pragma unroll
  for (int i = 0; i < QS_CHUNKS; ++i) {
    const int c = tt + i * QMV_WARPS * 32, which = c >= 2 * groups, o = 8 * (c - which * 2 * groups);
    s_off[i] = (which * 16 + o / groups) * s_pitch + 2 * (o % groups);
  }
  auto fetch_scales = [&](int tile) {
#pragma unroll
    for (int i = 0; i < QS_CHUNKS; ++i) {
      if (i * QMV_WARPS * 32 >= 4 * groups) break;
      const int c = tt + i * QMV_WARPS * 32, which = c >= 2 * groups;
      const size_t at = (size_t)tile * 32 * groups + 16 * (c - which * 2 * groups);
      if (c >= 4 * groups || tile >= tiles || at >= s_end) continue;
      const unsigned char* src = reinterpret_cast<const unsigned char*>(which ? p.biases : p.scales) + at;
      if (VEC || at + 16 <= s_end) {
        sc[i] = __ldg(reinterpret_cast<const uint4*>(src));
      } else {  // the arrays end inside the piece
        uint32_t w[4] = {};
        for (int e = 0; e < 8; ++e)
          if (at + 2 * e < s_end) w[e >> 1] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(src) + e) << (16 * (e & 1));
        sc[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  auto store_scales = [&](int buf) {
    unsigned char* dst = scb + (size_t)buf * 32 * s_pitch;
#pragma unroll
    for (int i = 0; i < QS_CHUNKS; ++i) {
      if (i * QMV_WARPS * 32 >= 4 * groups) break;
      const int c = tt + i * QMV_WARPS * 32;
      if (c >= 4 * groups) continue;
      if (VEC) {
        *reinterpret_cast<uint4*>(dst + s_off[i]) = sc[i];
      } else {
        const int which = c >= 2 * groups, o = 8 * (c - which * 2 * groups);
        const uint32_t w[4] = {sc[i].x, sc[i].y, sc[i].z, sc[i].w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint16_t*>(dst + (which * 16 + (o + e) / groups) * s_pitch + 2 * ((o + e) % groups)) =
              (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    }
  };
  fetch_scales(tile0);

  // ---- x: each row's largest magnitude, then its values in operand order
  const int per = p.k >> 3;  // vectors of 8 values
  if (!F16) {
    if (threadIdx.x < 8 * NT) rowmax[threadIdx.x] = 0;
    __syncthreads();
    for (int i0 = threadIdx.x - lane; i0 < p.t * per; i0 += THREADS) {  // whole warps
      const int i = min(i0 + lane, p.t * per - 1), r = i / per;
      const uint4 v = *reinterpret_cast<const uint4*>(p.x + (size_t)r * p.x_stride + 8 * (i % per));
      // magnitudes compare as whole numbers, infinity and NaN last
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7FFF0000u, w[e] << 16 & 0x7FFF0000u));
      if (__all_sync(~0u, r == __shfl_sync(~0u, r, 0))) {
        m = __reduce_max_sync(~0u, m);
        if (lane == 0) atomicMax(rowmax + r, (int)m);
      } else {
        atomicMax(rowmax + r, (int)m);
      }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < p.t * per; i += THREADS) {
    const int r = i / per, c = i % per;
    uint4 o;
    if (F16) {
      const uint2 v = *reinterpret_cast<const uint2*>(p.xc + (size_t)r * p.k + 8 * c);
      const int8_t* b = reinterpret_cast<const int8_t*>(&v);
      auto pair = [&](int e, float f) {
        const __half2 h = __floats2half2_rn(f * b[e], f * b[e + 4]);
        return *reinterpret_cast<const uint32_t*>(&h);
      };
      o = make_uint4(pair(0, 1.f), pair(1, 0.0625f), pair(2, 1.f), pair(3, 0.0625f));
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(p.x + (size_t)r * p.x_stride + 8 * c);
      const int ex = rowmax[r] >> 23, up = ex == 255 || rowmax[r] == 0 ? 0 : 120 + 127 - max(ex, 1);
      auto pair = [&](uint32_t lo, uint32_t hi, bool odd, int sh) {
        const float a = sh ? bf16hi(lo) : bf16lo(lo), b = sh ? bf16hi(hi) : bf16lo(hi);
        return pack_bf16x2(times_pow2(a, up - 4 * odd), times_pow2(b, up - 4 * odd));
      };
      o = make_uint4(pair(v.x, v.z, false, 0), pair(v.x, v.z, true, 1), pair(v.y, v.w, false, 0),
                     pair(v.y, v.w, true, 1));
    }
    *reinterpret_cast<uint4*>(xsm + (size_t)r * x_pitch + 16 * c) = o;
  }
  __syncthreads();
  // lanes past the rows read the last row; their columns are not stored
  const unsigned char* xrow[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) xrow[nt] = xsm + (size_t)min(8 * nt + g, p.t - 1) * x_pitch + 32 * j;
  // X of every group: with a constant for A (1, and 16 where x was divided)
  // each row of the product is the sums of x, in the scale of the others.
  constexpr uint32_t C1 = 0x00010001u, C16 = 0x00100010u;
  const uint32_t ones[4] = {C1, C1, C16, C16};
  for (int gr = threadIdx.x >> 5; gr < groups; gr += TEAMS * QMV_WARPS)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const unsigned char* xr = xrow[nt] + gr * 128;
      const uint4 v[2] = {*reinterpret_cast<const uint4*>(xr), *reinterpret_cast<const uint4*>(xr + 16)};
      float X[4];
      mma_first<F16>(X, ones, v[0].x, v[0].y);
      mma_16816(X, ones, v[0].z, v[0].w, F16);
      mma_16816(X, ones, v[1].x, v[1].y, F16);
      mma_16816(X, ones, v[1].z, v[1].w, F16);
      if (g == 0) {
        float* to = xsum + (gr * NT + nt) * (F16 ? 16 : 8) + 2 * j;
        if (F16) {  // and the 8-bit rows' scales of this group
          const int c = 8 * nt + 2 * j;
          const float f0 = c < p.t ? __ldg(p.xs + (size_t)c * groups + gr) : 0.f;
          const float f1 = c + 1 < p.t ? __ldg(p.xs + (size_t)(c + 1) * groups + gr) : 0.f;
          *reinterpret_cast<float2*>(to + 8) = make_float2(f0, f1);
          X[0] *= f0;
          X[1] *= f1;
        }
        *reinterpret_cast<float2*>(to) = make_float2(X[0], X[1]);
      }
    }
  store_scales(0);
  __syncthreads();

  int stage = 0, buf = 0;
  for (int tile = tile0; tile < tiles; tile += step) {
    fetch_scales(tile + step);
    const unsigned char* srow = scb + (size_t)buf * 32 * s_pitch + g * s_pitch;
    float acc[NT][4] = {};
    for (int u = ub; u < ue; ++u) {
      cp_async_wait<S - 2>();
      __syncwarp();  // this unit is there, and the last one is read by every lane
      issue(stage == 0 ? S - 1 : stage - 1);
      const unsigned char* src = ring + stage * QS_STAGE;
      stage = stage + 1 == S ? 0 : stage + 1;
      // scales and biases of rows g and g + 8; past the last group: not used
      const uint2 As = *reinterpret_cast<const uint2*>(srow + 8 * u);
      const uint2 Bs = *reinterpret_cast<const uint2*>(srow + 8 * u + 8 * s_pitch);
      const uint2 Ab = *reinterpret_cast<const uint2*>(srow + 8 * u + 16 * s_pitch);
      const uint2 Bb = *reinterpret_cast<const uint2*>(srow + 8 * u + 24 * s_pitch);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int gr = 4 * u + q;
        if (!VEC && gr >= groups) break;
        const uint2 wa = *reinterpret_cast<const uint2*>(src + g * QS_ROW + 32 * q + 8 * j);
        const uint2 wb = *reinterpret_cast<const uint2*>(src + (8 + g) * QS_ROW + 32 * q + 8 * j);
        uint32_t pa[2][4], pb[2][4];
        codes_raw(wa.x, pa[0]);
        codes_raw(wa.y, pa[1]);
        codes_raw(wb.x, pb[0]);
        codes_raw(wb.y, pb[1]);
        // scale and bias of group q: halves q of the row's 4 and 4
        auto half_of = [](uint32_t w, int hi) { return __half2float(__ushort_as_half((uint16_t)(hi ? w >> 16 : w))); };
        const float s0 = half_of(q < 2 ? As.x : As.y, q & 1), s1 = half_of(q < 2 ? Bs.x : Bs.y, q & 1);
        const float b0 = half_of(q < 2 ? Ab.x : Ab.y, q & 1), b1 = half_of(q < 2 ? Bb.x : Bb.y, q & 1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const unsigned char* xr = xrow[nt] + gr * 128;
          const uint4 v[2] = {*reinterpret_cast<const uint4*>(xr), *reinterpret_cast<const uint4*>(xr + 16)};
          const float* xg = xsum + (gr * NT + nt) * (F16 ? 16 : 8) + 2 * j;
          const float2 X = *reinterpret_cast<const float2*>(xg);
          const uint32_t xo[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
          float P[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const int w = s >> 1, h = 2 * (s & 1);
            const uint32_t a[4] = {pa[w][h], pb[w][h], pa[w][h + 1], pb[w][h + 1]};
            if (s == 0)
              mma_first<F16>(P, a, xo[0], xo[1]);
            else
              mma_16816(P, a, xo[2 * s], xo[2 * s + 1], F16);
          }
          float(&d)[4] = acc[nt];
          if (F16) {
            const float2 f = *reinterpret_cast<const float2*>(xg + 8);
            P[0] *= f.x, P[1] *= f.y, P[2] *= f.x, P[3] *= f.y;
          }
          d[0] = fmaf(s0, P[0], fmaf(b0, X.x, d[0]));
          d[1] = fmaf(s0, P[1], fmaf(b0, X.y, d[1]));
          d[2] = fmaf(s1, P[2], fmaf(b1, X.x, d[2]));
          d[3] = fmaf(s1, P[3], fmaf(b1, X.y, d[3]));
        }
      }
    }
    // the warps' sums, in a buffer that alternates: one barrier a tile
    float* mine = red + (size_t)(buf * QMV_WARPS + warp) * 8 * NT * 16;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float* q = mine + (8 * nt + 2 * j) * 16 + g;
      q[0] = acc[nt][0];
      q[16] = acc[nt][1];
      q[8] = acc[nt][2];
      q[24] = acc[nt][3];
    }
    store_scales(buf ^ 1);  // read since the last barrier but one by nobody
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(QMV_WARPS * 32) : "memory");
    for (int i = tt; i < p.t * 16; i += QMV_WARPS * 32) {
      const int c = i & 15, r = i >> 4, col = tile * 16 + c;
      if (col >= p.n) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < QMV_WARPS; ++w) v += red[((size_t)(buf * QMV_WARPS + w) * 8 * NT + r) * 16 + c];
      if (F16) {
        v *= 0x1p24f;
      } else {
        const int ex = rowmax[r] >> 23, up = ex == 255 || rowmax[r] == 0 ? 0 : 120 + 127 - max(ex, 1);
        v = times_pow2(v, 133 - up);
      }
      const size_t o = (size_t)r * p.n + col;
      if (out32)
        static_cast<float*>(p.y)[o] = v;
      else
        static_cast<uint16_t*>(p.y)[o] = f2bf(v);
    }
    buf ^= 1;
  }
  cp_async_wait<0>();
}

// What a CTA may have, static and dynamic together; bf16 rows have their largest
// magnitudes in static memory, which takes as much as the dynamic part's
// alignment (in the dynamic part they cost 1.5% of 4 rows of 4096 with 131072
// weight rows).
constexpr size_t QS_MAX_SMEM = 227 * 1024;
constexpr size_t QS_ALIGN = 128;
template <bool F16>
constexpr size_t QS_STATIC = F16 ? 0 : QS_ALIGN;
static_assert(8 * 2 * sizeof(int) <= QS_ALIGN, "rowmax of 16 rows");

template <int NT, int TEAMS, int S, bool F16>
bool try_config(const QmvParams& p, bool out32, cudaStream_t s, cudaError_t& e) {
  const size_t smem = qs_smem(p, NT, TEAMS, S);
  if (smem + QS_STATIC<F16> > QS_MAX_SMEM || p.k > QS_MAX_K) return false;
  const int tiles = (p.n + 15) / 16, ctas = (tiles + TEAMS - 1) / TEAMS;
  auto* kern = p.k % 512 == 0 ? qmv_stream_kernel<NT, TEAMS, S, F16, true> : qmv_stream_kernel<NT, TEAMS, S, F16, false>;
  if ((e = set_smem_limit_once(kern, (int)smem)) != cudaSuccess) return true;
  const dim3 grid(ctas < sm_count() ? ctas : sm_count()), block(TEAMS * QMV_WARPS * 32);
  MOE_LAUNCH("qmv_stream", s, { e = launch_k(kern, grid, block, smem, s, p, out32); });
  return true;
}

// The streaming kernel, if the rows of x fit beside its rings.  With more
// tiles than SMs it wants two teams a CTA; one team is then no match for the
// tile kernel below (8 rows of 8192 with 32768 weight rows: 66.6 us against
// 55.3), but for rows where that one pads most (9 rows of 4096 with 65536:
// 60.7 against 68.8, 16 rows 76.7 against 69.0) and for 8-bit rows (56.5
// against 73.2, 63.3 against 73.6).
template <int NT, bool F16>
bool try_stream(const QmvParams& p, bool out32, cudaStream_t s, cudaError_t& e) {
  if ((p.n + 15) / 16 > sm_count()) {
    if (try_config<NT, 2, 4, F16>(p, out32, s, e) || try_config<NT, 2, 3, F16>(p, out32, s, e)) return true;
    if (p.t <= 8 || (p.t > 12 && !F16)) return false;
  }
  return try_config<NT, 1, 4, F16>(p, out32, s, e) || try_config<NT, 1, 3, F16>(p, out32, s, e);
}

// ---------------------------------------------------------------------------
// More rows.
// ---------------------------------------------------------------------------

constexpr int QM_STAGES = 3;
template <int MT>
constexpr int qm_stage() { return MT * 16 * (QS_ROW + 16); }  // a unit: codes, then 4 scales and 4 biases a row
constexpr int QM_X_PITCH = 512 + 16;                           // bytes of a row's 4 groups of x, and a shift of banks
template <int NT, int MT>
constexpr int qm_smem() {
  return QMV_WARPS * QM_STAGES * qm_stage<MT>() + 2 * 8 * NT * QM_X_PITCH + 2 * 4 * 8 * NT * 8;
}

// y for 8 NT rows of x (a tile of them per blockIdx.y): a CTA owns 128 MT
// weight rows, 16 MT a warp, over all of k, in units of 4 groups.  Each warp's
// codes and scales come through a ring of its own, as in the streaming
// kernel; x comes unit by unit through two buffers that all warps share.
// What costs here is what is done per row of x, so codes are converted to
// 1 + q / 16, exact in bf16 and fp16, which needs nothing of x but the order of
// its values; P = sum q' x and X = sum x of a group add 16 s P + (b - 16 s) X.
// MT = 2 reads every value of x from shared memory once per 32 weight rows.
template <int NT, int MT, bool F16, bool VEC>
__global__ void __launch_bounds__(QMV_WARPS * 32, 1) qmv_tile_kernel(QmvParams p, bool out32) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int STAGE = qm_stage<MT>(), ROWS = 16 * MT, S = QM_STAGES;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, j = lane & 3;
  unsigned char* ring = smem + (size_t)warp * S * STAGE;
  unsigned char* xsm = smem + (size_t)QMV_WARPS * S * STAGE;                  // [2][8 NT rows]
  float2* xsum = reinterpret_cast<float2*>(xsm + 2 * 8 * NT * QM_X_PITCH);    // [2][4 groups][8 NT]: X, the row's scale
  const int groups = p.k >> 6, units = (groups + 3) >> 2;
  const int row0 = (blockIdx.x * QMV_WARPS + warp) * ROWS, t0 = blockIdx.y * 8 * NT;
  const size_t row_bytes = (size_t)p.k >> 1;
  pdl_wait();
  pdl_trigger();

  auto issue = [&](int u) {
    if (u < units && row0 < p.n) {
      unsigned char* dst = ring + (u % S) * STAGE;
      const int g0 = 4 * u, c = lane & 7;
#pragma unroll
      for (int i = 0; i < ROWS / 4; ++i) {
        const int r = 4 * i + (lane >> 3);
        // rows past the end read the last row; their results are not stored
        if (VEC || g0 + (c >> 1) < groups)
          cp_async16(dst + r * QS_ROW + 16 * c, p.codes + min(row0 + r, p.n - 1) * row_bytes + g0 * 32 + 16 * c);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int r = 16 * i + (lane >> 1);
        const uint16_t* src = (lane & 1 ? p.biases : p.scales) + (size_t)min(row0 + r, p.n - 1) * groups + g0;
        unsigned char* to = dst + ROWS * QS_ROW + r * 16 + 8 * (lane & 1);
        if (VEC) {
          cp_async8(to, src);
        } else {
          uint32_t v[4] = {};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (g0 + e < groups) v[e] = __ldg(src + e);
          *reinterpret_cast<uint2*>(to) = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
        }
      }
    }
    cp_async_commit();
  };

  // x of a unit: vector i of a thread is 8 values of row i * 8 + warp, so that
  // a warp reads one row's 256 and eight lanes hold a group
  uint4 xv[NT];
  float xf[NT];
  auto load_x = [&](int u) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = t0 + 8 * i + warp, gr = 4 * u + (lane >> 3);
      xv[i] = make_uint4(0, 0, 0, 0);
      xf[i] = 0.f;
      if (r < p.t && gr < groups) {
        if (F16) {
          const uint2 v = *reinterpret_cast<const uint2*>(p.xc + (size_t)r * p.k + u * 256 + 8 * lane);
          xv[i].x = v.x, xv[i].y = v.y;
          xf[i] = __ldg(p.xs + (size_t)r * groups + gr);
        } else {
          xv[i] = *reinterpret_cast<const uint4*>(p.x + (size_t)r * p.x_stride + u * 256 + 8 * lane);
        }
      }
    }
  };
  auto store_x = [&](int u) {
    unsigned char* xb = xsm + (u & 1) * 8 * NT * QM_X_PITCH;
    float2* sb = xsum + (u & 1) * 4 * 8 * NT;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      uint4 o;
      float sum;
      if (F16) {
        const uint2 v = make_uint2(xv[i].x, xv[i].y);
        const int8_t* b = reinterpret_cast<const int8_t*>(&v);
        auto pair = [&](int e) {
          const __half2 h = __floats2half2_rn(b[e], b[e + 4]);
          return *reinterpret_cast<const uint32_t*>(&h);
        };
        o = make_uint4(pair(0), pair(1), pair(2), pair(3));
        sum = (float)(((b[0] + b[1]) + (b[2] + b[3])) + ((b[4] + b[5]) + (b[6] + b[7])));
      } else {
        const uint4 v = xv[i];
        o = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                       __byte_perm(v.y, v.w, 0x7632));
        sum = ((bf16lo(v.x) + bf16hi(v.x)) + (bf16lo(v.y) + bf16hi(v.y))) +
              ((bf16lo(v.z) + bf16hi(v.z)) + (bf16lo(v.w) + bf16hi(v.w)));
      }
#pragma unroll
      for (int s = 1; s < 8; s *= 2) sum += __shfl_xor_sync(~0u, sum, s);
      *reinterpret_cast<uint4*>(xb + (8 * i + warp) * QM_X_PITCH + 16 * lane) = o;
      if ((lane & 7) == 0) sb[(lane >> 3) * 8 * NT + 8 * i + warp] = make_float2(sum, F16 ? xf[i] : 1.f);
    }
  };

#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);
  load_x(0);
  store_x(0);
  __syncthreads();
  float acc[MT][NT][4] = {};
  for (int u = 0; u < units; ++u) {
    if (u + 1 < units) load_x(u + 1);
    cp_async_wait<S - 2>();
    __syncwarp();  // this unit is there, and the last one is read by every lane
    issue(u + S - 1);
    const unsigned char* src = ring + (u % S) * STAGE;
    const unsigned char* xb = xsm + (u & 1) * 8 * NT * QM_X_PITCH;
    const float2* sums = xsum + (u & 1) * 4 * 8 * NT;
    uint4 sb[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        sb[m][e] = *reinterpret_cast<const uint4*>(src + ROWS * QS_ROW + (16 * m + 8 * e + g) * 16);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (!VEC && 4 * u + q >= groups) break;
      uint32_t pa[MT][2][4], pb[MT][2][4];
      float s[MT][2], b[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint2 wa = *reinterpret_cast<const uint2*>(src + (16 * m + g) * QS_ROW + 32 * q + 8 * j);
        const uint2 wb = *reinterpret_cast<const uint2*>(src + (16 * m + 8 + g) * QS_ROW + 32 * q + 8 * j);
        codes_to_pairs<F16>(wa.x, pa[m][0]);
        codes_to_pairs<F16>(wa.y, pa[m][1]);
        codes_to_pairs<F16>(wb.x, pb[m][0]);
        codes_to_pairs<F16>(wb.y, pb[m][1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t sw = q < 2 ? sb[m][e].x : sb[m][e].y, bw = q < 2 ? sb[m][e].z : sb[m][e].w;
          s[m][e] = 16.f * __half2float(__ushort_as_half((uint16_t)(q & 1 ? sw >> 16 : sw)));
          b[m][e] = __half2float(__ushort_as_half((uint16_t)(q & 1 ? bw >> 16 : bw))) - s[m][e];
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const unsigned char* xr = xb + (8 * nt + g) * QM_X_PITCH + q * 128 + 32 * j;
        const uint4 v0 = *reinterpret_cast<const uint4*>(xr), v1 = *reinterpret_cast<const uint4*>(xr + 16);
        const uint32_t xo[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        const float4 X = *reinterpret_cast<const float4*>(sums + q * 8 * NT + 8 * nt + 2 * j);  // rows 2 j, 2 j + 1
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float P[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int w = i >> 1, h = 2 * (i & 1);
            const uint32_t a[4] = {pa[m][w][h], pb[m][w][h], pa[m][w][h + 1], pb[m][w][h + 1]};
            if (i == 0)
              mma_first<F16>(P, a, xo[0], xo[1]);
            else
              mma_16816(P, a, xo[2 * i], xo[2 * i + 1], F16);
          }
          float(&d)[4] = acc[m][nt];
          if (F16) {
            d[0] = fmaf(X.y, fmaf(s[m][0], P[0], b[m][0] * X.x), d[0]);
            d[1] = fmaf(X.w, fmaf(s[m][0], P[1], b[m][0] * X.z), d[1]);
            d[2] = fmaf(X.y, fmaf(s[m][1], P[2], b[m][1] * X.x), d[2]);
            d[3] = fmaf(X.w, fmaf(s[m][1], P[3], b[m][1] * X.z), d[3]);
          } else {
            d[0] = fmaf(s[m][0], P[0], fmaf(b[m][0], X.x, d[0]));
            d[1] = fmaf(s[m][0], P[1], fmaf(b[m][0], X.z, d[1]));
            d[2] = fmaf(s[m][1], P[2], fmaf(b[m][1], X.x, d[2]));
            d[3] = fmaf(s[m][1], P[3], fmaf(b[m][1], X.z, d[3]));
          }
        }
      }
    }
    if (u + 1 < units) store_x(u + 1);  // its buffer was read up to the last barrier
    __syncthreads();
  }
  cp_async_wait<0>();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = row0 + 16 * m + 8 * (e >> 1) + g, r = t0 + 8 * nt + 2 * j + (e & 1);
        if (col >= p.n || r >= p.t) continue;
        const size_t o = (size_t)r * p.n + col;
        if (out32)
          static_cast<float*>(p.y)[o] = acc[m][nt][e];
        else
          static_cast<uint16_t*>(p.y)[o] = f2bf(acc[m][nt][e]);
      }
}

template <int NT, int MT, bool F16>
cudaError_t launch_tile(const QmvParams& p, bool out32, cudaStream_t s) {
  auto* kern = p.k % 256 == 0 ? qmv_tile_kernel<NT, MT, F16, true> : qmv_tile_kernel<NT, MT, F16, false>;
  cudaError_t e = set_smem_limit_once(kern, qm_smem<NT, MT>());
  if (e != cudaSuccess) return e;
  const dim3 grid((p.n + 128 * MT - 1) / (128 * MT), (p.t + 8 * NT - 1) / (8 * NT)), block(QMV_WARPS * 32);
  MOE_LAUNCH("qmv_tile", s, { e = launch_k(kern, grid, block, (size_t)qm_smem<NT, MT>(), s, p, out32); });
  return e;
}

template <bool F16>
cudaError_t launch_rows(const QmvParams& p, bool out32, cudaStream_t s) {
  // 32 weight rows a warp where that still gives every SM a CTA
  const bool wide = p.n >= 256 * sm_count();
  // Few rows stream the weights, unless k is so short that a tile's end comes
  // too often (4 rows with 131072 weight rows: k = 512 29.0 us streaming,
  // 17.8 in tiles; k = 1024 32.0 and 29.9).
  cudaError_t e;
  if (!(wide && p.k <= 1024) &&
      (p.t <= 8 ? try_stream<1, F16>(p, out32, s, e) : p.t <= 16 && try_stream<2, F16>(p, out32, s, e)))
    return e;
  if (p.t <= 8) return wide ? launch_tile<1, 2, F16>(p, out32, s) : launch_tile<1, 1, F16>(p, out32, s);
  if (p.t <= 16) return wide ? launch_tile<2, 2, F16>(p, out32, s) : launch_tile<2, 1, F16>(p, out32, s);
  if (p.t <= 32) return wide ? launch_tile<4, 2, F16>(p, out32, s) : launch_tile<4, 1, F16>(p, out32, s);
  return wide ? launch_tile<8, 2, F16>(p, out32, s) : launch_tile<8, 1, F16>(p, out32, s);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_qmv(const uint16_t* x, int64_t x_stride, const int8_t* x_codes, const float* x_scales,
                       const moe_qweights* w, int32_t t, int32_t n, int32_t k, void* y, int32_t y_fp32,
                       void* stream) {
  if (t < 1 || t > 65536) return set_error(MOE_ESHAPE, "t=%d outside [1, 65536]", t);
  if (n < 1 || n > 1048576) return set_error(MOE_ESHAPE, "n=%d outside [1, 1048576]", n);
  if (k < 64 || k > 65536 || k % 64)
    return set_error(MOE_ESHAPE, "k=%d must be a multiple of 64 in [64, 65536]", k);
  if (!w) return set_error(MOE_EINVAL, "w is NULL");
  if (!x == !x_codes || !x_codes != !x_scales)
    return set_error(MOE_EINVAL, "rows come as x, or as x_codes with x_scales");
  if (x && (x_stride < 0 || x_stride % 8))
    return set_error(MOE_ESHAPE, "x_stride must be a multiple of 8 elements, not negative");
  TRY(check_ptr(x, "x", 16, true));
  TRY(check_ptr(x_codes, "x_codes", 16, true));
  TRY(check_ptr(x_scales, "x_scales", 4, true));
  TRY(check_ptr(w->codes, "w->codes", 16));
  TRY(check_ptr(w->scales, "w->scales", 16));
  TRY(check_ptr(w->biases, "w->biases", 16));
  TRY(check_ptr(y, "y", y_fp32 ? 4 : 2));
  const QmvParams p{x, x_stride, x_codes, x_scales, w->codes, w->scales, w->biases, t, n, k, y};
  cudaStream_t s = (cudaStream_t)stream;
  const bool f = x_codes != nullptr, o = y_fp32 != 0;
  return cuda_status(f ? launch_rows<true>(p, o, s) : launch_rows<false>(p, o, s), "moe_qmv launch");
}
