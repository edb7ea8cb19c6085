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

// 16 row values k = 16 j .. 16 j + 15 of one group as the B operands of its
// four products: o[2 s], o[2 s + 1] hold the pairs (k0 + i, k0 + i + 4) that
// meet pairs 2 (s & 1) and 2 (s & 1) + 1 of the code word s >> 1.
__device__ __forceinline__ void row_pairs(const uint4 (&u)[2], uint32_t (&o)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    o[4 * h + 0] = __byte_perm(u[h].x, u[h].z, 0x5410);
    o[4 * h + 1] = __byte_perm(u[h].x, u[h].z, 0x7632);
    o[4 * h + 2] = __byte_perm(u[h].y, u[h].w, 0x5410);
    o[4 * h + 3] = __byte_perm(u[h].y, u[h].w, 0x7632);
  }
}

// The same from 16 signed 8-bit codes, to fp16: 1024 + (c + 128) is exact
// under the exponent of 1024, and so is the difference to 1152.
__device__ __forceinline__ void code_pairs(uint4 u, uint32_t (&o)[8]) {
  const uint32_t w[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
  const __half2 off = __floats2half2_rn(1152.f, 1152.f);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // bytes i of both words, each in the low byte of a half
      const uint32_t v = (__byte_perm(w[2 * h], w[2 * h + 1], i | (4 + i) << 8) & 0x00FFu) |
                         ((w[2 * h + 1] >> (8 * i)) & 0xFFu) << 16 | 0x64006400u;
      const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), off);
      o[4 * h + i] = *reinterpret_cast<const uint32_t*>(&r);
    }
}

constexpr int QMV_WARPS = 8;

// y = x W^T with W as the A operand of m16n8k16: a warp owns a tile of 16
// weight rows and 8 NT rows of x, and walks its share of the 64-wide groups.
// Per group a lane loads 8 bytes of codes of two weight rows (a quad covers a
// group's 32 bytes) straight into the fragment layout -- the order of k
// within a group is free as long as both operands agree -- so weights never
// pass through shared memory.  With q' = 1 + q / 16 the products give
// P = sum q' x and, from a constant operand of ones, X = sum x, and the
// group adds 16 s P + (b - 16 s) X, exactly s sum q x + b sum x.
// KS warps share a tile, each with a contiguous part of the groups; their
// sums meet in shared memory in a fixed order.
template <int NT, bool F16, bool OUT32>
__global__ void __launch_bounds__(QMV_WARPS * 32) qmv_kernel(QmvParams p, int KS) {
  extern __shared__ float red[];  // [warp][16][8 NT]
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, j = lane & 3;
  const int tiles = QMV_WARPS / KS, ks = warp % KS;
  const int row0 = (blockIdx.x * tiles + warp / KS) * 16;
  const int t0 = blockIdx.y * 8 * NT;
  const int groups = p.k >> 6;
  const int gb = (int)((int64_t)groups * ks / KS), ge = (int)((int64_t)groups * (ks + 1) / KS);
  // rows past the end read the last row; their results are not stored
  const int ra = min(row0 + g, p.n - 1), rb = min(row0 + g + 8, p.n - 1);
  const uint8_t* ca = p.codes + (size_t)ra * (p.k >> 1) + 8 * j;
  const uint8_t* cb = p.codes + (size_t)rb * (p.k >> 1) + 8 * j;
  const uint16_t* sa = p.scales + (size_t)ra * groups;
  const uint16_t* sb = p.scales + (size_t)rb * groups;
  const uint16_t* ba = p.biases + (size_t)ra * groups;
  const uint16_t* bb = p.biases + (size_t)rb * groups;
  constexpr uint32_t ONES = F16 ? 0x3C003C00u : 0x3F803F80u;
  const uint32_t ones[4] = {ONES, ONES, ONES, ONES};
  float acc[NT][4] = {};
  if (row0 < p.n)
#pragma unroll 4
    for (int gr = gb; gr < ge; ++gr) {
      const uint2 wa = __ldg(reinterpret_cast<const uint2*>(ca + gr * 32));
      const uint2 wb = __ldg(reinterpret_cast<const uint2*>(cb + gr * 32));
      const float s0 = 16.f * __half2float(__ushort_as_half(__ldg(sa + gr)));
      const float s1 = 16.f * __half2float(__ushort_as_half(__ldg(sb + gr)));
      const float b0 = __half2float(__ushort_as_half(__ldg(ba + gr))) - s0;
      const float b1 = __half2float(__ushort_as_half(__ldg(bb + gr))) - s1;
      uint32_t pa[2][4], pb[2][4];
      codes_to_pairs<F16>(wa.x, pa[0]);
      codes_to_pairs<F16>(wa.y, pa[1]);
      codes_to_pairs<F16>(wb.x, pb[0]);
      codes_to_pairs<F16>(wb.y, pb[1]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = t0 + 8 * nt + g;
        uint32_t xo[8];
        if (F16) {
          uint4 u = make_uint4(0, 0, 0, 0);
          if (r < p.t) u = *reinterpret_cast<const uint4*>(p.xc + (size_t)r * p.k + gr * 64 + 16 * j);
          code_pairs(u, xo);
        } else {
          uint4 u[2] = {};
          if (r < p.t) {
            const uint4* q = reinterpret_cast<const uint4*>(p.x + (size_t)r * p.x_stride + gr * 64 + 16 * j);
            u[0] = q[0];
            u[1] = q[1];
          }
          row_pairs(u, xo);
        }
        float P[4] = {}, X[4] = {};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int w = s >> 1, q = 2 * (s & 1);
          const uint32_t a[4] = {pa[w][q], pb[w][q], pa[w][q + 1], pb[w][q + 1]};
          mma_16816(P, a, xo[2 * s], xo[2 * s + 1], F16);
          mma_16816(X, ones, xo[2 * s], xo[2 * s + 1], F16);
        }
        float f0 = 1.f, f1 = 1.f;
        if (F16) {  // the rows' scales of this group
          const int c = t0 + 8 * nt + 2 * j;
          f0 = c < p.t ? p.xs[(size_t)c * groups + gr] : 0.f;
          f1 = c + 1 < p.t ? p.xs[(size_t)(c + 1) * groups + gr] : 0.f;
        }
        acc[nt][0] = fmaf(f0, fmaf(s0, P[0], b0 * X[0]), acc[nt][0]);
        acc[nt][1] = fmaf(f1, fmaf(s0, P[1], b0 * X[1]), acc[nt][1]);
        acc[nt][2] = fmaf(f0, fmaf(s1, P[2], b1 * X[2]), acc[nt][2]);
        acc[nt][3] = fmaf(f1, fmaf(s1, P[3], b1 * X[3]), acc[nt][3]);
      }
    }
  // sums of the KS parts, rows of x outermost, weight rows contiguous
  float* mine = red + (size_t)warp * 16 * 8 * NT;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float* q = mine + (8 * nt + 2 * j) * 16;
    q[g] = acc[nt][0];
    q[16 + g] = acc[nt][1];
    q[g + 8] = acc[nt][2];
    q[16 + g + 8] = acc[nt][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tiles * 16 * 8 * NT; i += blockDim.x) {
    const int c = i % 16, tile = i / 16 % tiles, r = i / (16 * tiles);
    const int col = (blockIdx.x * tiles + tile) * 16 + c;
    if (t0 + r >= p.t || col >= p.n) continue;
    float v = 0.f;
    for (int s = 0; s < KS; ++s) v += red[((size_t)(tile * KS + s) * 8 * NT + r) * 16 + c];
    const size_t o = (size_t)(t0 + r) * p.n + col;
    if (OUT32)
      static_cast<float*>(p.y)[o] = v;
    else
      static_cast<uint16_t*>(p.y)[o] = f2bf(v);
  }
}

// ---------------------------------------------------------------------------
// Few rows: weights streamed through shared memory.
// ---------------------------------------------------------------------------

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
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

// The products of qmv_kernel for t <= 8 NT rows, when what counts is how
// fast the weights come.  The CTA stages x once; then each of its TEAMS teams
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

constexpr size_t QS_MAX_SMEM = 227 * 1024;

template <int NT, int TEAMS, int S, bool F16>
bool try_config(const QmvParams& p, bool out32, cudaStream_t s, cudaError_t& e) {
  const size_t smem = qs_smem(p, NT, TEAMS, S);
  if (smem > QS_MAX_SMEM || p.k > QS_MAX_K) return false;
  const int tiles = (p.n + 15) / 16, ctas = (tiles + TEAMS - 1) / TEAMS;
  auto* kern = p.k % 512 == 0 ? qmv_stream_kernel<NT, TEAMS, S, F16, true> : qmv_stream_kernel<NT, TEAMS, S, F16, false>;
  if ((e = set_smem_limit_once(kern, (int)smem)) != cudaSuccess) return true;
  const dim3 grid(ctas < sm_count() ? ctas : sm_count()), block(TEAMS * QMV_WARPS * 32);
  MOE_LAUNCH("qmv_stream", s, { e = launch_k(kern, grid, block, smem, s, p, out32); });
  return true;
}

// The streaming kernel, if the rows of x fit beside its rings: two teams a
// CTA when there are tiles for them.
template <int NT, bool F16>
bool try_stream(const QmvParams& p, bool out32, cudaStream_t s, cudaError_t& e) {
  if ((p.n + 15) / 16 > sm_count() && (try_config<NT, 2, 4, F16>(p, out32, s, e) || try_config<NT, 2, 3, F16>(p, out32, s, e)))
    return true;
  return try_config<NT, 1, 4, F16>(p, out32, s, e) || try_config<NT, 1, 3, F16>(p, out32, s, e);
}

template <int NT, bool F16>
cudaError_t launch_qmv(const QmvParams& p, bool out32, cudaStream_t s) {
  const int tiles = (p.n + 15) / 16, groups = p.k / 64;
  // as few parts of k as keep every SM's warps busy
  int KS = 1;
  while (KS < QMV_WARPS && KS * 2 <= groups && (int64_t)tiles * KS < (int64_t)sm_count() * 16) KS *= 2;
  const int per = QMV_WARPS / KS;
  const dim3 grid((tiles + per - 1) / per, (p.t + 8 * NT - 1) / (8 * NT)), block(QMV_WARPS * 32);
  const size_t smem = (size_t)QMV_WARPS * 16 * 8 * NT * 4;
  cudaError_t e;
  auto* kern = out32 ? qmv_kernel<NT, F16, true> : qmv_kernel<NT, F16, false>;
  if (smem > 48 * 1024 && (e = set_smem_limit_once(kern, (int)smem)) != cudaSuccess) return e;
  MOE_LAUNCH("qmv", s, { e = launch_k(kern, grid, block, smem, s, p, KS); });
  return e;
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
  const int nt = (t + 7) / 8;
  cudaError_t e;
  if (t <= 8 ? (f ? try_stream<1, true>(p, o, s, e) : try_stream<1, false>(p, o, s, e))
             : t <= 16 && (f ? try_stream<2, true>(p, o, s, e) : try_stream<2, false>(p, o, s, e)))
    return cuda_status(e, "moe_qmv launch");
  if (nt <= 1)
    e = f ? launch_qmv<1, true>(p, o, s) : launch_qmv<1, false>(p, o, s);
  else if (nt <= 2)
    e = f ? launch_qmv<2, true>(p, o, s) : launch_qmv<2, false>(p, o, s);
  else if (nt <= 4)
    e = f ? launch_qmv<4, true>(p, o, s) : launch_qmv<4, false>(p, o, s);
  else
    e = f ? launch_qmv<8, true>(p, o, s) : launch_qmv<8, false>(p, o, s);
  return cuda_status(e, "moe_qmv launch");
}
