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
  TRY(check_ptr(w->scales, "w->scales", 2));
  TRY(check_ptr(w->biases, "w->biases", 2));
  TRY(check_ptr(y, "y", y_fp32 ? 4 : 2));
  const QmvParams p{x, x_stride, x_codes, x_scales, w->codes, w->scales, w->biases, t, n, k, y};
  cudaStream_t s = (cudaStream_t)stream;
  const bool f = x_codes != nullptr, o = y_fp32 != 0;
  const int nt = (t + 7) / 8;
  cudaError_t e;
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
