// Residual addition, RMS norm and 8-bit output (moe_add_rms_norm).
#include <math.h>

#include "api_checks.cuh"

namespace moe {

namespace {

constexpr int NORM_MAX_H = 16384;

struct NormParams {
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* residual;
  int64_t r_stride;
  const uint16_t* gamma;
  float eps;
  int t, h;
  uint16_t* sum;
  uint16_t* y;
  int8_t* codes;
  float* scales;
};

// One row per group of `rt` threads (a multiple of 32), `blockDim.x / rt`
// rows per CTA.  Thread i of a row holds the 16-byte vectors i, i + rt, ...
// of it (VPT of them) in registers between the sum of squares and the
// scaling, so that memory is read and written once: 2 bytes in per operand
// and 2 out per output and channel, which is what bounds the kernel.  Eight
// neighbouring lanes hold the 64 channels of one 8-bit group.
template <int VPT, bool Q8>
__global__ void __launch_bounds__(512) norm_kernel(NormParams p, int rt) {
  __shared__ float part[16];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ti = threadIdx.x % rt, rw = rt >> 5;
  const int row = blockIdx.x * (blockDim.x / rt) + threadIdx.x / rt;
  const bool live = row < p.t;
  const int nv = p.h >> 3;
  float a[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = ti + i * rt;
    const bool on = live && v < nv;
    uint4 u = make_uint4(0, 0, 0, 0), w = make_uint4(0, 0, 0, 0);
    if (on) {
      u = *reinterpret_cast<const uint4*>(p.x + (size_t)row * p.x_stride + 8 * v);
      if (p.residual) w = *reinterpret_cast<const uint4*>(p.residual + (size_t)row * p.r_stride + 8 * v);
    }
    const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[i][2 * j] = bf16lo(uu[j]) + bf16lo(ww[j]);
      a[i][2 * j + 1] = bf16hi(uu[j]) + bf16hi(ww[j]);
      ss = fmaf(a[i][2 * j], a[i][2 * j], ss);
      ss = fmaf(a[i][2 * j + 1], a[i][2 * j + 1], ss);
    }
    if (on && p.sum)
      *reinterpret_cast<uint4*>(p.sum + (size_t)row * p.h + 8 * v) =
          make_uint4(pack_bf16x2(a[i][0], a[i][1]), pack_bf16x2(a[i][2], a[i][3]), pack_bf16x2(a[i][4], a[i][5]),
                     pack_bf16x2(a[i][6], a[i][7]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
  if (rw > 1) {
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < rw; ++i) ss += part[warp / rw * rw + i];
  }
  const float rstd = 1.f / sqrtf(ss / (float)p.h + p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = ti + i * rt;
    const bool on = live && v < nv;
    const uint4 g = on ? *reinterpret_cast<const uint4*>(p.gamma + 8 * v) : make_uint4(0, 0, 0, 0);
    const uint32_t gg[4] = {g.x, g.y, g.z, g.w};
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[2 * j] = a[i][2 * j] * rstd * bf16lo(gg[j]);
      y[2 * j + 1] = a[i][2 * j + 1] * rstd * bf16hi(gg[j]);
    }
    if (on && p.y)
      *reinterpret_cast<uint4*>(p.y + (size_t)row * p.h + 8 * v) =
          make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                     pack_bf16x2(y[6], y[7]));
    if (Q8) {
      // the group's largest magnitude; fmaxf drops NaN, so finiteness (of
      // the 127-fold, which is what gets divided) is carried apart
      float m = 0.f;
      bool bad = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m = fmaxf(m, fabsf(y[j]));
        bad |= !isfinite(y[j] * 127.f);
      }
#pragma unroll
      for (int o = 4; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
      const uint32_t vote = __ballot_sync(~0u, bad);
      bad = (vote >> (lane & 24)) & 0xFFu;
      uint32_t c[2] = {0, 0};
      if (m > 0.f && !bad) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          c[j >> 2] |= (uint32_t)(uint8_t)(int8_t)__float2int_rn(y[j] * 127.f / m) << (8 * (j & 3));
      }
      if (on) {
        *reinterpret_cast<uint2*>(p.codes + (size_t)row * p.h + 8 * v) = make_uint2(c[0], c[1]);
        if ((lane & 7) == 0)
          p.scales[(size_t)row * (p.h >> 6) + (v >> 3)] = bad ? __int_as_float(0x7fffffff) : m / 127.f;
      }
    }
  }
}

template <int VPT>
cudaError_t launch_norm(const NormParams& p, int rt, cudaStream_t s) {
  const int rows = rt >= 256 ? 1 : 256 / rt;  // rows per CTA
  const dim3 grid((p.t + rows - 1) / rows), block(rt * rows);
  cudaError_t e = cudaSuccess;
  MOE_LAUNCH("add_rms_norm", s, {
    e = p.codes ? launch_k(norm_kernel<VPT, true>, grid, block, 0, s, p, rt)
                : launch_k(norm_kernel<VPT, false>, grid, block, 0, s, p, rt);
  });
  return e;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_add_rms_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual,
                                int64_t residual_stride, const uint16_t* gamma, float eps, int32_t t, int32_t h,
                                uint16_t* sum, uint16_t* y, int8_t* codes, float* scales, void* stream) {
  if (t < 1 || t > 65536) return set_error(MOE_ESHAPE, "t=%d outside [1, 65536]", t);
  if (h < 8 || h > NORM_MAX_H || h % 8)
    return set_error(MOE_ESHAPE, "h=%d must be a multiple of 8 in [8, %d]", h, NORM_MAX_H);
  if (x_stride < 0 || x_stride % 8 || (residual && (residual_stride < 0 || residual_stride % 8)))
    return set_error(MOE_ESHAPE, "row strides must be multiples of 8 elements, not negative");
  TRY(check_ptr(x, "x", 16));
  TRY(check_ptr(residual, "residual", 16, true));
  TRY(check_ptr(gamma, "gamma", 16));
  TRY(check_ptr(sum, "sum", 16, true));
  TRY(check_ptr(y, "y", 16, true));
  TRY(check_ptr(codes, "codes", 8, true));
  TRY(check_ptr(scales, "scales", 4, true));
  if (!sum && !y && !codes) return set_error(MOE_EINVAL, "no output asked for");
  if (!codes != !scales) return set_error(MOE_EINVAL, "codes and scales come together");
  if (codes && h % 64) return set_error(MOE_ESHAPE, "h=%d must be a multiple of 64 for 8-bit rows", h);
  if (!(eps >= 0.f)) return set_error(MOE_EINVAL, "eps=%g must not be negative", (double)eps);
  const NormParams p{x, x_stride, residual, residual_stride, gamma, eps, t, h, sum, y, codes, scales};
  // Vectors of a thread: up to 256 threads a row.  4096 rows of 4096 channels
  // took 24.9 us with one each, 22.5 with two (0.89 of the copy rate), 26.9
  // with four.
  const int nv = h / 8, vpt = nv <= 256 ? 1 : nv <= 512 ? 2 : 4;
  int rt = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
  if (rt < 256) {  // a power of two, so that rows tile the CTA
    int r = 32;
    while (r < rt) r *= 2;
    rt = r;
  }
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = vpt == 1 ? launch_norm<1>(p, rt, s) : vpt == 2 ? launch_norm<2>(p, rt, s)
                                                                        : launch_norm<4>(p, rt, s);
  return cuda_status(e, "moe_add_rms_norm launch");
}
