// Residual addition, RMS norm and 8-bit output (moe_add_rms_norm); the norms
// behind and before a block with its gate (moe_gated_rms_norm).
#include <math.h>

#include <type_traits>

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

__device__ __forceinline__ uint4 pack8(const float (&a)[8]) {
  return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                    pack_bf16x2(a[6], a[7]));
}

// Vector v of a normed row, y = a * rstd * gamma: as bf16 (y, if asked for)
// and, with Q8, as codes and its group's scale.  Whole warps call it.
template <bool Q8>
__device__ __forceinline__ void store_normed(uint16_t* yp, int8_t* codes, float* scales, int h, int row, int v, bool on,
                                             int lane, const float (&a)[8], float rstd, uint4 gamma) {
  const uint32_t gg[4] = {gamma.x, gamma.y, gamma.z, gamma.w};
  float y[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[2 * j] = a[2 * j] * rstd * bf16lo(gg[j]);
    y[2 * j + 1] = a[2 * j + 1] * rstd * bf16hi(gg[j]);
  }
  if (on && yp) *reinterpret_cast<uint4*>(yp + (size_t)row * h + 8 * v) = pack8(y);
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
      *reinterpret_cast<uint2*>(codes + (size_t)row * h + 8 * v) = make_uint2(c[0], c[1]);
      if ((lane & 7) == 0) scales[(size_t)row * (h >> 6) + (v >> 3)] = bad ? __int_as_float(0x7fffffff) : m / 127.f;
    }
  }
}

// Sum over the `rw` warps of a row; `part` has 16 places of its own per call.
__device__ __forceinline__ float row_sum(float v, float* part, int lane, int warp, int rw) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if (rw > 1) {
    if (lane == 0) part[warp] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < rw; ++i) v += part[warp / rw * rw + i];
  }
  return v;
}

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
      *reinterpret_cast<uint4*>(p.sum + (size_t)row * p.h + 8 * v) = pack8(a[i]);
  }
  ss = row_sum(ss, part, lane, warp, rw);
  const float rstd = 1.f / sqrtf(ss / (float)p.h + p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = ti + i * rt;
    const bool on = live && v < nv;
    const uint4 g = on ? *reinterpret_cast<const uint4*>(p.gamma + 8 * v) : make_uint4(0, 0, 0, 0);
    store_normed<Q8>(p.y, p.codes, p.scales, p.h, row, v, on, lane, a[i], rstd, g);
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

struct GatedParams {
  NormParams n;  // x is the block's output
  const uint16_t* post_gamma;
  float residual_scale;
  moe_gate gate;
};

enum { GATE_NONE, GATE_ROW, GATE_CHANNEL };  // a gate value for each row, or for each channel

// As norm_kernel, with two sums of squares: the block's output is normed,
// gated and added to the scaled residual in registers, and that sum is normed
// again.  All of a row's loads are issued before the first sum, so that the
// second one waits on the barrier alone.
template <int VPT, bool Q8, int GATE>
__global__ void __launch_bounds__(512) gated_norm_kernel(GatedParams gp, int rt) {
  __shared__ float part[2][16];
  pdl_wait();
  pdl_trigger();
  const NormParams& p = gp.n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ti = threadIdx.x % rt, rw = rt >> 5;
  const int row = blockIdx.x * (blockDim.x / rt) + threadIdx.x / rt;
  const bool live = row < p.t;
  const int nv = p.h >> 3;
  float a[VPT][8];
  uint4 r[VPT], g[GATE == GATE_CHANNEL ? VPT : 1];
  float row_gate = 1.f;
  if (GATE == GATE_ROW && live) row_gate = bf16f(gp.gate.values[(size_t)row * gp.gate.row_stride]);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = ti + i * rt;
    const bool on = live && v < nv;
    uint4 u = make_uint4(0, 0, 0, 0);
    r[i] = u;
    if (GATE == GATE_CHANNEL) g[i] = u;
    if (on) {
      u = *reinterpret_cast<const uint4*>(p.x + (size_t)row * p.x_stride + 8 * v);
      if (p.residual) r[i] = *reinterpret_cast<const uint4*>(p.residual + (size_t)row * p.r_stride + 8 * v);
      if (GATE == GATE_CHANNEL)
        g[i] = *reinterpret_cast<const uint4*>(gp.gate.values + (size_t)row * gp.gate.row_stride + 8 * v);
    }
    const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[i][2 * j] = bf16lo(uu[j]);
      a[i][2 * j + 1] = bf16hi(uu[j]);
      ss = fmaf(a[i][2 * j], a[i][2 * j], ss);
      ss = fmaf(a[i][2 * j + 1], a[i][2 * j + 1], ss);
    }
  }
  float rstd = 1.f;
  if (gp.post_gamma) {
    ss = row_sum(ss, part[0], lane, warp, rw);
    rstd = 1.f / sqrtf(ss / (float)p.h + p.eps);
  }
  if (GATE == GATE_ROW && gp.gate.sigmoid) row_gate = 1.f / (1.f + expf(-row_gate));
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = ti + i * rt;
    const bool on = live && v < nv;
    const uint4 w = on && gp.post_gamma ? *reinterpret_cast<const uint4*>(gp.post_gamma + 8 * v)
                                        : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w}, rr[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
    uint32_t gg[4] = {};
    if (GATE == GATE_CHANNEL) gg[0] = g[i].x, gg[1] = g[i].y, gg[2] = g[i].z, gg[3] = g[i].w;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float b = a[i][j] * rstd * (j & 1 ? bf16hi(ww[j >> 1]) : bf16lo(ww[j >> 1]));
      if (GATE == GATE_ROW) b *= row_gate;
      if (GATE == GATE_CHANNEL) {
        const float z = j & 1 ? bf16hi(gg[j >> 1]) : bf16lo(gg[j >> 1]);
        b *= gp.gate.sigmoid ? 1.f / (1.f + expf(-z)) : z;
      }
      a[i][j] = p.residual ? fmaf(gp.residual_scale, j & 1 ? bf16hi(rr[j >> 1]) : bf16lo(rr[j >> 1]), b) : b;
      ss = fmaf(a[i][j], a[i][j], ss);
    }
    if (on && p.sum) *reinterpret_cast<uint4*>(p.sum + (size_t)row * p.h + 8 * v) = pack8(a[i]);
  }
  if (!p.y && !Q8) return;  // the same for the whole grid
  ss = row_sum(ss, part[1], lane, warp, rw);
  rstd = 1.f / sqrtf(ss / (float)p.h + p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = ti + i * rt;
    const bool on = live && v < nv;
    const uint4 w = on ? *reinterpret_cast<const uint4*>(p.gamma + 8 * v) : make_uint4(0, 0, 0, 0);
    store_normed<Q8>(p.y, p.codes, p.scales, p.h, row, v, on, lane, a[i], rstd, w);
  }
}

template <int VPT>
cudaError_t launch_gated(const GatedParams& p, int rt, cudaStream_t s) {
  const int rows = rt >= 256 ? 1 : 256 / rt;  // rows per CTA
  const dim3 grid((p.n.t + rows - 1) / rows), block(rt * rows);
  const auto go = [&](auto q8, auto gate) {
    cudaError_t e = cudaSuccess;
    MOE_LAUNCH("gated_rms_norm", s,
               { e = launch_k(gated_norm_kernel<VPT, decltype(q8)::value, decltype(gate)::value>, grid, block, 0, s, p, rt); });
    return e;
  };
  const auto by_gate = [&](auto q8) {
    if (!p.gate.values) return go(q8, std::integral_constant<int, GATE_NONE>{});
    return p.gate.per_channel ? go(q8, std::integral_constant<int, GATE_CHANNEL>{})
                              : go(q8, std::integral_constant<int, GATE_ROW>{});
  };
  return p.n.codes ? by_gate(std::true_type{}) : by_gate(std::false_type{});
}

// Arguments that the two calls share, checked, and the threads of a row.
int check_norm(const NormParams& p) {
  if (p.t < 1 || p.t > 65536) return set_error(MOE_ESHAPE, "t=%d outside [1, 65536]", p.t);
  if (p.h < 8 || p.h > NORM_MAX_H || p.h % 8)
    return set_error(MOE_ESHAPE, "h=%d must be a multiple of 8 in [8, %d]", p.h, NORM_MAX_H);
  if (p.x_stride < 0 || p.x_stride % 8 || (p.residual && (p.r_stride < 0 || p.r_stride % 8)))
    return set_error(MOE_ESHAPE, "row strides must be multiples of 8 elements, not negative");
  TRY(check_ptr(p.x, "x", 16));
  TRY(check_ptr(p.residual, "residual", 16, true));
  TRY(check_ptr(p.gamma, "gamma", 16));
  TRY(check_ptr(p.sum, "sum", 16, true));
  TRY(check_ptr(p.y, "y", 16, true));
  TRY(check_ptr(p.codes, "codes", 8, true));
  TRY(check_ptr(p.scales, "scales", 4, true));
  if (!p.sum && !p.y && !p.codes) return set_error(MOE_EINVAL, "no output asked for");
  if (!p.codes != !p.scales) return set_error(MOE_EINVAL, "codes and scales come together");
  if (p.codes && p.h % 64) return set_error(MOE_ESHAPE, "h=%d must be a multiple of 64 for 8-bit rows", p.h);
  if (!(p.eps >= 0.f)) return set_error(MOE_EINVAL, "eps=%g must not be negative", (double)p.eps);
  return MOE_OK;
}

int row_threads(int h, int vpt) {
  int rt = ((h / 8 + vpt - 1) / vpt + 31) / 32 * 32;
  if (rt < 256) {  // a power of two, so that rows tile the CTA
    int r = 32;
    while (r < rt) r *= 2;
    rt = r;
  }
  return rt;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_add_rms_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual,
                                int64_t residual_stride, const uint16_t* gamma, float eps, int32_t t, int32_t h,
                                uint16_t* sum, uint16_t* y, int8_t* codes, float* scales, void* stream) {
  const NormParams p{x, x_stride, residual, residual_stride, gamma, eps, t, h, sum, y, codes, scales};
  TRY(check_norm(p));
  // Vectors of a thread: up to 256 threads a row.  4096 rows of 4096 channels
  // took 24.9 us with one each, 22.5 with two (0.89 of the copy rate), 26.9
  // with four.
  const int nv = h / 8, vpt = nv <= 256 ? 1 : nv <= 512 ? 2 : 4, rt = row_threads(h, vpt);
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = vpt == 1 ? launch_norm<1>(p, rt, s) : vpt == 2 ? launch_norm<2>(p, rt, s)
                                                                        : launch_norm<4>(p, rt, s);
  return cuda_status(e, "moe_add_rms_norm launch");
}

extern "C" int moe_gated_rms_norm(const uint16_t* x, int64_t x_stride, const uint16_t* post_gamma, const moe_gate* gate,
                                  const uint16_t* residual, int64_t residual_stride, float residual_scale,
                                  const uint16_t* gamma, float eps, int32_t t, int32_t h, uint16_t* sum, uint16_t* y,
                                  int8_t* codes, float* scales, void* stream) {
  GatedParams p{{x, x_stride, residual, residual_stride, gamma, eps, t, h, sum, y, codes, scales},
                post_gamma,
                residual_scale,
                gate ? *gate : moe_gate{}};
  TRY(check_norm(p.n));
  TRY(check_ptr(post_gamma, "post_gamma", 16, true));
  if (gate) {
    TRY(check_ptr(gate->values, "gate->values", gate->per_channel ? 16 : 2));
    if (gate->row_stride < 0 || (gate->per_channel && gate->row_stride % 8))
      return set_error(MOE_ESHAPE, "gate rows must be a multiple of 8 elements apart, not negative");
  }
  if (!isfinite(residual_scale)) return set_error(MOE_EINVAL, "residual_scale is not finite");
  const int nv = h / 8, vpt = nv <= 256 ? 1 : nv <= 512 ? 2 : 4, rt = row_threads(h, vpt);
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = vpt == 1 ? launch_gated<1>(p, rt, s) : vpt == 2 ? launch_gated<2>(p, rt, s)
                                                                         : launch_gated<4>(p, rt, s);
  return cuda_status(e, "moe_gated_rms_norm launch");
}
