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

// A gate value for each row, or for each channel as it is or through the sigmoid
// (apart: chosen inside the loop, both were worked out for every value).
enum { GATE_NONE, GATE_ROW, GATE_CHANNEL, GATE_SIGMOID };

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

__device__ __forceinline__ void copy16(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
               : "memory");
}

// As norm_kernel, with two sums of squares: the block's output is normed,
// gated and added to the scaled residual in registers, and that sum is normed
// again.
//
// MANY: the grid fills the SMs and each row group walks its rows, the next
// STAGES - 1 of them on their way into shared memory (a thread copies what it
// reads itself, so that its own copies are all that it waits for), the weights
// in registers.  4096 rows of 4096 channels, 8 bytes a channel (19.8 us at the
// copy rate): 25.9 us, 29.7 with a gate (31.9 and 30.7 with a CTA for each row,
// whose weights are as much L2 traffic as its rows).  No unit is at its limit
// (issue slots 60 %, ALU 41 %, of the warps 35 %): what is left is the
// latency of a row's steps, conversions and two sums with barriers one after
// another, with as many warps as the registers leave room for.  Three CTAs of 256 threads an SM, two
// vectors a thread: four or one vectors, two CTAs or 512 threads took 27.8 to
// 38 us.  Otherwise a group takes one row: a decoded token's call (2.1 us),
// which is bound by the latency of its loads and two sums.
template <int VPT, bool Q8, int GATE, bool MANY>
__global__ void __launch_bounds__(VPT == 4 ? 512 : 256, VPT == 4 ? 1 : 3) gated_norm_kernel(GatedParams gp, int rt, int stages) {
  __shared__ float part[2][16];
  extern __shared__ uint4 ring[];  // [stage][x, residual, gate][vector][thread]
  pdl_wait();
  pdl_trigger();
  const NormParams& p = gp.n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x;
  const int ti = threadIdx.x % rt, rw = rt >> 5;
  const int step = gridDim.x * (threads / rt);
  int row = blockIdx.x * (threads / rt) + threadIdx.x / rt;
  const int nv = p.h >> 3;
  const bool rows_gate = GATE >= GATE_CHANNEL && gp.gate.row_stride > 0;  // a row of gates for each row
  const uint4 none = make_uint4(0, 0, 0, 0), ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  uint4 post[VPT], gamma[VPT], gate[GATE >= GATE_CHANNEL ? VPT : 1];
  uint4* const mine = ring + threadIdx.x;
  const auto fetch = [&](int r, int stage) {
    uint4* to = mine + stage * 3 * VPT * threads;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = ti + i * rt;
      if (r < p.t && v < nv) {
        copy16(to + i * threads, p.x + (size_t)r * p.x_stride + 8 * v);
        if (p.residual) copy16(to + (VPT + i) * threads, p.residual + (size_t)r * p.r_stride + 8 * v);
        if (rows_gate) copy16(to + (2 * VPT + i) * threads, gp.gate.values + (size_t)r * gp.gate.row_stride + 8 * v);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (MANY)
    for (int i = 0; i < stages - 1; ++i) fetch(row + i * step, i);
  uint4 u[VPT], r[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = ti + i * rt;
    const bool on = v < nv && row < p.t;
    if (!MANY) {
      u[i] = on ? *reinterpret_cast<const uint4*>(p.x + (size_t)row * p.x_stride + 8 * v) : none;
      r[i] = on && p.residual ? *reinterpret_cast<const uint4*>(p.residual + (size_t)row * p.r_stride + 8 * v) : none;
    }
    if (GATE >= GATE_CHANNEL)
      gate[i] = on && !(MANY && rows_gate)
                    ? *reinterpret_cast<const uint4*>(gp.gate.values + (size_t)row * gp.gate.row_stride + 8 * v)
                    : none;
    post[i] = on && gp.post_gamma ? *reinterpret_cast<const uint4*>(gp.post_gamma + 8 * v) : ones;
    gamma[i] = on ? *reinterpret_cast<const uint4*>(p.gamma + 8 * v) : none;
  }
  int stage = 0;
  do {
    const bool live = row < p.t;
    float row_gate = 1.f;
    if (GATE == GATE_ROW && live) row_gate = bf16f(gp.gate.values[(size_t)row * gp.gate.row_stride]);
    if (MANY) {
      if (stages == 2)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      const uint4* from = mine + stage * 3 * VPT * threads;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const bool on = live && ti + i * rt < nv;
        u[i] = on ? from[i * threads] : none;
        r[i] = on && p.residual ? from[(VPT + i) * threads] : none;
        if (GATE >= GATE_CHANNEL && rows_gate) gate[i] = on ? from[(2 * VPT + i) * threads] : none;
      }
      const int free = stage == 0 ? stages - 1 : stage - 1;  // read in the last step
      fetch(row + (stages - 1) * step, free);
      stage = stage + 1 == stages ? 0 : stage + 1;
    }
    float a[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t uu[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
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
    if (GATE == GATE_ROW) rstd *= gp.gate.sigmoid ? sigmoid(row_gate) : row_gate;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = ti + i * rt;
      const uint32_t ww[4] = {post[i].x, post[i].y, post[i].z, post[i].w}, rr[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
      uint32_t gg[4] = {};
      if (GATE >= GATE_CHANNEL) gg[0] = gate[i].x, gg[1] = gate[i].y, gg[2] = gate[i].z, gg[3] = gate[i].w;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float b = a[i][j] * rstd * (j & 1 ? bf16hi(ww[j >> 1]) : bf16lo(ww[j >> 1]));
        if (GATE >= GATE_CHANNEL) {
          const float z = j & 1 ? bf16hi(gg[j >> 1]) : bf16lo(gg[j >> 1]);
          b *= GATE == GATE_SIGMOID ? sigmoid(z) : z;
        }
        a[i][j] = p.residual ? fmaf(gp.residual_scale, j & 1 ? bf16hi(rr[j >> 1]) : bf16lo(rr[j >> 1]), b) : b;
        ss = fmaf(a[i][j], a[i][j], ss);
      }
      if (live && v < nv && p.sum) *reinterpret_cast<uint4*>(p.sum + (size_t)row * p.h + 8 * v) = pack8(a[i]);
    }
    if (p.y || Q8) {  // the same for the whole grid
      ss = row_sum(ss, part[1], lane, warp, rw);
      rstd = 1.f / sqrtf(ss / (float)p.h + p.eps);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = ti + i * rt;
        store_normed<Q8>(p.y, p.codes, p.scales, p.h, row, v, live && v < nv, lane, a[i], rstd, gamma[i]);
      }
    }
    row += step;
    // a CTA's groups go on together: the sums have barriers, and one between
    // two uses of the same places where only one of the sums is taken
    if (MANY && rw > 1 && !(gp.post_gamma && (p.y || Q8))) __syncthreads();
  } while (MANY && row - (int)(threadIdx.x / rt) < p.t);
}

template <int VPT>
cudaError_t launch_gated(const GatedParams& p, int rt, cudaStream_t s) {
  const int rows = rt >= 256 ? 1 : 256 / rt, threads = rt * rows;  // rows at a time of a CTA
  const int stage_bytes = 3 * VPT * threads * 16, stages = 3 * stage_bytes <= 108 * 1024 ? 3 : 2;
  // as many CTAs an SM as their rings leave room for, two at least where the registers do
  const int fit = 220 * 1024 / (stages * stage_bytes), most = VPT < 4 ? 3 : threads > 256 ? 1 : 2;
  const int full = sm_count() * (fit < most ? fit : most);
  // rows of the walk: three steps and more, below that a CTA for each row is as good
  const bool many = p.n.t >= 3 * full * rows;
  const dim3 grid(many ? full : (p.n.t + rows - 1) / rows), block(threads);
  const int ring = many ? stages * stage_bytes : 0;
  const auto go = [&](auto q8, auto gate, auto walk) {
    const auto kern = gated_norm_kernel<VPT, decltype(q8)::value, decltype(gate)::value, decltype(walk)::value>;
    cudaError_t e = ring ? set_smem_limit_once(kern, ring) : cudaSuccess;
    if (e != cudaSuccess) return e;
    MOE_LAUNCH("gated_rms_norm", s, { e = launch_k(kern, grid, block, (size_t)ring, s, p, rt, stages); });
    return e;
  };
  const auto by_size = [&](auto q8, auto gate) { return many ? go(q8, gate, std::true_type{}) : go(q8, gate, std::false_type{}); };
  const auto by_gate = [&](auto q8) {
    if (!p.gate.values) return by_size(q8, std::integral_constant<int, GATE_NONE>{});
    if (!p.gate.per_channel) return by_size(q8, std::integral_constant<int, GATE_ROW>{});
    return p.gate.sigmoid ? by_size(q8, std::integral_constant<int, GATE_SIGMOID>{})
                          : by_size(q8, std::integral_constant<int, GATE_CHANNEL>{});
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
  // As above (so that without a norm or a gate behind the block the two calls
  // agree to the last bit), but of many short rows a warp takes each: its sums
  // have no barriers (65536 rows of 512 channels: 59 -> 48 us; of 1024: 112 -> 97;
  // 8192 rows, launch and cold caches in it: 16.5 -> 14.5 and 23 -> 21).
  const int nv = h / 8;
  const bool by_warp = t >= 8192 && nv <= 128;
  const int vpt = by_warp ? (nv <= 32 ? 1 : nv <= 64 ? 2 : 4) : nv <= 256 ? 1 : nv <= 512 ? 2 : 4;
  const int rt = row_threads(h, vpt);
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = vpt == 1 ? launch_gated<1>(p, rt, s) : vpt == 2 ? launch_gated<2>(p, rt, s)
                                                                         : launch_gated<4>(p, rt, s);
  return cuda_status(e, "moe_gated_rms_norm launch");
}
