// Append to the paged 8-bit key/value cache (moe_kv_append).
#include <math.h>

#include "kv_common.cuh"

namespace moe {

namespace {

constexpr int APPEND_THREADS = 256;

// A bf16 pair with each value whose 127-fold is not finite replaced by zero.
__device__ __forceinline__ uint32_t finite_pair(uint32_t u, bool& bad) {
  if (!isfinite(bf16lo(u) * 127.f)) u &= 0xFFFF0000u, bad = true;
  if (!isfinite(bf16hi(u) * 127.f)) u &= 0x0000FFFFu, bad = true;
  return u;
}
__device__ __forceinline__ uint4 finite_vec(uint4 u, bool& bad) {
  return make_uint4(finite_pair(u.x, bad), finite_pair(u.y, bad), finite_pair(u.z, bad), finite_pair(u.w, bad));
}

// v * 127 / m to the nearest whole number, ties to even, exactly: with an
// approximate quotient rounded to q, the remainder x - q m is exact in one
// fma (q and the bf16 m have 7 and 8 bits), and it says whether q is the
// nearest.  rm = 1 / m.  A true division costs about twice the instructions.
__device__ __forceinline__ int nearest_code(float v, float m, float rm) {
  const float x = v * 127.f;
  const float q = rintf(x * rm);
  const float r = fmaf(-q, m, x), over = fabsf(r) + fabsf(r) - m;
  const int c = (int)q;
  return over > 0.f || (over == 0.f && (c & 1)) ? c + (r > 0.f ? 1 : -1) : c;
}

// One CTA per (touched block, head, keys or values): the block's values stay
// in registers (VPT 16-byte vectors a thread) between the maximum and the
// codes, so every token is read once and every code written once; the bytes
// moved bound it.  Block slots are numbered without a scan: sequence s owns
// the slots from starts[s] / block + 2 s on, which is enough for n new
// tokens, as they touch at most (n - 1) / block + 2 blocks.
template <int VPT>
__global__ void __launch_bounds__(APPEND_THREADS)
    kv_append_kernel(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const int32_t* starts,
                     int t, moe_kv_cache c, DeviceStatus* st) {
  __shared__ float part[APPEND_THREADS / 32];
  __shared__ int owner;
  pdl_wait();
  pdl_trigger();
  const int slot = blockIdx.x, head = blockIdx.y, isv = blockIdx.z, tid = threadIdx.x;
  // the sequence that owns the slot: every thread looks at some, one answers
  if (tid == 0) owner = -1;
  __syncthreads();
  for (int i = tid; i < c.n_seq; i += APPEND_THREADS)
    if (starts[i] / c.block + 2 * i <= slot && slot < starts[i + 1] / c.block + 2 * (i + 1)) owner = i;
  __syncthreads();
  const int s = owner;
  if (s < 0) {  // past the last sequence, or starts out of order
    if (tid == 0 && slot < starts[c.n_seq] / c.block + 2 * c.n_seq) raise_flag(st, FLAG_BAD_CACHE);
    return;
  }
  int row0, n, len;
  if (!kv_sequence(c, starts, t, s, row0, n, len)) {
    if (tid == 0) raise_flag(st, FLAG_BAD_CACHE);
    return;
  }
  if (n == 0) return;
  const int old = len - n, first = old / c.block, last = (len - 1) / c.block;
  const int b = first + slot - (row0 / c.block + 2 * s);
  if (b < first || b > last) return;
  const int page = c.table[(size_t)s * c.max_blocks + b];
  const uint16_t* src = isv ? v : k;
  const int64_t stride = isv ? v_stride : k_stride;
  const int ring = 2 * c.block;
  uint16_t* tail = c.tail + (((size_t)s * 2 + isv) * c.hkv + head) * ring * c.d;
  const int vd = c.d >> 3, nv = c.block * vd;  // vectors of a token and of the block
  uint4 u[VPT];
  bool bad = false, lost = false;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = tid + i * APPEND_THREADS, r = e / vd, x = e % vd;
    const int pos = b * c.block + r;
    u[i] = make_uint4(0, 0, 0, 0);
    if (e < nv && pos < len) {
      if (pos < old)
        u[i] = finite_vec(*reinterpret_cast<const uint4*>(tail + (size_t)(pos % ring) * c.d + 8 * x), lost);
      else
        u[i] = finite_vec(*reinterpret_cast<const uint4*>(src + (size_t)(row0 + pos - old) * stride +
                                                          (size_t)head * c.d + 8 * x), bad);
    }
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) m = fmaxf(m, fmaxf(fabsf(bf16lo(w[q])), fabsf(bf16hi(w[q]))));
  }
  if (bad) raise_flag(st, FLAG_NOT_FINITE);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  if ((tid & 31) == 0) part[tid >> 5] = m;
  __syncthreads();  // also: what this block reads of the tail is in registers
#pragma unroll
  for (int i = 0; i < APPEND_THREADS / 32; ++i) m = fmaxf(m, part[i]);
  if (page < 0 || page >= c.n_pages) {
    if (tid == 0) raise_flag(st, FLAG_BAD_CACHE);
  } else {
    const size_t blk = ((size_t)isv * c.n_pages + page) * c.hkv + head;
    if (tid == 0) c.scales[blk] = m / 127.f;
    int8_t* out = c.codes + blk * c.block * c.d;
    // a maximum whose reciprocal is not a normal number is scaled up first
    const float up = m < 0x1p-100f ? 0x1p100f : 1.f, mu = m * up, rm = 1.f / mu;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = tid + i * APPEND_THREADS;
      if (e >= nv) continue;
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      uint32_t o[2] = {0, 0};
      if (m > 0.f)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float f = q & 1 ? bf16hi(w[q >> 1]) : bf16lo(w[q >> 1]);
          o[q >> 2] |= (uint32_t)(uint8_t)(int8_t)nearest_code(f * up, mu, rm) << (8 * (q & 3));
        }
      *reinterpret_cast<uint2*>(out + (size_t)e * 8) = make_uint2(o[0], o[1]);
    }
  }
  // The new tokens of the last two blocks go to the tail.  Only the first
  // touched block's CTA reads the tail, in that block's half of the ring, so a
  // block in the other half, and the first itself, is written from here; one
  // in the same half waits for the first block's CTA, which copies it.
  if (b >= last - 1 && (b == first || ((b - first) & 1))) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = tid + i * APPEND_THREADS, r = e / vd, x = e % vd, pos = b * c.block + r;
      if (e < nv && pos >= old && pos < len) *reinterpret_cast<uint4*>(tail + (size_t)(pos % ring) * c.d + 8 * x) = u[i];
    }
  }
  const int other = (last - first) & 1 ? last - 1 : last;
  if (b == first && other > first) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = tid + i * APPEND_THREADS, pos = other * c.block + e / vd;
      u[i] = make_uint4(0, 0, 0, 0);
      if (e < nv && pos < len)
        u[i] = *reinterpret_cast<const uint4*>(src + (size_t)(row0 + pos - old) * stride + (size_t)head * c.d + 8 * (e % vd));
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = tid + i * APPEND_THREADS, pos = other * c.block + e / vd;
      bool again = false;
      if (e < nv && pos < len)
        *reinterpret_cast<uint4*>(tail + (size_t)(pos % ring) * c.d + 8 * (e % vd)) = finite_vec(u[i], again);
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                             const int32_t* starts, int t, const moe_kv_cache& c, DeviceStatus* st,
                             cudaStream_t s) {
  const dim3 grid(t / c.block + 2 * c.n_seq, c.hkv, 2);
  const int vpt = (c.block * c.d / 8 + APPEND_THREADS - 1) / APPEND_THREADS;
  cudaError_t e;
  auto* kern = vpt <= 1 ? kv_append_kernel<1> : vpt <= 2 ? kv_append_kernel<2> : vpt <= 4 ? kv_append_kernel<4>
                                                                                      : kv_append_kernel<8>;
  MOE_LAUNCH("kv_append", s,
             { e = launch_k(kern, grid, dim3(APPEND_THREADS), 0, s, k, k_stride, v, v_stride, starts, t, c, st); });
  return e;
}

}  // namespace moe
