// Append to the paged 8-bit key/value cache (moe_kv_append).
#include <math.h>

#include "kv_common.cuh"

namespace moe {

namespace {

constexpr int APPEND_THREADS = 256;

// The largest magnitude, in the bits of a bf16, whose 127-fold is a finite
// fp32 number; what is above is taken as zero.
constexpr uint32_t MOST_BITS = 0x7C00 + 0x0001;  // 1.0078125 * 2^121: 127 times it is 2^127.99

__device__ __forceinline__ uint32_t finite_pair(uint32_t u, bool& bad) {
  if ((u & 0x7FFFu) > MOST_BITS) u &= 0xFFFF0000u, bad = true;
  if ((u >> 16 & 0x7FFFu) > MOST_BITS) u &= 0x0000FFFFu, bad = true;
  return u;
}
__device__ __forceinline__ uint4 finite_vec(uint4 u, bool& bad) {
  return make_uint4(finite_pair(u.x, bad), finite_pair(u.y, bad), finite_pair(u.z, bad), finite_pair(u.w, bad));
}
// The larger of m and the magnitudes of eight values, as bits in both halves.
__device__ __forceinline__ uint32_t most_of(uint32_t m, uint4 u) {
  m = __vmaxu2(m, __vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu));
  return __vmaxu2(m, __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
}

// v * 127 / m to the nearest whole number, ties to even, exactly: with an
// approximate quotient rounded to q, the remainder x - q m is exact in one
// fma (q and the bf16 m have 7 and 8 bits), and it says whether q is the
// nearest.  rm = 1 / m.
__device__ __forceinline__ int nearest_code(float v, float m, float rm) {
  const float x = v * 127.f;
  const float q = rintf(x * rm);
  const float r = fmaf(-q, m, x), over = fabsf(r) + fabsf(r) - m;
  const int c = (int)q;
  return over > 0.f || (over == 0.f && (c & 1)) ? c + (r > 0.f ? 1 : -1) : c;
}

// Codes of eight values.  k = 127 / m rounded, so v k is off by 2^-24 of at
// most 127: adding 1.5 * 2^23 rounds it to the nearest whole number, which then
// stands in the sum's low byte, and only where the remainder comes within
// 2^-13 of a half does nearest_code decide.
__device__ __forceinline__ uint2 codes_of(uint4 u, float up, float m, float rm, float k) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t t[8];
  float far = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float f = (q & 1 ? bf16hi(w[q >> 1]) : bf16lo(w[q >> 1])) * up;
    const float s = fmaf(f, k, 12582912.f);
    far = fmaxf(far, fabsf(fmaf(f, k, 12582912.f - s)));
    t[q] = __float_as_uint(s);
  }
  if (far > 0.5f - 0x1p-13f) {
#pragma unroll 1
    for (int q = 0; q < 8; ++q) {
      const uint32_t x = q < 4 ? (q < 2 ? w[0] : w[1]) : (q < 6 ? w[2] : w[3]);
      const int c = nearest_code((q & 1 ? bf16hi(x) : bf16lo(x)) * up, m, rm);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e == q) t[e] = (uint32_t)c;
    }
  }
  uint32_t o[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    o[h] = __byte_perm(__byte_perm(t[4 * h], t[4 * h + 1], 0x0040), __byte_perm(t[4 * h + 2], t[4 * h + 3], 0x0040), 0x5410);
  return make_uint2(o[0], o[1]);
}

// One CTA per (touched block, head, keys or values): the block's values stay
// in registers (VPT 16-byte vectors a thread) between the maximum and the
// codes, so every token is read once and every code written once.  Three
// prompts of 2311 tokens, 8 heads: 23 us for 38 MB; what bounds it is the
// quantiser's instructions (some 12 a value, issued in 0.61 of the cycles) and
// the barriers around the maximum, not the bytes.  Block slots are numbered without a scan: sequence s owns
// the slots from starts[s] / block + 2 s on, which is enough for n new
// tokens, as they touch at most (n - 1) / block + 2 blocks.
template <int VPT>
__global__ void __launch_bounds__(APPEND_THREADS)
    kv_append_kernel(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const int32_t* starts,
                     int t, moe_kv_cache c, int32_t* held, DeviceStatus* st) {
  __shared__ uint32_t part[APPEND_THREADS / 32];
  __shared__ int owner;
  pdl_wait();
  pdl_trigger();
  const int slot = blockIdx.x, head = blockIdx.y, isv = blockIdx.z, tid = threadIdx.x;
  // the sequence that owns the slot: every thread looks at some, one answers
  if (tid == 0) owner = -1;
  __syncthreads();
  for (int i = tid; i < c.n_seq; i += APPEND_THREADS) {
    const int from = starts[i], to = starts[i + 1];
    if (from / c.block + 2 * i <= slot && slot < to / c.block + 2 * (i + 1)) owner = i;
    if (to < from && slot == 0) raise_flag(st, FLAG_BAD_CACHE);  // may own no slot that would say so
  }
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
  // Whether the tail holds what this call reads of it, and what it holds
  // afterwards: by one thread a sequence.
  if (held && b == first && head == 0 && isv == 0 && tid == 0) {
    int32_t* filled = held + 2 * (size_t)s;
    if (old > first * c.block) {
      const int end = filled[first & 1];
      if (end && (end < old || (end - 1) / c.block != first)) raise_flag(st, FLAG_BAD_TAIL);
    }
    for (int e = max(first, last - 1); e <= last; ++e) filled[e & 1] = min(len, (e + 1) * c.block);
  }
  const int page = c.table[(size_t)s * c.max_blocks + b];
  const uint16_t* src = isv ? v : k;
  const int64_t stride = isv ? v_stride : k_stride;
  const int ring = 2 * c.block;
  uint16_t* tail = c.tail + (((size_t)s * 2 + isv) * c.hkv + head) * ring * c.d;
  const int vd = c.d >> 3, nv = c.block * vd;  // vectors of a token and of the block
  uint4 u[VPT];
  uint32_t m2 = 0;  // maxima of the low and of the high halves
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = tid + i * APPEND_THREADS, r = e / vd, x = e % vd;
    const int pos = b * c.block + r;
    u[i] = make_uint4(0, 0, 0, 0);
    if (e < nv && pos < len)
      u[i] = *reinterpret_cast<const uint4*>(
          pos < old ? tail + (size_t)(pos % ring) * c.d + 8 * x
                    : src + (size_t)(row0 + pos - old) * stride + (size_t)head * c.d + 8 * x);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) m2 = most_of(m2, u[i]);
  auto block_most = [&](uint32_t v) {  // also: what this block reads of the tail is in registers
    v = __reduce_max_sync(~0u, max(v & 0xFFFFu, v >> 16));
    if ((tid & 31) == 0) part[tid >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < APPEND_THREADS / 32; ++i) v = max(v, part[i]);
    return v;
  };
  uint32_t bits = block_most(m2);
  if (bits > MOST_BITS) {  // the whole block: something in it is not finite
    bool bad = false;
    m2 = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      bool lost = false;
      u[i] = finite_vec(u[i], lost);
      const int e = tid + i * APPEND_THREADS;
      if (lost && b * c.block + e / vd >= old) bad = true;  // older ones have been reported
      m2 = most_of(m2, u[i]);
    }
    if (bad) raise_flag(st, FLAG_NOT_FINITE);
    __syncthreads();
    bits = block_most(m2);
  }
  const float m = __uint_as_float(bits << 16);
  if (page < 0 || page >= c.n_pages) {
    if (tid == 0) raise_flag(st, FLAG_BAD_CACHE);
  } else {
    const size_t blk = ((size_t)isv * c.n_pages + page) * c.hkv + head;
    if (tid == 0) c.scales[blk] = m / 127.f;
    int8_t* out = c.codes + blk * c.block * c.d;
    // a maximum whose reciprocal is not a normal number is scaled up first
    const float up = m < 0x1p-100f ? 0x1p100f : 1.f, mu = m * up, rm = 1.f / mu, k127 = 127.f / mu;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = tid + i * APPEND_THREADS;
      if (e >= nv) continue;
      *reinterpret_cast<uint2*>(out + (size_t)e * 8) = m > 0.f ? codes_of(u[i], up, mu, rm, k127) : make_uint2(0, 0);
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
                             const int32_t* starts, int t, const moe_kv_cache& c, int32_t* held, DeviceStatus* st,
                             cudaStream_t s) {
  const dim3 grid(t / c.block + 2 * c.n_seq, c.hkv, 2);
  const int vpt = (c.block * c.d / 8 + APPEND_THREADS - 1) / APPEND_THREADS;
  cudaError_t e;
  auto* kern = vpt <= 1 ? kv_append_kernel<1> : vpt <= 2 ? kv_append_kernel<2> : vpt <= 4 ? kv_append_kernel<4>
                                                                                      : kv_append_kernel<8>;
  MOE_LAUNCH("kv_append", s, {
    e = launch_k(kern, grid, dim3(APPEND_THREADS), 0, s, k, k_stride, v, v_stride, starts, t, c, held, st);
  });
  return e;
}

}  // namespace moe
