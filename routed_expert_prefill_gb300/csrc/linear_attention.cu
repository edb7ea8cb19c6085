// Linear attention with a decay for each head (moe_linear_attention): the
// recurrent kernel, argument checks and the choice of kernel.
#include <math.h>

#include "api_checks.cuh"
#include "linear_common.cuh"

namespace moe {

namespace {

// One sequence and head a CTA, one column j of its state S a thread: S[.][j]
// stays in D registers while the rows pass, each of which decays it, adds
// k_i v_j and sums q_i S[i][j].  Columns do not mix, so nothing is joined.
// With one row a sequence the state's bytes bound it, read and written once
// (D independent loads of a thread hide the latency); with more, 3 D
// operations a row and column do.
template <int D>
__global__ void __launch_bounds__(D) linear_recurrent_kernel(LinearParams p) {
  __shared__ __align__(16) float kq[2][2][D];
  pdl_wait();
  pdl_trigger();
  const int j = threadIdx.x, head = blockIdx.x % p.hv, s = blockIdx.x / p.hv;
  int row, n, slot_in, slot_out;
  if (!linear_sequence(p, s, row, n, slot_in, slot_out)) {
    if (j == 0) raise_flag(p.st, FLAG_BAD_STATE);
    return;
  }
  if (n == 0 && slot_in == slot_out) return;
  float S[D];
  if (slot_in >= 0) {
    const float* from = p.states + ((size_t)slot_in * p.hv + head) * D * D + j;
#pragma unroll
    for (int i = 0; i < D; ++i) S[i] = __ldcs(from + i * D);
  } else {
#pragma unroll
    for (int i = 0; i < D; ++i) S[i] = 0.f;
  }
  const int hk = head / (p.hv / p.hk);
  const uint16_t* q = p.q + (size_t)row * p.q_stride + hk * D + j;
  const uint16_t* k = p.k + (size_t)row * p.k_stride + hk * D + j;
  const uint16_t* v = p.v + (size_t)row * p.v_stride + head * D + j;
  const float* g = p.log_decay + (size_t)row * p.decay_stride + head;
  uint16_t* out = p.out + ((size_t)row * p.hv + head) * D + j;
  uint16_t nq = 0, nk = 0, nv = 0;
  float ng = 0.f;
  if (n) nq = *q, nk = *k, nv = *v, ng = *g;
  for (int r = 0; r < n; ++r) {
    float(*at)[D] = kq[r & 1];
    at[0][j] = bf16f(nk);
    at[1][j] = bf16f(nq);
    const float vj = bf16f(nv), gr = decay_of(ng);
    __syncthreads();
    if (r + 1 < n) {
      q += p.q_stride, k += p.k_stride, v += p.v_stride, g += p.decay_stride;
      nq = *q, nk = *k, nv = *v, ng = *g;
    }
    float o[4] = {};
    // S exp(g) is S + S (exp(g) - 1) for a slow decay: exp(g) rounded to fp32
    // would be off by the same 2^-25 in every row, over 1 / (1 - exp(g)) rows
    const bool slow = gr > -0.5f;
    const float f = slow ? expm1f(gr) : expf(gr);
#define MOE_LINEAR_ROW(STEP)                                                                                          \
  _Pragma("unroll") for (int i = 0; i < D; i += 4) {                                                                  \
    const float4 kk = *reinterpret_cast<const float4*>(&at[0][i]), qq = *reinterpret_cast<const float4*>(&at[1][i]);  \
    S[i] = STEP(S[i], kk.x), o[0] = fmaf(qq.x, S[i], o[0]);                                                           \
    S[i + 1] = STEP(S[i + 1], kk.y), o[1] = fmaf(qq.y, S[i + 1], o[1]);                                               \
    S[i + 2] = STEP(S[i + 2], kk.z), o[2] = fmaf(qq.z, S[i + 2], o[2]);                                               \
    S[i + 3] = STEP(S[i + 3], kk.w), o[3] = fmaf(qq.w, S[i + 3], o[3]);                                               \
  }
#define MOE_LINEAR_SLOW(s, kk) fmaf(s, f, fmaf(kk, vj, s))
#define MOE_LINEAR_FAST(s, kk) fmaf(s, f, kk * vj)
    if (slow) {
      MOE_LINEAR_ROW(MOE_LINEAR_SLOW)
    } else {
      MOE_LINEAR_ROW(MOE_LINEAR_FAST)
    }
    *out = f2bf(p.scale * ((o[0] + o[1]) + (o[2] + o[3])));
    out += (size_t)p.hv * D;
  }
  if (slot_out >= 0) {
    float* to = p.states + ((size_t)slot_out * p.hv + head) * D * D + j;
#pragma unroll
    for (int i = 0; i < D; ++i) __stcs(to + i * D, S[i]);
  }
}

}  // namespace

cudaError_t launch_linear_recurrent(const LinearParams& p, int d, cudaStream_t s) {
  const dim3 grid((unsigned)p.n_seq * p.hv);
  cudaError_t e = cudaSuccess;
  MOE_LAUNCH("linear_recurrent", s, {
    e = d == 128 ? launch_k(linear_recurrent_kernel<128>, grid, dim3(128), 0, s, p)
                 : launch_k(linear_recurrent_kernel<64>, grid, dim3(64), 0, s, p);
  });
  return e;
}

size_t linear_chunk_ws_bytes(int d);  // linear_chunk.cu
cudaError_t launch_linear_chunk(const LinearParams& p, int d, unsigned char* ws, cudaStream_t s);

namespace {

size_t linear_ws_bytes(int d) { return sizeof(DeviceStatus) + linear_chunk_ws_bytes(d); }

// Rows of a sequence on average, from which on the chunk kernel takes the call.
constexpr int CHUNK_ROWS = 24;

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_linear_workspace_bytes(int32_t d) { return d == 64 || d == 128 ? linear_ws_bytes(d) : 0; }

int moe_linear_attention(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                         int64_t v_stride, const float* log_decay, int64_t decay_stride, const int32_t* starts, int32_t t,
                         int32_t n_seq, int32_t hk, int32_t hv, int32_t d, float scale, float* states, int32_t n_slots,
                         const int32_t* slots, const int32_t* slots_out, uint16_t* out, void* ws, size_t ws_bytes,
                         void* stream) {
  if (t < 1 || t > 65536) return set_error(MOE_ESHAPE, "t=%d outside [1, 65536]", t);
  if (d != 64 && d != 128) return set_error(MOE_ESHAPE, "d=%d must be 64 or 128", d);
  if (n_seq < 1 || n_seq > 65536) return set_error(MOE_ESHAPE, "n_seq=%d outside [1, 65536]", n_seq);
  if (hv < 1 || hv > 1024) return set_error(MOE_ESHAPE, "hv=%d outside [1, 1024]", hv);
  if (hk < 1 || hv % hk) return set_error(MOE_ESHAPE, "hv=%d must be a multiple of hk=%d", hv, hk);
  if (n_slots < 1) return set_error(MOE_ESHAPE, "n_slots=%d must be positive", n_slots);
  if (!slots && n_slots < n_seq) return set_error(MOE_ESHAPE, "n_slots=%d: fewer than the %d sequences", n_slots, n_seq);
  if (q_stride < 0 || q_stride % 8 || k_stride < 0 || k_stride % 8 || v_stride < 0 || v_stride % 8)
    return set_error(MOE_ESHAPE, "row strides must be multiples of 8 elements, not negative");
  if (decay_stride < 0) return set_error(MOE_ESHAPE, "decay_stride must not be negative");
  if (!isfinite(scale)) return set_error(MOE_EINVAL, "scale is not finite");
  TRY(check_ptr(q, "q", 16));
  TRY(check_ptr(k, "k", 16));
  TRY(check_ptr(v, "v", 16));
  TRY(check_ptr(log_decay, "log_decay", 4));
  TRY(check_ptr(starts, "starts", 4));
  TRY(check_ptr(states, "states", 16));
  TRY(check_ptr(slots, "slots", 4, true));
  TRY(check_ptr(slots_out, "slots_out", 4, true));
  TRY(check_ptr(out, "out", 16));
  if (!ws) return set_error(MOE_EWORKSPACE, "workspace is NULL");
  if ((uintptr_t)ws % 256) return set_error(MOE_EWORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < linear_ws_bytes(d))
    return set_error(MOE_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, linear_ws_bytes(d));
  const LinearParams p{q, k, v, q_stride, k_stride, v_stride, log_decay, decay_stride, starts, t, n_seq, hk, hv, scale,
                       states, n_slots, slots, slots_out, out, (DeviceStatus*)ws};
  cudaStream_t s = (cudaStream_t)stream;
  // rows that lie over one another (one row for all) are no tiles
  const bool apart = q_stride >= (int64_t)hk * d && k_stride >= (int64_t)hk * d && v_stride >= (int64_t)hv * d;
  const cudaError_t e = apart && t > (int64_t)CHUNK_ROWS * n_seq
                            ? launch_linear_chunk(p, d, (unsigned char*)ws + sizeof(DeviceStatus), s)
                            : launch_linear_recurrent(p, d, s);
  return cuda_status(e, "moe_linear_attention launch");
}

}  // extern "C"
