// Linear attention with a decay for each head (moe_linear_attention): the
// recurrent kernel, argument checks and the choice of kernel.
#include <math.h>

#include <type_traits>

#include "api_checks.cuh"
#include "linear_common.cuh"

namespace moe {

namespace {

// One sequence and head a CTA, half of two columns of its state S a thread:
// lanes 16 apart share the columns j, j + 1 and hold the rows i below and from
// D / 2 on.  They stay in D registers while the tokens pass, each of which
// decays them, adds k_i v_j and sums q_i S[i][j]; the halves of a sum are
// joined by a shuffle.  With one token a sequence the state's bytes bound it,
// read and written once, D / 2 independent loads of a thread on their way (64
// sequences of 32 heads, 268 MB: 0.87 of the copy rate); with more, three
// operations a value and token do, and the reads of keys and queries from
// shared memory, one of 16 bytes for eight values.
template <int D>
__global__ void __launch_bounds__(D) linear_recurrent_kernel(LinearParams p) {
  __shared__ __align__(16) float kq[2][2][D];
  constexpr int H = D / 2;  // rows of a thread
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, head = blockIdx.x % p.hv, s = blockIdx.x / p.hv;
  const int i0 = (lane >> 4) * H, j = 2 * ((tid >> 5) * 16 + (lane & 15));
  int row, n, slot_in, slot_out;
  if (!linear_sequence(p, s, row, n, slot_in, slot_out)) {
    if (tid == 0) raise_flag(p.st, FLAG_BAD_STATE);
    return;
  }
  if (n == 0 && slot_in == slot_out) return;
  float2 S[H];
  if (slot_in >= 0) {
    const float2* from = reinterpret_cast<const float2*>(p.states + ((size_t)slot_in * p.hv + head) * D * D + i0 * D + j);
#pragma unroll
    for (int i = 0; i < H; ++i) S[i] = __ldcs(from + i * (D / 2));
  } else {
#pragma unroll
    for (int i = 0; i < H; ++i) S[i] = make_float2(0.f, 0.f);
  }
  const int hk = head / (p.hv / p.hk);
  const uint16_t* q = p.q + (size_t)row * p.q_stride + hk * D + tid;
  const uint16_t* k = p.k + (size_t)row * p.k_stride + hk * D + tid;
  const uint32_t* v = reinterpret_cast<const uint32_t*>(p.v + (size_t)row * p.v_stride + head * D + j);
  const float* g = p.log_decay + (size_t)row * p.decay_stride + head;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + ((size_t)row * p.hv + head) * D + j);
  uint16_t nq = 0, nk = 0;
  uint32_t nv = 0;
  float ng = 0.f;
  if (n) nq = *q, nk = *k, nv = *v, ng = *g;
  for (int r = 0; r < n; ++r) {
    float(*at)[D] = kq[r & 1];
    at[0][tid] = bf16f(nk);
    at[1][tid] = bf16f(nq);
    const float va = bf16lo(nv), vb = bf16hi(nv), gr = decay_of(ng);
    __syncthreads();
    if (r + 1 < n) {
      q += p.q_stride, k += p.k_stride, v += p.v_stride / 2, g += p.decay_stride;
      nq = *q, nk = *k, nv = *v, ng = *g;
    }
    // S exp(g) is S + S (exp(g) - 1) for a slow decay: exp(g) rounded to fp32
    // would be off by the same 2^-25 for every token, over 1 / (1 - exp(g)) of them
    const bool slow = gr > -0.5f;
    const float f = slow ? expm1f(gr) : expf(gr);
    float x = 0.f, y = 0.f;
    const auto take = [&](auto is_slow) {
      float oa[2] = {}, ob[2] = {};
#pragma unroll
      for (int i = 0; i < H; i += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&at[0][i0 + i]), q4 = *reinterpret_cast<const float4*>(&at[1][i0 + i]);
        const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float2& a = S[i + h];
          a.x = fmaf(a.x, f, decltype(is_slow)::value ? fmaf(kk[h], va, a.x) : kk[h] * va);
          a.y = fmaf(a.y, f, decltype(is_slow)::value ? fmaf(kk[h], vb, a.y) : kk[h] * vb);
          oa[h & 1] = fmaf(qq[h], a.x, oa[h & 1]);
          ob[h & 1] = fmaf(qq[h], a.y, ob[h & 1]);
        }
      }
      x = oa[0] + oa[1];
      y = ob[0] + ob[1];
    };
    if (slow)  // the same for the whole CTA
      take(std::true_type{});
    else
      take(std::false_type{});
    x += __shfl_xor_sync(~0u, x, 16);
    y += __shfl_xor_sync(~0u, y, 16);
    if (lane < 16) *out = pack_bf16x2(p.scale * x, p.scale * y);
    out += (size_t)p.hv * D / 2;
  }
  if (slot_out >= 0) {
    float2* to = reinterpret_cast<float2*>(p.states + ((size_t)slot_out * p.hv + head) * D * D + i0 * D + j);
#pragma unroll
    for (int i = 0; i < H; ++i) __stcs(to + i * (D / 2), S[i]);
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

// Rows of a sequence on average, above which the chunk kernel takes the call (a
// chunk of 128 takes as long however few of them are rows).  With 32 heads of
// 128, recurrent against chunk kernel, caches cold: 64 sequences of 16 rows 118
// and 138 us, of 24 155 and 140; 8 sequences of 16 26 and 31, of 24 33 and 32.
// Heads of 64: 64 sequences of 40 71 and 81, of 56 93 and 80; 8 sequences of 16
// 19 and 22, of 40 33 and 23.
// What the host knows of a call is t and n_seq, not the lengths: the recurrent
// kernel's time is that of the longest sequence, so that a prompt among many
// sequences of a row is slow in it (256 of one row and one of 4096: 3430 us;
// the two calls apart 167 and 78).
constexpr int chunk_rows(int d) { return d == 128 ? 24 : 40; }

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
  const cudaError_t e = apart && t > (int64_t)chunk_rows(d) * n_seq
                            ? launch_linear_chunk(p, d, (unsigned char*)ws + sizeof(DeviceStatus), s)
                            : launch_linear_recurrent(p, d, s);
  return cuda_status(e, "moe_linear_attention launch");
}

}  // extern "C"
