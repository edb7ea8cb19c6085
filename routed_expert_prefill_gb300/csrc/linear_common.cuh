// What the kernels of linear attention share (internal).
#pragma once
#include "common.cuh"

namespace moe {

struct LinearParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;
  const float* log_decay;
  int64_t decay_stride;  // 0: one value a head for all rows
  const int32_t* starts;
  int t, n_seq, hk, hv;
  float scale;
  float* states;
  int n_slots;
  const int32_t* slots;      // null: sequence s has slot s
  const int32_t* slots_out;  // null: the same slots
  uint16_t* out;
  DeviceStatus* st;
};

// One sequence's rows and slots, checked; slot_in or slot_out -1: none.
// False (and a flag) where they are out of range: the sequence is left out.
__device__ __forceinline__ bool linear_sequence(const LinearParams& p, int s, int& row, int& n, int& slot_in, int& slot_out) {
  row = p.starts[s];
  const int end = p.starts[s + 1];
  slot_in = p.slots ? p.slots[s] : s;
  slot_out = p.slots_out ? p.slots_out[s] : slot_in;
  n = end - row;
  return row >= 0 && end >= row && end <= p.t && slot_in >= -1 && slot_in < p.n_slots && slot_out >= -1 &&
         slot_out < p.n_slots;
}

// A log decay as it counts: above zero it is zero.
__device__ __forceinline__ float decay_of(float g) { return g > 0.f ? 0.f : g; }

// Two fp32 values at a time.
__device__ __forceinline__ unsigned long long bits2(float2 v) { return *reinterpret_cast<unsigned long long*>(&v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

}  // namespace moe
