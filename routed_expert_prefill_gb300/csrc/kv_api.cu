// C ABI of the paged 8-bit key/value cache: argument checks and dispatch.
#include <math.h>

#include "api_checks.cuh"
#include "kv_common.cuh"

namespace moe {

cudaError_t launch_kv_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                             const int32_t* starts, int t, const moe_kv_cache& c, int32_t* held, DeviceStatus* st,
                             cudaStream_t s);
cudaError_t launch_kv_attention(const uint16_t* q, int64_t q_stride, const int32_t* starts, int t, int hq,
                                float scale, const moe_kv_cache& c, uint16_t* out, unsigned char* ws,
                                cudaStream_t s);

namespace {

int check_cache(const moe_kv_cache* c, const int32_t* starts, int32_t t, const void* ws, size_t ws_bytes) {
  if (!c) return set_error(MOE_EINVAL, "cache is NULL");
  if (t < 1 || t > 65536) return set_error(MOE_ESHAPE, "t=%d outside [1, 65536]", t);
  if (c->d != 64 && c->d != 128) return set_error(MOE_ESHAPE, "d=%d must be 64 or 128", c->d);
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128)
    return set_error(MOE_ESHAPE, "block=%d must be 16, 32, 64 or 128", c->block);
  if (c->hkv < 1 || c->hkv > 1024) return set_error(MOE_ESHAPE, "hkv=%d outside [1, 1024]", c->hkv);
  if (c->n_seq < 1 || c->n_seq > 65536) return set_error(MOE_ESHAPE, "n_seq=%d outside [1, 65536]", c->n_seq);
  if (c->n_pages < 1) return set_error(MOE_ESHAPE, "n_pages=%d must be positive", c->n_pages);
  if (c->max_blocks < 1 || (int64_t)c->max_blocks * c->block > (1 << 30))
    return set_error(MOE_ESHAPE, "max_blocks=%d: at most 2^30 tokens a sequence", c->max_blocks);
  TRY(check_ptr(c->codes, "cache->codes", 16));
  TRY(check_ptr(c->scales, "cache->scales", 4));
  TRY(check_ptr(c->tail, "cache->tail", 16));
  TRY(check_ptr(c->table, "cache->table", 4));
  TRY(check_ptr(c->lens, "cache->lens", 4));
  TRY(check_ptr(starts, "starts", 4));
  if (!ws) return set_error(MOE_EWORKSPACE, "workspace is NULL");
  if ((uintptr_t)ws % 256) return set_error(MOE_EWORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < kv_ws_bytes(c->d))
    return set_error(MOE_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, kv_ws_bytes(c->d));
  return MOE_OK;
}

int check_rows(const void* p, int64_t stride, const char* name) {
  TRY(check_ptr(p, name, 16));
  if (stride < 0 || stride % 8)
    return set_error(MOE_ESHAPE, "%s: the row stride must be a multiple of 8 elements, not negative", name);
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_kv_workspace_bytes(int32_t d) { return d == 64 || d == 128 ? kv_ws_bytes(d) : 0; }

int moe_kv_append_held(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const int32_t* starts,
                       int32_t t, const moe_kv_cache* cache, int32_t* held, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_cache(cache, starts, t, ws, ws_bytes));
  TRY(check_rows(k, k_stride, "k"));
  TRY(check_rows(v, v_stride, "v"));
  TRY(check_ptr(held, "held", 4, true));
  return cuda_status(launch_kv_append(k, k_stride, v, v_stride, starts, t, *cache, held, (DeviceStatus*)ws,
                                      (cudaStream_t)stream),
                     "moe_kv_append launch");
}

int moe_kv_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const int32_t* starts,
                  int32_t t, const moe_kv_cache* cache, void* ws, size_t ws_bytes, void* stream) {
  return moe_kv_append_held(k, k_stride, v, v_stride, starts, t, cache, nullptr, ws, ws_bytes, stream);
}

int moe_kv_attention(const uint16_t* q, int64_t q_stride, const int32_t* starts, int32_t t, int32_t hq, float scale,
                     const moe_kv_cache* cache, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_cache(cache, starts, t, ws, ws_bytes));
  TRY(check_rows(q, q_stride, "q"));
  TRY(check_ptr(out, "out", 16));
  if (hq < cache->hkv || hq % cache->hkv || hq > 32768)
    return set_error(MOE_ESHAPE, "hq=%d must be a multiple of hkv=%d, at most 32768", hq, cache->hkv);
  if (!isfinite(scale)) return set_error(MOE_EINVAL, "scale is not finite");
  return cuda_status(launch_kv_attention(q, q_stride, starts, t, hq, scale, *cache, out, (unsigned char*)ws,
                                         (cudaStream_t)stream),
                     "moe_kv_attention launch");
}

}  // extern "C"
