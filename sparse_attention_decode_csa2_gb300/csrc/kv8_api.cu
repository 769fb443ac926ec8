// C ABI of the 8-bit paged KV cache: argument checks and launches.
#include <math.h>

#include "kv8.cuh"

namespace csa2 {
namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

// The 8-bit cache and the step's batch; fills the kernels' arguments.
csa2_status check_kv8(const csa2_kv8_cache* c, const csa2_kv8_batch* b, void* ws, Kv8Args* a) {
  if (!c || !b) return CSA2_ERR_INVALID_ARG;
  if (c->n_pages < 0 || c->H_kv < 1 || b->S < 0 || b->T < 0 || b->max_pages < 0)
    return CSA2_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return CSA2_ERR_UNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
    return CSA2_ERR_UNSUPPORTED;
  if (c->n_pages > INT32_MAX || (int64_t)b->max_pages * c->page > (int64_t)1 << 30)
    return CSA2_ERR_UNSUPPORTED;
  // a tensor of T rows and the slots of S sequences are indexed with 32 bits in places
  if (b->T > 1 << 28 || b->S > 1 << 24 || c->H_kv > 1 << 14) return CSA2_ERR_UNSUPPORTED;
  if (b->S == 0 && b->T > 0) return CSA2_ERR_INVALID_ARG;
  if (!b->cu_rows && b->S > 0 && b->T % b->S != 0) return CSA2_ERR_INVALID_ARG;
  if (b->S > 0 && b->T > 0) {
    if (!b->kv_len || (b->max_pages > 0 && !b->block_table)) return CSA2_ERR_INVALID_ARG;
    if (c->n_pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale))
      return CSA2_ERR_INVALID_ARG;
  }
  if (!aligned16(c->k) || !aligned16(c->v)) return CSA2_ERR_INVALID_ARG;
  for (const void* p : {(const void*)c->k_scale, (const void*)c->v_scale,
                        (const void*)b->block_table, (const void*)b->kv_len,
                        (const void*)b->cu_rows})
    if (!aligned(p, 4)) return CSA2_ERR_INVALID_ARG;
  a->k = c->k;
  a->v = c->v;
  a->k_scale = c->k_scale;
  a->v_scale = c->v_scale;
  a->n_pages = c->n_pages;
  a->table = b->block_table;
  a->kv_len = b->kv_len;
  a->cu = b->cu_rows;
  a->status = static_cast<int32_t*>(ws);
  a->H_kv = c->H_kv;
  a->D = c->D;
  a->page_shift = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  a->S = b->S;
  a->T = b->T;
  a->max_pages = b->max_pages;
  return CSA2_OK;
}

// Rows [T][heads][D] whose tokens are `stride` elements apart: 16-byte vectors.
csa2_status check_rows(const void* p, int type, int64_t stride, int heads, int D) {
  if (type != CSA2_BF16 && type != CSA2_FP16 && type != CSA2_FP32) return CSA2_ERR_INVALID_ARG;
  const int64_t size = type == CSA2_FP32 ? 4 : 2;
  if (stride < (int64_t)heads * D || stride > (int64_t)1 << 40) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(p) || stride * size % 16 != 0) return CSA2_ERR_INVALID_ARG;
  return CSA2_OK;
}

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" {

size_t csa2_kv8_workspace_size(const csa2_kv8_cache* c, const csa2_kv8_batch* b, int H) {
  if (!c || !b || c->H_kv < 1 || H < 1 || b->S < 1 || b->T < 1) return kStatusBytes;
  return kStatusBytes + kv8_attn_scratch_bytes(b->S, b->T, H, c->H_kv, c->D);
}

csa2_status csa2_kv8_append(const csa2_kv8_cache* cache, const csa2_kv8_batch* batch,
                            const void* k, const void* v, int type, int64_t k_stride,
                            int64_t v_stride, void* ws, size_t ws_bytes, cudaStream_t stream) {
  Kv8Args a;
  csa2_status s = check_kv8(cache, batch, ws, &a);
  if (s != CSA2_OK) return s;
  if ((s = check_rows(k, type, k_stride, a.H_kv, a.D)) != CSA2_OK) return s;
  if ((s = check_rows(v, type, v_stride, a.H_kv, a.D)) != CSA2_OK) return s;
  if (a.T > 0 && (!k || !v)) return CSA2_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 4) || ws_bytes < kStatusBytes) return CSA2_ERR_WORKSPACE;
  if (a.S == 0 || a.T == 0) return CSA2_OK;
  return check_launch(launch_kv8_append(a, k, v, type, k_stride, v_stride, stream));
}

csa2_status csa2_kv8_read(const csa2_kv8_cache* cache, const csa2_kv8_batch* batch, void* k,
                          void* v, int type, void* ws, size_t ws_bytes, cudaStream_t stream) {
  Kv8Args a;
  csa2_status s = check_kv8(cache, batch, ws, &a);
  if (s != CSA2_OK) return s;
  const int64_t stride = (int64_t)a.H_kv * a.D;
  if ((s = check_rows(k, type, stride, a.H_kv, a.D)) != CSA2_OK) return s;
  if ((s = check_rows(v, type, stride, a.H_kv, a.D)) != CSA2_OK) return s;
  if (a.T > 0 && (!k || !v)) return CSA2_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 4) || ws_bytes < kStatusBytes) return CSA2_ERR_WORKSPACE;
  if (a.S == 0 || a.T == 0) return CSA2_OK;
  return check_launch(launch_kv8_read(a, k, v, type, stream));
}

csa2_status csa2_kv8_attn(const void* q, int type, int64_t q_stride, int H,
                          const csa2_kv8_cache* cache, const csa2_kv8_batch* batch, int causal,
                          int window, float softmax_scale, void* out, float* lse, void* ws,
                          size_t ws_bytes, cudaStream_t stream) {
  Kv8AttnArgs a;
  csa2_status s = check_kv8(cache, batch, ws, &a.c);
  if (s != CSA2_OK) return s;
  if (H < 1 || H % a.c.H_kv != 0) return CSA2_ERR_INVALID_ARG;
  a.H = H;
  a.G = H / a.c.H_kv;
  if (a.G > 256) return CSA2_ERR_UNSUPPORTED;
  if (type != CSA2_BF16 && type != CSA2_FP16) return CSA2_ERR_INVALID_ARG;
  if ((s = check_rows(q, type, q_stride, H, a.c.D)) != CSA2_OK) return s;
  if (window < 0 || (window > 0 && !causal)) return CSA2_ERR_INVALID_ARG;
  a.scale_log2 = softmax_scale * 1.44269504088896340736f;
  if (!(softmax_scale > 0.0f) || !(a.scale_log2 < INFINITY)) return CSA2_ERR_INVALID_ARG;
  if (a.c.T > 0 && (!q || !out)) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned(lse, 4)) return CSA2_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws) || ws_bytes < csa2_kv8_workspace_size(cache, batch, H))
    return CSA2_ERR_WORKSPACE;
  if (a.c.S == 0 || a.c.T == 0) return CSA2_OK;
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.lse = lse;
  a.causal = causal ? 1 : 0;
  a.window = window < 3 << 29 ? window : 3 << 29;  // (past any length; token - window fits an int)
  a.uncut = 0;
  a.tpu = 0;
  a.g_inv = (65536 + a.G - 1) / a.G;
  a.scratch = reinterpret_cast<uint8_t*>(ws) + kStatusBytes;
  return check_launch(launch_kv8_attn(a, type, stream));
}

}  // extern "C"
