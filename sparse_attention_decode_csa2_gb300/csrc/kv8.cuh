// The 8-bit paged KV cache: geometry shared by its kernels (append, read
// back, attention) and the launchers' declarations.
#pragma once

#include "csa2_internal.cuh"

namespace csa2 {

// The cache and the step's batch as the kernels see them (validated by the C
// ABI: page is 1 << page_shift in 16..128, max_pages << page_shift < 2^31).
struct Kv8Args {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t n_pages;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;  // null: T / S rows for every sequence
  int32_t* status;
  int H_kv, D, page_shift, S, T, max_pages;
};

// A sequence's rows of the step.  Row i (of n) is token len - n + i; tokens
// below zero do not exist (their rows belong to no token).  A sequence whose
// entries make no sense has no rows (`bad`).
struct Kv8Seq {
  int row0, n, len;
  bool bad;
};

// From its entries cu[s], cu[s + 1] (with cu) and kv_len[s].
__device__ __forceinline__ Kv8Seq kv8_seq_of(const Kv8Args& a, int r0, int r1, int len) {
  Kv8Seq q;
  q.bad = r0 < 0 || r1 < r0 || r1 > a.T;
  q.row0 = q.bad ? 0 : r0;
  q.n = q.bad ? 0 : r1 - r0;
  // a length past the block table: the tokens the table has no entry for are skipped
  q.bad = q.bad || len < 0 || len > (int)((int64_t)a.max_pages << a.page_shift);
  q.len = len < 0 ? 0 : len;
  return q;
}
__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8Args& a, int s) {
  const int n = a.T / a.S;
  return a.cu ? kv8_seq_of(a, a.cu[s], a.cu[s + 1], a.kv_len[s])
              : kv8_seq_of(a, s * n, s * n + n, a.kv_len[s]);
}

// Page id of column `col` (< max_pages) of sequence s, or -1 (and the
// bad-index bit) for an entry outside the cache.
__device__ __forceinline__ int64_t kv8_page(const Kv8Args& a, int s, int col) {
  const int32_t p = a.table[(int64_t)s * a.max_pages + col];
  if (p >= 0 && p < a.n_pages) return p;
  set_status(a.status, kStatusBadIndex);
  return -1;
}

// 2^e for whole e in [-126, 127], and 1 / 2^e's exponent arithmetic from bits.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {
  return half2_bits_to_float2(e4m3x2_to_f16x2(v));
}

// Two floats -> two E4M3 bytes (low byte = lo), nearest even, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

cudaError_t launch_kv8_append(const Kv8Args& a, const void* k, const void* v, int type,
                              int64_t k_stride, int64_t v_stride, cudaStream_t stream);
cudaError_t launch_kv8_read(const Kv8Args& a, void* k, void* v, int type, cudaStream_t stream);

struct Kv8AttnArgs {
  Kv8Args c;
  const void* q;       // [T][H][D], token stride q_stride elements
  int64_t q_stride;
  void* out;           // [T][H][D], q's type
  float* lse;          // [T][H] or null
  int H, G, causal, window;
  int g_inv;           // ceil(2^16 / G)
  int tpu;             // tokens of a unit's rows (the kernel's rows a unit / G)
  int uncut;           // every unit is one worker's: no parts, no merge kernel
  float scale_log2;    // softmax scale * log2(e)
  uint8_t* scratch;    // kv8_attn_scratch_bytes(...)
};

// Tokens that a row can see at most, from what the host knows.
inline int64_t kv8_most_tokens(const Kv8AttnArgs& a) {
  const int64_t table = (int64_t)a.c.max_pages << a.c.page_shift;
  return a.window > 0 && a.window < table ? a.window : table;
}

size_t kv8_attn_scratch_bytes(int S, int T, int H, int H_kv, int D);
// The kernels for many query rows per sequence (chosen by launch_kv8_attn).
size_t kv8_attn_tc_scratch_bytes(int D);
cudaError_t launch_kv8_attn_tc(const Kv8AttnArgs& a, int type, cudaStream_t stream);
cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, int type, cudaStream_t stream);

}  // namespace csa2
