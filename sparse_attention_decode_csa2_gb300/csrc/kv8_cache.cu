// The 8-bit paged KV cache's writer and reader.
//
// Cache: E4M3 codes [n_pages][H_kv][page][D] for K and for V, one fp32 scale
// per page and head.  The scale of a block (a page's tokens of one head) is
// the power of two 2^e with the least e such that absmax <= 448 * 2^e.  E4M3
// is a floating-point format, so any scale keeps the same relative precision
// above its subnormals; a power of two makes x / scale and a later change of
// scale exact, and the only rounding left is that to the 3-bit mantissa.
//
// A page fills over several steps.  Its scale only grows: when a step's rows
// need a larger one, the rows that the page holds are decoded, divided and
// rounded again (exact except where a code becomes subnormal).  A step that
// writes a page's first token starts the scale anew, whatever the page held.
//
// One team of threads (a warp for small blocks or a few rows per sequence, else
// 128) owns the rows of one (sequence, page, head) of K or V: it reads them once
// into registers, reduces absmax, settles the scale and stores the codes.  No two
// teams touch the same block, so there are no atomics.  The team first follows a
// chain of dependent loads (sequence, page, rows), so what bounds the writer of
// prompts is how many rows the resident teams hold in flight: 128 threads with
// four 32-byte pieces each keep a page of 64 rows of 128 channels in 64 registers
// a thread, eight teams to an SM.  Measured (GB300): 20011 bf16 rows of 8 heads x
// 128 channels, page 64, in 24.6 us, 5.0 TB/s of rows read and codes written (the
// copy peak is 6.77; 18.2 us); with 256 threads a team 32.8 us.  Maxima by packed
// 16-bit instructions, half as many, took 26.5 us: instructions do not bound it.
// Steps of a few tokens take the call's own time (12 us through the binding; 3 to 4 us
// on the device).
#include <cuda_bf16.h>

#include "kv8.cuh"

namespace csa2 {
namespace {

constexpr int kTeamBig = 128;             // threads of a team (and of its block)
constexpr int kBlockSmall = 256;          // threads of a block of warp teams
constexpr int kEMin = -100, kEMax = 120;  // scale exponents

template <typename T>
struct Vec16;  // 16 consecutive values
template <>
struct Vec16<float> {
  float4 r[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ void get(float* x) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = r[i].x;
      x[4 * i + 1] = r[i].y;
      x[4 * i + 2] = r[i].z;
      x[4 * i + 3] = r[i].w;
    }
  }
};
template <typename T>
struct Vec16Half {
  uint4 r[2];
  __device__ __forceinline__ void load(const T* p) {
    r[0] = __ldg(reinterpret_cast<const uint4*>(p));
    r[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float* x) const;
};
template <>
__device__ __forceinline__ void Vec16Half<__nv_bfloat16>::get(float* x) const {
  const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void Vec16Half<__half>::get(float* x) const {
  const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = half2_bits_to_float2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <>
struct Vec16<__nv_bfloat16> : Vec16Half<__nv_bfloat16> {};
template <>
struct Vec16<__half> : Vec16Half<__half> {};

// Least e with amax <= 448 * 2^e (448 = 1.75 * 2^8), clamped; infinity gives kEMax.
__device__ __forceinline__ int scale_exponent(float amax) {
  if (!(amax > 0.0f)) return kEMin;
  int m_bits = (int)(__float_as_uint(amax) & 0x7FFFFFu);
  const int E = (int)(__float_as_uint(amax) >> 23) - 127;  // -127: subnormal, far below kEMin
  int e = E - 8 + (m_bits > 0x600000 ? 1 : 0);
  return e < kEMin ? kEMin : (e > kEMax ? kEMax : e);
}

// 16 codes of the values x * inv.
__device__ __forceinline__ uint4 encode16(const float* x, float inv) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = f32x2_to_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) |
           (f32x2_to_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void decode16(uint4 c, float* x) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4m3x2_to_float2((uint16_t)(w[i] & 0xFFFFu));
    const float2 b = e4m3x2_to_float2((uint16_t)(w[i] >> 16));
    x[4 * i] = a.x;
    x[4 * i + 1] = a.y;
    x[4 * i + 2] = b.x;
    x[4 * i + 3] = b.y;
  }
}

// Work items: (slot, head, K or V).  Each sequence has enough slots for the
// pages its rows can touch: n rows touch at most (n + page - 2) / page + 1
// pages.  With equal shares that is the count; with cu, sequence s owns slots
// [cu[s] / page + 2 s, cu[s + 1] / page + 2 s + 2), which is at least as many
// and needs no prefix sum, so a slot finds its sequence by bisection.  Offsets
// that decrease or leave [0, T] break the order that the bisection goes by: the
// slots that it then misses are the last block's (lost_slots).
__host__ __device__ inline int64_t pages_of(int64_t n, int page_shift) {
  return ((n + ((int64_t)1 << page_shift) - 2) >> page_shift) + 1;
}
__host__ __device__ inline int64_t slots_of(int S, int T, bool cu, int page_shift) {
  if (cu) return ((int64_t)T >> page_shift) + 2 * (int64_t)S;
  return (int64_t)S * pages_of(T / S, page_shift);
}
// Sequence s's first slot, from its entry of cu.
__device__ __forceinline__ int64_t slot_base(const Kv8Args& a, int s, int cu) {
  return (int64_t)(min(max(cu, 0), a.T) >> a.page_shift) + 2 * (int64_t)s;
}

// The rows of the step that slot j of sequence s stands for: page column `col`,
// tokens [pos, pos + rows), the first of them row `row` of the step.  rows = 0:
// nothing to do.
struct Slot {
  int s, j, col, pos, rows, row;
  Kv8Seq q;
};

// r.s, r.j and r.q are set.
__device__ __forceinline__ void slot_rows(const Kv8Args& a, Slot& r) {
  const int cap = (int)min((int64_t)r.q.len, (int64_t)a.max_pages << a.page_shift);
  const int64_t first = (int64_t)r.q.len - r.q.n;  // token of the sequence's row 0
  const int p0 = first < 0 ? 0 : (int)first;
  const int64_t col = (int64_t)(p0 >> a.page_shift) + r.j;
  r.col = col >= a.max_pages ? a.max_pages : (int)col;
  const int64_t start = col << a.page_shift, end = start + ((int64_t)1 << a.page_shift);
  const int64_t lo = start > p0 ? start : p0, hi = end < cap ? end : cap;
  r.pos = (int)(lo < cap ? lo : cap);
  r.rows = r.q.n > 0 && r.col < a.max_pages && hi > lo ? (int)(hi - lo) : 0;
  r.row = r.q.row0 + (int)(lo - first);
}

// With cu: the last sequence s whose first slot is not past `slot`, 32 candidates a
// round (every lane of a warp has the same slot); the last round has the
// sequence's entries.
__device__ __forceinline__ void search_slot(const Kv8Args& a, int64_t slot, Slot& r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.S, step;
  do {
    step = (hi - lo + 31) / 32;
    const int c = lo + lane * step;
    int cu = 0, next = 0, len = 0;
    bool le = false;
    if (c < hi) {
      cu = a.cu[c];
      if (step == 1) {
        next = a.cu[c + 1];
        len = a.kv_len[c];
      }
      le = lane == 0 || slot_base(a, c, cu) <= slot;
    }
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));  // the highest that is not past the slot
    lo += k * step;
    hi = min(hi, lo + step);
    if (step == 1) {
      cu = __shfl_sync(0xffffffffu, cu, k);
      next = __shfl_sync(0xffffffffu, next, k);
      len = __shfl_sync(0xffffffffu, len, k);
      r.q = kv8_seq_of(a, cu, next, len);
      const int64_t j = slot - slot_base(a, lo, cu);
      r.j = j < 0 || j > INT32_MAX ? INT32_MAX : (int)j;
    }
  } while (step > 1);
  r.s = lo;
}

__device__ __forceinline__ Slot find_slot(const Kv8Args& a, int64_t slot) {
  Slot r;
  if (a.cu) {
    search_slot(a, slot, r);
  } else {
    const int64_t per = pages_of(a.T / a.S, a.page_shift);
    r.s = (int)(slot / per);
    r.j = (int)(slot % per);
    r.q = kv8_seq(a, r.s);
  }
  slot_rows(a, r);
  return r;
}

// The last block: raises the bad-index bit if any sequence's entries make no sense.
// True (to all threads) if it is cu's, so that slots may be lost.
__device__ __forceinline__ bool check_batch(const Kv8Args& a) {
  bool bad = false, order = false;
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
    bad |= kv8_seq(a, s).bad;
    if (a.cu) order |= a.cu[s] < 0 || a.cu[s + 1] < a.cu[s] || a.cu[s + 1] > a.T;
  }
  if (bad) set_status(a.status, kStatusBadIndex);
  return __syncthreads_or(order);
}

// The slots of sound sequences that the search gives to others, one after the other
// (every thread of the block; `take` has the slot).  For a batch that should not be:
// it may take its time.
template <class Take>
__device__ __forceinline__ void lost_slots(const Kv8Args& a, Take&& take) {
  const int64_t slots = slots_of(a.S, a.T, true, a.page_shift);
  for (int s = 0; s < a.S; ++s) {
    Slot r;
    r.s = s;
    r.q = kv8_seq(a, s);
    if (r.q.n == 0) continue;
    const int64_t base = slot_base(a, s, a.cu[s]);
    const int n = (int)pages_of(r.q.n, a.page_shift);
    for (r.j = 0; r.j < n; ++r.j) {
      if (base + r.j < slots) {
        Slot at;
        search_slot(a, base + r.j, at);
        if (at.s == s) continue;  // a team has it
      }
      slot_rows(a, r);
      take(r);
    }
  }
}

template <int kTeam>
constexpr int block_of() {
  return kTeam == 32 ? kBlockSmall : kTeam;
}

template <int kTeam>
__device__ __forceinline__ float team_max(float x, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if (kTeam > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTeam / 32; ++i) x = fmaxf(x, red[i]);
  }
  return x;
}

// Rows of the step into one block: (page of the slot, head, K or V), by one team.
// One pass over the rows: the first kHold chunks of a thread stay in registers (four: a
// page of 64 rows of 128 channels for a team of 128), the rest are read again.
template <typename T, int kTeam, int kHold>
__device__ __forceinline__ void append_block(const Kv8Args& a, const T* __restrict__ k,
                                             const T* __restrict__ v, int64_t k_stride,
                                             int64_t v_stride, const Slot& sl, int h, bool is_v,
                                             float* red) {
  const int t = threadIdx.x % kTeam;
  if (sl.rows == 0) return;
  const int64_t page_id = kv8_page(a, sl.s, sl.col);
  if (page_id < 0) return;
  const int D = a.D, cpr = D / 16;  // 16-value chunks per row
  const int off = sl.pos & ((1 << a.page_shift) - 1);
  const int64_t stride = is_v ? v_stride : k_stride;
  const T* src = (is_v ? v : k) + (int64_t)sl.row * stride + (int64_t)h * D;
  uint8_t* blk = (is_v ? a.v : a.k) + ((page_id * a.H_kv + h) << a.page_shift) * D;
  float* scale = (is_v ? a.v_scale : a.k_scale) + page_id * a.H_kv + h;

  Vec16<T> held[kHold > 0 ? kHold : 1];
  const int chunks = sl.rows * cpr;
  const int shift = D == 128 ? 3 : 2;
  auto at = [&](int c) { return src + (int64_t)(c >> shift) * stride + (c & (cpr - 1)) * 16; };
  float amax = 0.0f;
  auto take = [&](const Vec16<T>& w) {
    float x[16];
    w.get(x);
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (t + i * kTeam < chunks) held[i].load(at(t + i * kTeam));
  const float old = off > 0 ? *scale : 0.0f;  // a page that starts forgets its scale
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (t + i * kTeam < chunks) take(held[i]);
  for (int c = t + kHold * kTeam; c < chunks; c += kTeam) {
    Vec16<T> w;
    w.load(at(c));
    take(w);
  }
  amax = team_max<kTeam>(amax, red);  // every thread has read the old scale by here
  const float need = pow2f(scale_exponent(amax));
  const float sc = fmaxf(old, need), inv = 1.0f / sc;

  uint8_t* dst = blk + (int64_t)off * D;
  auto put = [&](int c, const Vec16<T>& w) {
    float x[16];
    w.get(x);
    *reinterpret_cast<uint4*>(dst + (int64_t)c * 16) = encode16(x, inv);
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (t + i * kTeam < chunks) put(t + i * kTeam, held[i]);
  for (int c = t + kHold * kTeam; c < chunks; c += kTeam) {
    Vec16<T> w;
    w.load(at(c));
    put(c, w);
  }
  if (off > 0 && sc > old) {  // the rows that the page held
    const float r = old * inv;
    for (int c = t; c < off * cpr; c += kTeam) {
      uint4* p = reinterpret_cast<uint4*>(blk) + c;
      float x[16];
      decode16(*p, x);
      *p = encode16(x, r);
    }
  }
  __syncwarp();
  if (t == 0 && sc != old) *scale = sc;
}

template <typename T, int kTeam>
__device__ __noinline__ void append_lost(const Kv8Args& a, const T* k, const T* v, int64_t k_stride,
                                         int64_t v_stride, float* red) {
  lost_slots(a, [&](const Slot& sl) {
    for (int i = threadIdx.x / kTeam; i < 2 * a.H_kv; i += block_of<kTeam>() / kTeam) {
      append_block<T, kTeam, 0>(a, k, v, k_stride, v_stride, sl, i >> 1, i & 1, red);
      if (kTeam > 32) __syncthreads();  // the maxima of the next block
    }
  });
}

template <typename T, int kTeam>
__global__ void __launch_bounds__(block_of<kTeam>(), (kTeam == 32 ? 4 : 8) / (sizeof(T) / 2))
kv8_append_kernel(const __grid_constant__ Kv8Args a, const T* __restrict__ k,
                  const T* __restrict__ v, int64_t k_stride, int64_t v_stride, int64_t items) {
  __shared__ float red[kTeam / 32];
  const int64_t item = (int64_t)blockIdx.x * (block_of<kTeam>() / kTeam) + threadIdx.x / kTeam;
  if (blockIdx.x == gridDim.x - 1) {  // past the items
    if (check_batch(a)) append_lost<T, kTeam>(a, k, v, k_stride, v_stride, red);
    return;
  }
  if (item >= items) return;
  append_block<T, kTeam, 4>(a, k, v, k_stride, v_stride, find_slot(a, (item >> 1) / a.H_kv),
                            (int)((item >> 1) % a.H_kv), item & 1, red);
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const float* x);
template <>
__device__ __forceinline__ void store16<float>(float* p, const float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    __stcs(reinterpret_cast<float4*>(p) + i,
           make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
}
template <>
__device__ __forceinline__ void store16<__half>(__half* p, const float* x) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(reinterpret_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
}
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float* x) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(reinterpret_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
}

// Values of the step's rows: code * scale, rounded once to T.  Teams and
// items as the writer's; rows of tokens below zero, and of pages outside the
// cache, read as zeros.  Bound by its writes, twice its reads: 8 sequences of 16384
// tokens (8 heads x 128, bf16) 140 us, 5.7 TB/s in all, of which a plain fill of
// the 537 MB written takes 136.
template <typename T, int kTeam>
__device__ __forceinline__ void read_block(const Kv8Args& a, T* __restrict__ k, T* __restrict__ v,
                                           const Slot& sl, int h, bool is_v) {
  const int t = threadIdx.x % kTeam;
  const int D = a.D, cpr = D / 16, shift = D == 128 ? 3 : 2;
  const int64_t stride = (int64_t)a.H_kv * D;
  T* out = (is_v ? v : k) + (int64_t)h * D;
  auto dst = [&](int row, int64_t c) {
    return out + (row + (c >> shift)) * stride + (c & (cpr - 1)) * 16;
  };
  if (sl.j == 0) {  // rows without a token, or past the block table
    const float zero[16] = {};
    const int64_t cap = (int64_t)a.max_pages << a.page_shift;
    const int before = min(sl.q.n, max(0, sl.q.n - sl.q.len));
    for (int64_t c = t; c < (int64_t)before * cpr; c += kTeam) store16<T>(dst(sl.q.row0, c), zero);
    const int past = (int)min((int64_t)sl.q.n, max((int64_t)0, (int64_t)sl.q.len - cap));
    for (int64_t c = t; c < (int64_t)past * cpr; c += kTeam)
      store16<T>(dst(sl.q.row0 + sl.q.n - past, c), zero);
  }
  if (sl.rows == 0) return;
  const int64_t page_id = kv8_page(a, sl.s, sl.col);
  const int off = sl.pos & ((1 << a.page_shift) - 1);
  const int64_t b = (page_id < 0 ? 0 : page_id) * a.H_kv + h;
  const uint8_t* src = (is_v ? a.v : a.k) + ((b << a.page_shift) + off) * D;
  const float sc = page_id < 0 ? 0.0f : (is_v ? a.v_scale : a.k_scale)[b];
  for (int c = t; c < sl.rows * cpr; c += kTeam) {
    float x[16];
    decode16(page_id < 0 ? make_uint4(0, 0, 0, 0)
                         : __ldg(reinterpret_cast<const uint4*>(src) + c), x);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= sc;
    store16<T>(dst(sl.row, c), x);
  }
}

template <typename T, int kTeam>
__device__ __noinline__ void read_lost(const Kv8Args& a, T* k, T* v) {
  lost_slots(a, [&](const Slot& sl) {
    for (int i = threadIdx.x / kTeam; i < 2 * a.H_kv; i += block_of<kTeam>() / kTeam)
      read_block<T, kTeam>(a, k, v, sl, i >> 1, i & 1);
  });
}

template <typename T, int kTeam>
__global__ void __launch_bounds__(block_of<kTeam>(), kTeam == 32 ? 5 : 16)
kv8_read_kernel(const __grid_constant__ Kv8Args a, T* __restrict__ k, T* __restrict__ v,
                int64_t items) {
  const int64_t item = (int64_t)blockIdx.x * (block_of<kTeam>() / kTeam) + threadIdx.x / kTeam;
  if (blockIdx.x == gridDim.x - 1) {
    if (check_batch(a)) read_lost<T, kTeam>(a, k, v);
    return;
  }
  if (item >= items) return;
  read_block<T, kTeam>(a, k, v, find_slot(a, (item >> 1) / a.H_kv), (int)((item >> 1) % a.H_kv),
                       item & 1);
}

// A warp per item where a block's rows are few, or few of it are written: up to
// four 16-value pieces a lane, as many as it holds.  Measured: one token of 256
// sequences, a call by itself, 20 us with warps and 26 with teams of 128; the
// prompts above 36.6 us with warps and 24.6 with teams; the reader 145 and 140.
inline bool small_items(const Kv8Args& a) {
  const int64_t rows = ((int64_t)a.T + a.S - 1) / a.S, page = (int64_t)1 << a.page_shift;
  return (rows < page ? rows : page) * (a.D / 16) <= 128;
}
// Blocks of a launch: the items', and one that checks the batch's entries.
inline int64_t blocks_of(int64_t items, bool small) {
  return (small ? (items + kBlockSmall / 32 - 1) / (kBlockSmall / 32) : items) + 1;
}

template <typename T>
cudaError_t append_t(const Kv8Args& a, const void* k, const void* v, int64_t ks, int64_t vs,
                     cudaStream_t stream) {
  const int64_t items = slots_of(a.S, a.T, a.cu != nullptr, a.page_shift) * a.H_kv * 2;
  const T* kp = static_cast<const T*>(k);
  const T* vp = static_cast<const T*>(v);
  const bool small = small_items(a);
  const int64_t blocks = blocks_of(items, small);
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (small)
    kv8_append_kernel<T, 32><<<(unsigned)blocks, kBlockSmall, 0, stream>>>(a, kp, vp, ks, vs, items);
  else
    kv8_append_kernel<T, kTeamBig><<<(unsigned)blocks, kTeamBig, 0, stream>>>(a, kp, vp, ks, vs,
                                                                              items);
  return cudaGetLastError();
}

template <typename T>
cudaError_t read_t(const Kv8Args& a, void* k, void* v, cudaStream_t stream) {
  const int64_t items = slots_of(a.S, a.T, a.cu != nullptr, a.page_shift) * a.H_kv * 2;
  T* kp = static_cast<T*>(k);
  T* vp = static_cast<T*>(v);
  const bool small = small_items(a);
  const int64_t blocks = blocks_of(items, small);
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (small)
    kv8_read_kernel<T, 32><<<(unsigned)blocks, kBlockSmall, 0, stream>>>(a, kp, vp, items);
  else
    kv8_read_kernel<T, kTeamBig><<<(unsigned)blocks, kTeamBig, 0, stream>>>(a, kp, vp, items);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Args& a, const void* k, const void* v, int type,
                              int64_t k_stride, int64_t v_stride, cudaStream_t stream) {
  switch (type) {
    case CSA2_BF16: return append_t<__nv_bfloat16>(a, k, v, k_stride, v_stride, stream);
    case CSA2_FP16: return append_t<__half>(a, k, v, k_stride, v_stride, stream);
    default: return append_t<float>(a, k, v, k_stride, v_stride, stream);
  }
}

cudaError_t launch_kv8_read(const Kv8Args& a, void* k, void* v, int type, cudaStream_t stream) {
  switch (type) {
    case CSA2_BF16: return read_t<__nv_bfloat16>(a, k, v, stream);
    case CSA2_FP16: return read_t<__half>(a, k, v, stream);
    default: return read_t<float>(a, k, v, stream);
  }
}

}  // namespace csa2
