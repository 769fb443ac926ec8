// How the attention over the 8-bit cache is dealt out.  A unit of work is
// (sequence, block of up to kUnit query rows = tokens x G heads, KV head); its
// keys are cut into granules.  The batch's granules, in the order (sequence,
// block, head, key), are dealt to the grid's CTAs ("workers") as equal
// contiguous ranges.  What a unit costs beside its keys (its queries, its output)
// counts as kCost granules before its first: without them a worker with many
// short units took twice the mean (prompts through a window of 1024).  Everything is computed on the device from kv_len and cu:
// there is no host plan, nothing to keep up to date, no CTA for tokens that a
// sequence does not have, and a captured graph follows the lengths.
#pragma once

#include "kv8.cuh"

namespace csa2 {
namespace kv8 {

constexpr float kLn2 = 0.69314718055994530942f;

struct Dims {
  int n, row0, len, cap;  // the sequence's rows and tokens; tokens the table has room for
  int tpu, nm;            // tokens of a block of rows, blocks
};

// What the kernels of one kind share: query rows of a unit, keys of a granule, a
// unit's fixed cost in granules.
template <int kUnit_, int kGranule_, int kCost_>
struct Shape {
  static constexpr int kUnit = kUnit_, kGranule = kGranule_, kCost = kCost_;
};

template <class Sh>
__device__ __forceinline__ Dims seq_dims(const Kv8AttnArgs& a, int s) {
  const Kv8Seq q = kv8_seq(a.c, s);
  Dims d;
  d.n = q.n;
  d.row0 = q.row0;
  d.len = q.len;
  d.cap = (int)min((int64_t)q.len, (int64_t)a.c.max_pages << a.c.page_shift);
  d.tpu = a.tpu;
  d.nm = q.n <= d.tpu ? (q.n > 0 ? 1 : 0) : (q.n + d.tpu - 1) / d.tpu;
  return d;
}

// Tokens [lo, hi) that some row of block m sees, and the granules that cover them.
struct Span {
  int lo, hi, g0, ng;
};

template <class Sh>
__device__ __forceinline__ Span unit_span(const Kv8AttnArgs& a, const Dims& d, int m) {
  Span u;
  u.lo = 0;
  u.hi = d.cap;
  if (a.causal) {
    const int i0 = m * d.tpu, i1 = min(d.n, i0 + d.tpu);
    const int64_t p0 = (int64_t)d.len - d.n + i0, p1 = (int64_t)d.len - d.n + i1 - 1;
    u.hi = (int)max((int64_t)0, min((int64_t)d.cap, p1 + 1));
    if (a.window > 0) u.lo = (int)max((int64_t)0, p0 - a.window + 1);
  }
  if (u.lo > u.hi) u.lo = u.hi;
  u.g0 = u.lo / Sh::kGranule;
  u.ng = max(1, (u.hi + Sh::kGranule - 1) / Sh::kGranule - u.g0);  // one at least: it writes the rows
  return u;
}

// Places of a unit in the batch's order: its granules after its fixed cost, or one
// where units are not cut.
template <class Sh>
__device__ __forceinline__ int unit_places(const Kv8AttnArgs& a, const Span& u) {
  return a.uncut ? 1 : u.ng + Sh::kCost;
}

// A worker's range [w0, w1) of the batch's granules (fixed costs included) and
// where it starts: place c0 of unit (s, m, h).  s < 0: no range.
struct Range {
  int64_t w0, w1;
  int64_t q;   // every worker has q places, the first r one more
  int r;
  int s, m, h, c0;
};

template <int kWarps>
struct RangeSmem {
  int64_t warp_sum[kWarps];
  int s, m, h, c0;
  Dims d;
  Span u;
};

// (A 64-bit division takes some hundred cycles; the numbers are small but for
// batches of billions of places.)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// The worker that has place x.
__device__ __forceinline__ int owner(const Range& r, int64_t x) {
  const int64_t big = (int64_t)r.r * (r.q + 1);
  return x < big ? (int)quotient(x, r.q + 1) : r.r + (int)quotient(x - big, r.q);
}

// Sums one value per lane of each warp; every lane gets the warp's total.
__device__ __forceinline__ int64_t warp_total(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// All threads of the block.  A warp takes a contiguous share of the sequences,
// 32 at a time: a lane per sequence where the sequences have one block of rows,
// else the lanes go over a sequence's blocks together.
template <class Sh, int kWarps>
__device__ Range find_range(const Kv8AttnArgs& a, int worker, int workers,
                            RangeSmem<kWarps>& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.c.S + kWarps - 1) / kWarps;
  const int s0 = min(a.c.S, warp * per), s1 = min(a.c.S, s0 + per);
  bool bad = false;  // some sequence's entries make no sense
  // granules of the blocks of sequence s, every KV head
  auto lane_work = [&](const Dims& d) -> int64_t {  // a lane's sequence with one block (or none)
    return d.nm == 1 ? (int64_t)unit_places<Sh>(a, unit_span<Sh>(a, d, 0)) * a.c.H_kv : 0;
  };
  auto warp_work = [&](const Dims& d) -> int64_t {  // the warp's sequence, any number of blocks
    if (!a.causal) return (int64_t)d.nm * unit_places<Sh>(a, unit_span<Sh>(a, d, 0)) * a.c.H_kv;
    int64_t w = 0;
    for (int m = lane; m < d.nm; m += 32) w += unit_places<Sh>(a, unit_span<Sh>(a, d, m));
    return warp_total(w) * a.c.H_kv;
  };
  // work of sequence base + lane (0 past s1), and its dimensions
  auto chunk = [&](int base, Dims& d) -> int64_t {
    const int s = base + lane;
    d.nm = 0;
    if (s < s1) {
      d = seq_dims<Sh>(a, s);
      bad |= kv8_seq(a.c, s).bad;
    }
    int64_t w = lane_work(d);
    uint32_t big = __ballot_sync(0xffffffffu, d.nm > 1);
    while (big) {
      const int l = __ffs(big) - 1;
      big &= big - 1;
      const int64_t x = warp_work(seq_dims<Sh>(a, base + l));
      if (lane == l) w = x;
    }
    return w;
  };
  Dims d0;  // of the warp's first 32 sequences
  const int64_t first = chunk(s0, d0), first_inc = warp_scan(first, lane);
  int64_t mine = __shfl_sync(0xffffffffu, first_inc, 31);
  if (s0 + 32 < s1) {
    int64_t more = 0;
    for (int b = s0 + 32; b < s1; b += 32) {
      Dims d;
      more += chunk(b, d);
    }
    mine += warp_total(more);
  }
  if (bad) set_status(a.c.status, kStatusBadIndex);
  if (lane == 0) sm.warp_sum[warp] = mine;
  if (tid == 0) sm.s = -1;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += sm.warp_sum[w];
    total += sm.warp_sum[w];
  }
  Range r;
  r.q = quotient(total, workers);
  r.r = (int)(total - r.q * workers);
  r.w0 = worker * r.q + min(worker, r.r);
  r.w1 = r.w0 + r.q + (worker < r.r ? 1 : 0);
  if (r.w0 < r.w1 && r.w0 >= base && r.w0 < base + mine) {  // this warp's sequences hold w0
    int64_t at = base;
    for (int b = s0; b < s1; b += 32) {
      Dims db;
      const int64_t w = b == s0 ? first : chunk(b, db);
      const int64_t inc = b == s0 ? first_inc : warp_scan(w, lane);
      const uint32_t past = __ballot_sync(0xffffffffu, r.w0 < at + inc);
      if (past) {
        const int l = __ffs(past) - 1;
        const int s = b + l;
        // (the short way takes 1000 cycles less before a CTA's first load)
        if (b == s0 && __shfl_sync(0xffffffffu, d0.nm, l) == 1) {
          if (lane == l) {
            const int64_t rem = r.w0 - at - (inc - w);
            const Span u = unit_span<Sh>(a, d0, 0);
            const int n = unit_places<Sh>(a, u);
            sm.s = s;
            sm.m = 0;
            sm.h = (int)quotient(rem, n);
            sm.c0 = (int)(rem - (int64_t)sm.h * n);
            sm.d = d0;
            sm.u = u;
          }
          break;
        }
        int64_t rem = r.w0 - at - __shfl_sync(0xffffffffu, inc - w, l);
        const Dims d = seq_dims<Sh>(a, s);
        // the block of rows: 32 at a time
        for (int m0 = 0; m0 < d.nm; m0 += 32) {
          const int ng = m0 + lane < d.nm ? unit_places<Sh>(a, unit_span<Sh>(a, d, m0 + lane)) : 0;
          const int64_t x = (int64_t)ng * a.c.H_kv, xi = warp_scan(x, lane);
          const uint32_t pm = __ballot_sync(0xffffffffu, rem < xi);
          if (pm) {
            const int k = __ffs(pm) - 1;
            rem -= __shfl_sync(0xffffffffu, xi - x, k);
            const int n = __shfl_sync(0xffffffffu, ng, k);
            if (lane == 0) {
              sm.s = s;
              sm.m = m0 + k;
              sm.h = (int)quotient(rem, n);
              sm.c0 = (int)(rem - (int64_t)sm.h * n);
              sm.d = d;
              sm.u = unit_span<Sh>(a, d, m0 + k);
            }
            break;
          }
          rem -= __shfl_sync(0xffffffffu, xi, 31);
        }
        break;
      }
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  r.s = sm.s;
  r.m = sm.m;
  r.h = sm.h;
  r.c0 = sm.c0;
  return r;
}

// Scratch: a record for each worker, then its parts of cut units, out [kUnit][D] (as if
// the part's keys were all), max [kUnit], sum [kUnit]: [0] a part that continues a unit,
// [1] one that starts it.  (out is stored small: a value of 448 * 2^120, as append stores an
// infinity, is past fp32 and would be NaN by a weight of zero.)  The record of the worker that starts a cut unit says how to
// join it, so that the merge kernel need not find its way again.
constexpr float kPartOut = 0.0625f;
struct Cut {
  int last;  // the worker with the unit's last part; -1: this worker starts no cut unit
  int token, head, rows;  // the unit's first row in q and out, its KV head's first query head
};

// Walks the units of a range that it has granules of: unit (s, m, h), granules
// [t0, t1) of its span.
template <class Sh>
struct Walk {
  int s, m, h, t0, t1;
  int64_t pos, end;  // the batch's places: of the unit, of the range's end
  Dims d;
  Span u;

  // To the range's first unit; false if it has none.
  template <int kWarps>
  __device__ __forceinline__ bool start(const Kv8AttnArgs& a, const Range& r,
                                        const RangeSmem<kWarps>& sm) {
    s = r.s;
    m = r.m;
    h = r.h;
    end = r.w1;
    d = sm.d;
    u = sm.u;
    pos = r.w0 - r.c0;
    return clip(a, r.c0) || next(a);
  }
  // To the next unit of the range; false at its end.
  __device__ __forceinline__ bool next(const Kv8AttnArgs& a) {
    while (true) {
      pos += unit_places<Sh>(a, u);
      if (pos >= end) return false;
      if (++h == a.c.H_kv) {
        h = 0;
        if (++m < d.nm) {
          u = unit_span<Sh>(a, d, m);
        } else {
          m = 0;
          do {
            if (++s >= a.c.S) return false;
            d = seq_dims<Sh>(a, s);
          } while (d.nm == 0);
          u = unit_span<Sh>(a, d, 0);
        }
      }
      if (clip(a, 0)) return true;
    }
  }
  // The unit's granules from place c0 to the range's end; false if none.
  __device__ __forceinline__ bool clip(const Kv8AttnArgs& a, int c0) {
    if (a.uncut) {
      t0 = 0;
      t1 = u.ng;
      return true;
    }
    t0 = max(0, c0 - Sh::kCost);
    t1 = (int)min((int64_t)u.ng, end - pos - Sh::kCost);
    return t1 > t0;
  }
  // The record of a unit that this range starts and does not end.
  __device__ __forceinline__ Cut cut(const Kv8AttnArgs& a, const Range& r) const {
    const int64_t past = pos + unit_places<Sh>(a, u);  // the place behind its last
    return Cut{owner(r, past - 1), d.row0 + first_row(), h * a.G, rows(a.G)};
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == u.ng; }
  __device__ __forceinline__ int first_row() const { return m * d.tpu; }  // its first token's row
  __device__ __forceinline__ int rows(int G) const {
    return (min(d.n, (m + 1) * d.tpu) - m * d.tpu) * G;
  }
};

__host__ __device__ constexpr size_t part_floats(int unit, int D) {
  return (size_t)unit * D + 2 * (size_t)unit;
}
__host__ __device__ inline size_t scratch_bytes(int workers, int unit, int D) {
  return align_up((size_t)workers * sizeof(Cut), 256) + (size_t)workers * 2 * part_floats(unit, D) * 4;
}
__device__ __forceinline__ float* scratch_part(const Kv8AttnArgs& a, int workers, int worker,
                                               bool starts, int unit, int D) {
  return reinterpret_cast<float*>(a.scratch + align_up((size_t)workers * sizeof(Cut), 256)) +
         ((size_t)worker * 2 + (starts ? 1 : 0)) * part_floats(unit, D);
}
// One thread of a worker (first a record without a unit, then the unit it starts).
__device__ __forceinline__ void write_cut(const Kv8AttnArgs& a, const Cut& c) {
  if (!a.uncut)
    *reinterpret_cast<int4*>(a.scratch + (size_t)blockIdx.x * sizeof(Cut)) =
        make_int4(c.last, c.token, c.head, c.rows);
}

// A warp's walk in shared memory (kept out of registers): one lane moves it.
template <class Sh, int kWarps>
__device__ __forceinline__ bool warp_start(Walk<Sh>& w, const Kv8AttnArgs& a, const Range& r,
                                           const RangeSmem<kWarps>& sm) {
  bool any = false;
  if ((threadIdx.x & 31) == 0 && r.s >= 0) any = w.start(a, r, sm);
  any = __shfl_sync(0xffffffffu, any, 0);
  __syncwarp();
  return any;
}
template <class Sh>
__device__ __forceinline__ bool warp_next(Walk<Sh>& w, const Kv8AttnArgs& a) {
  __syncwarp();
  bool more = false;
  if ((threadIdx.x & 31) == 0) more = w.next(a);
  more = __shfl_sync(0xffffffffu, more, 0);
  __syncwarp();
  return more;
}

// 2^x by the hardware's approximation (relative error about 2^-22); results
// below 2^-126 are zeros (the form that keeps them costs three more instructions).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Is one of 16 E4M3 codes a NaN (0x7F, 0xFF)?
__device__ __forceinline__ bool has_nan(uint4 x) {
  auto sevens = [](uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; };
  return ((sevens(x.x) | sevens(x.y) | sevens(x.z) | sevens(x.w)) & 0x80808080u) != 0;
}

// The NaN of 16 codes, the others zero.
__device__ __forceinline__ uint4 only_nan(uint4 x) {
  auto f = [](uint32_t w) {
    return ((((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0x7Fu;
  };
  return make_uint4(f(x.x), f(x.y), f(x.z), f(x.w));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool kBf16>
__device__ __forceinline__ float2 pair_to_float2(uint32_t w) {
  if (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return half2_bits_to_float2(w);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pair_from_floats(float lo, float hi) {
  if (!kBf16) return pack_f16(lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Exponent that brings a row's largest magnitude mx to [1, 2) (0 for a row of zeros).
__device__ __forceinline__ int row_exponent(float mx) {
  const int E = (int)(__float_as_uint(mx) >> 23) - 127;
  return mx > 0.0f ? max(-126, min(126, E)) : 0;
}

// V scales far apart.  O is held in units of 2^E, a V scale enters the weights as its
// ratio to 2^E, and E follows the blocks as their keys come: it stays where the ratio is
// in [2^-6, 4), so that fp16 weights lose no logits to a scale, and moves to the
// block's exponent otherwise, O scaled by the (exact) power of two between.  Down it goes
// to 2^60 below the largest only, so that O (2^55 and less, for 2^30 tokens) cannot
// overflow.  Blocks that are smaller still count in the sum with a ratio of 1, and
// their values (below 2^-51 of the largest scale) are left out, but for NaN.
constexpr int kSpan = 60;
__device__ __forceinline__ bool near_unit(float ratio) {
  return __float_as_uint(ratio) - 0x3C800000u < 0x40800000u - 0x3C800000u;
}
// E for a block: its ratio is in [2^-2, 2^-1), so that blocks a few powers of two to either
// side do not move it.
__device__ __forceinline__ int unit_exp(float scale) {
  return max(-126, min(126, (int)((__float_as_uint(scale) >> 23) & 0xFFu) - 125));
}
// E of 2^-E; kNoUnit for 2^127.
__device__ __forceinline__ int unit_of(float unit) { return 127 - (int)(__float_as_uint(unit) >> 23); }
// 2^e, zero below fp32's normal numbers.
__device__ __forceinline__ float pow2_or_zero(int e) { return e < -126 ? 0.0f : pow2f(e); }
// E and the largest exponent so far; a unit starts without.
struct VUnit {
  int e, top;
};
constexpr int kNoUnit = -127;
// The block's ratio, and what O is to be multiplied by before it.  far: its values are
// left out.
__device__ __forceinline__ float follow(VUnit& u, float scale, float& factor, bool& far) {
  const int e = unit_exp(scale);
  factor = 1.0f;
  far = false;
  if (u.e == kNoUnit) {
    u.e = u.top = e;
  } else if (e > u.e + 3 || e < u.e - 4) {
    u.top = max(u.top, e);
    const int to = max(e, u.top - kSpan);
    if (e < to - 4) {
      far = true;
      return 1.0f;
    }
    factor = pow2_or_zero(u.e - to);
    u.e = to;
  }
  return scale * pow2f(-u.e);
}

// row / G for row < 256, by the host's reciprocal ceil(2^16 / G): row times its
// excess (below G) stays below 2^16.
__device__ __forceinline__ int over_g(const Kv8AttnArgs& a, int row) {
  return (row * a.g_inv) >> 16;
}
// Row of q, out and lse (token x H + head) of a unit's row.
__device__ __forceinline__ int64_t out_row(const Kv8AttnArgs& a, int token, int head, int row) {
  const int t = over_g(a, row);
  return (int64_t)(token + t) * a.H + head + (row - t * a.G);
}

// Joins the parts of the cut units: block (x, y) takes the unit that worker x
// starts, every gridDim.y-th group of its rows.  A part counts by its share of the sum so
// far, so the result stays a mean of the parts' outputs and cannot overflow, whatever
// scales the parts' values have.  Few parts: a thread has four
// channels of a row and goes through them.  Many (a long context with few units):
// a warp has 32 channels of a row; its lanes share out the parts' maxima and sums,
// 32 at a time, and four groups of eight lanes sum a quarter of the parts each, all
// loads independent.  (A thread that goes through the parts takes 0.35 us a part;
// for two parts of 256 rows the shared form takes twice as long as it.  No shared
// memory: a block with some has its SM's memory divided anew, which waits for the
// blocks of the attention and delays the next call's.)
template <class Sh, int D>
constexpr int merge_rows() {  // rows of a block of four warps
  return 4 / (D / 32);
}
// Blocks for a worker's unit: a row group each for up to 16 rows, or, where the units
// are few and so of many parts, up to 128.  (One token of 60000, 64 heads over 1, D =
// 128: 31 us with 128, 42 with 16; two of 50000, 128 heads: 52 and 114.  Batches of
// many units would start thousands of blocks for nothing.)
template <class Sh, int D>
int merge_blocks(const Kv8AttnArgs& a, int workers) {
  const int64_t most = a.c.cu ? Sh::kUnit : (int64_t)(a.c.T / a.c.S) * a.G;
  const int rows = (int)(most < Sh::kUnit ? most : Sh::kUnit);
  const int64_t units = ((int64_t)a.c.S + a.c.T / a.tpu) * a.c.H_kv;
  const int cap = units * 4 <= workers ? 128 : 16;
  return ((rows < cap ? rows : cap) + merge_rows<Sh, D>() - 1) / merge_rows<Sh, D>();
}
template <class Sh, int D, bool kBf16>
__device__ __forceinline__ void merge_parts(const Kv8AttnArgs& a, int workers, float headroom) {
  constexpr int kUnit = Sh::kUnit, kRowsPer = merge_rows<Sh, D>();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane >> 3;
  const int sub = warp / (D / 32), ch = (warp % (D / 32)) * 32 + (lane & 7) * 4;
  pdl_wait();
  const int4 cut = __ldcg(reinterpret_cast<const int4*>(a.scratch) + blockIdx.x);
  const int last = cut.x, nrow = last < 0 ? 0 : cut.w;
  auto write = [&](int row, int c4, float4 x, float m, float l) {
    const int64_t orow = out_row(a, cut.y, cut.z, row);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + c4) =
        make_uint2(pair_from_floats<kBf16>(x.x / kPartOut, x.y / kPartOut),
                   pair_from_floats<kBf16>(x.z / kPartOut, x.w / kPartOut));
    if (a.lse && c4 == 0)
      a.lse[orow] =
          l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) - headroom + __log2f(l)) * kLn2;
  };
  if (last - (int)blockIdx.x < 4) {
    constexpr int kTpr = D / 4, kRows = 128 / kTpr;
    const int c4 = (threadIdx.x % kTpr) * 4;
    for (int row = blockIdx.y * kRows + threadIdx.x / kTpr; row < nrow; row += gridDim.y * kRows) {
      float m = -INFINITY, l = 0.0f;
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int p = blockIdx.x; p <= last; ++p) {
        const float* src = scratch_part(a, workers, p, p == (int)blockIdx.x, kUnit, D);
        const float pm = __ldcg(src + kUnit * D + row), pl = __ldcg(src + kUnit * D + kUnit + row);
        const float4 y = __ldcg(reinterpret_cast<const float4*>(src + (size_t)row * D + c4));
        const float nm = fmaxf(m, pm), z = nm == -INFINITY ? 0.0f : nm;
        float f0 = l * ex2(m - z), f1 = pl * ex2(pm - z);
        m = nm;
        l = f0 + f1;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no visible token: zeros
        f0 *= inv;
        f1 *= inv;
        x.x = x.x * f0 + y.x * f1;
        x.y = x.y * f0 + y.y * f1;
        x.z = x.z * f0 + y.z * f1;
        x.w = x.w * f0 + y.w * f1;
      }
      write(row, c4, x, m, l);
    }
    return;
  }
  for (int row = blockIdx.y * kRowsPer + sub; row < nrow; row += gridDim.y * kRowsPer) {
    float m = -INFINITY, l = 0.0f;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p0 = blockIdx.x; p0 <= last; p0 += 32) {
      const int n = min(32, last + 1 - p0);
      auto part = [&](int i) {
        return scratch_part(a, workers, p0 + i, p0 + i == (int)blockIdx.x, kUnit, D);
      };
      float pm = -INFINITY, pl = 0.0f;
      if (lane < n) {
        pm = __ldcg(part(lane) + kUnit * D + row);
        pl = __ldcg(part(lane) + kUnit * D + kUnit + row);
      }
      float4 y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = group + 4 * k;
        y[k] = i < n ? __ldcg(reinterpret_cast<const float4*>(part(i) + (size_t)row * D + ch))
                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      float top = fmaxf(m, pm);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float z = top == -INFINITY ? 0.0f : top, g = pl * ex2(pm - z);
      float old = l * ex2(m - z), sum = g;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l = old + sum;
      m = top;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l, f = g * inv;
      old *= inv;
      x.x *= old;
      x.y *= old;
      x.z *= old;
      x.w *= old;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float h = __shfl_sync(0xffffffffu, f, group + 4 * k);
        x.x = fmaf(y[k].x, h, x.x);
        x.y = fmaf(y[k].y, h, x.y);
        x.z = fmaf(y[k].z, h, x.z);
        x.w = fmaf(y[k].w, h, x.w);
      }
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
      x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
      x.z += __shfl_xor_sync(0xffffffffu, x.z, o);
      x.w += __shfl_xor_sync(0xffffffffu, x.w, o);
    }
    if (group == 0) write(row, ch, x, m, l);
  }
}

}  // namespace kv8
}  // namespace csa2
