// Attention of a few query rows per sequence over the 8-bit paged KV cache:
//   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale * q . k_j)
// over the tokens j that row t sees.  A KV head's G query heads share its
// tokens, so a unit of work is (sequence, up to 16 query rows = tokens x G
// heads, KV head) and each cache byte is read once per unit: the kernel is
// bound by reading the cache, 2 bytes of codes per channel and token.
//
// Arithmetic.  E4M3 codes are exact in fp16, and so are queries once their row
// is scaled by a power of two to a largest value in [1, 2) (bf16 rows; values
// 2^-17 below the row's largest lose bits of no weight).  The matrix
// instructions (fp16 in, fp32 accumulate) therefore form q . codes with only
// fp32 rounding.  The block scales enter in the exponent: with K scale ks and V
// scale vs of key j's block,
//   s_j = scale log2(e) ks (q . kcode_j) + log2(vs / 2^E),   w_j = 2^(s_j - ref + 7),
//   out = 2^E sum_j w_j vcode_j / sum_j (w_j 2^E / vs),
// with a reference near the largest s, and a unit 2^E near the blocks' V scales that
// moves where they lie far apart (kv8_sched.cuh).  So the weights fit fp16, and
// applying both scales costs one fused multiply-add.  The weights are
// rounded to fp16 as the operand of the second product (2^-11 relative; the
// factor 2^7 keeps those of 2^-21 and more of the reference normal, so that a long
// tail of small ones is not lost); sums and maxima are fp32.
//
// Work split.  The units' keys are cut into granules of 128 keys and the whole
// batch's granules are dealt to the grid's CTAs as equal contiguous ranges
// (computed from kv_len on the device: no host plan, no empty CTAs for short
// sequences in a long table).  A CTA that holds a whole unit writes its output;
// parts of a unit that is cut go to scratch (at most two per CTA) and the merge
// kernel joins them in order, so results do not depend on timing.
//
// A warp takes 32 keys at a time through its own ring of shared-memory stages
// (16-byte asynchronous copies, swizzled); the warps of a CTA do not wait for one
// another before they join their sums.  K fragments are plain 16-byte shared loads
// (the channel order of the contraction is permuted so that a lane's 16 bytes are
// its four k-steps), V fragments come from transposing matrix loads of bytes, whose
// four bytes are a lane's keys of a k-step when S's columns are permuted to match;
// both are converted in registers (E4M3 -> fp16 is one instruction for two values).
//
// The running maximum is lazy: weights are formed with the old one, which gives
// the key at the reference a weight of 2^7, and only where a sum of them leaves
// fp16's range (seen from the sums that are needed anyway) does it move and O is
// rescaled.
//
// Measured (GB300; the copy peak is 6.77 TB/s):
//   one token of 32 sequences of up to 64K tokens (64 heads over 8, D = 128):
//     465 us, 6.8 TB/s: the copy's rate
//   17 sequences of up to 9K tokens (40 heads over 8, D = 64): 34.8 us (3.2 TB/s).
//     Of them 5 us go before the first tile (ranges, pages, first loads) and 4 to
//     the merge; between, the warps wait for their own loads and results
//     (12 warps an SM: the registers of O and of the codes in flight)
//   4 drafted tokens of 24 sequences of up to 16K tokens (32 heads over 4, D = 128;
//     32 rows a KV head): 90 us (3.3 TB/s), tensor pipe 40 % busy, 35 % of issue
//     slots: the same waits, with eight warps an SM
// Following the V scales costs 463 -> 465, 32.8 -> 34.8 and 86 -> 90 us of these: a
// comparison a tile and the code of the rare case.  (Tiles whose second half came by
// itself by going round the loop once more: 494, 35.8 and 94.)
#include <type_traits>

#include "kv8_sched.cuh"

namespace csa2 {
namespace {

using namespace kv8;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTileKeys = 32;
// log2 of the weight at the reference, and the largest sum of eight weights: no
// weight is above it, which fp16 holds (65504)
constexpr float kHeadroom = 7.0f, kMostSum = 57344.0f;

// A warp has kMt matrix tiles of 16 query rows, and its own keys and ring.
template <int D, int kMt>
struct Cfg {
  static constexpr int unit = 16 * kMt;                    // query rows
  static constexpr int granule = kWarps * kTileKeys;       // keys
  // a unit's queries and output count as three granules (17 sequences of 9K tokens, D =
  // 64, with none to four: 43.6, 34.3, 32.9, 32.8, 32.8 us; drafts 89, 88, 86.4, 86.0, 86.5)
  using Work = Shape<unit, granule, 3>;
  static constexpr int stages = D == 128 ? 3 : 4;
  static constexpr int tile = kTileKeys * D;               // bytes of K (or V) of a stage
  static constexpr int stage = 2 * tile;
  static constexpr int ring = kWarps * stages * stage;
  static constexpr int scales = kWarps * stages * 16;      // ks, vs of two 16-key halves
  // kMt > 1: the fragments of Q (in registers otherwise)
  static constexpr int q = kMt > 1 ? unit * D * 2 : 0;
  static constexpr int smem = ring + scales + q;
  // per SM, as the registers allow: with fewer of them a thread and one CTA more, both
  // D were slower
  static constexpr int ctas = D == 64 && kMt == 1 ? 3 : 2;
  // the join of the warps uses kMt stages of each ring, the next unit's first tiles
  // the others
  static_assert(kMt * stage == unit * D * 4 && kMt < stages && kWarps == 4, "join");
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes into shared memory, zeros where !ok.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0));
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 4 : 0));
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float* c, const uint32_t* x, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk ch of key r in a tile: 128-byte lines, chunks
// exclusive-or'ed so that eight lanes that read one chunk of eight keys, or all
// chunks of the two neighbouring keys of a quarter-warp, meet different banks.
template <int D>
__device__ __forceinline__ uint32_t tile_off(int r, int ch) {
  if (D == 128) return (uint32_t)(r * 128 + ((ch ^ ((r & 1) << 2) ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)((r >> 1) * 128 + (((((r & 1) << 2) | ch) ^ ((r >> 1) & 3)) << 4));
}
// Key of column n of 8-key matrix nt of a tile: columns 2c, 2c + 1 of matrices
// 2b, 2b + 1 are keys 16 b + 4 c .. + 3, the four bytes that a transposing matrix
// load of V gives lane c.
__device__ __forceinline__ int key_of(int nt, int n) {
  return (nt >> 1) * 16 + (n >> 1) * 4 + (nt & 1) * 2 + (n & 1);
}

// 4 E4M3 codes -> fp16.
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t x) {
  uint2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(x));
  return r;
}

// 16 rows of Q as loaded: of this lane's rows row, row + 8 (where the unit has
// them) channels 64 j + 16 c .. + 15.
template <int D>
struct QRows {
  uint4 x[2][D / 64][2];
};
template <int D>
__device__ __forceinline__ QRows<D> fetch_q(const Kv8AttnArgs& a, int row0, int head0, int row,
                                            int nrow, int c) {
  QRows<D> q;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int rr = row + 8 * r;
    const bool ok = rr < nrow;
    const int tok = over_g(a, ok ? rr : 0), head = head0 + (ok ? rr - tok * a.G : 0);
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(a.q) + (int64_t)(row0 + tok) * a.q_stride + (int64_t)head * D);
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
        q.x[r][j][hf] = ok ? __ldg(src + 8 * j + 2 * c + hf) : make_uint4(0, 0, 0, 0);
  }
  return q;
}
// Their fragments: k-step 4 j + i contracts channels 64 j + 16 c + 4 i .. + 3.
// bf16 rows are scaled to a largest magnitude in [1, 2); crow: the rows' logit
// factors.
template <int D, bool kBf16>
__device__ __forceinline__ void make_q(const QRows<D>& q, float scale, uint32_t (*qf)[4],
                                       float* crow) {
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    uint32_t x[D / 64][8];
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        x[j][4 * hf] = q.x[r][j][hf].x;
        x[j][4 * hf + 1] = q.x[r][j][hf].y;
        x[j][4 * hf + 2] = q.x[r][j][hf].z;
        x[j][4 * hf + 3] = q.x[r][j][hf].w;
      }
    crow[r] = scale;
    if (kBf16) {
      float mx = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = pair_to_float2<true>(x[j][i]);
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int E = row_exponent(mx);
      const float down = pow2f(-E);
      crow[r] *= pow2f(E);
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = pair_to_float2<true>(x[j][i]);
          x[j][i] = pack_f16(f.x * down, f.y * down);
        }
    }
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qf[4 * j + i][r] = x[j][2 * i];
        qf[4 * j + i][2 + r] = x[j][2 * i + 1];
      }
  }
}

template <int D, int kMt, bool kBf16>
__global__ void __launch_bounds__(kThreads, Cfg<D, kMt>::ctas)
kv8_attn_kernel(const __grid_constant__ Kv8AttnArgs a) {
  using C = Cfg<D, kMt>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RangeSmem<kWarps> rsm;
  __shared__ float row_max[kWarps][C::unit], row_sum[kWarps][C::unit], row_c[C::unit];
  __shared__ int v_exp[kWarps];  // of the warp's V scales: the largest exponent; at the join, E
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  pdl_trigger();
  const Range rg = find_range<typename C::Work, kWarps>(a, blockIdx.x, gridDim.x, rsm);
  if (tid == 0) write_cut(a, Cut{-1, 0, 0, 0});
  __shared__ Walk<typename C::Work> walks[kWarps][2];  // of the unit, and of the next
  Walk<typename C::Work>& w = walks[warp][0];
  Walk<typename C::Work>& ahead = walks[warp][1];
  if (!warp_start(w, a, rg, rsm)) return;

  uint8_t* ring = smem + warp * (C::stages * C::stage);
  float* ring_scale = reinterpret_cast<float*>(smem + C::ring) + warp * (C::stages * 4);
  uint4* qs = reinterpret_cast<uint4*>(smem + C::ring + C::scales);  // [matrix tile][k-step][lane]
  const uint32_t ring_u = smem_u32(ring), scale_u = smem_u32(ring_scale);
  const int page_mask = (1 << a.c.page_shift) - 1;

  // ---- the unit's tiles: pages, copies ----
  constexpr int kJoin = kMt;  // stages of each ring that the join of the warps uses
  int key_first;              // the warp's first key of granule 0 of the span
  int issue = 0, slot = 0;    // the next tile to request (of the unit's), its stage
  int pids, pids_next;        // pages of the requested block of 16 tiles and of the next
  // page ids of tiles i .. i + 15 of the unit's: lane l has tile i + l % 16, its
  // 16-key half l / 16; -1: nothing of the half is seen, or the entry is outside the cache
  // (in two steps, the table's entry and its check, for what may run between them)
  auto seen_key = [&](const Walk<typename C::Work>& u, int i) -> int {  // -1: nothing is seen
    const int t = u.t0 + i + (lane & 15);
    const int key = (u.u.g0 + t) * C::granule + warp * kTileKeys + (lane & 16);
    return t < u.t1 && key < u.u.hi && key + 16 > u.u.lo ? key : -1;
  };
  auto entry = [&](const Walk<typename C::Work>& u, int key) -> int {
    return key < 0 ? 0 : a.c.table[(int64_t)u.s * a.c.max_pages + (key >> a.c.page_shift)];
  };
  auto page_or_none = [&](int key, int p) -> int {
    if (key < 0) return -1;
    if (p >= 0 && p < a.c.n_pages) return p;
    set_status(a.c.status, kStatusBadIndex);
    return -1;
  };
  auto pages = [&](const Walk<typename C::Work>& u, int i) -> int {
    const int key = seen_key(u, i);
    return page_or_none(key, entry(u, key));
  };
  // Requests the unit's next tile (an empty group of copies past its last).  A half
  // is 16 * D contiguous bytes of a page.
  auto request = [&]() {
    constexpr int kCh = D / 16, kPerIt = 32 / kCh;  // chunks a key, keys an instruction
    constexpr int kIts = 16 / kPerIt;               // instructions a half
    if ((issue & 15) == 0 && issue > 0) {
      pids = pids_next;
      pids_next = pages(w, issue + 16);
    }
    const int t = w.t0 + issue;
    if (t < w.t1) {
      const int key0 = key_first + t * C::granule;
      const uint32_t kd = ring_u + slot * C::stage, vd = kd + C::tile;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int p = __shfl_sync(0xffffffffu, pids, (issue & 15) + 16 * hf);
        const int first = key0 + 16 * hf;
        const int64_t off =
            ((((int64_t)max(p, 0) * a.c.H_kv + w.h) << a.c.page_shift) + (first & page_mask)) * D +
            lane * 16;
        const uint8_t *ksrc = a.c.k + off, *vsrc = a.c.v + off;
        if (p >= 0 && first >= w.u.lo && first + 16 <= w.u.hi) {
#pragma unroll
          for (int it = 0; it < kIts; ++it) {
            const uint32_t so = tile_off<D>(16 * hf + it * kPerIt + lane / kCh, lane % kCh);
            copy16(kd + so, ksrc + it * 512, true);
            copy16(vd + so, vsrc + it * 512, true);
          }
        } else {  // keys that no row sees, or without a page, are zeros
#pragma unroll
          for (int it = 0; it < kIts; ++it) {
            const int r = it * kPerIt + lane / kCh;
            const bool ok = p >= 0 && first + r >= w.u.lo && first + r < w.u.hi;
            const uint32_t so = tile_off<D>(16 * hf + r, lane % kCh);
            copy16(kd + so, ksrc + it * 512, ok);
            copy16(vd + so, vsrc + it * 512, ok);
          }
        }
      }
      // ks of half 0, 1, vs of half 0, 1 (zeros: no page)
      const int p = __shfl_sync(0xffffffffu, pids, (issue & 15) + (lane & 1) * 16);
      if (lane < 4)
        copy4(scale_u + (slot * 4 + lane) * 4,
              ((lane & 2) ? a.c.v_scale : a.c.k_scale) +
                  (p >= 0 ? (int64_t)p * a.c.H_kv + w.h : 0),
              p >= 0);
    }
    copy_commit();
    ++issue;
    if (++slot == C::stages) slot = 0;
  };
  auto open_unit = [&](int first_pages) {
    key_first = w.u.g0 * C::granule + warp * kTileKeys;
    issue = 0;
    pids = first_pages;
    pids_next = pages(w, 16);
  };
  const int qtile = kMt == 1 ? 0 : warp;  // the matrix tile of Q that this warp takes
  QRows<D> qrows;
  auto fetch = [&]() {
    if (qtile < C::unit / 16)
      qrows = fetch_q<D>(a, w.d.row0 + w.first_row(), w.h * a.G, qtile * 16 + g, w.rows(a.G), c);
  };

  // the unit's first loads, all in flight together: the pages, which the copies wait
  // for, then Q, ahead of the copies, which fill the memory's queues
  const int key0 = seen_key(w, 0), entry0 = entry(w, key0);
  fetch();
  open_unit(page_or_none(key0, entry0));
#pragma unroll 1
  for (int i = 0; i < C::stages - 1; ++i) request();
  int st = 0;
  while (true) {
    // the next unit and its first pages, while this one's tiles arrive
    if (lane == 0) ahead = w;
    const bool more = warp_next(ahead, a);
    const int pids_ahead = more ? pages(ahead, 0) : -1;
    const int i0 = w.first_row(), nrow = w.rows(a.G);
    // ---- Q ----
    uint32_t qf[kMt == 1 ? D / 16 : 1][4];
    float crow[kMt][2];
    if constexpr (kMt == 1) {
      make_q<D, kBf16>(qrows, a.scale_log2, qf, crow[0]);
    } else {
      if (warp < C::unit / 16) {
        uint32_t f[D / 16][4];
        float cr[2];
        make_q<D, kBf16>(qrows, a.scale_log2, f, cr);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          qs[(warp * (D / 16) + k) * 32 + lane] = make_uint4(f[k][0], f[k][1], f[k][2], f[k][3]);
        if (c == 0) {
          row_c[warp * 16 + g] = cr[0];
          row_c[warp * 16 + g + 8] = cr[1];
        }
      }
      __syncthreads();
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        crow[mt][0] = row_c[16 * mt + g];
        crow[mt][1] = row_c[16 * mt + g + 8];
      }
    }
    // each row's token (rows that the unit does not have: its first row's), and the
    // tokens [all_lo, all_hi) that every row of the warp sees
    int rpos[kMt][2];
    int all_lo = w.u.lo, all_hi = w.u.hi;
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 16 * mt + g + 8 * r;
        rpos[mt][r] = w.d.len - w.d.n + i0 + over_g(a, row < nrow ? row : 0);
        if (a.causal) {
          all_hi = min(all_hi, rpos[mt][r] + 1);
          if (a.window > 0) all_lo = max(all_lo, rpos[mt][r] - a.window + 1);
        }
      }
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);
    all_hi = __reduce_min_sync(0xffffffffu, all_hi);

    float o[kMt][D / 8][4];
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[mt][i][0] = o[mt][i][1] = o[mt][i][2] = o[mt][i][3] = 0.0f;
    float mrow[kMt][2], lrow[kMt][2];
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt) {
      mrow[mt][0] = mrow[mt][1] = -INFINITY;
      lrow[mt][0] = lrow[mt][1] = 0.0f;
    }

    // a tile's keys (kHalves = 1: its first half): V scales as ratios to 2^E; what O is to be
    // multiplied by, where `moved`
    auto attend = [&](auto halves, const uint8_t* kt, uint32_t vt, int key0, float2 ks, bool half0,
                      bool half1, const float (&ratio)[2], bool masked, bool moved, float factor) {
      constexpr int kHalves = decltype(halves)::value;
      // ---- S = Q K^T ----
      float sc[kMt][2 * kHalves][4];
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2 * kHalves; ++nt) sc[mt][nt][0] = sc[mt][nt][1] = sc[mt][nt][2] = sc[mt][nt][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        [[maybe_unused]] uint4 qv[kMt][4];
        if constexpr (kMt > 1) {
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              qv[mt][i] = qs[(mt * (D / 16) + 4 * j + i) * 32 + lane];
        }
        uint4 b[2 * kHalves];
#pragma unroll
        for (int nt = 0; nt < 2 * kHalves; ++nt)
          b[nt] = *reinterpret_cast<const uint4*>(kt + tile_off<D>(key_of(nt, g), 4 * j + c));
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (4 kMt independent products in a row)
#pragma unroll
          for (int nt = 0; nt < 2 * kHalves; ++nt) {
            const uint2 f = e4m3x4_to_f16x4(i == 0 ? b[nt].x : i == 1 ? b[nt].y : i == 2 ? b[nt].z : b[nt].w);
            if constexpr (kMt == 1) {
              mma16816(sc[0][nt], qf[4 * j + i], f.x, f.y);
            } else {
#pragma unroll
              for (int mt = 0; mt < kMt; ++mt) {
                const uint32_t x[4] = {qv[mt][i].x, qv[mt][i].y, qv[mt][i].z, qv[mt][i].w};
                mma16816(sc[mt][nt], x, f.x, f.y);
              }
            }
          }
      }
      // ---- masks ----
      if (masked) {
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int nt = 0; nt < 2 * kHalves; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + key_of(nt, 2 * c + (e & 1)), pos = rpos[mt][e >> 1];
              if (key < w.u.lo || key >= w.u.hi || (a.causal && key > pos) ||
                  (a.window > 0 && key <= pos - a.window) || !(nt < 2 ? half0 : half1))
                sc[mt][nt][e] = -INFINITY;
            }
      }
      // ---- weights ----
      const float lv[2] = {__log2f(ratio[0]), __log2f(ratio[1])};
      const float rv[2] = {1.0f / ratio[0], 1.0f / ratio[1]};
      // exponents: the logit in powers of two plus log2 of the V scale's ratio.  (Subtracting
      // the reference from the rounded exponent, not inside the fused multiply-add,
      // makes the reference's own weight exact however large the logits are.)
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2 * kHalves; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[mt][nt][e] = fmaf(sc[mt][nt][e],
                                 fmaxf(crow[mt][e >> 1] * (nt < 2 ? ks.x : ks.y), 1.17549435e-38f),
                                 lv[nt >> 1]);
      uint32_t pf[kMt][kHalves][4];
      float ls[kMt][2][kHalves];  // sums [row][half]
      bool fresh = false;
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) fresh |= mrow[mt][0] == -INFINITY || mrow[mt][1] == -INFINITY;
      bool move = moved || __any_sync(0xffffffffu, fresh);
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        if (move) {  // the reference moves to the tile's largest exponent where that is past it
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) {
            float alpha[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float x = -INFINITY;
#pragma unroll
              for (int nt = 0; nt < 2 * kHalves; ++nt)
                x = fmaxf(x, fmaxf(sc[mt][nt][2 * r], sc[mt][nt][2 * r + 1]));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
              alpha[r] = x > mrow[mt][r] ? ex2(mrow[mt][r] - x) : 1.0f;
              mrow[mt][r] = fmaxf(mrow[mt][r], x);
              lrow[mt][r] *= alpha[r];
              alpha[r] *= factor;  // (1 but where E moves, which is always a first pass)
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[mt][i][0] *= alpha[0];
              o[mt][i][1] *= alpha[0];
              o[mt][i][2] *= alpha[1];
              o[mt][i][3] *= alpha[1];
            }
          }
        }
        float most = 0.0f;
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float base = (mrow[mt][r] == -INFINITY ? 0.0f : mrow[mt][r]) - kHeadroom;
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf) {
              float p[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                p[i] = ex2(sc[mt][2 * hf + (i >> 1)][2 * r + (i & 1)] - base);
              ls[mt][r][hf] = (p[0] + p[1]) + (p[2] + p[3]);
              most = fmaxf(most, ls[mt][r][hf]);
              pf[mt][hf][r] = pack_f16(p[0], p[1]);
              pf[mt][hf][2 + r] = pack_f16(p[2], p[3]);
            }
          }
        // a weight may leave fp16's range only where a sum does, and only with a
        // reference that has not moved
        if (move || !__any_sync(0xffffffffu, most > kMostSum)) break;
        move = true;
      }
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int hf = kHalves - 1; hf >= 0; --hf)
            lrow[mt][r] = fmaf(ls[mt][r][hf], rv[hf], lrow[mt][r]);
      // ---- O += P V ----
#pragma unroll
      for (int kk = 0; kk < kHalves; ++kk) {
        const int r = kk * 16 + (lane & 15);
#pragma unroll
        for (int cb = 0; cb < D / 16; cb += 2) {
          // two 16-key x 16-channel blocks: v[2 b + e] holds keys 4c .. 4c + 3 of
          // channel 16 (cb + b) + 8 e + g
          uint32_t v[4];
          asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                       : "r"(vt + tile_off<D>(r, cb + (lane >> 4)))
                       : "memory");
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint2 f = e4m3x4_to_f16x4(v[b]);
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt) mma16816(o[mt][2 * cb + b], pf[mt][kk], f.x, f.y);
          }
        }
      }
    };
    // E from the first tile
    copy_wait<C::stages - 2>();
    __syncwarp();
    float unit;  // 2^-E
    {
      const float2 vs = *reinterpret_cast<const float2*>(ring_scale + st * 4 + 2);
      const float s = vs.x != 0.0f ? vs.x : vs.y;
      const int e = s != 0.0f ? unit_exp(s) : kNoUnit;
      unit = pow2f(-e);
      if (lane == 0) v_exp[warp] = e;
    }
#pragma unroll 1
    for (int t = w.t0; t < w.t1; ++t) {
      copy_wait<C::stages - 2>();
      // every lane's copies of tile t are there, and it is done with tile t - 1, whose
      // stage takes the next copies
      __syncwarp();
      request();
      const float4 bs = *reinterpret_cast<const float4*>(ring_scale + st * 4);
      const uint8_t* kt = ring + st * C::stage;
      const uint32_t vt = ring_u + st * C::stage + C::tile;
      if (++st == C::stages) st = 0;
      const int key0 = key_first + t * C::granule;
      // the halves' V scales as ratios to 2^E
      float ratio[2] = {bs.z * unit, bs.w * unit}, factor = 1.0f;
      bool half0 = true, half1 = true, moved = false;
      const bool masked = !(near_unit(ratio[0]) && near_unit(ratio[1]) && key0 >= all_lo &&
                            key0 + kTileKeys <= all_hi);
      if (masked) {
        half0 = bs.z != 0.0f;
        half1 = bs.w != 0.0f;
        if (!half0 && !half1) continue;
        // A weight of zero does not hide a NaN of V: where some rows see a key and
        // others do not, its V codes become zeros and its K codes NaN, which the mask
        // hides.  (Keys that no row sees are zeros.)
        const int key = key0 + lane;
        uint8_t* codes = ring + (vt - C::tile - ring_u);
        if (key < all_lo || key >= all_hi) {
          bool nan = false;
#pragma unroll 1
          for (int ch = 0; ch < D / 16; ++ch) {
            uint4* x = reinterpret_cast<uint4*>(codes + C::tile + tile_off<D>(lane, ch));
            if (has_nan(*x)) {
              *x = make_uint4(0, 0, 0, 0);
              nan = true;
            }
          }
          if (nan) *reinterpret_cast<uint32_t*>(codes + tile_off<D>(lane, 0)) = 0x7F7F7F7Fu;
        }
        __syncwarp();
        moved = (half0 && !near_unit(ratio[0])) || (half1 && !near_unit(ratio[1]));
        if (moved) {
          VUnit u = {unit_of(unit), v_exp[warp]};
          float f1 = 1.0f;
          bool far0 = false, far1 = false;
          if (half0) ratio[0] = follow(u, bs.z, factor, far0);
          if (half1) ratio[1] = follow(u, bs.w, f1, far1);
          unit = pow2f(-u.e);
          __syncwarp();
          if (lane == 0) v_exp[warp] = u.top;
          if (lane < 16 ? far0 : far1) {  // of values that are left out, the NaN stay
#pragma unroll 1
            for (int ch = 0; ch < D / 16; ++ch) {
              uint4* x = reinterpret_cast<uint4*>(codes + C::tile + tile_off<D>(lane, ch));
              *x = only_nan(*x);
            }
          }
          __syncwarp();
          if (half0 && half1 && f1 != 1.0f) {  // E moves between the halves (pages of 16 tokens)
            attend(std::integral_constant<int, 1>{}, kt, vt, key0, make_float2(bs.x, bs.y), true,
                   true, ratio, true, true, factor);
            half0 = false;
            factor = 1.0f;
          }
          factor *= f1;
        }
        if (!half0) ratio[0] = 1.0f;
        if (!half1) ratio[1] = 1.0f;
      }
      attend(std::integral_constant<int, 2>{}, kt, vt, key0, make_float2(bs.x, bs.y), half0, half1,
             ratio, masked, moved, factor);
    }
    copy_wait<0>();
    __syncwarp();  // the warp is done with its ring

    // ---- the next unit's first tiles, into the stages that the join leaves ----
    const bool whole = w.whole(), starts = w.t0 == 0;
    const int token0 = w.d.row0 + i0, head0 = w.h * a.G;
    if (starts && !whole && tid == 0) write_cut(a, w.cut(a, rg));
    __syncwarp();
    if (more) {
      if (lane == 0) w = ahead;
      __syncwarp();
      open_unit(pids_ahead);
      slot = st = kJoin;
#pragma unroll 1
      for (int i = 0; i < min(C::stages - kJoin, C::stages - 1); ++i) request();
    }

    // ---- join the warps ----
    float* obuf = reinterpret_cast<float*>(ring);  // [row][D], of each warp
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        lrow[mt][r] += __shfl_xor_sync(0xffffffffu, lrow[mt][r], 1);
        lrow[mt][r] += __shfl_xor_sync(0xffffffffu, lrow[mt][r], 2);
        const int row = 16 * mt + g + 8 * r;
        if (c == 0) {
          row_max[warp][row] = mrow[mt][r];
          row_sum[warp][row] = lrow[mt][r];
        }
        if (lane == 0 && mt == 0 && r == 0) v_exp[warp] = max(-126, unit_of(unit));
        float* dst = obuf + (size_t)row * D + 2 * c;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)  // (8-channel blocks exclusive-or'ed with the row: other banks)
          *reinterpret_cast<float2*>(dst + 8 * (i ^ (row & 3))) =
              make_float2(o[mt][i][2 * r], o[mt][i][2 * r + 1]);
      }
    if (more) fetch();
    __syncthreads();
    float* pw = scratch_part(a, gridDim.x, blockIdx.x, starts, C::unit, D);
    // (a warp without keys has O = 0 and the least E)
    const int e_top = max(max(v_exp[0], v_exp[1]), max(v_exp[2], v_exp[3]));
    const float to_one = pow2f(e_top);
    constexpr int kTpr = D / 4;  // threads per row
#pragma unroll 1
    for (int i = 0; i < C::unit * kTpr / kThreads; ++i) {
      const int row = (i * kThreads + tid) / kTpr, ch = (tid % kTpr) * 4;
      if (row >= nrow) continue;
      float m = row_max[0][row];
#pragma unroll
      for (int q = 1; q < kWarps; ++q) m = fmaxf(m, row_max[q][row]);
      const float mz = m == -INFINITY ? 0.0f : m;
      float l = 0.0f;
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < kWarps; ++q) {
        float f = ex2(row_max[q][row] - mz);
        l = fmaf(row_sum[q][row], f, l);
        f *= pow2_or_zero(v_exp[q] - e_top);
        const float4 y = *reinterpret_cast<const float4*>(
            smem + q * (C::stages * C::stage) + ((size_t)row * D + (ch ^ ((row & 3) * 8))) * 4);
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
      }
      // no visible token: zeros
      const float inv = l == 0.0f ? 0.0f : (whole ? 1.0f : kPartOut) / l;
      x.x = x.x * inv * to_one;
      x.y = x.y * inv * to_one;
      x.z = x.z * inv * to_one;
      x.w = x.w * inv * to_one;
      if (whole) {
        const int64_t orow = out_row(a, token0, head0, row);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + ch) =
            make_uint2(pair_from_floats<kBf16>(x.x, x.y), pair_from_floats<kBf16>(x.z, x.w));
        if (a.lse && ch == 0)
          a.lse[orow] = l == 0.0f ? -INFINITY : (mz - kHeadroom + __log2f(l)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(pw + (size_t)row * D + ch) = x;
        if (ch == 0) {
          pw[C::unit * D + row] = m;
          pw[C::unit * D + C::unit + row] = l;
        }
      }
    }
    if (!more) break;
    __syncthreads();  // the joined stages may be written again
#pragma unroll 1
    for (int i = min(C::stages - kJoin, C::stages - 1); i < C::stages - 1; ++i) request();
  }
}

template <int D, int kMt, bool kBf16>
__global__ void __launch_bounds__(kThreads)
kv8_merge_kernel(const __grid_constant__ Kv8AttnArgs a, int workers) {
  using C = Cfg<D, kMt>;
  merge_parts<typename C::Work, D, kBf16>(a, workers, kHeadroom);
}

template <int D, int kMt, bool kBf16>
cudaError_t attn_t(const Kv8AttnArgs& args, cudaStream_t stream) {
  using C = Cfg<D, kMt>;
  Kv8AttnArgs a = args;
  a.tpu = C::unit / a.G;
  cudaError_t e = cudaFuncSetAttribute(kv8_attn_kernel<D, kMt, kBf16>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  const int workers = device_sm_count() * C::ctas;
  e = launch_kernel(kv8_attn_kernel<D, kMt, kBf16>, dim3(workers), dim3(kThreads), C::smem,
                    stream, /*pdl=*/false, a);
  if (e != cudaSuccess || a.uncut) return e;
  const dim3 grid(workers, merge_blocks<typename C::Work, D>(a, workers));
  return launch_kernel(kv8_merge_kernel<D, kMt, kBf16>, grid, dim3(kThreads), 0, stream,
                       /*pdl=*/true, a, workers);
}

// Rows of a KV head (per sequence, on average) up to which the kernel of 16 rows
// and that of 32 are taken.  Measured: one token of 32 sequences of 64K (8 rows) 464
// us with 16, 700 with 32; 17 sequences of 9K (5 rows, D = 64) 34.4 and 45.2; drafts
// (32 rows, D = 128) 103 with 16, whose units read the cache twice, 88 with 32 and
// 114 with the tcgen05 kernel.  Of 40 to 64 rows there the tcgen05 kernel takes 122
// us (D = 64: 97), units of 32 rows 152 (101); two warps of 32 rows that share the keys
// took 146 (both convert every tile).
constexpr int64_t kRows1 = 16, kRows2 = 32;
// Units of up to so many keys are not cut: one CTA takes 3 to 4 us for 512 keys,
// what the merge kernel would add (128 sequences of 1000 tokens: 58 us cut, 64 us
// with units of 1024 keys left whole).
constexpr int64_t kUncut = 512;

// Query rows of a KV head per sequence, on average.
int64_t mean_rows(int S, int T, int G) {
  return max((int64_t)G, ((int64_t)T * G + S - 1) / S);
}

}  // namespace

size_t kv8_attn_scratch_bytes(int S, int T, int H, int H_kv, int D) {
  if (D != 64 && D != 128) return 0;
  if (mean_rows(S, T, H / H_kv) > kRows2) return kv8_attn_tc_scratch_bytes(D);
  return align_up(scratch_bytes(device_sm_count() * 3, 32, D), 256);
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& args, int type, cudaStream_t stream) {
  Kv8AttnArgs a = args;
  const int64_t rows = mean_rows(a.c.S, a.c.T, a.G);
  a.uncut = kv8_most_tokens(a) <= kUncut;
  if (rows > kRows2) return launch_kv8_attn_tc(a, type, stream);
  const bool one = rows <= kRows1, bf16 = type == CSA2_BF16;
  if (a.c.D == 128)
    return one ? (bf16 ? attn_t<128, 1, true>(a, stream) : attn_t<128, 1, false>(a, stream))
               : (bf16 ? attn_t<128, 2, true>(a, stream) : attn_t<128, 2, false>(a, stream));
  return one ? (bf16 ? attn_t<64, 1, true>(a, stream) : attn_t<64, 1, false>(a, stream))
             : (bf16 ? attn_t<64, 2, true>(a, stream) : attn_t<64, 2, false>(a, stream));
}

}  // namespace csa2
