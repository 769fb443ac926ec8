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
//   s_j = scale log2(e) ks (q . kcode_j) + log2(vs),   w_j = 2^(s_j - max s + 15),
//   out = sum_j w_j vcode_j / sum_j (w_j / vs),
// so every weight is at most 2^15 whatever the scales, and applying both scales
// costs one fused multiply-add.  The weights are rounded to fp16 as the operand
// of the second product (2^-11 relative; the factor 2^15 keeps weights down to
// 2^-29 of the largest normal, so that a long tail of small ones is not lost);
// sums and maxima are fp32.
//
// Work split.  The units' keys are cut into granules of 128 keys and the whole
// batch's granules are dealt to the grid's CTAs as equal contiguous ranges
// (computed from kv_len on the device: no host plan, no empty CTAs for short
// sequences in a long table).  A CTA that holds a whole unit writes its output;
// parts of a unit that is cut go to scratch (at most two per CTA) and the merge
// kernel joins them in order, so results do not depend on timing.
//
// A warp takes 32 keys of a granule through its own ring of shared-memory
// stages (16-byte asynchronous copies, swizzled), with no barrier between warps:
// K fragments are plain 16-byte shared loads (the channel order of the
// contraction is permuted so that a lane's 16 bytes are its four k-steps), V
// fragments come from transposing matrix loads of byte pairs, both converted in
// registers (E4M3 -> fp16 is one instruction for two values).
#include "kv8_sched.cuh"

namespace csa2 {
namespace {

using namespace kv8;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTileKeys = 32;
constexpr float kHeadroom = 15.0f;  // log2 of the largest weight

// kRg warps share a tile's keys, 16 query rows each; 4 / kRg groups of warps
// have rings of their own.  The ring of a CTA has the same size for every kRg.
template <int D, int kRg>
struct Cfg {
  static constexpr int unit = 16 * kRg;                    // query rows
  static constexpr int kgs = kWarps / kRg;                 // key groups
  static constexpr int granule = kgs * kTileKeys;          // keys
  // a unit's queries and output take about as long as 128 keys
  using Work = Shape<unit, granule, kRg>;
  static constexpr int stages = (D == 128 ? 3 : 4) * kRg;
  static constexpr int tile = kTileKeys * D;               // bytes of K (or V) of a stage
  static constexpr int stage = 2 * tile;
  static constexpr int ring = kgs * stages * stage;
  static constexpr int scales = kgs * stages * 16;         // ks, vs of two 16-key halves
  static constexpr int smem = ring + scales;
  static constexpr int ctas = D == 128 ? 2 : 3;            // per SM
  static_assert(ring >= kWarps * 16 * D * 4, "the merge of the warps reuses the ring");
  static_assert(stages <= 16, "two bits a stage in a word");
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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk ch of key r in a tile: 128-byte lines, chunks
// exclusive-or'ed with the line so that eight lanes reading one chunk of eight
// keys, or all chunks of two keys, meet eight different banks.
template <int D>
__device__ __forceinline__ uint32_t tile_off(int r, int ch) {
  if (D == 128) return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4));
  return (uint32_t)((r >> 1) * 128 + (((((r & 1) << 2) | ch) ^ ((r >> 1) & 7)) << 4));
}
// Key of column n of an 8-key matrix: at D = 128 two neighbouring columns are
// four keys apart, so that a quarter-warp's two keys swizzle to different halves
// of a line.
template <int D>
__device__ __forceinline__ int key_of(int n) {
  return D == 128 ? (n >> 1) | ((n & 1) << 2) : n;
}

// The warps of key group kg.
template <int kRg>
__device__ __forceinline__ void group_sync(int kg) {
  if (kRg == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + kg), "n"(kRg * 32) : "memory");
}

template <int D, int kRg, bool kBf16>
__global__ void __launch_bounds__(kThreads, Cfg<D, kRg>::ctas)
kv8_attn_kernel(const __grid_constant__ Kv8AttnArgs a) {
  using C = Cfg<D, kRg>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RangeSmem<kWarps> rsm;
  __shared__ float row_max[C::kgs][C::unit], row_sum[C::kgs][C::unit];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int kg = warp / kRg, rq = warp % kRg;  // key group, row group
  pdl_trigger();
  if (blockIdx.x == 0) kv8_check_batch(a.c);
  const Range rg = find_range<typename C::Work, kWarps>(a, blockIdx.x, gridDim.x, rsm);
  if (rg.s < 0) return;

  uint8_t* ring = smem + kg * (C::stages * C::stage);
  float* ring_scale = reinterpret_cast<float*>(smem + C::ring) + kg * (C::stages * 4);
  const uint32_t ring_u = smem_u32(ring), scale_u = smem_u32(ring_scale);
  const int page_mask = (1 << a.c.page_shift) - 1;
  float* part =
      reinterpret_cast<float*>(a.scratch) + (size_t)blockIdx.x * 2 * part_floats(C::unit, D);

  Walk<typename C::Work> w;
  if (!w.start(a, rg)) return;
  do {
    const int i0 = w.first_row(), nrow = w.rows(a.G);

    // ---- this lane's two rows of Q (g and g + 8) ----
    uint32_t qf[D / 16][4];
    float crow[2];       // logit factor of the row, without the block's K scale
    int rlo[2], rhi[2];  // tokens the row sees
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = rq * 16 + g + 8 * r;
      const bool ok = row < nrow;
      const int tok = i0 + (ok ? row : 0) / a.G, head = w.h * a.G + (ok ? row % a.G : 0);
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          static_cast<const uint16_t*>(a.q) + (int64_t)(w.d.row0 + tok) * a.q_stride +
          (int64_t)head * D);
      uint32_t x[D / 64][8];
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint4 t = ok ? __ldg(reinterpret_cast<const uint4*>(src + 32 * j + 8 * c + 4 * hf))
                             : make_uint4(0, 0, 0, 0);
          x[j][4 * hf] = t.x;
          x[j][4 * hf + 1] = t.y;
          x[j][4 * hf + 2] = t.z;
          x[j][4 * hf + 3] = t.w;
        }
      }
      crow[r] = a.scale_log2;
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
      // k-step 4 j + i contracts channels 64 j + 16 c + 4 i .. + 3
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qf[4 * j + i][r] = x[j][2 * i];
          qf[4 * j + i][2 + r] = x[j][2 * i + 1];
        }
      rlo[r] = w.u.lo;
      rhi[r] = w.u.hi;
      if (a.causal && ok) {
        const int64_t p = (int64_t)w.d.len - w.d.n + tok;
        rhi[r] = (int)max((int64_t)0, min((int64_t)w.u.hi, p + 1));
        if (a.window > 0) rlo[r] = (int)max((int64_t)rlo[r], p - a.window + 1);
      }
    }

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float mrow[2] = {-INFINITY, -INFINITY}, lrow[2] = {0.0f, 0.0f};

    const int32_t* table = a.c.table + (int64_t)w.s * a.c.max_pages;
    // page ids of a tile's two 16-key halves (one page where pages are longer);
    // -1: nothing of the half is seen, or the entry is outside the cache
    auto tile_page = [&](int t) -> int {
      const int key = (w.u.g0 + t) * C::granule + kg * kTileKeys + (lane & 16);
      int p = -1;
      if (t < w.t1 && key < w.u.hi && key + 16 > w.u.lo) {
        p = table[key >> a.c.page_shift];
        if (p < 0 || p >= a.c.n_pages) {
          set_status(a.c.status, kStatusBadIndex);
          p = -1;
        }
      }
      return p;
    };
    auto load_tile = [&](int t, int pid) {
      const int st = (t - w.t0) % C::stages;
      const int p0 = __shfl_sync(0xffffffffu, pid, 0), p1 = __shfl_sync(0xffffffffu, pid, 16);
      if (t < w.t1) {
        const int key0 = (w.u.g0 + t) * C::granule + kg * kTileKeys;
        const uint32_t kd = ring_u + st * C::stage, vd = kd + C::tile;
        constexpr int kCh = D / 16;              // 16-byte chunks per key
        constexpr int kPerIt = 32 / kCh;         // keys per instruction
        constexpr int kMine = kTileKeys / kRg;   // keys that this warp copies
#pragma unroll
        for (int it = 0; it < kMine / kPerIt; ++it) {
          const int r = rq * kMine + it * kPerIt + lane / kCh, ch = lane % kCh;
          const int key = key0 + r;
          const int p = r < 16 ? p0 : p1;
          const bool ok = p >= 0 && key >= w.u.lo && key < w.u.hi;
          const int64_t off =
              ok ? ((((int64_t)p * a.c.H_kv + w.h) << a.c.page_shift) + (key & page_mask)) * D + ch * 16
                 : 0;
          const uint32_t so = tile_off<D>(r, ch);
          copy16(kd + so, a.c.k + off, ok);
          copy16(vd + so, a.c.v + off, ok);
        }
        if (rq == 0 && lane < 4) {  // ks of half 0, 1, vs of half 0, 1
          const int p = (lane & 1) ? p1 : p0;
          const bool ok = p >= 0;
          const int64_t off = ok ? (int64_t)p * a.c.H_kv + w.h : 0;
          copy4(scale_u + (st * 4 + lane) * 4, ((lane & 2) ? a.c.v_scale : a.c.k_scale) + off, ok);
        }
      }
      copy_commit();
    };

    int pid_next = tile_page(w.t0);
    uint32_t live = 0;  // two bits per stage: its halves hold a page
#pragma unroll
    for (int i = 0; i < C::stages - 1; ++i) {
      const int pid = pid_next;
      pid_next = tile_page(w.t0 + i + 1);
      load_tile(w.t0 + i, pid);
      const uint32_t b = __ballot_sync(0xffffffffu, pid >= 0);
      live |= ((b & 1u) | ((b >> 15) & 2u)) << (2 * i);
    }
    for (int t = w.t0; t < w.t1; ++t) {
      const int rel = t - w.t0, st = rel % C::stages;
      copy_wait<C::stages - 2>();
      // the group's copies of tile t are there, and it is done with tile t - 1,
      // whose stage takes the next copies
      group_sync<kRg>(kg);
      {
        const int pid = pid_next;
        pid_next = tile_page(t + C::stages);
        load_tile(t + C::stages - 1, pid);
        const int ns = (rel + C::stages - 1) % C::stages;
        const uint32_t b = __ballot_sync(0xffffffffu, pid >= 0);
        live = (live & ~(3u << (2 * ns))) | (((b & 1u) | ((b >> 15) & 2u)) << (2 * ns));
      }
      const uint32_t halves = (live >> (2 * st)) & 3u;
      if (halves != 0) {
        const uint8_t* kt = ring + st * C::stage;
        const uint32_t vt = ring_u + st * C::stage + C::tile;
        const int key0 = (w.u.g0 + t) * C::granule + kg * kTileKeys;
        // ---- S = Q K^T ----
        float sc[4][4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;
          const int r = nt * 8 + key_of<D>(g);
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            const uint4 b = *reinterpret_cast<const uint4*>(kt + tile_off<D>(r, 4 * j + c));
            const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma16816(sc[nt], qf[4 * j + i], e4m3x2_to_f16x2((uint16_t)(bw[i] & 0xFFFFu)),
                       e4m3x2_to_f16x2((uint16_t)(bw[i] >> 16)));
          }
        }
        // ---- block scales, masks, running maximum ----
        const float4 bs = *reinterpret_cast<const float4*>(ring_scale + st * 4);
        const float ks[2] = {bs.x, bs.y};
        const float lv[2] = {(halves & 1u) ? __log2f(bs.z) : 0.0f, (halves & 2u) ? __log2f(bs.w) : 0.0f};
        const float rv[2] = {(halves & 1u) ? 1.0f / bs.z : 0.0f, (halves & 2u) ? 1.0f / bs.w : 0.0f};
        float tmax[2] = {-INFINITY, -INFINITY};
        const bool whole = halves == 3u && key0 >= max(rlo[0], rlo[1]) &&
                           key0 + kTileKeys <= min(rhi[0], rhi[1]);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const int hf = nt >> 1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = e >> 1;
            float x = fmaf(sc[nt][e], crow[r] * ks[hf], lv[hf]);
            if (!whole) {
              const int key = key0 + nt * 8 + key_of<D>(2 * c + (e & 1));
              if (key < rlo[r] || key >= rhi[r] || !((halves >> hf) & 1u)) x = -INFINITY;
            }
            sc[nt][e] = x;
            tmax[r] = fmaxf(tmax[r], x);
          }
        }
        float alpha[2], mu[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x = tmax[r];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          const float m = fmaxf(mrow[r], x), z = m == -INFINITY ? 0.0f : m;
          mu[r] = z - kHeadroom;
          alpha[r] = ex2(mrow[r] - z);
          mrow[r] = m;
        }
        // ---- weights ----
        float ls[2][2] = {};
        uint32_t pf[2][4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2(sc[nt][e] - mu[e >> 1]);
            ls[nt >> 1][e >> 1] += p[e];
          }
          pf[nt >> 1][(nt & 1) * 2] = pack_f16(p[0], p[1]);
          pf[nt >> 1][(nt & 1) * 2 + 1] = pack_f16(p[2], p[3]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
          lrow[r] = fmaf(lrow[r], alpha[r], fmaf(ls[0][r], rv[0], ls[1][r] * rv[1]));
        if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= alpha[0];
            o[i][1] *= alpha[0];
            o[i][2] *= alpha[1];
            o[i][3] *= alpha[1];
          }
        }
        // ---- O += P V ----
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const int r = kk * 16 + ((lane >> 3) & 1) * 8 + key_of<D>(lane & 7);
#pragma unroll
          for (int cb = 0; cb < D / 16; cb += 2) {
            uint32_t v[4];
            asm volatile(
                "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                : "r"(vt + tile_off<D>(r, cb + (lane >> 4)))
                : "memory");
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              // bytes (key, channel): (2c, 2g) (2c, 2g+1) (2c+1, 2g) (2c+1, 2g+1)
              const uint32_t x0 = __byte_perm(v[2 * b], 0, 0x3120);
              const uint32_t x1 = __byte_perm(v[2 * b + 1], 0, 0x3120);
              mma16816(o[2 * (cb + b)], pf[kk], e4m3x2_to_f16x2((uint16_t)(x0 & 0xFFFFu)),
                       e4m3x2_to_f16x2((uint16_t)(x1 & 0xFFFFu)));
              mma16816(o[2 * (cb + b) + 1], pf[kk], e4m3x2_to_f16x2((uint16_t)(x0 >> 16)),
                       e4m3x2_to_f16x2((uint16_t)(x1 >> 16)));
            }
          }
        }
      }
    }
    copy_wait<0>();

    // ---- join the key groups ----
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      lrow[r] += __shfl_xor_sync(0xffffffffu, lrow[r], 1);
      lrow[r] += __shfl_xor_sync(0xffffffffu, lrow[r], 2);
      if (c == 0) {
        row_max[kg][rq * 16 + g + 8 * r] = mrow[r];
        row_sum[kg][rq * 16 + g + 8 * r] = lrow[r];
      }
    }
    __syncthreads();  // every warp is done with its ring
    float* obuf = reinterpret_cast<float*>(smem);  // [key group][row][D]
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = rq * 16 + g + 8 * r;
      float m = row_max[0][row];
#pragma unroll
      for (int i = 1; i < C::kgs; ++i) m = fmaxf(m, row_max[i][row]);
      const float f = ex2(mrow[r] - (m == -INFINITY ? 0.0f : m));
      float* dst = obuf + ((size_t)kg * C::unit + row) * D;
#pragma unroll
      for (int cb = 0; cb < D / 16; ++cb)
        *reinterpret_cast<float4*>(dst + 16 * cb + 4 * c) =
            make_float4(o[2 * cb][2 * r] * f, o[2 * cb + 1][2 * r] * f, o[2 * cb][2 * r + 1] * f,
                        o[2 * cb + 1][2 * r + 1] * f);
    }
    __syncthreads();
    float* pw = part + (w.t0 == 0 ? part_floats(C::unit, D) : 0);
    constexpr int kTpr = D / 4;  // threads per row
#pragma unroll
    for (int i = 0; i < C::unit * kTpr / kThreads; ++i) {
      const int row = (i * kThreads + tid) / kTpr, ch = (tid % kTpr) * 4;
      float m = row_max[0][row];
#pragma unroll
      for (int q = 1; q < C::kgs; ++q) m = fmaxf(m, row_max[q][row]);
      const float mz = m == -INFINITY ? 0.0f : m;
      float l = 0.0f;
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < C::kgs; ++q) {
        l = fmaf(row_sum[q][row], ex2(row_max[q][row] - mz), l);
        const float4 y =
            *reinterpret_cast<const float4*>(obuf + ((size_t)q * C::unit + row) * D + ch);
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      if (row >= nrow) continue;
      if (w.whole()) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no visible token: zeros
        const int64_t orow = (int64_t)(w.d.row0 + i0 + row / a.G) * a.H + w.h * a.G + row % a.G;
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + ch) =
            make_uint2(pair_from_floats<kBf16>(x.x * inv, x.y * inv),
                       pair_from_floats<kBf16>(x.z * inv, x.w * inv));
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
    __syncthreads();  // the buffers are read before the next unit's copies
  } while (w.next(a));
}

template <int D, int kRg, bool kBf16>
__global__ void __launch_bounds__(kThreads)
kv8_merge_kernel(const __grid_constant__ Kv8AttnArgs a, int workers) {
  using C = Cfg<D, kRg>;
  merge_parts<typename C::Work, kWarps, D, kBf16>(a, workers, kHeadroom);
}

template <int D>
int grid_workers() {
  return device_sm_count() * Cfg<D, 1>::ctas;
}

template <int D, int kRg, bool kBf16>
cudaError_t attn_t(const Kv8AttnArgs& a, cudaStream_t stream) {
  using C = Cfg<D, kRg>;
  cudaError_t e = cudaFuncSetAttribute(kv8_attn_kernel<D, kRg, kBf16>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  const int workers = grid_workers<D>();
  kv8_attn_kernel<D, kRg, kBf16><<<workers, kThreads, C::smem, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  constexpr int kRowsPer = kThreads / (D / 4);
  return launch_kernel(kv8_merge_kernel<D, kRg, kBf16>, dim3(workers, C::unit / kRowsPer),
                       dim3(kThreads), 0, stream, /*pdl=*/true, a, workers);
}

template <int D, bool kBf16>
cudaError_t attn_rows(const Kv8AttnArgs& a, int row_groups, cudaStream_t stream) {
  switch (row_groups) {
    case 1: return attn_t<D, 1, kBf16>(a, stream);
    case 2: return attn_t<D, 2, kBf16>(a, stream);
    default: return attn_t<D, 4, kBf16>(a, stream);
  }
}

// Query rows of a KV head per sequence, on average.
int64_t mean_rows(int S, int T, int G) {
  return max((int64_t)G, ((int64_t)T * G + S - 1) / S);
}

}  // namespace

size_t kv8_attn_scratch_bytes(int S, int T, int H, int H_kv, int D) {
  if (D != 64 && D != 128) return 0;
  if (mean_rows(S, T, H / H_kv) > 64) return kv8_attn_tc_scratch_bytes(D);
  const int workers = D == 128 ? grid_workers<128>() : grid_workers<64>();
  return align_up((size_t)workers * 2 * part_floats(64, D) * 4, 256);
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, int type, cudaStream_t stream) {
  const int64_t rows = mean_rows(a.c.S, a.c.T, a.G);
  if (rows > 64) return launch_kv8_attn_tc(a, type, stream);
  const int rg = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  if (a.c.D == 128)
    return type == CSA2_BF16 ? attn_rows<128, true>(a, rg, stream)
                             : attn_rows<128, false>(a, rg, stream);
  return type == CSA2_BF16 ? attn_rows<64, true>(a, rg, stream)
                           : attn_rows<64, false>(a, rg, stream);
}

}  // namespace csa2
