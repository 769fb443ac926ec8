// Attention of many query rows per sequence (prompts and prompt chunks) over
// the 8-bit paged KV cache, on the 5th-generation tensor cores.  The arithmetic
// is that of the kernel for few rows (kv8_attn.cu): rows scaled by powers of
// two, block scales in the exponent, weights in fp16, sums and maxima in fp32.
//
// One persistent CTA per SM walks its range of units (kv8_sched.cuh): a unit is
// a KV head's query rows of a block, two tiles of 128 rows (row = token x G +
// head), against tiles of 128 keys:
//   S_t[row][key]  = sum_c Q_t[row][c] K[key][c]     A = Q_t (shared memory), B = K
//   O_t[row][c]   += sum_key P_t[row][key] V[key][c] A = P_t (tensor memory), B = V MN-major
// Tensor memory holds S_0, S_1 (128 columns each; P_t overwrites S_t as fp16)
// and O_0, O_1 (D columns each).  While the softmax of one row tile runs, the
// tensor pipe works on the other: O_0(j) S_0(j+1) O_1(j) S_1(j+1).
//
// Warp roles (512 threads):
//   warps 0-3, 4-7  softmax of row tile 0, 1: a thread owns a row (a tensor-memory
//                   lane), so row maxima and sums need no exchange.  The reference
//                   maximum is lazy: weights are formed in one pass with the old
//                   reference, which gives a logit at the reference a weight of 2^7;
//                   only where they grow past fp16's range (seen from their sums)
//                   does it move, O is rescaled and the weights are formed again.
//                   It moves to the largest logit, whose weight is exact then; in a
//                   tile's second half by whole powers of two, so that the fp16 weights
//                   of the first half are scaled without a second rounding
//   warps 8-11      dequantisers: E4M3 codes to fp16, 128-byte swizzled, double
//                   buffered; keys that no row of the unit may see, and those of
//                   pages outside the cache, become zeros
//   warps 12, 14    issue the MMAs of row tile 0, 1 (12: tensor memory too).  An
//                   issuing warp is held until the tensor pipe has room, so that one
//                   warp would come late to every barrier: the second issuer took
//                   the chunk below from 825 to 787 us
//   warp 13         loader: the block table and scales, and the codes of a tile's
//                   pages into shared memory by bulk copies (through L2, where the
//                   units of a sequence share them); a tile's K is requested while
//                   its predecessor's V is converted and the reverse
//   (warp 15 only completes its warpgroup, for the register split)
// Measured (GB300; cuBLAS bf16 1.89 PFLOP/s): a chunk of 4096 rows over 16K tokens
// (32 heads over 8, D = 128) 776 us, 1.24 PFLOP/s of products that the mask leaves,
// 65 %; tensor pipe 55 % busy, XU 28 %, 47 % of issue slots.  A tile of keys takes
// 3300 to 3700 cycles, of which its MMAs 2048 (D = 128); each row tile goes through
// softmax (1950 cycles, two warps a scheduler), P to O, S again, one after the other,
// since P overwrites S.  Prompts of 10007 rows through a window of 1024 (16 heads
// over 4, D = 64): 102 us.  There a unit has 8 clean tiles (softmax-bound as above:
// D = 64 halves only the MMAs), 2 to 3 at the mask's edges with 1200 cycles more, and
// 5000 cycles from its last tile to the next unit's first.
// Before the loader had a warp of its own (the dequantisers looked up pages and
// scales and loaded to registers): 6600 cycles a pair of tiles, 3000 of them in
// those dependent loads.
// V scales far apart (kv8_sched.cuh): the loader marks such a tile, the softmax scales O
// and adds the groups of 16 keys by phases.  Ordinary tiles pay for the check: prompts
// through the window 97 -> 102 us, the chunk nothing.
// Every wait is bounded (about 2 s): a role that gives up sets the timeout
// status and leaves, the others follow, and tensor memory is freed.
#include "kv8_sched.cuh"
#include "tc_common.cuh"

namespace csa2 {
namespace {

using namespace kv8;
using namespace tc;

constexpr int kSoftWarps = 8, kDeqWarp0 = 8, kDeqWarps = 4, kMmaWarp = 12, kLoadWarp = 13,
              kMmaWarp1 = 14;
constexpr int kWarps = 16, kThreads = kWarps * 32;
// Registers a thread after the roles part (four warpgroups, 512 in all: the 128
// a thread of the launch): a softmax thread holds a row of P and a part of S.
constexpr int kSoftRegs = 184, kDeqRegs = 80, kMmaRegs = 64;
static_assert(2 * kSoftRegs + kDeqRegs + kMmaRegs <= 512, "register split");
constexpr int kUnit = 256;      // query rows of a unit
constexpr int kTileE = 128;     // keys of a tile (and rows of a row tile)
// log2 of the weight at the reference, and the largest sum of 16 weights: no weight is
// above it, which fp16 holds (65504)
constexpr float kHeadroom = 7.0f, kMostSum = 57344.0f;
// The largest reference with which exponents are formed by one fused
// multiply-add: its rounding is then at most 2^-8 of a power of two, that of the
// logits themselves.
constexpr float kFused = 65536.0f;
// (a unit's queries and output count as two granules: prompts of 10007 rows through a
// window of 1024 with one to three 104.5, 96.6, 97.6 us when they took 97)
using Work = Shape<kUnit, kTileE, 2>;
constexpr uint32_t kAtom = 128 * 128;            // bytes: 128 rows of 64 fp16 channels

template <int D>
struct Lay {
  static constexpr uint32_t tile = (D / 64) * kAtom;  // bytes of Q_t, of a K or a V stage
  static constexpr uint32_t raw = kTileE * D;         // bytes of a tile's codes of K (or V)
  static constexpr uint32_t q = 0, k = 2 * tile, v = 4 * tile, rk = 6 * tile, rv = rk + raw;
  static constexpr uint32_t ctl = rv + raw;
  static constexpr uint32_t alloc = ctl + 2048 + 1024;  // slack to align the base to 1 KiB
};
static_assert(Lay<128>::alloc <= 232448, "shared memory");

struct Ctl {
  // of a tile's 16-key groups: K scale, log2 of the V scale's ratio to the unit of O, the
  // ratio's reciprocal (0: nothing of it is seen).  Four tiles: the loader is at most one ahead of the dequantisers, which
  // are at most two ahead of the slower softmax
  float4 sc[4][8];
  int32_t marks[4];       // of a tile: kRagged, kEdge, kMoved; see there
  uint16_t phase[4][8];   // of a tile with kMoved: groups, and the power of two of O before them
  uint64_t rk_full, rk_empty, rv_full, rv_empty;  // the codes of a tile
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2];
  uint64_t phase_ready[2], phase_done[2];
  uint8_t phases[kSoftWarps];  // waits of each warp for phase_done so far
  int32_t* status;
  uint64_t done;
  Walk<Work> walk[kMmaWarp1 + 1];  // each warp's own (kept out of registers)
  uint32_t tmem;
};
static_assert(sizeof(Ctl) <= 2048, "control block");

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(su32(bar), parity, status));
}

template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Arrives for the warp: its generic writes to shared memory (read by the tensor
// cores) and its tensor-memory accesses come before.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  proxy_fence();
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(su32(bar));
}

// One lane of the warp.  The tensor-core instructions stand in a branch on it: the
// compiler then keeps their operands in uniform registers.  Measured for eight
// MMAs of 128 x 128 x 16 in a row: 283 cycles to issue them so, 566 behind
// `lane == 0`, 725 as a loop with the instruction predicated.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}"
               : "=r"(p));
  return p != 0;
}
// Instruction descriptor of P to O: B (V) MN-major.
__device__ __forceinline__ uint32_t idesc_o(int D) { return idesc_f16(D, false) | (1u << 16); }
// MMA with A from tensor memory.
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

#define CSA2_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), \
                      "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define CSA2_I8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), \
                      "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
// 32 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : CSA2_R8(x, 0), CSA2_R8(x, 8), CSA2_R8(x, 16), CSA2_R8(x, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      CSA2_I8(x, 0), CSA2_I8(x, 8), CSA2_I8(x, 16), CSA2_I8(x, 24)
      : "memory");
}

// Waits for the loads from tensor memory; x is theirs.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]),
                 "+r"(x[6]), "+r"(x[7]), "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]),
                 "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]), "+r"(x[16]), "+r"(x[17]),
                 "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]), "+r"(x[23]),
                 "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27]), "+r"(x[28]), "+r"(x[29])
               :
               : "memory");
  asm volatile("" : "+r"(x[30]), "+r"(x[31]));
}

// Pairs of fp32 operations in one instruction.
struct F2 {
  float lo, hi;
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.lo), "=f"(r.hi)
      : "f"(a.lo), "f"(a.hi), "f"(b.lo), "f"(b.hi), "f"(c.lo), "f"(c.hi));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.lo), "=f"(r.hi)
      : "f"(a.lo), "f"(a.hi), "f"(b.lo), "f"(b.hi));
  return r;
}

// Marks of a tile: keys that no row of the unit sees; keys that some rows see and
// others do not; V scales that the unit 2^E of O has to follow.  From bit 16 on E + 128,
// behind the tile; with kMoved also, from bit 4, the number of phases in which P to O runs
// (the groups of a phase share an E; between two the softmax scales O) and, from bit 8, the
// groups whose values are left out (their weights are zeros: a NaN among them is seen).
constexpr int kRagged = 1, kEdge = 2, kMoved = 4;

// Columns of S (a tile's, from address ts) outside the row's [lo, hi) become
// -infinity.  Not inlined: the code of the roles shares the SM's instruction cache,
// and the softmax keeps its registers.
__device__ __noinline__ void mask_tile(uint32_t ts, int lo, int hi) {
#pragma unroll 1
  for (int i = 0; i < kTileE; i += 32) {
    if (!__any_sync(0xffffffffu, lo > i || hi < i + 32)) continue;
    const int l = max(0, min(32, lo - i)), h = max(0, min(32, hi - i));
    const uint32_t seen = __funnelshift_lc(0xFFFFFFFFu, 0u, h) & __funnelshift_lc(0u, 0xFFFFFFFFu, l);
    uint32_t x[32];
    tmem_ld32(ts + i, x);
    tmem_wait_ld32(x);
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (!((seen >> k) & 1)) x[k] = 0xFF800000u;
    tmem_st32(ts + i, x);
  }
  tmem_wait_st();
}

// O's row (from address to) times f.
template <int D>
__device__ __noinline__ void scale_o(uint32_t to, float f) {
#pragma unroll 1
  for (int i = 0; i < D; i += 16) {
    float o[16];
    tmem_ld16(to + i, o);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] *= f;
    tmem_st16(to + i, o);
  }
}
// Zeros into 8, 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_zero8(uint32_t addr) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(addr),
               "r"(0)
               : "memory");
}
__device__ __forceinline__ void tmem_zero32(uint32_t addr) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,"
      "%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(addr),
      "r"(0)
      : "memory");
}

// `bytes` contiguous bytes of global memory into shared memory, completing on bar.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
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

// 16 E4M3 codes -> fp16, into 16-byte chunks 2 c4, 2 c4 + 1 of key e of an atom.
__device__ __forceinline__ void put16(uint8_t* atom, int e, int c4, uint4 w) {
  uint8_t* row = atom + (e >> 3) * 1024 + (e & 7) * 128;
  const uint2 a = e4m3x4_to_f16x4(w.x), b = e4m3x4_to_f16x4(w.y);
  const uint2 c = e4m3x4_to_f16x4(w.z), d = e4m3x4_to_f16x4(w.w);
  *reinterpret_cast<uint4*>(row + (((2 * c4) ^ (e & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
  *reinterpret_cast<uint4*>(row + (((2 * c4 + 1) ^ (e & 7)) << 4)) = make_uint4(c.x, c.y, d.x, d.y);
}

// 32 rows of a unit's Q (from row `first`), scaled to a largest magnitude in [1, 2),
// into the warp's part of their row tile; returns the exponent of the lane's row.
// D / 8 lanes take a row (a lane that takes a row of its own touches 32 lines an
// instruction).  Not inlined: the softmax keeps its registers.
template <int D, bool kBf16>
__device__ __noinline__ int load_rows(const Kv8AttnArgs& a, uint8_t* qt, int first, int row0,
                                      int head0, int nrow) {
  constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // lanes a row, rows an instruction
  const int lane = threadIdx.x & 31;
  int e = 0;
#pragma unroll 1
  for (int b = 0; b < 32; b += 8 * kAt) {
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = first + b + kAt * i + lane / kLanes, rt = over_g(a, r);
      x[i] = r < nrow ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                            (int64_t)(row0 + rt) * a.q_stride +
                                                            (int64_t)(head0 + r - rt * a.G) * D) +
                              lane % kLanes)
                      : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      if (kBf16) {
        float mx = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = pair_to_float2<true>(y[j]);
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const int E = row_exponent(mx);
        const int mine = __shfl_sync(0xffffffffu, E, (lane % kAt) * kLanes);
        if (lane / kAt == b / kAt + i) e = mine;
        const float down = pow2f(-E);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = pair_to_float2<true>(y[j]);
          y[j] = pack_f16(f.x * down, f.y * down);
        }
      }
      *reinterpret_cast<uint4*>(qt + sw128_off((first & 127) + b + kAt * i + lane / kLanes,
                                               8 * (lane % kLanes), kAtom)) =
          make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  return e;
}

// The loader's warp, for a tile with V scales that are not near the unit of O (lane g < 8
// has group g's; live: the groups that are seen): the lane's ratio, the lane's phase, and
// what the tile's marks say of them.
struct Phases {
  VUnit u;
  float ratio;
  int phase, marks;
};
__device__ __noinline__ Phases phases_of(VUnit u, float vs, uint32_t live) {
  const int lane = threadIdx.x & 31, e = unit_exp(vs);
  float ratio = 1.0f;
  int phase = 0;
  uint32_t todo = live, far = 0;
  int n = 0;
  while (todo) {
    auto near = [&]() {
      return __ballot_sync(0xffffffffu, ((todo >> lane) & 1) && e >= u.e - 4 && e <= u.e + 3);
    };
    uint32_t now = near();
    int by = 0;
    if (!now) {  // to the first of them
      const int l = __ffs(todo) - 1, was = u.e;
      float factor;
      bool left_out;
      follow(u, __shfl_sync(0xffffffffu, vs, l), factor, left_out);
      if (left_out) {
        far |= 1u << l;
        todo &= ~(1u << l);
        continue;
      }
      by = max(-127, was - u.e);
      now = near();
    }
    if (lane == n) phase = (int)now | ((by & 0xFF) << 8);
    if ((now >> lane) & 1) ratio = vs * pow2f(-u.e);
    todo &= ~now;
    ++n;
  }
  return {u, ratio, phase, kMoved | (max(n, 1) << 4) | (int)(far << 8)};
}

// A tile with kMoved, its softmax warps with their weights written: P to O of all phases
// but the last, and the weights of their groups zero after it, so that the issuer adds
// the last one as it does any tile.  False: a wait gave up.  (Not inlined, with what it
// needs in shared memory, and nothing of it in the issuers' loop: the roles share the SM's
// instruction cache and the softmax has no register to spare.  A branch on the marks in
// the issuers' loop cost the chunk below 3 %, more arguments here 2 %.)
template <int D>
__device__ __noinline__ bool add_phases(Ctl& ctl, uint32_t it) {
  const int warp = threadIdx.x >> 5, t = warp >> 2;
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t ts = ctl.tmem + t * 128, to = ctl.tmem + 256 + t * D;
  const int marks = ctl.marks[it & 3], n = (marks >> 4) & 15;
  int zero = (marks >> 8) & 0xFF;  // groups without weight from here on
  for (int i = 0;; ++i) {
#pragma unroll 1
    for (int g = 0; g < 8; ++g)
      if ((zero >> g) & 1) tmem_zero8(ts + lane_base + 8 * g);
    const int phase = ctl.phase[it & 3][i], by = (int8_t)(phase >> 8);
    if (by != 0) scale_o<D>(to + lane_base, pow2_or_zero(by));
    tmem_wait_st();
    if (i + 1 == n) return true;
    const uint32_t parity = ctl.phases[warp] & 1u;
    warp_arrive(&ctl.phase_ready[t]);
    if ((warp & 3) == 0) {
      if (!warp_wait(&ctl.phase_ready[t], parity, ctl.status) ||
          !warp_wait(&ctl.v_full[it & 1u], (it >> 1) & 1u, ctl.status))
        return false;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t v = su32(&ctl) - Lay<D>::ctl + Lay<D>::v + (it & 1u) * Lay<D>::tile;
        const uint64_t vb = sw128_desc(v, kAtom, 1024);
#pragma unroll 1
        for (int x = 0; x < 8; ++x)
          if ((phase >> x) & 1) mma_f16_ta(to, ts + 8 * x, vb + x * (2048 >> 4), idesc_o(D), 1);
        mma_commit(su32(&ctl.phase_done[t]));
      }
      __syncwarp();
    }
    if (!warp_wait(&ctl.phase_done[t], parity, ctl.status)) return false;
    tc_fence_after();
    if ((threadIdx.x & 31) == 0) ++ctl.phases[warp];
    __syncwarp();
    zero = phase & 0xFF;
  }
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
kv8_attn_tc_kernel(const __grid_constant__ Kv8AttnArgs a) {
  using L = Lay<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = su32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + L::ctl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* status = a.c.status;
  pdl_trigger();
  // (in the loader's space, which is free until the roles part)
  RangeSmem<kWarps>& rsm = *reinterpret_cast<RangeSmem<kWarps>*>(smem + L::rk);
  const Range rg = find_range<Work, kWarps>(a, blockIdx.x, gridDim.x, rsm);
  Walk<Work>& w = ctl.walk[min(warp, kMmaWarp1)];
  bool any = false;
  if (warp <= kMmaWarp1) any = warp_start(w, a, rg, rsm);
  proxy_fence();  // (of the range's record, before the loader's copies land on it)
  if (!__syncthreads_or(any)) {  // no range, or one that ends within a unit's fixed cost
    if (tid == 0) write_cut(a, Cut{-1, 0, 0, 0});
    return;
  }

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
        su32(&ctl.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(su32(&ctl.q_full[i]), 4);
      mbar_init(su32(&ctl.p_full[i]), 4);
      mbar_init(su32(&ctl.k_full[i]), kDeqWarps);
      mbar_init(su32(&ctl.v_full[i]), kDeqWarps);
      mbar_init(su32(&ctl.k_empty[i]), 2);
      mbar_init(su32(&ctl.v_empty[i]), 2);
      mbar_init(su32(&ctl.s_full[i]), 1);
      mbar_init(su32(&ctl.o_full[i]), 1);
      mbar_init(su32(&ctl.phase_ready[i]), 4);
      mbar_init(su32(&ctl.phase_done[i]), 1);
    }
    for (int i = 0; i < kSoftWarps; ++i) ctl.phases[i] = 0;
    ctl.status = status;
    mbar_init(su32(&ctl.done), 2);
    mbar_init(su32(&ctl.rk_full), 1);
    mbar_init(su32(&ctl.rv_full), 1);
    mbar_init(su32(&ctl.rk_empty), kDeqWarps);
    mbar_init(su32(&ctl.rv_empty), kDeqWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm_s = ctl.tmem, tm_o = ctl.tmem + 256;
  uint32_t it = 0;  // tiles of keys so far, over all units
  bool alive = true;

  if (warp < kSoftWarps) {
    // ================= softmax =================
    more_registers<kSoftRegs>();
    const int t = warp >> 2, quad = warp & 3;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t ts = tm_s + t * 128 + lane_base, to = tm_o + t * D + lane_base;
    const int row = t * 128 + quad * 32 + lane;
    uint8_t* qt = smem + L::q + t * L::tile;
    uint32_t cnt = 0, units = 0;
    // the unit's row of this thread
    bool ok;
    int64_t orow;       // of out, lse
    float crow;         // logit factor, without the block's K scale
    int rlo, rhi;       // tokens it sees
    // To the next unit that has row tile t (`first`: this one, if it has it).
    auto advance = [&](bool first) -> bool {
      while (true) {
        if (!first && !warp_next(w, a)) return false;
        first = false;
        if (t == 0 || w.rows(a.G) > 128) return true;
        it += w.t1 - w.t0;
      }
    };
    auto load_q = [&]() {
      const int i0 = w.first_row(), nrow = w.rows(a.G);
      ok = row < nrow;
      const int tok = i0 + (ok ? row : 0) / a.G, head = w.h * a.G + (ok ? row % a.G : 0);
      orow = (int64_t)(w.d.row0 + tok) * a.H + head;
      crow = a.scale_log2 * pow2f(load_rows<D, kBf16>(a, qt, row & ~31, w.d.row0 + i0, w.h * a.G, nrow));
      warp_arrive(&ctl.q_full[t]);
      rlo = w.u.lo;
      rhi = w.u.hi;
      if (a.causal && ok) {
        const int64_t p = (int64_t)w.d.len - w.d.n + tok;
        rhi = (int)max((int64_t)0, min((int64_t)w.u.hi, p + 1));
        if (a.window > 0) rlo = (int)max((int64_t)rlo, p - a.window + 1);
      }
    };
    bool have = advance(true);
    if (have) load_q();
#pragma unroll 1
    for (int i = 0; i < D; i += 32) tmem_zero32(to + i);
    while (have) {
      const int t0 = w.t0, t1 = w.t1;
      float m_ref = -INFINITY, l = 0.0f;
      int marks = 0;
      for (int j = t0, key0 = (w.u.g0 + t0) * kTileE; j < t1; ++j, ++it, ++cnt, key0 += kTileE) {
        if (!warp_wait(&ctl.s_full[t], cnt & 1u, status)) {
          alive = false;
          break;
        }
        tc_fence_after();
        const float4* sc = ctl.sc[it & 3];
        if (__any_sync(0xffffffffu, key0 < rlo || key0 + kTileE > rhi)) {
          mask_tile(ts, rlo - key0, rhi - key0);
        }
        // two halves of 64 keys (a loop: the code of all roles shares the SM's
        // instruction cache, and unrolled it misses)
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          // with a reference (and logits small enough for the fused form below to be
          // as exact as they are): the weights in one pass
          bool slow = __any_sync(0xffffffffu, !(fabsf(m_ref) <= kFused));
          if (!slow) {
            uint32_t p[32], s[2][32];
            const float base = m_ref - kHeadroom;
            float sum = 0.0f, most = 0.0f;  // `most`: the largest sum of a group
            tmem_ld32(ts + 64 * half, s[0]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t* x = s[i];
              tmem_wait_ld32(x);
              if (i == 0) tmem_ld32(ts + 64 * half + 32, s[1]);
#pragma unroll
              for (int gi = 0; gi < 2; ++gi) {
                const float4 b = sc[4 * half + 2 * i + gi];
                const float c = fmaxf(crow * b.x, 1.17549435e-38f), d = b.y - base;
                F2 part[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  const F2 y = fma2(
                      {__uint_as_float(x[16 * gi + k]), __uint_as_float(x[16 * gi + k + 1])}, {c, c},
                      {d, d});
                  const F2 w2 = {ex2(y.lo), ex2(y.hi)};
                  part[(k >> 1) & 1] = add2(part[(k >> 1) & 1], w2);
                  p[16 * i + 8 * gi + k / 2] = pack_f16(w2.lo, w2.hi);
                }
                const F2 both = add2(part[0], part[1]);
                const float one = both.lo + both.hi;
                most = fmaxf(most, one);
                sum = fmaf(one, b.z, sum);
              }
            }
            // a weight may leave fp16's range only in a group whose sum does
            slow = __any_sync(0xffffffffu, most > kMostSum);
            if (!slow) {
              l += sum;
              tmem_st32(ts + 32 * half, p);
            }
          }
          if (slow) {  // the reference moves to the half's largest exponent where that is past it
            // The first half's weights, and O as the first half left it, are read
            // back below: their stores are waited for (loads from tensor memory are
            // not ordered behind stores).
            tmem_wait_st();
            float x = -INFINITY;
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              uint32_t y[32];
              tmem_ld32(ts + 64 * half + 32 * i, y);
              tmem_wait_ld32(y);
#pragma unroll
              for (int gi = 0; gi < 2; ++gi) {
                const float4 b = sc[4 * half + 2 * i + gi];
                float mx = __uint_as_float(y[16 * gi]);
#pragma unroll
                for (int k = 1; k < 16; ++k) mx = fmaxf(mx, __uint_as_float(y[16 * gi + k]));
                x = fmaxf(x, fmaf(mx, fmaxf(crow * b.x, 1.17549435e-38f), b.y));
              }
            }
            // in the second half by whole powers of two, so that the first half's weights keep
            // their bits (past 2^64 nothing of them is left)
            float up = fmaxf(m_ref, x);
            if (half == 1 && up - m_ref < 64.0f) up = m_ref + ceilf(up - m_ref);
            const float alpha = up > m_ref ? ex2(m_ref - up) : 1.0f;
            m_ref = up;
            l *= alpha;
            // S_t(j) is done, so O_t(j - 1), issued before it, is too
            if (j > t0) scale_o<D>(to, alpha);
            if (half == 1) {  // the first half's weights had the old reference
              uint32_t y[32];
              tmem_ld32(ts, y);
              tmem_wait_ld32(y);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const float2 f = half2_bits_to_float2(y[k]);
                y[k] = pack_f16(f.x * alpha, f.y * alpha);
              }
              tmem_st32(ts, y);
            }
            // the weights, the reference subtracted from the rounded exponent: the largest
            // logit's weight is exact however large it is.  P's columns are those of
            // keys that have been read
            const float base = (m_ref == -INFINITY ? 0.0f : m_ref) - kHeadroom;
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              uint32_t y[32];
              float p[16];
              tmem_ld32(ts + 64 * half + 32 * i, y);
              tmem_wait_ld32(y);
#pragma unroll
              for (int gi = 0; gi < 2; ++gi) {
                const float4 b = sc[4 * half + 2 * i + gi];
                const float c = fmaxf(crow * b.x, 1.17549435e-38f);
                float one = 0.0f;
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  const float w0 = ex2(fmaf(__uint_as_float(y[16 * gi + k]), c, b.y) - base);
                  const float w1 = ex2(fmaf(__uint_as_float(y[16 * gi + k + 1]), c, b.y) - base);
                  one += w0 + w1;
                  p[8 * gi + k / 2] = __uint_as_float(pack_f16(w0, w1));
                }
                l = fmaf(one, b.z, l);
              }
              tmem_st16(ts + 32 * half + 16 * i, p);
            }
          }
        }
        marks = ctl.marks[it & 3];
        tmem_wait_st();
        if (marks & kMoved) {
          alive = add_phases<D>(ctl, it);
          if (!alive) break;
        }
        warp_arrive(&ctl.p_full[t]);
      }
      if (!alive) break;
      // the next unit's Q (every S_t of this one is done): its first product runs
      // while this unit's output is written
      const bool whole = w.whole(), out_ok = ok;
      const int64_t out_row = orow;
      have = advance(false);
      if (have) load_q();
      if (!warp_wait(&ctl.o_full[t], units & 1u, status)) {
        alive = false;
        break;
      }
      ++units;
      tc_fence_after();
      // ---- output, or a part of it ----
      // no visible token: zeros
      const float inv = l == 0.0f ? 0.0f : (whole ? 1.0f : kPartOut) / l;
      float f = inv;
      const int e = (marks >> 16) - 128;
      if (abs(e) <= 60) {
        f *= pow2f(e);
      } else {  // (one number need not hold both)
        scale_o<D>(to, inv);
        tmem_wait_st();
        f = pow2_or_zero(e);
      }
      float* part = scratch_part(a, gridDim.x, blockIdx.x, t0 == 0, kUnit, D);
#pragma unroll 1
      for (int i = 0; i < D; i += 32) {
        uint32_t o[32];
        tmem_ld32(to + i, o);
        tmem_wait_ld();
        tmem_zero32(to + i);  // for the next unit
        if (!out_ok) continue;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + out_row * D + i);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
              y[n] = pair_from_floats<kBf16>(__uint_as_float(o[8 * k + 2 * n]) * f,
                                             __uint_as_float(o[8 * k + 2 * n + 1]) * f);
            dst[k] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(part + (size_t)row * D + i);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t y[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
              y[n] = __float_as_uint(__uint_as_float(o[4 * k + n]) * f);
            dst[k] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      if (out_ok) {
        if (whole) {
          if (a.lse)
            a.lse[out_row] = l == 0.0f ? -INFINITY
                                    : ((m_ref == -INFINITY ? 0.0f : m_ref) - kHeadroom + __log2f(l)) * kLn2;
        } else {
          part[kUnit * D + row] = m_ref;
          part[kUnit * D + kUnit + row] = l;
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ================= dequantisers =================
    fewer_registers<kDeqRegs>();
    // a lane converts 16 channels (chunk c of the key's codes) of D / 16 lanes a
    // key: it reads 16 bytes and writes two 16-byte chunks of atom c / 4.  The lanes
    // of the second atom take the key beside (e ^ 1), so that the eight lanes of a
    // phase meet the eight different 16-byte slots of the swizzle in both
    constexpr int kCh = D / 16, kKeys = 32 / kCh;  // lanes a key, keys an instruction
    const int dw = warp - kDeqWarp0, c = lane % kCh, sub = (lane / kCh) ^ (c >> 2);
    do {
      const int t1 = w.t1, g0 = w.u.g0, lo = w.u.lo, hi = w.u.hi;
      for (int j = w.t0; j < t1; ++j, ++it) {
        const uint32_t st = it & 1u, par = ((it >> 1) & 1u) ^ 1u;
        const int key0 = (g0 + j) * kTileE;
#pragma unroll 1
        for (int kv = 0; kv < 2 && alive; ++kv) {  // K, V
          uint64_t* bars = kv ? &ctl.rv_full : &ctl.rk_full;  // full, empty
          uint64_t* full = kv ? ctl.v_full : ctl.k_full;
          uint64_t* empty = kv ? ctl.v_empty : ctl.k_empty;
          alive = warp_wait(bars, it & 1u, status) && warp_wait(empty + st, par, status);
          if (!alive) break;
          const int marks = ctl.marks[it & 3] & (kRagged | kEdge);
          if ((marks & kEdge) && !(alive = warp_wait(&ctl.rv_full, it & 1u, status))) break;
          const uint8_t* raw = smem + L::rk + kv * L::raw;
          uint8_t* to = smem + L::k + (2 * kv + st) * L::tile;
          if (marks == 0) {
#pragma unroll 4
            for (int i = 0; i < 32 / kKeys; ++i) {
              const int e = 32 * dw + kKeys * i + sub;
              put16(to + (c >> 2) * kAtom, e, c & 3,
                    *reinterpret_cast<const uint4*>(raw + e * D + 16 * c));
            }
          } else {
            const uint8_t* raw_v = smem + L::rv;
#pragma unroll 4
            for (int i = 0; i < 32 / kKeys; ++i) {
              const int e = 32 * dw + kKeys * i + sub;
              uint4 x = *reinterpret_cast<const uint4*>(raw + e * D + 16 * c);
              if (key0 + e < lo || key0 + e >= hi || ctl.sc[it & 3][e >> 4].z == 0.0f) {
                x = make_uint4(0, 0, 0, 0);
              } else if ((marks & kEdge) &&  // (only there have V's codes been waited for)
                         has_nan(*reinterpret_cast<const uint4*>(raw_v + e * D + 16 * c))) {
                // A weight of zero does not hide a NaN of V: where some rows see a key
                // and others do not, its V codes become zeros and its K codes NaN,
                // which the mask hides
                x = kv ? make_uint4(0, 0, 0, 0) : make_uint4(0x7F7F7F7Fu, 0, 0, 0);
              }
              put16(to + (c >> 2) * kAtom, e, c & 3, x);
            }
          }
          warp_arrive(full + st);
          if (lane == 0) mbar_arrive(su32(bars + 1));
        }
        if (!alive) break;
      }
    } while (alive && warp_next(w, a));
  } else {
    fewer_registers<kMmaRegs>();
  }
  if (warp == kLoadWarp) {
    // ================= loader =================
    // lanes 0-7: a 16-key group of the tile each; the first of a page's groups
    // (a run) requests the page's codes
    const int page = 1 << a.c.page_shift, run = min(page, kTileE);
    if (lane == 0) write_cut(a, Cut{-1, 0, 0, 0});
    const uint32_t run_bytes = (uint32_t)(run * D);
    const bool leads = lane < 8 && (16 * lane) % run == 0;
    uint32_t ks_out = 0, vs_out = 0;  // tiles whose K, V have been requested
    do {
      if (w.t0 == 0 && w.t1 < w.u.ng && lane == 0) write_cut(a, w.cut(a, rg));
      const int t1 = w.t1, g0 = w.u.g0, lo = w.u.lo, hi = w.u.hi, h = w.h;
      const int32_t* table = a.c.table + (int64_t)w.s * a.c.max_pages;
      // tokens that every row sees
      int all_lo = lo, all_hi = hi;
      if (a.causal) {
        const int first = w.d.len - w.d.n + w.first_row();
        all_hi = min(hi, first + 1);
        if (a.window > 0) all_lo = max(lo, first + min(w.d.n - w.first_row(), w.d.tpu) - a.window);
      }
      // page of the lane's group in tile j: -1 where no key of its run is seen or the
      // entry is outside the cache
      auto find = [&](int j) -> int {
        const int key = (g0 + j) * kTileE + 16 * lane, from = key & ~(run - 1);
        if (j >= t1 || lane >= 8 || from >= hi || from + run <= lo) return -1;
        const int p = table[key >> a.c.page_shift];
        if (p >= 0 && p < a.c.n_pages) return p;
        set_status(status, kStatusBadIndex);
        return -1;
      };
      VUnit vu = {kNoUnit, kNoUnit};
      float unit = 0.0f;  // 2^-E
      float ks = 0.0f, vs = 0.0f;
      auto scales = [&](int p) {
        if (p >= 0) {
          ks = __ldg(a.c.k_scale + (int64_t)p * a.c.H_kv + h);
          vs = __ldg(a.c.v_scale + (int64_t)p * a.c.H_kv + h);
        }
      };
      int pid = find(w.t0), next = find(w.t0 + 1);
      scales(pid);
      // the unit's queries, for which the softmax would wait at the unit's start
      for (int row = lane; row < w.rows(a.G); row += 32) {
        const int tok = over_g(a, row);
        const uint16_t* src = static_cast<const uint16_t*>(a.q) +
                              (int64_t)(w.d.row0 + w.first_row() + tok) * a.q_stride +
                              (int64_t)(h * a.G + row - tok * a.G) * D;
#pragma unroll
        for (int i = 0; i < D; i += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i));
      }
      for (int j = w.t0; j < t1; ++j, ++it) {
        const int key0 = (g0 + j) * kTileE, key = key0 + 16 * lane;
        const bool seen = pid >= 0 && key < hi && key + 16 > lo;
        const uint32_t all = __ballot_sync(0xffffffffu, seen || lane >= 8);
        const uint32_t live = __ballot_sync(0xffffffffu, seen);
        if (vu.e == kNoUnit && live) {
          vu.e = vu.top = unit_exp(__shfl_sync(0xffffffffu, vs, __ffs(live) - 1));
          unit = pow2f(-vu.e);
        }
        float ratio = vs * unit;
        const bool moved = __any_sync(0xffffffffu, seen && !near_unit(ratio));
        int how = 0, phase = 0;
        if (moved) {
          const Phases ph = phases_of(vu, vs, live);
          vu = ph.u;
          unit = pow2f(-vu.e);
          ratio = ph.ratio;
          how = ph.marks;
          phase = ph.phase;
        }
        const float4 sc = seen ? make_float4(ks, __log2f(ratio), 1.0f / ratio, 0.0f)
                               : make_float4(1.0f, -INFINITY, 0.0f, 0.0f);
        const int64_t off = ((((int64_t)pid * a.c.H_kv + h) << a.c.page_shift) + (key & (page - 1))) * D;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, leads && pid >= 0)) * run_bytes;
        if (!warp_wait(&ctl.rk_empty, (it & 1u) ^ 1u, status)) {
          alive = false;
          break;
        }
        if (lane < 8) {
          ctl.sc[it & 3][lane] = sc;
          if (moved) ctl.phase[it & 3][lane] = (uint16_t)phase;
        }
        if (lane == 0)
          ctl.marks[it & 3] =
              ((vu.e + 128) << 16) | how | (all != 0xffffffffu || key0 < lo || key0 + kTileE > hi ? kRagged : 0) |
              (max(key0, lo) < all_lo || min(key0 + kTileE, hi) > all_hi ? kEdge : 0);
        __syncwarp();
        if (lane == 0) mbar_expect_tx(su32(&ctl.rk_full), bytes);
        __syncwarp();
        if (leads && pid >= 0)
          bulk_load(su32(smem + L::rk) + 16 * lane * D, a.c.k + off, run_bytes, su32(&ctl.rk_full));
        ++ks_out;
        if (!warp_wait(&ctl.rv_empty, (it & 1u) ^ 1u, status)) {
          alive = false;
          break;
        }
        if (lane == 0) mbar_expect_tx(su32(&ctl.rv_full), bytes);
        __syncwarp();
        if (leads && pid >= 0)
          bulk_load(su32(smem + L::rv) + 16 * lane * D, a.c.v + off, run_bytes, su32(&ctl.rv_full));
        ++vs_out;
        pid = next;
        scales(pid);
        next = find(j + 2);
      }
    } while (alive && warp_next(w, a));
    // no copy is in flight when the CTA ends: the last ones are waited for
    if (ks_out > 0) warp_wait(&ctl.rk_full, (ks_out - 1) & 1u, status);
    if (vs_out > 0) warp_wait(&ctl.rv_full, (vs_out - 1) & 1u, status);
  }
  if (warp == kMmaWarp || warp == kMmaWarp1) {
    // ================= MMA issuers =================
    const uint32_t id_s = idesc_f16(kTileE, false);
    const uint32_t id_o = idesc_o(D);
    const int t = warp == kMmaWarp ? 0 : 1;                  // row tile
    const uint32_t sb = su32(smem), ts = tm_s + t * 128, to = tm_o + t * D;
    const uint64_t dq = sw128_desc(sb + L::q + t * L::tile, 16, 1024);
    const uint64_t dk = sw128_desc(sb + L::k, 16, 1024);
    const uint64_t dv = sw128_desc(sb + L::v, kAtom, 1024);
    uint32_t cnt = 0, units = 0;
    do {
      const int n = w.t1 - w.t0;
      const bool mine = t == 0 || w.rows(a.G) > 128;  // else the unit has one row tile
      if (mine) {
        alive = warp_wait(&ctl.q_full[t], units & 1u, status);
        ++units;
      }
      // S_t(0) of the unit, then for each tile j of keys O_t(j) and S_t(j + 1)
#pragma unroll 1
      for (int j = -1; j < n && alive; ++j) {
        const uint32_t o = it + j, s2 = o + 1;  // tiles of the CTA: of O, of S
        if (j >= 0) alive = warp_wait(&ctl.v_full[o & 1u], (o >> 1) & 1u, status);
        if (alive && j + 1 < n) alive = warp_wait(&ctl.k_full[s2 & 1u], (s2 >> 1) & 1u, status);
        if (!mine) {  // only releases the tiles
          if (alive && lane == 0) {
            if (j >= 0) mbar_arrive(su32(&ctl.v_empty[o & 1u]));
            if (j + 1 < n) mbar_arrive(su32(&ctl.k_empty[s2 & 1u]));
          }
          __syncwarp();
          continue;
        }
        if (alive && j >= 0) {  // P_t(j) is written and O_t rescaled
          alive = warp_wait(&ctl.p_full[t], cnt & 1u, status);
          ++cnt;
        }
        if (!alive) break;
        tc_fence_after();
        if (elect_one()) {
          if (j >= 0) {
            const uint64_t vb = dv + (o & 1u) * (L::tile >> 4);
#pragma unroll
            for (int x = 0; x < kTileE / 16; ++x)  // 16 keys: 8 columns of P, 2048 bytes of V
              mma_f16_ta(to, ts + 8 * x, vb + x * (2048 >> 4), id_o, 1);  // (O starts as zeros)
            mma_commit(su32(&ctl.v_empty[o & 1u]));
            if (j + 1 == n) mma_commit(su32(&ctl.o_full[t]));
          }
          if (j + 1 < n) {
            const uint64_t kb = dk + (s2 & 1u) * (L::tile >> 4);
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {  // 16 channels: 32 bytes of atom x / 4
              const uint32_t off = ((x >> 2) * kAtom + (x & 3) * 32) >> 4;
              mma_f16(ts, dq + off, kb + off, id_s, x != 0);
            }
            mma_commit(su32(&ctl.s_full[t]));
            mma_commit(su32(&ctl.k_empty[s2 & 1u]));
          }
        }
        __syncwarp();
      }
      it += n;
    } while (alive && warp_next(w, a));
    // nothing is in flight when tensor memory is freed
    if (elect_one()) mma_commit(su32(&ctl.done));
    __syncwarp();
    warp_wait(&ctl.done, 0u, status);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm_s));
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(128)
kv8_merge_tc_kernel(const __grid_constant__ Kv8AttnArgs a, int workers) {
  merge_parts<Work, D, kBf16>(a, workers, kHeadroom);
}

template <int D, bool kBf16>
cudaError_t attn_tc_t(const Kv8AttnArgs& args, cudaStream_t stream) {
  using L = Lay<D>;
  Kv8AttnArgs a = args;
  a.tpu = kUnit / a.G;
  cudaError_t e = cudaFuncSetAttribute(kv8_attn_tc_kernel<D, kBf16>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, L::alloc);
  if (e != cudaSuccess) return e;
  const int workers = device_sm_count();
  e = launch_kernel(kv8_attn_tc_kernel<D, kBf16>, dim3(workers), dim3(kThreads), L::alloc, stream,
                    /*pdl=*/false, a);
  if (e != cudaSuccess || a.uncut) return e;
  const dim3 grid(workers, merge_blocks<Work, D>(a, workers));
  return launch_kernel(kv8_merge_tc_kernel<D, kBf16>, grid, dim3(128), 0, stream, /*pdl=*/true, a,
                       workers);
}

}  // namespace

size_t kv8_attn_tc_scratch_bytes(int D) {
  return align_up(scratch_bytes(device_sm_count(), kUnit, D), 256);
}

cudaError_t launch_kv8_attn_tc(const Kv8AttnArgs& a, int type, cudaStream_t stream) {
  if (a.c.D == 128)
    return type == CSA2_BF16 ? attn_tc_t<128, true>(a, stream) : attn_tc_t<128, false>(a, stream);
  return type == CSA2_BF16 ? attn_tc_t<64, true>(a, stream) : attn_tc_t<64, false>(a, stream);
}

}  // namespace csa2
