// Verification attention over a cache held in 8 or 4 bits (va_quant.cuh), on the
// 5th-generation tensor cores with the KEYS on the TMEM lanes.  For blocks of NR
// packed query rows (GQA group x draft tokens) and tiles of 128 keys:
//
//   S^T (128 keys x NR) = K (128 x d) . Q^T     A = K in TMEM, B = Q, K-major
//   O^T (d x NR)       += V^T . P^T             A = V tile, MN-major; B = P^T, MN-major
//
// K and V become halves on their way: a code times its group scale has at most six
// significant bits and lies in 2^-18 .. 2^12, so that is exact, and the row scale, a
// power of two, stays out of the operands.  It multiplies a key's scores (one key is
// one thread), and a key's P for the value row.  Nothing of a row is read twice.
//
// Roundings.  Q is scaled by one power of two for the block, its largest element to
// 2^14 .. 2^15, and rounded to half: an element keeps all its 8 bits down to 2^-31 of the
// largest and is off by 2^-39 of it at most (2^-25 of 2^14).  P is rounded to half: relative
// 2^-11, an eighth of the 2^-8 that the bf16 output is rounded by.  Weights are
// 2^6 at the row's reference and at most 2^14; times the ratio of the key's value scale to
// the largest one that the row sees they are rounded once, below 2^-14 by 2^-25 at most.
// Scores, row sums, O and the merge are fp32.
//
// The softmax reference of a row is its maximum over the first tile and moves when a score
// exceeds it by more than 2^8 in weight, and with it the largest value scale.  The rows of a
// block see the same keys, and so the same value scales, up to the draft keys.  A tile of those
// with a larger scale shifts each row's reference by the largest scale that the row sees (with
// one scale for the block, a draft row of 2^30 on one branch of a tree took all weights of the
// others): P = weight 2^shift * scale / unit, and the row sums are in units of 2^shift as well.
//
// Roles, one CTA per SM, persistent over the stream-K cut of all tiles, cooperative:
//   softmax    up to 64 rows a warpgroup (64: two) for even and one for odd tiles, so that two
//              tiles are under way, each parity with its own references, sums and O, joined
//              at the end of a part; 128 rows four warpgroups for every tile (TMEM holds one
//              O).  A thread owns a key and up to 32 rows
//   K          a warpgroup (up to 32 rows: two, for even and odd tiles): a thread takes its
//              key's row from the ring, makes halves and stores them to TMEM (two buffers)
//   V          as many: the same into a swizzled tile in shared memory (two buffers)
//   producers  two warps, K and V each: TMA boxes of whole rows (dense; pages of 8 rows
//              and more), or 16-byte cp.async gathers
//   issuers    a warp for S (and TMEM), one for PV
// K needs no shared memory this way: the tile's 32 KB of halves would be written once
// and read once, at 128 bytes a cycle as long as HBM takes for a whole 4-bit tile.
//
// Barriers of tile j (buffer j % 2, scales j % 4):
//   full_k/v[stage]   the ring's rows have landed;  empty_k/v[stage] they are in registers
//   k_full[j % 4]     K in TMEM, the scales of K and V in shared memory
//   v_full[j % 2]     V's tile
//   s_full[j % 2]     S of the tile (and its K buffer is free)
//   p_full[j % 2]     P written, S read;  o_done[j % 2] PV done (P and V buffers free)
// A scale buffer is written again for tile j + 4, behind the wait for PV of tile j + 1 (V;
// two warpgroups: of tile j) or S of tile j + 2 (K), which come after the softmax of tile j.
// Every wait is bounded; a role that gives up goes on without waiting.
//
// What bounds it (one GB300; a tile is 20.5 KB of 4-bit rows, 0.44 us of an SM's share of the
// measured copy rate): neither bytes nor tensor cores, but the warp instructions of a tile and
// the waits between its roles.  131072 keys, 8 kv-heads; instructions a tile and the part of the
// schedulers' slots that issue (profiled; long scoreboard is the largest stall of all):
//   16 rows    3780, 58%: one token 47 us (over a 16-bit cache 83)
//   32 rows    4150, 49%: 8 tokens 55 us (84)
//   64 rows    5590, 48%: 16 tokens 77 us over 8-bit rows, 82 over 4-bit ones (89)
//   128 rows   8690, 62%: 64 tokens 208 us (108: there a thread has a row, one sum and one
//              reference, and nothing is converted; over 8 bits four blocks of 64 rows, 268)
//   short calls  12 us of launch, plan, first tile, unit ends and merge, most of it code
//              fetched for the first time (8 tokens over 32K keys: 24.6 us, ten of them tiles)
// Above 16 rows the softmax spills (48 to 112 bytes of stores in the code), 10 to 24 of a tile's
// instructions, 88 with 128 rows.
// Steps that led here, 131072 keys, 8 kv-heads, 4 bits, one token / 8 / 64 tokens in us:
// one softmax warpgroup of 32 rows, everything unrolled 75 / 83 / 352; two issuers and
// descriptors in uniform registers 53 / 62 / 283; parities, 32-bit shared addresses, waits
// that sleep, maxima of the first tile 53 / 60 / 308; P scaled without selects 52 / 58 / 261;
// blocks of 128 rows - / - / 217; two pairs of converting warpgroups up to 32 rows 46 / 54 / -.
#pragma once

#include <cuda.h>
#include <math.h>

#include "va_attn_quant.h"
#include "va_common.cuh"
#include "va_kernels.h"
#include "va_merge.cuh"
#include "va_pipeline.cuh"
#include "va_quant.cuh"
#include "va_rowreduce.cuh"
#include "va_tcgen05.cuh"

namespace va {

constexpr int kTqKeys = 128;    // keys per tile
constexpr int kTqStages = 8;    // most stages of the ring
constexpr float kTqBias = 6.f;  // log2 of the weight at the reference
constexpr float kTqMove = 8.f;  // a score this far above the reference moves it
// References shifted by value scales: the unit is the largest scale that a row of the block
// sees, or 2^40, and a shift at most 2^80, so that weights and sums stay within fp32 (2^30 keys of
// weight 2^14).  A row whose own scale is above 2^-80 of the unit, 2^-100 with the room that
// halves have below 2^6, loses nothing.  (With the unit at 2^-60 of the largest, shifts of 60
// everywhere, the lse of every short sequence was off by up to 7e-6.)
constexpr float kTqShift = 80.f, kTqUnit = 0x1p40f;

template <int NR, bool kTma = true>
struct TqCfg {
  static constexpr int kRowGroups = NR > 32 ? NR / 32 : 1;  // of NW rows, each with
  static constexpr int kParities = NR > 64 ? 1 : 2;         // one warpgroup, or one for even and one for odd tiles
  static constexpr int NW = NR / kRowGroups;                // rows of a softmax thread
  static constexpr int kGroups = kParities * kRowGroups;    // softmax warpgroups
  static constexpr int kSoft = 128 * kGroups;
  // warpgroups that convert K, and V: up to 32 rows one for even and one for odd tiles
  static constexpr int kPairs = NR <= 32 ? 2 : 1;
  // (the last warpgroup: two producers and two issuers, of S and of PV)
  static constexpr int kKWarp = 4 * kGroups, kVWarp = kKWarp + 4 * kPairs, kProducer = kVWarp + 4 * kPairs,
                       kMmaWarp = kProducer + 2;
  static constexpr int kThreads = (kProducer + 4) * 32;
  // Registers a thread: the launch's, and what the warpgroups divide them into.
  static constexpr int kWarpgroups = kGroups + 2 * kPairs + 1;
  static constexpr int kRegsLaunch = 72;
  // (128 rows with 88, 48 and 56: 64 tokens over 131072 4-bit keys 218 us; with 96, 40 and 40
  // 208, but gathers, whose addresses live in the rest, 269 instead of 251 over 2 x 65536 keys)
  static constexpr bool kWide = NR == 128 && kTma;
  static constexpr int kRegsSoft = NR == 16 ? 96 : NR == 32 ? 128 : kWide ? 96 : 88,
                       kRegsKv = NR == 16 ? 64 : kWide ? 40 : 48, kRegsRest = kWide ? 40 : 56;
  static_assert(kGroups * kRegsSoft + 2 * kPairs * kRegsKv + kRegsRest <= kWarpgroups * kRegsLaunch,
                "within the launch's registers");
  static_assert(kThreads * kRegsLaunch <= 65536, "a block's registers");
};

// Shared memory by its 32-bit address: the roles' loops are short, and 64-bit address
// arithmetic was a third of their instructions.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 lds128f(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float2 lds64f(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts32f(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// role_wait in few instructions: most warps wait most of the time, a try comes back after
// some hundred cycles whatever time it is given, and looking at the clock after each took
// a third of all instructions.
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)  // ns
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool tq_wait_on(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint64_t limit_ns,
                                        int *status) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_sleep(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      record_status(status, VA_ERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int FMT, int D, int NR>
struct TqSmem {
  static constexpr int kRow = QRow<FMT, D>::kBytes;
  static constexpr int kRaw = kTqKeys * kRow;              // K (or V) rows of a stage
  static constexpr int kVBytes = (D / 64) * kTqKeys * 128; // V tile in halves
  // (d 64: the PV MMA keeps M = 128; its lanes 64 .. 127 multiply the 16 KB that follow
  // the tile, inside the plan, and nobody reads them)
  static constexpr int kPOff = 2 * kVBytes;                // P^T: per key a 128-byte row, for 64 rows of Q each
  static constexpr int kPBytes = (NR > 64 ? 2 : 1) * kTqKeys * 128;
  static constexpr int kQOff = kPOff + 2 * kPBytes;
  static constexpr int kQBytes = (D / 64) * NR * 128;
  static constexpr int kBarOff = kQOff + kQBytes;
  static constexpr int kNumBars = 4 * kTqStages + 4 + 2 + 2 + 2 + 2 + 2;
  static constexpr int kMiscOff = (kBarOff + kNumBars * 8 + 15) & ~15;  // tmem base, abort flag, merge flag
  static constexpr int kRowMaskOff = kMiscOff + 16;      // u64 [64]: draft visibility rows
  static constexpr int kKeyMaskOff = kRowMaskOff + 512;  // u32 [4][64]: per 32 rows and draft key, the rows that see it
  static constexpr int kRedOff = kKeyMaskOff + 1024;     // float4 [2 NR]: per-warp row maxima and sums of each tile parity
  static constexpr int kVRedOff = kRedOff + 2 * NR * 16; // float [2][16]: per-warp largest value scales (also Q maxima), those of the prefix
  static constexpr int kRefOff = kVRedOff + 128;         // float [2 NR]: bias less the reference of a row
  static constexpr int kAlphaOff = kRefOff + 2 * NR * 4; // float [2 NR]: what a moved reference scales by; then 1 / l factors
  static constexpr int kVRowOff = kAlphaOff + 2 * NR * 4; // float [NR] (one parity): largest value scale that a row has seen
  static constexpr int kKsOff = kVRowOff + (TqCfg<NR>::kParities == 1 ? NR * 4 : 0);  // float2 [4][128]: scales of the tile's K and V rows
  static constexpr int kRingOff = (kKsOff + 4 * 1024 + 127) & ~127;
  // fewest stages, beside the largest plan
  static constexpr int kStages = (kSmemLimit - 1024 - kRingOff - (kMaxSegments + 1) * 4) / (2 * kRaw);
  static_assert(kStages >= 2, "a ring");
  static constexpr int kNC = NR < 32 ? 32 : NR;          // TMEM columns per region
  // O (of even and of odd tiles), two S, two K of D/2 columns
  static constexpr int kSCol = TqCfg<NR>::kParities * kNC, kKCol = kSCol + 2 * kNC;
  static constexpr int kTmemCols = kKCol + D <= 256 ? 256 : 512;
  static_assert(kKCol + D <= 512, "TMEM plan");
  static_assert(kQOff % 1024 == 0 && kPOff % 1024 == 0 && kQBytes % 1024 == 0, "swizzle atoms");
  static_assert(kRefOff % 16 == 0 && kAlphaOff % 16 == 0 && kKsOff % 16 == 0, "vector loads");
  // d 64: what the unused lanes of the second V buffer read is the P buffers
  static_assert(D == 128 || kPOff + 16384 <= kQOff, "unused lanes stay inside");
};

// Instruction descriptor of kind::f16 with half operands and fp32 accumulation.
__host__ __device__ constexpr uint32_t umma_idesc_half(int M, int N, int a_mn_major, int b_mn_major) {
  return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }

// 16 bytes of codes as halves, two to a register: 32 values of e2m1 (groups 2c and 2c + 1
// of the row's group scales) or 16 of e4m3.
template <int FMT>
struct CodeChunk {
  static constexpr int kRegs = FMT == VA_KV_E4M3 ? 8 : 16;
};
template <int FMT>
__device__ __forceinline__ void codes_to_halves(const uint4 &v, uint32_t two_groups, uint32_t (&h)[CodeChunk<FMT>::kRegs]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (FMT == VA_KV_E4M3) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = half2_bits(e4m3x2_to_half2(w[i / 2] >> (16 * (i & 1)) & 0xffffu));
  } else {
    const __half2 g = e4m3x2_to_half2(two_groups & 0xffffu);
    const __half2 g0 = __low2half2(g), g1 = __high2half2(g);
#pragma unroll
    for (int i = 0; i < 4; ++i) e2m1x8_to_half2(w[i], h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = half2_bits(__hmul2(*reinterpret_cast<__half2 *>(h + i), i < 8 ? g0 : g1));
  }
}

// log2 of a power of two.
__device__ __forceinline__ float exponent_of(float pow2) { return (float)((__float_as_int(pow2) >> 23) - 127); }

// The row scale out of a row's tail.
template <int FMT, int D>
__device__ __forceinline__ float tail_scale(const uint4 &tail) {
  return __uint_as_float(FMT == VA_KV_E4M3 ? tail.x : D == 128 ? tail.z : tail.y);
}

// Tile i0 of part c when `total` tiles are cut into G near-equal ranges, [c total / G], in 32
// bits (G <= 2^10: 64-bit divisions are long calls), and the part that owns tile t.
__device__ __forceinline__ int tq_first_tile(int c, int total, int G) { return c * (total / G) + c * (total % G) / G; }
__device__ __forceinline__ int tq_owner(int t, int total, int G) {
  int c = min(G - 1, (int)((float)t * (float)G / (float)total));
  while (c > 0 && tq_first_tile(c, total, G) > t) --c;
  while (c + 1 < G && tq_first_tile(c + 1, total, G) <= t) ++c;
  return c;
}

// The CTA's share.  The kv-heads and row blocks of a sequence (`lanes` of them) lie side by
// side in memory, a row of 48 to 144 bytes each: CTAs go through the sequences in step,
// CTA c with lane c % lanes and part c / lanes of the lane's tiles, so that what one of
// them reads of a DRAM page or a cache line the others need at that moment.  With each
// lane's tiles after the other (lanes = 1: segments are units), 64 single-token
// sequences over 8192 keys read 1.4 times their bytes from HBM: 262 us, in step 190 (now 168).
struct TqRange {
  int units, lanes, lane;  // unit u of this lane is segment u * lanes + lane
  int total, G, part;      // tiles of the lane, parts they are cut into, this CTA's
  int t0, t1, u0;          // its tiles [t0, t1), the first unit that reaches past t0
  __device__ __forceinline__ int segment(int u) const { return u * lanes + lane; }
  // this CTA's tiles [lt0, lt1) of unit u
  __device__ __forceinline__ void tiles(const int *tstart, int u, int &lt0, int &lt1) const {
    const int first = tstart[u];
    lt0 = max(first, t0) - first;
    lt1 = min(tstart[u + 1], t1) - first;
  }
};

__device__ __forceinline__ TqRange tq_plan(const AttnParams &p, int *tstart) {
  TqRange r;
  r.lanes = p.lanes;
  r.units = p.S / p.lanes;
  r.lane = blockIdx.x % p.lanes;
  r.part = blockIdx.x / p.lanes;
#pragma unroll 1
  for (int u = threadIdx.x; u < r.units; u += blockDim.x) {
    const Seg g = seg_info(p, r.segment(u), true);
    tstart[u] = (g.nkeys + kTqKeys - 1) / kTqKeys;
  }
  __syncthreads();
  if (threadIdx.x < 32) warp_scan_inplace(tstart, r.units);
  __syncthreads();
  r.total = tstart[r.units];
  r.G = min((int)gridDim.x / r.lanes, r.total);
  r.t0 = r.t1 = r.u0 = 0;
  if (r.part < r.G) {
    r.t0 = tq_first_tile(r.part, r.total, r.G);
    r.t1 = tq_first_tile(r.part + 1, r.total, r.G);
    int lo = 0, hi = r.units - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (tstart[mid + 1] > r.t0) hi = mid; else lo = mid + 1;
    }
    r.u0 = lo;
  }
  return r;
}

// ---------------------------------------------------------------------------
// producer: one warp fills the K (or V) half of the ring with raw rows
// ---------------------------------------------------------------------------
template <int FMT, int D, bool kTma>
__device__ __forceinline__ void produce_raw(const AttnParams &p, const CUtensorMap *tm, const uint8_t *cache,
                                            const int *tstart, const TqRange &cr, uint8_t *ring, uint64_t *full,
                                            uint64_t *empty, volatile int *abort_flag) {
  constexpr int RB = QRow<FMT, D>::kBytes;
  constexpr int TK = kTqKeys;
  const int lane = threadIdx.x & 31;
  const uint64_t policy = l2_evict_first_policy();
  const bool paged = p.layout == VA_LAYOUT_PAGED;
  bool ok = true;
  int st = 0, it = 0;
  uint32_t ph = 0;
  for (int u = cr.u0; u < cr.units && tstart[u] < cr.t1; ++u) {
    const int s = cr.segment(u);
    const Seg g = seg_info(p, s, false);
    int lt0, lt1;
    cr.tiles(tstart, u, lt0, lt1);
    // Page entries of 32 boxes at a time, a lane each (2 to 32 tiles'), and those of the next
    // 32 on their way: an entry a tile ahead made a tile take the latency of its load
    // (64 single-token sequences over 8192 keys in 64-row pages: 188 us, now 167).
    const int BR = p.tma_box;
    const int boxes = kTma ? TK / BR : 1, ahead = 32 / boxes;  // of a tile; tiles
    auto box_pages = [&](int lt) {
      const int k = lt * TK + lane * BR;
      if (!kTma || !paged || k >= g.nkeys) return 0;
      return __ldg(p.page_table + (size_t)g.b * p.max_pages + (k >> p.page_shift));
    };
    int lt_pages = lt0, pages = box_pages(lt0), pages_next = box_pages(lt0 + ahead);
    // (gather) the page entries of a tile's rows, four a lane, on their way while the tile
    // before is copied: turned into addresses at once, a tile took their latency too (64
    // single-token sequences over 8192 keys in 4-row pages: 503 us, now 234)
    int entries[TK / 32];
    auto look_up = [&](int lt) {
#pragma unroll
      for (int j = 0; j < TK / 32; ++j) {
        const int k = lt * TK + 32 * j + lane;
        entries[j] = lt < lt1 && k < g.nkeys ? __ldg(p.page_table + (size_t)g.b * p.max_pages + (k >> p.page_shift)) : 0;
      }
    };
    if constexpr (!kTma) look_up(lt0);
    for (int lt = lt0; lt < lt1; ++lt, ++it) {
      if (kTma && lt == lt_pages + ahead) {
        lt_pages = lt;
        pages = pages_next;
        pages_next = box_pages(lt + ahead);
      }
      if (__builtin_expect(ok && !mbar_sleep(smem_u32(empty + st), ph ^ 1u), 0))
        ok = tq_wait_on(smem_u32(empty + st), ph ^ 1u, abort_flag, p.wait_ns, p.status);
      ok = __all_sync(0xffffffffu, ok);  // (a gather passes addresses between the lanes)
      if (ok) {
        uint8_t *dst = ring + (size_t)st * (2 * TK * RB);
        const int k0 = lt * TK;
        if constexpr (kTma) {
          // dense: one box; rows past the segment's end arrive too (other tokens, or
          // zeros past the cache) and are masked.  Paged: a box a page; boxes that
          // start past the end are not loaded.
          const int nb = paged ? min(boxes, (g.nkeys - k0 + BR - 1) / BR) : 1;
          const int page_now = __shfl_sync(0xffffffffu, pages, ((lt - lt_pages) * boxes + lane) & 31);
          if (lane == 0) mbar_arrive_expect_tx(full + st, (uint32_t)(nb * BR * RB));
          __syncwarp();
          if (lane < nb) {
            int row;
            if (paged) {
              int page = page_now;
              if (page < 0 || page >= p.num_pages) {
                record_status(p.status, VA_ERR_DEVICE_BOUNDS);
                page = 0;
              }
              row = (page << p.page_shift) + ((k0 + lane * BR) & ((1 << p.page_shift) - 1));
            } else {
              row = g.b * p.len_cap + k0;
            }
            tma_load_3d(dst + lane * BR * RB, tm, 0, g.hkv, row, full + st, policy);
          }
        } else {
          constexpr int CPR = RB / 16;  // 16-byte chunks of a row
          const uint8_t *now[TK / 32];
#pragma unroll
          for (int j = 0; j < TK / 32; ++j) {
            const int k = k0 + 32 * j + lane;
            int page = entries[j];
            if (page < 0 || page >= p.num_pages) {
              record_status(p.status, VA_ERR_DEVICE_BOUNDS);
              page = 0;
            }
            const size_t row = ((size_t)page << p.page_shift) + (k & ((1 << p.page_shift) - 1));
            now[j] = cache + (row * p.Hkv + g.hkv) * RB;
          }
          look_up(lt + 1);
#pragma unroll
          for (int j = 0; j < TK / 32; ++j) {
            const uint8_t *mine = now[j];
#pragma unroll
            for (int i = 0; i < CPR; ++i) {
              const int e = 32 * i + lane, r = e / CPR, c = e % CPR;
              const uintptr_t a = (uintptr_t)__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), r);
              cp_async_16(dst + (32 * j + r) * RB + c * 16, reinterpret_cast<const void *>(a + 16 * c),
                          k0 + 32 * j + r < g.nkeys ? 16u : 0u);
            }
          }
          cp_async_mbar_arrive(full + st);
        }
      }
      if (++st == p.stages) {
        st = 0;
        ph ^= 1u;
      }
    }
  }
  // the copies this warp issued land before it leaves (bounded)
  if constexpr (kTma) {
    for (int j = max(0, it - p.stages); j < it; ++j)
      mbar_wait(full + j % p.stages, (uint32_t)(j / p.stages) & 1u, p.wait_ns >> 4);
  } else {
    cp_async_wait_all();
  }
}

// Merge of rows [r0, r1) of a split segment (as merge_rows_warp) in few instructions, by
// groups of `wpr` warps to a row, each with every wpr-th part: a lane holds the weight of a
// part, then D/32 columns.  Straight code that runs once is fetched from far away: the
// unrolled merge took 3 us of a split call, about what four tiles take.  `part` is shared
// memory for n_warps x D floats; every softmax thread calls it (barrier `bar`).
template <int D>
__device__ __forceinline__ void merge_rows_compact(const AttnParams &p, int b, int hkv, int row_base, int slot0, int np,
                                                   int r0, int r1, int warp_id, int n_warps, int lane, float *part,
                                                   int bar) {
  constexpr int C = D / 32;
  const int group = p.Hq / p.Hkv, n = r1 - r0;
  const int wpr = n > 0 ? max(1, n_warps / n) : 1;  // warps to a row
  const int step = n_warps / wpr;                   // rows at once
  const int sub = warp_id % wpr;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += step) {
    const int row = r0 + i0 + warp_id / wpr;
    const bool act = warp_id / wpr < step && row < r1;
    float L = 0.f, M = -INFINITY, acc[C];
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] = 0.f;
    if (act) {
      const float *l = p.lse_part + (size_t)slot0 * p.rows_pad + row;
      const float *o = p.o_part + ((size_t)slot0 * p.rows_pad + row) * D + lane * C;
#pragma unroll 1
      for (int q0 = 0; q0 < np; q0 += 32) {
        const float ls = q0 + lane < np ? __ldcg(l + (size_t)(q0 + lane) * p.rows_pad) : -INFINITY;
        const int cnt = min(32, np - q0);
        float v[8][C];
        auto load = [&](int j0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float *src = o + (size_t)(q0 + min(j0 + j * wpr, cnt - 1)) * p.rows_pad * D;
            if constexpr (C == 4) {
              const float4 u = __ldcg(reinterpret_cast<const float4 *>(src));
              v[j][0] = u.x;
              v[j][1] = u.y;
              v[j][2] = u.z;
              v[j][3] = u.w;
            } else {
              const float2 u = __ldcg(reinterpret_cast<const float2 *>(src));
              v[j][0] = u.x;
              v[j][1] = u.y;
            }
          }
        };
        load(sub);  // (before the weights are known)
        float m = ls;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, x));
        m = max_nan(m, M);
        if (m == -INFINITY) continue;  // no part so far saw a key
        const float a = M == -INFINITY ? 0.f : __expf(M - m), w = ls == -INFINITY ? 0.f : __expf(ls - m);
        float sum = w;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        L = L * a + sum;
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] *= a;
#pragma unroll 1
        for (int j0 = sub; j0 < cnt; j0 += 8 * wpr) {
          if (j0 != sub) load(j0);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, min(j0 + j * wpr, cnt - 1));
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] = fmaf(j0 + j * wpr < cnt ? wj : 0.f, v[j][i], acc[i]);
          }
        }
        M = m;
      }
    }
    if (wpr > 1) {
#pragma unroll
      for (int i = 0; i < C; ++i) part[warp_id * D + lane * C + i] = acc[i];
      named_bar_sync(bar, n_warps * 32);
      if (act && sub == 0) {
#pragma unroll 1
        for (int w = 1; w < wpr; ++w)
#pragma unroll
          for (int i = 0; i < C; ++i) acc[i] += part[(warp_id + w) * D + lane * C + i];
      }
      named_bar_sync(bar, n_warps * 32);
    }
    if (!act || sub != 0) continue;
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const int t = (row_base + row) / group, hq = hkv * group + (row_base + row) - t * group;
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + (((size_t)b * p.T + t) * p.Hq + hq) * D + lane * C;
    if constexpr (C == 4)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    else
      *reinterpret_cast<uint32_t *>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
    if (lane == 0) p.lse[((size_t)b * p.Hq + hq) * p.T + t] = L != 0.f ? M + __logf(L) : -INFINITY;
  }
}

template <int FMT, int D, int NR, bool kTma>
__global__ void __launch_bounds__(TqCfg<NR, kTma>::kThreads, 1)
    verify_attn_quant_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmk,
                             const __grid_constant__ CUtensorMap tmv) {
  using SM = TqSmem<FMT, D, NR>;
  using Cfg = TqCfg<NR, kTma>;
  constexpr int TK = kTqKeys, NC = SM::kNC, WG = Cfg::kGroups, RG = Cfg::kRowGroups, PAR = Cfg::kParities, NW = Cfg::NW, kSoft = Cfg::kSoft,
                RB = SM::kRow;
  constexpr int kXRows = NR > 32 ? 16 : NW;  // scores a softmax thread holds at once (registers)
  constexpr int kChunks = QRow<FMT, D>::kCodeBytes / 16, kRegs = CodeChunk<FMT>::kRegs;
  constexpr int kBarQ = 1, kBarSoft = 3, kBarEnd = 4, kBarRed0 = 5;  // kBarRed0 + softmax warpgroup
  constexpr int kEndThreads = kSoft + 256 * Cfg::kPairs + 64;        // all but the producers
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *sV = smem, *sQ = smem + SM::kQOff, *ring = smem + SM::kRingOff;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SM::kBarOff);
  uint64_t *full = bars, *empty = bars + 2 * kTqStages;  // [K, V][stage]
  uint64_t *k_full = bars + 4 * kTqStages, *v_full = k_full + 4, *s_full = v_full + 2, *p_full = s_full + 2,
           *o_done = p_full + 2, *drains = o_done + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SM::kMiscOff);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SM::kMiscOff + 4);
  uint64_t *rowmask = reinterpret_cast<uint64_t *>(smem + SM::kRowMaskOff);
  uint32_t *keymask = reinterpret_cast<uint32_t *>(smem + SM::kKeyMaskOff);
  float4 *red = reinterpret_cast<float4 *>(smem + SM::kRedOff);
  float *vred = reinterpret_cast<float *>(smem + SM::kVRedOff);
  float *refs = reinterpret_cast<float *>(smem + SM::kRefOff), *alphas = reinterpret_cast<float *>(smem + SM::kAlphaOff);
  int *tstart = reinterpret_cast<int *>(ring + (size_t)p.stages * (2 * SM::kRaw));

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = blockIdx.x;
  // (addresses of the same barriers)
  const uint32_t smem_a = smem_u32(smem), bar_a = smem_a + SM::kBarOff;
  const uint32_t a_full = bar_a, a_empty = bar_a + 16 * kTqStages, a_k_full = a_empty + 16 * kTqStages, a_v_full = a_k_full + 32,
                 a_s_full = a_v_full + 16, a_p_full = a_s_full + 16, a_o_done = a_p_full + 16;
  if (kTma && tid == 32) {
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
  }
  if (tid < SM::kNumBars) {  // a barrier a thread, in the order of their addresses
    uint64_t *bar = bars + tid;
    const int n = bar < empty  ? (kTma ? 1 : 32)
                  : bar < k_full ? 4
                  : bar < v_full ? 8
                  : bar < s_full ? 4
                  : bar < p_full ? (c == p.test_stall ? kNever : 1)
                  : bar < o_done ? 128 * RG
                                 : 1;
    mbar_init(bar, n);
    if (tid == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  const TqRange cr = tq_plan(p, tstart);  // contains __syncthreads
  if (cr.part >= cr.G) return;
  const int t1 = cr.t1;

  bool ok = true;
  auto wait_ok = [&](uint32_t bar, uint32_t parity) {
    if (__builtin_expect(ok && !mbar_sleep(bar, parity), 0)) ok = tq_wait_on(bar, parity, abort_flag, p.wait_ns, p.status);
  };
  // TMEM is allocated: every role but the producers waits for its address here
  auto tmem_base = [&]() {
    tc_fence_before();
    named_bar_sync(kBarEnd, kEndThreads);
    tc_fence_after();
    return *tmem_slot;
  };

  if (warp >= Cfg::kProducer) {
    regs_dec<Cfg::kRegsRest>();
    if (warp < Cfg::kMmaWarp) {
      const bool is_v = warp != Cfg::kProducer;
      produce_raw<FMT, D, kTma>(p, is_v ? &tmv : &tmk, static_cast<const uint8_t *>(is_v ? p.v : p.k), tstart, cr,
                                ring + (is_v ? SM::kRaw : 0), full + (is_v ? kTqStages : 0),
                                empty + (is_v ? kTqStages : 0), abort_flag);
      return;
    }
    if (warp == Cfg::kMmaWarp) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(SM::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ================================ MMA issuer ================================
    // Whatever addresses are made of is the same in every lane, and said to be (a
    // shuffle from lane 0): descriptors then live in uniform registers, where the
    // MMA takes them from.  Unknown to be uniform, an MMA took 85 to 137 cycles to
    // issue beside the other roles, 48 alone.
    auto uni = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
    const uint32_t tmem = uni(tmem_base());
    const uint32_t base = uni(smem_u32(smem));
    uint32_t jt = 0;
    if (warp == Cfg::kMmaWarp) {
      const uint32_t id_s = umma_idesc_half(128, NR, 0, 0);
      const uint64_t dQ0 = umma_sdesc(base + SM::kQOff, 16, 1024);
      for (int u = cr.u0; u < cr.units && (int)uni(tstart[u]) < t1; ++u) {
        int lt0, lt1;
        cr.tiles(tstart, u, lt0, lt1);
        const int n = (int)uni(lt1 - lt0);
        named_bar_sync(kBarQ, kSoft + 32);  // Q of this segment is in shared memory
        for (int i = 0; i < n; ++i, ++jt) {
          const uint32_t b = jt & 1u;
          // (two tiles ahead of the softmax: S of tile j - 2 has been read)
          if (i >= 2) wait_ok(a_p_full + 8 * b, ((jt - 2) >> 1) & 1u);
          wait_ok(a_k_full + 8 * (jt & 3), (jt >> 2) & 1u);
          __syncwarp();
          tc_fence_after();
          const uint32_t tS = tmem + SM::kSCol + b * NC, tK = tmem + SM::kKCol + b * (D / 2);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t qoff = (uint64_t)(((kk >> 2) * (NR * 128) + (kk & 3) * 32) >> 4);
            umma_ts_warp(tS, tK + kk * 8, dQ0 + qoff, id_s, kk > 0 ? 1u : 0u);
          }
          umma_commit_warp(s_full + b);
          __syncwarp();
        }
      }
    } else {
      const uint32_t id_o = umma_idesc_half(128, NR, 1, 1);
      const uint64_t dV0 = umma_sdesc(base, TK * 128, 1024);
      const uint64_t dP0 = umma_sdesc(base + SM::kPOff, TK * 128, 1024);
      for (int u = cr.u0; u < cr.units && (int)uni(tstart[u]) < t1; ++u) {
        int lt0, lt1;
        cr.tiles(tstart, u, lt0, lt1);
        const int n = (int)uni(lt1 - lt0);
        for (int i = 0; i < n; ++i, ++jt) {
          const uint32_t b = jt & 1u;
          wait_ok(a_v_full + 8 * b, (jt >> 1) & 1u);
          wait_ok(a_p_full + 8 * b, (jt >> 1) & 1u);
          __syncwarp();
          tc_fence_after();
          const uint64_t dV = dV0 + (uint64_t)(b * (SM::kVBytes >> 4)), dP = dP0 + (uint64_t)(b * (SM::kPBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < TK / 16; ++kk) {
            const uint64_t off = (uint64_t)((kk * 2048) >> 4);
            umma_ss_warp(tmem + (PAR == 2 ? b * NC : 0), dV + off, dP + off, id_o, kk > 0 || i >= PAR ? 1u : 0u);
          }
          umma_commit_warp(o_done + b);
          __syncwarp();
        }
      }
    }
    // drain: every MMA issued has finished before TMEM is released
    uint64_t *drain = drains + (warp - Cfg::kMmaWarp);
    umma_commit_warp(drain);
    mbar_wait(drain, 0u, p.wait_ns);
    __syncwarp();
    tc_fence_before();
    named_bar_sync(kBarEnd, kEndThreads);
    if (warp != Cfg::kMmaWarp) return;
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SM::kTmemCols) : "memory");
    return;
  }

  if (warp >= Cfg::kKWarp) {
    // ============================ K and V to halves ============================
    regs_dec<Cfg::kRegsKv>();
    const uint32_t tmem = tmem_base();
    const bool is_v = warp >= Cfg::kVWarp;
    const int key = (warp & 3) * 32 + lane;
    const uint32_t fl = a_full + (is_v ? 8 * kTqStages : 0), em = fl + 16 * kTqStages;
    const uint32_t freed = is_v ? a_o_done : a_s_full;
    const uint32_t sc = smem_a + SM::kKsOff + key * 8 + (is_v ? 4 : 0);
    const uint32_t row0 = smem_a + SM::kRingOff + (is_v ? SM::kRaw : 0) + key * RB;
    // 16-byte chunk c of the key's V row: (vrow ^ 16 c), 16 KB further for the second half
    const uint32_t vrow = smem_a + key * 128 + ((key & 7) << 4);
    const uint32_t tK0 = tmem + ((uint32_t)((warp & 3) * 32) << 16) + SM::kKCol;
    const int n = t1 - cr.t0;
    const int jt0 = Cfg::kPairs == 2 ? (warp - Cfg::kKWarp) >> 2 & 1 : 0;  // its first tile
    // A wait for a phase also ends while the phase two before it is open.  With three stages
    // a stage goes back and forth between the two warpgroups, and the rows of tile j can have
    // landed, and been converted, before those of tile j - 1: what comes next in its stage
    // waits until tile j - 1 has left it.  (Two, and any even number: the same warpgroup had
    // the stage.  Five and more: the MMA of tile j - 4, waited for, is behind tile j - 5.)
    constexpr bool kBehind = Cfg::kPairs == 2 && SM::kStages <= 3;
    int st = jt0;
    uint32_t ph = 0, row = row0 + jt0 * (2 * SM::kRaw);
    for (int jt = jt0; jt < n; jt += Cfg::kPairs) {
      const uint32_t b = (uint32_t)jt & 1u;
      if constexpr (kBehind) wait_ok(em + 8 * st, ph ^ 1u);
      wait_ok(fl + 8 * st, ph);
      const uint4 tail = lds128(row + QRow<FMT, D>::kCodeBytes);
      const uint32_t sc_now = sc + (jt & 3) * 1024, kb = a_k_full + 8 * (jt & 3);
      if (is_v) {
        sts32f(sc_now, tail_scale<FMT, D>(tail));
        __syncwarp();
        if (lane == 0) mbar_arrive_at(kb);
      }
      if (jt >= 2) wait_ok(freed + 8 * b, (uint32_t)((jt - 2) >> 1) & 1u);
      __syncwarp();
      tc_fence_after();
      if (!is_v) sts32f(sc_now, tail_scale<FMT, D>(tail));
      // 64 elements a pass; one copy of the conversion for K and V, rolled: the warps of six
      // roles share the instruction caches
      constexpr int kPer = kChunks / (D / 64);
#pragma unroll 1
      for (uint32_t half = 0; half < D / 64; ++half) {
        const uint32_t dst = vrow + b * SM::kVBytes + half * (TK * 128), tK = tK0 + b * (D / 2) + half * 32;
        const uint32_t groups = half == 0 ? tail.x : tail.y;
        uint4 code[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) code[i] = lds128(row + half * (kPer * 16) + i * 16);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          uint32_t h[kRegs];
          codes_to_halves<FMT>(code[i], groups >> (16 * (i & 1)), h);
          if (is_v) {
#pragma unroll
            for (int u = 0; u < kRegs / 4; ++u)
              sts128(dst ^ ((i * (kRegs / 4) + u) << 4), h[4 * u], h[4 * u + 1], h[4 * u + 2], h[4 * u + 3]);
          } else if constexpr (kRegs == 16) {
            tmem_st16(tK + i * kRegs, h);
          } else {
            tmem_st8(tK + i * kRegs, h);
          }
        }
      }
      if (is_v)
        fence_proxy_async_smem();
      else
        tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        // (having given up on a wait, it frees no stage: the copies into it may be under way,
        // and its barrier takes no second announcement before they land)
        if (ok) mbar_arrive_at(em + 8 * st);
        mbar_arrive_at(is_v ? a_v_full + 8 * b : kb);
      }
      row += Cfg::kPairs * (2 * SM::kRaw);
      st += Cfg::kPairs;
      if (st >= p.stages) {
        st = Cfg::kPairs == 1 ? 0 : st - p.stages;
        row = Cfg::kPairs == 1 ? row0 : row0 + st * (2 * SM::kRaw);
        ph ^= 1u;
      }
    }
    tc_fence_before();
    named_bar_sync(kBarEnd, kEndThreads);
    return;
  }

  // ================================== softmax ==================================
  regs_inc<Cfg::kRegsSoft>();
  const uint32_t tmem = tmem_base();
  const int wg = warp >> 2, par = PAR == 2 ? wg / RG : 0;  // warpgroup; with two parities the tiles it takes: jt % 2 == par
  const int rg = wg % RG, r_wg = rg * NW;                  // its rows [r_wg, r_wg + NW) of the block
  const int wq = warp & 3, ktid = tid & 127;          // warp of the warpgroup; key of the tile, output column of the epilogue
  const int kBarRed = kBarRed0 + wg;
  const uint32_t tLane = tmem + ((uint32_t)(wq * 32) << 16);
  const uint32_t tO = tLane + par * NC + r_wg;
  float4 *my_red = red + par * NR + r_wg;             // [NW]
  float *ref = refs + par * NR + r_wg, *alpha = alphas + par * NR + r_wg;
  const uint32_t a_ref = smem_u32(ref), a_scale = smem_a + SM::kKsOff + ktid * 8;
  // 16-byte chunk cw of the thread's P^T row (8 rows of Q): (a_p0 ^ 16 cw)
  const uint32_t a_p0 = (smem_a + SM::kPOff + (r_wg / 64) * (TK * 128) + ktid * 128 + ((ktid & 7) << 4)) ^ ((r_wg / 8 & 7) << 4);
  const int group = p.Hq / p.Hkv;
  const float inv_group = 1.f / (float)group;
  auto token_of = [&](int r) { return __float2int_rd(((float)r + 0.5f) * inv_group); };  // r / group (r <= 4096)
  int jt = 0;
  // split segments this CTA holds a part of (at most its first and its last)
  int n_split = 0, ms[2] = {0, 0}, mslot[2] = {0, 0}, mnp[2] = {0, 0}, mpart[2] = {0, 0};
  for (int u = cr.u0; u < cr.units && tstart[u] < t1; ++u) {
    const int s = cr.segment(u);
    const Seg g = seg_info(p, s, false);
    int lt0, lt1;
    cr.tiles(tstart, u, lt0, lt1);
    const int jt0 = jt;
    const int base = g.rb * NR, R = min(NR, p.R - base);  // the packed rows [base, base + R) of the kv-head
    // bit r: row 32 w + r of this segment is one of draft token t
    auto token_rows = [&](int t, int w) -> uint32_t {
      const int lo = min(max(t * group - base - 32 * w, 0), 32), hi = min(max((t + 1) * group - base - 32 * w, 0), 32);
      return (hi == 32 ? ~0u : (1u << hi) - 1u) & (lo == 32 ? 0u : ~0u << lo);
    };

    // ---- Q of this segment: halves, scaled by a power of two, [D/64][NR rows][128 B], 128B swizzle ----
    float q_unit;  // what a product of the scaled Q stands for, in base-2 score units
    {
      const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(p.q);
      constexpr int kCh = D / 8, kQIt = (NR * kCh + kSoft - 1) / kSoft;
      uint4 v[kQIt];
      uint32_t top = 0;  // largest finite |bf16|
#pragma unroll
      for (int u = 0; u < kQIt; ++u) {
        const int e = tid + u * kSoft, row = e / kCh;
        v[u] = make_uint4(0, 0, 0, 0);
        if (row < R) {
          const int t = token_of(base + row), hq = g.hkv * group + (base + row) - t * group;
          v[u] = __ldg(reinterpret_cast<const uint4 *>(qb + (((size_t)g.b * p.T + t) * p.Hq + hq) * D) + (e % kCh));
        }
      }
#pragma unroll
      for (int u = 0; u < kQIt; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo = w[i] & 0x7fffu, hi = w[i] >> 16 & 0x7fffu;
          top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) reinterpret_cast<uint32_t *>(vred)[warp] = top;
      named_bar_sync(kBarSoft, kSoft);
#pragma unroll
      for (int i = 0; i < 4 * WG; ++i) top = max(top, reinterpret_cast<uint32_t *>(vred)[i]);
      const int k = top == 0 ? 0 : min(120, 141 - (int)(top >> 7));  // 14 - (exponent - 127)
      const float up = __uint_as_float((uint32_t)(127 + k) << 23);
      q_unit = p.scale * kLog2e * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
      for (int u = 0; u < kQIt; ++u) {
        const int e = tid + u * kSoft, row = e / kCh, ch = e % kCh;
        if (row >= NR) break;  // (16 rows of d 64 are fewer chunks than threads)
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          h[i] = half2_bits(__floats2half2_rn(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up));
        *reinterpret_cast<uint4 *>(sQ + (ch >> 3) * (NR * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) =
            make_uint4(h[0], h[1], h[2], h[3]);
      }
      fence_proxy_async_smem();
    }
    tc_fence_before();
    named_bar_sync(kBarQ, kSoft + 32);

    // ---- draft visibility, when this part holds draft keys ----
    const bool has_draft = lt1 * TK > g.n_prefix;
    if (has_draft) {
      if (warp == 0) {
        const DraftPre dpre = draft_prefetch(p, g.b);
        uint64_t lo, hi;
        draft_rows(p, dpre, lo, hi);
        if (lane < p.T) rowmask[lane] = lo;
        if (lane + 32 < p.T) rowmask[lane + 32] = hi;
      }
      named_bar_sync(kBarSoft, kSoft);
      for (int e = tid; e < 64 * (NR > 32 ? NR / 32 : 1); e += kSoft) {
        const int key = e & 63, w = e >> 6;
        uint32_t km = 0;
        if (key < p.T) {
#pragma unroll 1
          for (int t = 0; t < p.T; ++t)
            if ((rowmask[t] >> key) & 1ull) km |= token_rows(t, w);
        }
        const int left = R - 32 * w;  // rows past the block's see nothing
        keymask[e] = left >= 32 ? km : left <= 0 ? 0u : km & ((1u << left) - 1u);
      }
      named_bar_sync(kBarSoft, kSoft);
    }

    // Reference of row r: ref[r] = kTqBias less it (infinity: no key seen), log2 units; in
    // shared memory, where a vector load gives four rows to every thread.
    float lsum[NW];    // sums of P over this thread's keys
#pragma unroll
    for (int r = 0; r < NW; ++r) lsum[r] = 0.f;
    // unit of the value scales: the largest one seen (0: no tile yet), at most kTqUnit once rows
    // have shifts of their own (apart); and one over it
    float vref = 0.f, rvref = 0.f;
    [[maybe_unused]] bool apart = false;
    [[maybe_unused]] float *vrow = reinterpret_cast<float *>(smem + SM::kVRowOff) + r_wg;
    const int skip = PAR == 2 ? (jt ^ par) & 1 : 0, lt_first = lt0 + skip;
    jt += skip;

    for (int lt = lt_first; lt < lt1; lt += PAR, jt += PAR) {
      const bool masked = lt * TK + TK > g.n_prefix;
      const uint32_t b = PAR == 2 ? (uint32_t)par : (uint32_t)jt & 1u;  // buffer of the tile
      const uint32_t tS = tLane + SM::kSCol + b * NC + r_wg;
      uint32_t km = ~0u;   // the thread's rows that see this key
      bool any = true;     // some row of the block does
      if (__builtin_expect(masked, 0)) {
        const int key = lt * TK + ktid, d = key - g.n_prefix;
        if (key >= g.nkeys) {
          km = 0u;
          any = false;
        } else if (d >= 0) {
          km = keymask[64 * rg + d];
          uint32_t all = 0;
#pragma unroll
          for (int w = 0; w < (NR > 32 ? NR / 32 : 1); ++w) all |= keymask[64 * w + d];
          any = all != 0u;
        }
      }
      wait_ok(a_k_full + 8 * (jt & 3), (uint32_t)(jt >> 2) & 1u);
      const float2 sc = lds64f(a_scale + (jt & 3) * 1024);
      // (a value row that is NaN makes the scores of its key NaN)
      const float vsc = sc.y, cs = fmaf(sc.x, q_unit, vsc - vsc);
      wait_ok(a_s_full + 8 * b, (uint32_t)(jt >> 1) & 1u);
      __syncwarp();
      tc_fence_after();
      float x[kXRows];
      // scores of this key above the references (and 2^6 in weight), -inf where unseen: rows
      // [h, h + kXRows)
      auto load_scores = [&](int h) {
        tmem_ld_f<kXRows>(tS + h, x);
        if (__builtin_expect(masked, 0)) {
#pragma unroll
          for (int r = 0; r < kXRows; r += 4) {
            const float4 n4 = lds128f(a_ref + 4 * (h + r));
            const float nn[4] = {n4.x, n4.y, n4.z, n4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[r + i] = (km >> (h + r + i)) & 1u ? fmaf(x[r + i], cs, nn[i] == INFINITY ? kTqBias : nn[i]) : -INFINITY;
          }
        } else {
#pragma unroll
          for (int r = 0; r < kXRows; r += 4) {
            const float4 n4 = lds128f(a_ref + 4 * (h + r));
            const float2 y = fma2(make_float2(x[r], x[r + 1]), make_float2(cs, cs), make_float2(n4.x, n4.y));
            const float2 z = fma2(make_float2(x[r + 2], x[r + 3]), make_float2(cs, cs), make_float2(n4.z, n4.w));
            x[r] = y.x;
            x[r + 1] = y.y;
            x[r + 2] = z.x;
            x[r + 3] = z.y;
          }
        }
      };
      // First tile of the part: its row maxima are the references (the scores of one key as
      // a first guess were passed by 2^8 in some row of most parts, once or twice, and each
      // move costs as much as several tiles).  Later they move when a score passes one.
      const bool first = vref == 0.f;
      bool move = first;
      if (__builtin_expect(!first, 1)) {
        float dmax = -INFINITY;
#pragma unroll
        for (int h = 0; h < NW; h += kXRows) {
          load_scores(h);
#pragma unroll
          for (int r = 0; r < kXRows; r += 2) dmax = max3f(dmax, x[r], x[r + 1]);
          if (__builtin_expect(masked, 0)) {  // (a row's first key moves its reference, however small the score)
#pragma unroll
            for (int r = 0; r < kXRows; ++r)
              if (((km >> (h + r)) & 1u) && ref[h + r] == INFINITY) dmax = INFINITY;
          }
        }
        // (two parities: a draft of 64 tokens has one tile in each)
        move = bar_red_or(kBarRed, 128, dmax > kTqBias + kTqMove || ((vsc > vref || (PAR == 1 && apart)) && any));
      }
      if (__builtin_expect(move, 0)) {
        // the references to the row maxima seen so far, and the value scale to the largest
#pragma unroll
        for (int h = 0; h < NW; h += kXRows) {
          if (first) {
            tmem_ld_f<kXRows>(tS + h, x);
#pragma unroll
            for (int r = 0; r < kXRows; ++r) x[r] = (km >> (h + r)) & 1u ? fmaf(x[r], cs, kTqBias) : -INFINITY;
          } else {
            load_scores(h);
          }
          WarpScatterMax<kXRows, 16>::run(x, lane);
          if ((lane & (32 / kXRows - 1)) == 0)
            reinterpret_cast<float *>(my_red + h)[(lane / (32 / kXRows)) * 4 + wq] = x[0];
        }
        {  // (NaN and the scales of keys that nobody sees stay out)
          const uint32_t wm = __reduce_max_sync(0xffffffffu, any && vsc == vsc ? __float_as_uint(vsc) : 0u);
          if (lane == 0) vred[warp] = __uint_as_float(wm);
          if (NR <= 32 && masked) {  // of the prefix, which every row sees
            const bool prefix = lt * TK + ktid < g.n_prefix;
            const uint32_t wp = __reduce_max_sync(0xffffffffu, prefix && vsc == vsc ? __float_as_uint(vsc) : 0u);
            if (lane == 0) vred[16 + warp] = __uint_as_float(wp);
          }
        }
        named_bar_sync(kBarRed, 128);
        const float vtile = fmaxf(fmaxf(vred[4 * wg], vred[4 * wg + 1]), fmaxf(vred[4 * wg + 2], vred[4 * wg + 3]));
        const bool shift = masked && (first || (PAR == 1 && apart) || vtile > vref);
        float vnew = fmaxf(fmaxf(vref, vtile), 0x1p-126f);
        if (shift) vnew = fminf(vnew, kTqUnit);
        float up = 0.f, vmax = 0x1p-126f;  // of row ktid: its largest score above the reference (or zero), its largest value scale
        if (ktid < NW) {
          const float4 m4 = my_red[ktid];
          up = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)) - kTqBias;
        }
        if (__builtin_expect(shift, 0)) {
          // Largest value scale of the tile's keys that a row sees (NaN stays out).  Up to 32 rows
          // the row's own thread goes through the draft keys, above a reduction over the keys as
          // for the scores.  (What this block does to the registers of the loop around it: one
          // token over 131072 4-bit keys 46.2 us, with the reduction 47.5, 64 sequences of one
          // token over 8192 keys 168 and 173; 16 tokens over 8-bit keys 79.6 and 76.6, 64 over
          // 4-bit keys 222 and 216.)
          if constexpr (NR <= 32) {
            const float4 pre = *reinterpret_cast<const float4 *>(vred + 16 + 4 * wg);
            const int d0 = g.n_prefix - lt * TK;  // the tile's first draft key
            uint32_t a_sc = a_scale + (jt & 3) * 1024 - ktid * 8 + max(d0, 0) * 8 + 4;
            uint32_t a_km = smem_a + SM::kKeyMaskOff + 256 * rg + max(-d0, 0) * 4;
            vmax = fmaxf(fmaxf(pre.x, pre.y), fmaxf(pre.z, pre.w));
            if (ktid < NW) {
#pragma unroll 1
              for (int i = min(d0 + p.T, TK) - max(d0, 0); i > 0; --i, a_sc += 8, a_km += 4)
                if ((lds32(a_km) >> ktid) & 1u) vmax = fmaxf(vmax, __uint_as_float(lds32(a_sc)));
            }
          } else {
            named_bar_sync(kBarRed, 128);  // (the maxima of the scores have been read)
#pragma unroll
            for (int h = 0; h < NW; h += kXRows) {
#pragma unroll
              for (int r = 0; r < kXRows; ++r) x[r] = ((km >> (h + r)) & 1u) && vsc == vsc ? vsc : 0.f;
              WarpScatterMax<kXRows, 16>::run(x, lane);
              if ((lane & (32 / kXRows - 1)) == 0)
                reinterpret_cast<float *>(my_red + h)[(lane / (32 / kXRows)) * 4 + wq] = x[0];
            }
            named_bar_sync(kBarRed, 128);
            const float4 m4 = my_red[ktid & (NW - 1)];
            vmax = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
          }
          vmax = fmaxf(fmaxf(vmax, 0x1p-126f), PAR == 1 && apart ? vrow[ktid & (NW - 1)] : vref);
        }
        if (ktid < NW) {
          const float old = first ? INFINITY : ref[ktid];
          const bool none = old == INFINITY;
          const float was = PAR == 1 && apart ? fminf(exponent_of(vref) - exponent_of(vrow[ktid]), kTqShift) : 0.f;
          const float is = shift ? fminf(exponent_of(vnew) - exponent_of(vmax), kTqShift) : 0.f;
          const float now = (none ? kTqBias - up : old - was - fmaxf(up - was, 0.f)) + is;
          alpha[ktid] = none ? 0.f : ex2_approx(now - old);
          ref[ktid] = now;
          if (PAR == 1 && shift) vrow[ktid] = vmax;
        }
        const float vdown = vref * (1.f / vnew);
        vref = vnew;
        rvref = 1.f / vref;
        if (PAR == 1) apart = shift;
        named_bar_sync(kBarRed, 128);
        if (!first) {
#pragma unroll
          for (int r = 0; r < NW; ++r) lsum[r] *= alpha[r];
          // O holds every PV up to the previous tile (of this parity)
          if (PAR == 2)
            wait_ok(a_o_done + 8 * b, (uint32_t)((jt - 2) >> 1) & 1u);
          else
            wait_ok(a_o_done + 8 * (b ^ 1u), (uint32_t)((jt - 1) >> 1) & 1u);
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < NW; h += 16) {
            float a[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) a[r] = alpha[h + r] * vdown;
            tmem_scale_cols<16>(tO + h, a);
            tmem_st_wait();
          }
        }
        if (kXRows == NW) load_scores(0);
      }
      // PV of tile jt - 2: its P buffer is free (and the barrier stays within a phase of its waiters)
      if (jt >= 2) wait_ok(a_o_done + 8 * b, (uint32_t)((jt - 2) >> 1) & 1u);
      const uint32_t a_p = a_p0 + b * SM::kPBytes;
      // P^T row of this key: chunk cc holds rows 8cc .. 8cc + 7
      // A power of two, at most 2^80 where somebody sees the key (elsewhere it may be anything
      // and P is 0: the product has to be).  It multiplies in fp32: as a half it is 0 below
      // 2^-24, where its product with a weight is not.
      const float ratio = fminf(fabsf(vsc * rvref), 0x1p80f);
#pragma unroll
      for (int h0 = 0; h0 < NW; h0 += kXRows) {
        if (kXRows != NW) load_scores(h0);
#pragma unroll
        for (int cw = 0; cw < kXRows / 8; ++cw) {
          uint32_t h[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int xr = 8 * cw + 2 * q, r = h0 + xr;
            const float a = ex2_approx(x[xr]), e = ex2_approx(x[xr + 1]);  // (0 where unseen)
            const float2 s2 = add2(make_float2(lsum[r], lsum[r + 1]), make_float2(a, e));
            lsum[r] = s2.x;
            lsum[r + 1] = s2.y;
            const float2 w2 = mul2(make_float2(a, e), make_float2(ratio, ratio));
            h[q] = half2_bits(__floats2half2_rn(w2.x, w2.y));
          }
          sts128(a_p ^ ((h0 / 8 + cw) << 4), h[0], h[1], h[2], h[3]);
        }
      }
      if (__builtin_expect(!any, 0)) {
        // a key that no row sees: zero V, so that 0 * V stays 0 whatever it held
        wait_ok(a_v_full + 8 * b, (uint32_t)(jt >> 1) & 1u);
#pragma unroll
        for (int c0 = 0; c0 < D / 8 / RG; ++c0)
          *reinterpret_cast<uint4 *>(sV + b * SM::kVBytes + swz<TK>(ktid, rg * (D / 8 / RG) + c0)) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive_at(a_p_full + 8 * b);
    }
    // the lane's parts that share this segment, and this one's slot: a lane has units + G of them
    const int first_part = tq_owner(tstart[u], cr.total, cr.G);
    const int n_parts = tq_owner(tstart[u + 1] - 1, cr.total, cr.G) - first_part + 1;
    const int lane_slot = cr.lane * (cr.units + cr.G) + u;
    // ---- epilogue: the two parities' O and l of every row of this part joined ----
    // (a warpgroup waits for the PVs of its own tiles, whose phases it has followed, and
    // meets the others at the barrier below)
    const bool mine = lt_first < lt1;  // this parity had a tile
    if (PAR == 2) {
      if (mine) wait_ok(a_o_done + 8 * par, (uint32_t)((jt - 2) >> 1) & 1u);
    } else {  // (the barrier of the tile before the last has been followed up to two tiles ago)
      if (jt >= 2) wait_ok(a_o_done + 8 * (jt & 1), (uint32_t)((jt - 2) >> 1) & 1u);
      wait_ok(a_o_done + 8 * ((jt - 1) & 1), (uint32_t)((jt - 1) >> 1) & 1u);
    }
    __syncwarp();
    tc_fence_after();
    jt = jt0 + (lt1 - lt0);
    const size_t slot = (size_t)(lane_slot + cr.part);
#pragma unroll
    for (int h = 0; h < NW; h += 16) {
      WarpScatterSum<16, 16>::run(lsum + h, lane);
      if ((lane & 1) == 0) reinterpret_cast<float *>(my_red + h)[(lane / 2) * 4 + wq] = mine ? lsum[h] : 0.f;
    }
    if (!mine && ktid < NW) ref[ktid] = INFINITY;
    // (after the barrier: the other parity's readers of vred may still be in their last tile)
    tc_fence_before();
    named_bar_sync(kBarSoft, kSoft);
    tc_fence_after();
    if (lane == 0 && wq == 0) vred[wg] = mine ? vref : 0.f;
    named_bar_sync(kBarSoft, kSoft);
    if (tid < NR) {
      // row tid: O = f0 O_even + f1 O_odd, in units of the row sum
      const float4 e4 = red[tid];
      float l = (e4.x + e4.y) + (e4.z + e4.w), nm = refs[tid], f0 = 1.f, f1 = 0.f;
      if constexpr (PAR == 2) {
        const float4 d4 = red[NR + tid];
        const float l1 = (d4.x + d4.y) + (d4.z + d4.w), n0 = nm, n1 = refs[NR + tid];
        nm = fminf(n0, n1);
        f0 = n0 == INFINITY ? 0.f : ex2_approx(nm - n0);
        f1 = n1 == INFINITY ? 0.f : ex2_approx(nm - n1);
        l = l * f0 + l1 * f1;
      }
      const bool seen = !(l == 0.f);  // (NaN: a row that holds one)
      const float inv = tid < R && seen ? 1.f / l : 0.f;
      alphas[tid] = inv * f0 * vred[tid / NW];
      if constexpr (PAR == 2) alphas[NR + tid] = inv * f1 * vred[RG + tid / NW];
      if (tid < R && ok) {
        const int t = token_of(base + tid), hq = g.hkv * group + (base + tid) - t * group;
        const float lse_nat = seen ? (__log2f(l) - nm) * kLn2 : -INFINITY;
        if (n_parts == 1)
          p.lse[((size_t)g.b * p.Hq + hq) * p.T + t] = lse_nat;
        else
          p.lse_part[slot * p.rows_pad + tid] = lse_nat;
      }
    }
    named_bar_sync(kBarSoft, kSoft);
    constexpr int HR = NR / WG;            // rows that a warpgroup writes
    const int e0 = wg * HR;
    float ov[HR];
    tmem_ld_f<HR>(tLane + e0, ov);
    if constexpr (PAR == 2) {
      const bool has0 = lt0 + (jt0 & 1) < lt1, has1 = lt0 + ((jt0 & 1) ^ 1) < lt1;  // (TMEM of no tile holds anything)
      float od[HR];
      tmem_ld_f<HR>(tLane + NC + e0, od);
#pragma unroll
      for (int j = 0; j < HR; ++j)
        ov[j] = (has0 ? ov[j] * alphas[e0 + j] : 0.f) + (has1 ? od[j] * alphas[NR + e0 + j] : 0.f);
    } else {
#pragma unroll
      for (int j = 0; j < HR; ++j) ov[j] *= alphas[e0 + j];
    }
    if (n_parts > 1) {
      // fp32 part: thread d stores column d of the rows (a warp writes 128 contiguous bytes of a row)
      float *orow = p.o_part + (slot * p.rows_pad + e0) * D + ktid;
      if (ok && (D == 128 || ktid < D)) {
#pragma unroll
        for (int j = 0; j < HR; ++j) orow[j * D] = ov[j];
      }
      // publish the part (always, so the counters return to zero): the block barrier
      // orders every thread's stores before thread 0's release increment
      tc_fence_before();
      named_bar_sync(kBarSoft, kSoft);
      if (tid == 0 && c != p.test_drop_part)
        red_release_inc_gpu(reinterpret_cast<unsigned *>(&p.merge_cnt[s].x), 2u * n_parts - 1u);
      if (n_split < 2) {
        ms[n_split] = s;
        mslot[n_split] = lane_slot + first_part;
        mnp[n_split] = n_parts;
        mpart[n_split] = cr.part - first_part;
        ++n_split;
      }
    } else {
      // final bf16 rows, staged in the Q buffer: the group rows of one draft token are contiguous in out
      __nv_bfloat16 *stage_b = reinterpret_cast<__nv_bfloat16 *>(sQ);
      if (D == 128 || ktid < D) {
#pragma unroll
        for (int j = 0; j < HR; ++j) stage_b[(e0 + j) * D + ktid] = __float2bfloat16_rn(ov[j]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      named_bar_sync(kBarSoft, kSoft);
      if (ok && tid < p.T) {
        const int t = tid, r0 = max(t * group - base, 0), n = min((t + 1) * group - base, R) - r0;
        if (n > 0) {
          __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                               (((size_t)g.b * p.T + t) * p.Hq + g.hkv * group + (base + r0 - t * group)) * D;
          const __nv_bfloat16 *src = stage_b + (size_t)r0 * D;
          if (p.out_align16) {
            bulk_store_s2g(dst, src, (uint32_t)(n * D * 2));
            bulk_commit();
            bulk_wait_read_all();
          } else {
            for (int e = 0; e < n * D; ++e) dst[e] = src[e];
          }
        }
      }
      named_bar_sync(kBarSoft, kSoft);
    }
  }
  bulk_wait_all();

  // ---- merge of the split segments: each of a segment's CTAs merges a share of its rows ----
  volatile int *merge_ok = abort_flag + 1;
  for (int k = 0; k < n_split; ++k) {
    const int s = ms[k], np = mnp[k];
    if (tid == 0) *merge_ok = wait_parts_arrived(p, s, np) ? 1 : 0;
    named_bar_sync(kBarSoft, kSoft);  // thread 0's acquire, then the barrier, orders the reads below
    if (*merge_ok) {
      const int seg = s / p.NRB, base = s % p.NRB * NR, R = min(NR, p.R - base);
      const int r0 = mpart[k] * R / np, r1 = (mpart[k] + 1) * R / np;
      merge_rows_compact<D>(p, seg / p.Hkv, seg % p.Hkv, base, mslot[k], np, r0, r1, warp, 4 * WG, lane,
                            reinterpret_cast<float *>(smem + SM::kPOff), kBarSoft);
    }
    named_bar_sync(kBarSoft, kSoft);
    // leave: np arrivals and np departures wrap the counter back to zero
    if (tid == 0) red_relaxed_inc_gpu(reinterpret_cast<unsigned *>(&p.merge_cnt[s].x), 2u * np - 1u);
  }
  tc_fence_before();
  named_bar_sync(kBarEnd, kEndThreads);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Stages of the ring that fit beside the rest.
template <int FMT, int D, int NR>
static int tq_stages(const AttnParams &p) {
  using SM = TqSmem<FMT, D, NR>;
  const int n = (kSmemLimit - 1024 - SM::kRingOff - (p.S + 1) * 4) / (2 * SM::kRaw);  // S <= kMaxSegments
  return n > kTqStages ? kTqStages : n;
}

template <int FMT, int D, int NR, bool kTma>
static cudaError_t launch_tq_t(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                               cudaStream_t stream) {
  using SM = TqSmem<FMT, D, NR>;
  p.stages = tq_stages<FMT, D, NR>(p);
  auto kern = verify_attn_quant_kernel<FMT, D, NR, kTma>;
  cudaError_t e = allow_smem(kern);
  if (e != cudaSuccess) return e;
  // cooperative: every CTA is resident, so the wait for a segment's parts ends
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(TqCfg<NR>::kThreads);
  cfg.dynamicSmemBytes = 1024 + (size_t)SM::kRingOff + (size_t)p.stages * (2 * SM::kRaw) + (size_t)(p.S + 1) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, tmk, tmv);
}

template <int FMT, int D, bool kTma>
static cudaError_t launch_tq_blocks(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                    cudaStream_t stream) {
  if constexpr (quant_block_rows(128, FMT, D) == 128)
    return launch_tq_t<FMT, D, 128, kTma>(p, tmk, tmv, grid, stream);
  else
    return cudaErrorInvalidValue;
}

template <int FMT, int D>
static cudaError_t launch_tq(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                             cudaStream_t stream) {
  if (p.tma_box > 0)
    return p.rows_pad == 16   ? launch_tq_t<FMT, D, 16, true>(p, tmk, tmv, grid, stream)
           : p.rows_pad == 32 ? launch_tq_t<FMT, D, 32, true>(p, tmk, tmv, grid, stream)
           : p.rows_pad == 64 ? launch_tq_t<FMT, D, 64, true>(p, tmk, tmv, grid, stream)
                              : launch_tq_blocks<FMT, D, true>(p, tmk, tmv, grid, stream);
  return p.rows_pad == 16   ? launch_tq_t<FMT, D, 16, false>(p, tmk, tmv, grid, stream)
         : p.rows_pad == 32 ? launch_tq_t<FMT, D, 32, false>(p, tmk, tmv, grid, stream)
         : p.rows_pad == 64 ? launch_tq_t<FMT, D, 64, false>(p, tmk, tmv, grid, stream)
                            : launch_tq_blocks<FMT, D, false>(p, tmk, tmv, grid, stream);
}

}  // namespace va
