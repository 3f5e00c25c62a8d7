// Verification attention on the 5th-generation tensor cores with the KEYS on
// the TMEM lanes, for segments of at most 64 packed query rows (GQA group x T
// draft tokens; a chain of 8 drafts with group 4 gives 32 rows; d 64 with score
// shaping comes in blocks of 64 rows above that).  One MMA has
// M = 128, so rather than padding 32 query rows to 128 the products are taken
// transposed, with a 128-key tile as the M side:
//
//   S^T (128 keys x NR rows)   = K (128 x d) . Q^T       A = K tile, K-major; B = Q, K-major
//   O^T (128 d x 2NR)         += V^T . [P_hi | P_lo]^T   A = V tile, MN-major; B = P^T, MN-major
//   l   (2NR, every lane)     += 1 (128 x 128) . [P_hi | P_lo]^T   (64 rows only; A = ones in TMEM)
//
// (LongSpec 2.C: the unmasked prefix and the masked draft block are the same
// tile loop, the draft block being the last tiles of a segment; partial
// results of a segment split over CTAs are merged by the exact log-sum-exp
// combine.)  P is split into a bf16 high part and the bf16 rounding of its
// residual, and both are multiplied by ONE MMA whose N covers the two halves:
// the accumulator columns of O_hi and O_lo sit side by side and are added in
// the epilogue.  ~16 bits of every weight survive, so a row whose weight rests
// on a few keys (attention sinks) keeps the exact result to well below the
// bf16 output rounding, at no extra MMA: an MMA of N <= 128 costs the same
// issue time as one of half that width.
//
// Roles (6 warps, 7 when a second producer warp shares a gather; one CTA per
// SM, cooperative launch):
//   warps 0-3  softmax: thread k owns key k of the tile (TMEM lane k) and all
//              NR rows of it.  Scores are taken in log2 units against a
//              per-row reference max that moves only when some score of the
//              tile exceeds it by more than 2^8 (exact either way: the
//              exponentials stay below 2^8 and O, l are rescaled when it
//              moves); whether it must move is one block-wide vote (bar.red),
//              and only then are the row maxima reduced across the 128 keys.
//              P (bf16 hi and lo parts) is written as the MN-major P^T
//              operand over the K tile of the same stage, which the S MMA has
//              finished reading.  In the epilogue thread d owns output column d.
//   warp 4     producer: TMA boxes (dense, paged with pages of 8 rows or more)
//              or cp.async gathers (sparse, small pages) into a 3-stage ring
//              of 128-key K and V tiles (64 KB a stage)
//   warp 5     MMA issuer and TMEM owner: S of tile i+2 is issued as soon as
//              the softmax of tile i has released its S buffer.
// TMEM columns (NC = max(NR, 32)): O^T hi at 0 and lo at NR, S buffers at 2NC
// and 3NC, the ones operand at 4NC, l hi / lo (64 rows) at 5NC and 5NC + NR.
// Every wait is bounded; on timeout the CTA
// records VA_ERR_TIMEOUT, keeps the barrier sequence of all roles, drains and
// frees TMEM.
//
// With score shaping (va_mod.cuh) the raw products a softmax thread has loaded
// are capped and biased in its registers before anything else looks at them; a
// thread owns one key, so the key's position is one number and the rows' slopes
// and offsets are broadcast from shared memory.  What the cap adds, five packed
// instructions for two scores at least, made the four softmax warps the bound; above 16
// rows there are therefore eight (TkCfg), and the 1024-key window of 64 paged
// sequences went from 126 to 93 us, the capped 8-token chain over 32K from 39.7
// to 34.7 us.  What bounds them now: HBM for long prefixes (single tokens over
// 32 kv-heads: 98% of the measured copy rate), the segments' beginnings and ends
// for short ones (about four tiles' time each, see kSegCost).
#pragma once

#include <cuda.h>
#include <math.h>

#include "va_common.cuh"
#include "va_kernels.h"
#include "va_pipeline.cuh"
#include "va_merge.cuh"
#include "va_rope_fused.cuh"
#include "va_tcgen05.cuh"

namespace va {

constexpr int kTkKeys = 128;  // keys per tile
// Warps: 0-3 softmax, 4 producer, 5 MMA issuer, then NR <= 32 adds a second
// producer warp that shares the cp.async gather of the paged / sparse layouts
// (one warp's gather is limited by the copies it can keep in flight).  Seven
// warps leave at most two per SM sub-partition, so 255 registers stay available.
// kTma: 0 gathers, 1 TMA boxes, 2 TMA boxes issued by two producer warps (score
// shaping, pages below 64 rows).
// Two softmax warpgroups share a tile's rows (score shaping, more than 16 rows):
// each keeps half of them, so the two are two independent halves of the softmax
// on the same S, P and O buffers, and a tile takes a thread half the work.  Ten or
// eleven warps leave 168 registers a thread, which the 64-row instances exceed by
// some 90 bytes; loading the next segment's Q ahead cost 440 bytes of spills and
// took the window from 88 to 97 us, so it is not done.
template <int NR, int kTma, int kMod>
struct TkCfg {
  static constexpr int kProducers = kTma == 2 || (kTma == 0 && NR <= 32) ? 2 : 1;
  static constexpr int kGroups = kMod != 0 && NR >= 32 ? 2 : 1;  // softmax warpgroups
  static constexpr int kThreads = (4 * kGroups + 1 + kProducers) * 32;
};

// D = 64 (score shaping only): a stage is half the size, so the ring is twice as
// long.  P hi and lo of 64 rows need 32 KB, twice a 64-wide K tile: K gets that
// room in the stage.  The PV MMA keeps M = 128: its lanes 64 to 127 multiply
// whatever follows the V tile in shared memory (16 KB past the last stage are
// part of the plan) and nobody reads them.
template <int D, int NR>
struct TkSmem {
  using Geo = StageGeom<__nv_bfloat16, D, kTkKeys>;
  static constexpr int kVOff = D == 64 && NR > 32 ? 2 * Geo::kTileBytes : Geo::kTileBytes;  // V tile in a stage
  static constexpr int kStageBytes = kVOff + Geo::kTileBytes;  // 64 KB (D 64: 32 or 48)
  static constexpr int kStages = D == 128 ? 3 : NR > 32 ? 4 : 6;
  static constexpr int kQOff = kStages * kStageBytes;
  static constexpr int kQBytes = (D / 64) * NR * 128;  // 128-byte columns of NR rows
  static constexpr int kBarOff = kQOff + kQBytes;
  // barriers: full[NS], empty[NS], s_full[2], p_full[2], o_done[2], drain
  static constexpr int kNumBars = 2 * kStages + 7;
  static constexpr int kMiscOff = (kBarOff + kNumBars * 8 + 15) & ~15;  // tmem base, abort flag, merge flag
  static constexpr int kRowMaskOff = kMiscOff + 16;        // u64 [64]: draft visibility rows
  static constexpr int kKeyMaskOff = kRowMaskOff + 512;    // u64 [64]: per draft key, rows that see it
  static constexpr int kRedOff = kKeyMaskOff + 512;        // float4 [NR]: per-warp row maxima
  static constexpr int kRowInvOff = kRedOff + NR * 16;     // float [64]: 1 / l per row (epilogue)
  // then the rotary table of the segment (rope_table_bytes, 0 without
  // positions), or with score shaping float2 [64] (slope, offset) of the rows
  // and int [64] first visible keys of the draft tokens and the ranges of the
  // first sequences, and the tile starts of the work plan
  static constexpr int kRopeOff = kRowInvOff + 256;
  // (d 64, 64 rows: and uint64 [64] rows of the draft tokens)
  static constexpr int kTokRowsOff = 64 * 8 + 64 * 4 + kModCache * 16;
  static constexpr int kModBytes = kTokRowsOff + (D == 64 && NR == 64 ? 64 * 8 : 0);
  static_assert(kQOff % 1024 == 0 && kQBytes % 1024 == 0, "UMMA operands need 1024-byte aligned swizzle atoms");
  static_assert(kBarOff % 8 == 0 && kRowMaskOff % 8 == 0 && kKeyMaskOff % 8 == 0, "8-byte alignment");
  static_assert(kRedOff % 16 == 0, "float4 array needs 16-byte alignment");
  static_assert(kRowInvOff % 16 == 0, "vector loads of the row constants");
  static constexpr int kNC = NR < 32 ? 32 : NR;            // TMEM columns per region
  static constexpr int kTmemCols = NR <= 32 ? 256 : 512;
  // O_hi | O_lo take columns [0, 2NR): within O and the (unused) l region for
  // NR <= 32; for 64 rows l moves past the ones operand
  static constexpr int kLCol = NR <= 32 ? kNC : 5 * kNC;
  static_assert(2 * NR <= 2 * kNC && kLCol + 2 * NR <= kTmemCols, "TMEM plan");
};

// Row-wise block of a warp: v[N] per lane -> lane holds the warp maximum of
// max(N/32, 1) rows (row j + (N/32)*lane for N >= 32, lane / (32/N) below).
template <int N, int O>
struct WarpScatterMax {
  static __device__ __forceinline__ void run(float *v, int lane) {
    if constexpr (O == 0) {
      return;
    } else if constexpr (N >= 2) {
      constexpr int H = N / 2;
      const bool up = (lane & O) != 0;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float send = up ? v[i] : v[i + H];
        const float keep = up ? v[i + H] : v[i];
        v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, O));
      }
      WarpScatterMax<H, O / 2>::run(v, lane);
    } else {
      v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], O));
      WarpScatterMax<1, O / 2>::run(v, lane);
    }
  }
};

// The same reduce-scatter with sums: lane l ends with the warp's sum of the
// rows WarpScatterMax leaves it.
template <int N, int O>
struct WarpScatterSum {
  static __device__ __forceinline__ void run(float *v, int lane) {
    if constexpr (O == 0) {
      return;
    } else if constexpr (N >= 2) {
      constexpr int H = N / 2;
      const bool up = (lane & O) != 0;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float send = up ? v[i] : v[i + H];
        const float keep = up ? v[i + H] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, O);
      }
      WarpScatterSum<H, O / 2>::run(v, lane);
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], O);
      WarpScatterSum<1, O / 2>::run(v, lane);
    }
  }
};

// NR fp32 columns of this thread's TMEM lane.
template <int NR>
__device__ __forceinline__ void tmem_ld_f(uint32_t taddr, float (&x)[NR]) {
  if constexpr (NR == 8) {
    uint32_t u[8];
    tmem_ld8(taddr, u);
    tmem_ld_wait(u);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(u[j]);
  } else if constexpr (NR == 16) {
    uint32_t u[16];
    tmem_ld16(taddr, u);
    tmem_ld_wait(u);
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(u[j]);
  } else {
#pragma unroll
    for (int h = 0; h < NR / 32; ++h) {
      uint32_t u[32];
      tmem_ld32(taddr + 32 * h, u);
      tmem_ld_wait(u);
#pragma unroll
      for (int j = 0; j < 32; ++j) x[32 * h + j] = __uint_as_float(u[j]);
    }
  }
}

// O_hi + O_lo: N fp32 columns at taddr plus the N columns `lo` further on.
template <int N>
__device__ __forceinline__ void tmem_ld_hilo(uint32_t taddr, uint32_t lo, float (&x)[N]) {
  float y[N];
  tmem_ld_f<N>(taddr, x);
  tmem_ld_f<N>(taddr + lo, y);
#pragma unroll
  for (int j = 0; j < N; ++j) x[j] += y[j];
}

// Multiply column j of this lane's NR columns at taddr by a[j].
template <int NR>
__device__ __forceinline__ void tmem_scale_cols(uint32_t taddr, const float *a) {
  if constexpr (NR == 16) {
    uint32_t u[16];
    tmem_ld16(taddr, u);
    tmem_ld_wait(u);
#pragma unroll
    for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * a[j]);
    tmem_st16(taddr, u);
  } else {
    // 16 columns at a time, each stored before the next is loaded: this rare
    // path then needs few registers next to the 64-row softmax state
#pragma unroll
    for (int h = 0; h < NR / 16; ++h) {
      uint32_t u[16];
      tmem_ld16(taddr + 16 * h, u);
      tmem_ld_wait(u);
#pragma unroll
      for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * a[16 * h + j]);
      tmem_st16(taddr + 16 * h, u);
      tmem_st_wait();
    }
  }
}

// kMod: 0 without score shaping, 1 with a window or document start only (the
// scores are the plain ones), 2 with a cap or slopes.
template <int D, int NR, int kTma, bool kRope, int kMod>
__global__ void __launch_bounds__(TkCfg<NR, kTma, kMod>::kThreads, 1)
    verify_attn_tck_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmk,
                           const __grid_constant__ CUtensorMap tmv) {
  using SM = TkSmem<D, NR>;
  using Geo = typename SM::Geo;
  constexpr int TK = kTkKeys;
  constexpr int NS = SM::kStages;
  constexpr int NC = SM::kNC;
  using Cfg = TkCfg<NR, kTma, kMod>;
  constexpr int WG = Cfg::kGroups;
  constexpr int NW = NR / WG;  // rows of a softmax thread
  // d 64: more than 64 rows come as blocks of 64, each a segment of its own (d 128
  // has the kernel with the rows on the lanes for them)
  constexpr bool kBlocks = D == 64 && NR == 64 && kMod != 0;
  constexpr int kSoft = 128 * WG;
  // up to 32 rows a thread: the row sums l are kept by the softmax threads (each over its own
  // keys, reduced once per segment part) instead of a ones-operand MMA per tile
  constexpr bool kRegL = NW <= 32;
  static_assert(!(kRope && kMod != 0), "the two share their shared-memory table");
  constexpr int kProducerWarp = 4 * WG, kMmaWarp = 4 * WG + 1;
  constexpr int kBarQ = 1, kBarSoft = 3, kBarEnd = 4, kBarRed0 = 5;  // kBarRed0 + softmax warpgroup
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *stages = smem;
  uint8_t *sQ = smem + SM::kQOff;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SM::kBarOff);
  uint64_t *full = bars;
  uint64_t *empty = bars + NS;
  uint64_t *s_full = bars + 2 * NS;      // [b]
  uint64_t *p_full = bars + 2 * NS + 2;  // [b]
  uint64_t *o_done = bars + 2 * NS + 4;  // [tile & 1]
  uint64_t *drain = bars + 2 * NS + 6;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SM::kMiscOff);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SM::kMiscOff + 4);
  uint64_t *rowmask = reinterpret_cast<uint64_t *>(smem + SM::kRowMaskOff);
  uint64_t *keymask = reinterpret_cast<uint64_t *>(smem + SM::kKeyMaskOff);
  float4 *red = reinterpret_cast<float4 *>(smem + SM::kRedOff);
  float *row_inv = reinterpret_cast<float *>(smem + SM::kRowInvOff);
  float2 *rope_tab = reinterpret_cast<float2 *>(smem + SM::kRopeOff);
  int *tstart = reinterpret_cast<int *>(smem + SM::kRopeOff + (kRope ? rope_table_bytes(p) : kMod != 0 ? SM::kModBytes : 0));
  float2 *mod_row = reinterpret_cast<float2 *>(smem + SM::kRopeOff);       // (slope, offset) of row r
  int *mod_first = reinterpret_cast<int *>(smem + SM::kRopeOff + 64 * 8);  // first visible key of token t
  uint64_t *tok_rows = reinterpret_cast<uint64_t *>(smem + SM::kRopeOff + SM::kTokRowsOff);
  constexpr bool use_tma = kTma != 0;  // tiles by TMA boxes (dense, paged), else cp.async gathers

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int c = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, (use_tma ? 1 : 32) * Cfg::kProducers);
      mbar_init(empty + i, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full + b, c == p.test_stall ? kNever : 1);
      mbar_init(p_full + b, kSoft);
    }
    mbar_init(o_done + 0, 1);
    mbar_init(o_done + 1, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  const CtaRange cr = plan_cta<TK, kMod != 0>(
      p, tstart, reinterpret_cast<int4 *>(smem + SM::kRopeOff + 64 * 8 + 64 * 4));  // contains __syncthreads
  if (c >= cr.G) return;
  const int t1 = cr.t1, s0 = cr.s0;

  if (warp == kProducerWarp || warp > kMmaWarp) {
    bool pok = true;
    produce_tiles<__nv_bfloat16, D, NS, TK, NS - 1, Cfg::kProducers, kTma, kMod != 0, SM::kVOff>(
        p, &tmk, &tmv, tstart, cr, stages, full, empty, abort_flag, use_tma, pok,
        warp == kProducerWarp ? 0 : warp - kMmaWarp);
    return;
  }

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(SM::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  named_bar_sync(kBarEnd, kSoft + 32);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // scores stay raw until the exponential; capped or biased ones are in base-2 units already
  const float cl2 = kMod == 2 ? 1.f : p.scale * kLog2e;
  const int group = p.Hq / p.Hkv;

  bool ok = true;
  auto wait_ok = [&](uint64_t *bar, uint32_t parity) { role_wait(bar, parity, ok, abort_flag, p.wait_ns, p.status); };

  if (warp == kMmaWarp) {
    // (after giving up, too, this warp goes on issuing: no lane may leave the warp that
    // elects an issuer; the MMAs stay inside the buffers and nobody keeps their results)
    // ================================ MMA issuer ================================
    const uint32_t id_s = umma_idesc(128, NR, 0, 0);
    const uint32_t id_o = umma_idesc(128, 2 * NR, 1, 1);  // N = [P_hi | P_lo]
    const uint32_t id_l = umma_idesc(128, 2 * NR, 0, 1);
    const uint32_t tO = tmem, tL = tmem + SM::kLCol, tOnes = tmem + 4 * NC;
    int it = 0, jt = 0;
    // Shared-memory descriptors are built once; a K-step or stage offset is an
    // add to the start-address field (addresses stay below 256 KB, so the
    // 14-bit field never carries).
    const uint64_t dK0 = umma_sdesc(smem_u32(stages), 16, 1024);                      // K tile, K-major
    const uint64_t dQ0 = umma_sdesc(smem_u32(sQ), 16, 1024);                          // Q, K-major
    const uint64_t dV0 = umma_sdesc(smem_u32(stages) + SM::kVOff, TK * 128, 1024);  // V tile, MN-major
    // P^T over the K tile: per key a 128-byte row of the hi then lo parts (N =
    // 2NR <= 64, one swizzle atom wide), or for 64 rows hi and lo as two atoms
    // 16 KB apart
    const uint64_t dP0 = umma_sdesc(smem_u32(stages), TK * 128, 1024);
    constexpr uint64_t kStageStep = SM::kStageBytes >> 4;
    auto issue_s = [&](int b, int st, const Seg &g, int lt) {  // S^T(b) = K Q^T
      if (kRope && lt * TK + TK > g.n_prefix) {
        // the draft keys of this tile, rotated in place before the MMA reads them
        const int r0 = max(0, g.n_prefix - lt * TK), r1 = min(TK, g.nkeys - lt * TK);
        rope_rotate_tile_rows_bf16_call<D, TK>(stages + st * SM::kStageBytes, r0, r1, lt * TK + r0 - g.n_prefix,
                                               rope_tab, lane, 32);
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      const uint64_t dK = dK0 + (uint64_t)st * kStageStep;
      const uint32_t dS = tmem + (2 + b) * NC;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint64_t koff = (uint64_t)(((ks >> 2) * (TK * 128) + (ks & 3) * 32) >> 4);
        const uint64_t qoff = (uint64_t)(((ks >> 2) * (NR * 128) + (ks & 3) * 32) >> 4);
        umma_ss_warp(dS, dK + koff, dQ0 + qoff, id_s, ks > 0 ? 1u : 0u);
      }
      umma_commit_warp(s_full + b);
    };
    auto issue_pv = [&](int st, int b, bool first) {  // [O_hi|O_lo]^T += V^T [P_hi|P_lo]^T
      tc_fence_after();
      const uint64_t dV = dV0 + (uint64_t)st * kStageStep;
      const uint64_t dP = dP0 + (uint64_t)st * kStageStep;
      const uint32_t acc0 = first ? 0u : 1u;
#pragma unroll
      for (int kk = 0; kk < TK / 16; ++kk) {
        const uint64_t off = (uint64_t)((kk * 2048) >> 4);
        const uint32_t acc = kk > 0 ? 1u : acc0;
        umma_ss_warp(tO, dV + off, dP + off, id_o, acc);
        if constexpr (!kRegL) umma_ts_warp(tL, tOnes, dP + off, id_l, acc);
      }
      umma_commit_warp(o_done + b);
      umma_commit_warp(empty + st);  // the stage is free once these MMAs have read it
    };

    for (int s = s0; s < p.S && tstart[s] < t1; ++s) {
      const Seg g = seg_at<kMod != 0, TK>(p, s, cr);
      int lt0, lt1;
      seg_tiles<kMod != 0>(tstart, s, cr, lt0, lt1);
      if (kMod != 0 && lt0 >= lt1) continue;
      named_bar_sync(kBarQ, kSoft + 32);  // Q of this segment is in shared memory
      wait_ok(full + it % NS, (uint32_t)(it / NS) & 1u);
      issue_s(jt & 1, it % NS, g, lt0);
      if (lt0 + 1 < lt1) {
        wait_ok(full + (it + 1) % NS, (uint32_t)((it + 1) / NS) & 1u);
        issue_s((jt + 1) & 1, (it + 1) % NS, g, lt0 + 1);
      }
      for (int lt = lt0; lt < lt1; ++lt, ++it, ++jt) {
        const int b = jt & 1;
        wait_ok(p_full + b, (uint32_t)(jt >> 1) & 1u);
        issue_pv(it % NS, b, lt == lt0);
        if (lt + 2 < lt1) {
          wait_ok(full + (it + 2) % NS, (uint32_t)((it + 2) / NS) & 1u);
          issue_s(b, (it + 2) % NS, g, lt + 2);
        }
        __syncwarp();
      }
    }
    // drain: every MMA issued has finished before TMEM is released
    umma_commit_warp(drain);
    mbar_wait(drain, 0u, p.wait_ns);
    tc_fence_before();
    named_bar_sync(kBarEnd, kSoft + 32);
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SM::kTmemCols)
                 : "memory");
    return;
  }

  // ================================== softmax ==================================
  const int wg = WG == 1 ? 0 : warp >> 2;     // softmax warpgroup: rows [r_wg, r_wg + NW)
  const int r_wg = wg * NW;
  const int wq = WG == 1 ? warp : warp & 3;   // warp of the warpgroup
  const int ktid = WG == 1 ? tid : tid & 127;  // key of the tile, and output column of the epilogue
  const int kBarRed = kBarRed0 + wg;
  const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
  const uint32_t tO = tmem + lane_base, tL = tO + SM::kLCol;
  if constexpr (WG == 1) {  // the all-ones A operand of the row-sum MMA: 8 columns of bf16 pairs (1.0, 1.0)
    uint32_t ones[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) ones[j] = 0x3F803F80u;
    tmem_st8(tO + 4 * NC, ones);
    tmem_st_wait();
  }
  int it = 0, jt = 0;
  int rope_b = -1;  // sequence whose rotary table is in shared memory
  // split segments this CTA holds a part of (at most its first and its last):
  // merged after its last tile
  int n_split = 0, ms[2] = {0, 0}, mslot[2] = {0, 0}, mnp[2] = {0, 0}, mpart[2] = {0, 0};
  for (int s = s0; s < p.S && tstart[s] < t1; ++s) {
    const Seg g = seg_at<kMod != 0, TK>(p, s, cr);
    int lt0, lt1;
    seg_tiles<kMod != 0>(tstart, s, cr, lt0, lt1);
    if (kMod != 0 && lt0 >= lt1) continue;
    const int first_cta = owner_cta(tstart[s] + (kMod != 0 ? cr.cost : 0), cr.total, cr.G);
    const int n_parts = owner_cta(tstart[s + 1] - 1, cr.total, cr.G) - first_cta + 1;
    if (lt0 == 0 && tid == 0) p.meta[s] = make_int2(s + first_cta, n_parts);
    // the packed rows [base, base + R) of the kv-head
    const int base = kBlocks ? g.rb * NR : 0, R = kBlocks ? min(NR, p.R - base) : p.R;
    // bit r: this segment's row r is one of draft token t
    auto token_rows = [&](int t) -> uint64_t {
      if constexpr (kBlocks) {
        const int lo = max(t * group - base, 0), hi = min((t + 1) * group - base, 64);
        return hi <= lo ? 0ull : (hi - lo >= 64 ? ~0ull : (1ull << (hi - lo)) - 1) << lo;
      } else {
        return (group >= 64 ? ~0ull : (1ull << group) - 1) << (t * group);
      }
    };

    // ---- Q of this segment into shared memory: [2 columns][NR rows][128 B], 128B swizzle ----
    // (the previous segment's MMAs have completed: its epilogue waited for the last one)
    if constexpr (kRope) {
      // rotary table of this sequence's draft tokens (kept while the CTA stays
      // on the sequence), then q rotated on its way in
      if (g.b != rope_b) {
        rope_build_table(p, g.b, rope_tab, tid, kSoft);
        named_bar_sync(kBarSoft, kSoft);
        rope_b = g.b;
      }
      const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(p.q);
      constexpr int kQIt = (NR * 8 + kSoft - 1) / kSoft;
      uint4 lo[kQIt], hi[kQIt];
#pragma unroll
      for (int u = 0; u < kQIt; ++u) {  // loads first: one round trip
        const int e = tid + u * kSoft;
        const int row = e >> 3;
        lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
        if (e < NR * 8 && row < p.R) {
          const int t = row / group;
          const int hq = g.hkv * group + row % group;
          const uint4 *src = reinterpret_cast<const uint4 *>(qb + (((size_t)g.b * p.T + t) * p.Hq + hq) * D);
          lo[u] = __ldg(src + (e & 7));
          hi[u] = __ldg(src + (e & 7) + 8);
        }
      }
#pragma unroll
      for (int u = 0; u < kQIt; ++u) {
        const int e = tid + u * kSoft;
        if (e >= NR * 8) continue;
        const int row = e >> 3, ch = e & 7;
        if (row < p.R) rope_rotate8_bf16(lo[u], hi[u], rope_tab + (row / group) * (D / 2) + ch * 8);
        *reinterpret_cast<uint4 *>(sQ + row * 128 + ((ch ^ (row & 7)) << 4)) = lo[u];
        *reinterpret_cast<uint4 *>(sQ + NR * 128 + row * 128 + ((ch ^ (row & 7)) << 4)) = hi[u];
      }
      fence_proxy_async_smem();
    } else {
      // every load of the thread in flight before the first store
      const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(p.q);
      constexpr int kCh = D / 8;  // 16-byte chunks of a row
      constexpr int kQIt = NR * kCh / kSoft;
      uint4 v[kQIt];
#pragma unroll
      for (int u = 0; u < kQIt; ++u) {
        const int e = tid + u * kSoft;
        const int row = e / kCh;
        v[u] = make_uint4(0, 0, 0, 0);
        if (row < R) {
          const int t = (base + row) / group;
          const int hq = g.hkv * group + (base + row) % group;
          v[u] = __ldg(reinterpret_cast<const uint4 *>(qb + (((size_t)g.b * p.T + t) * p.Hq + hq) * D) + (e % kCh));
        }
      }
#pragma unroll
      for (int u = 0; u < kQIt; ++u) {
        const int e = tid + u * kSoft;
        const int row = e / kCh, ch = e % kCh;
        *reinterpret_cast<uint4 *>(sQ + (ch >> 3) * (NR * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = v[u];
      }
      fence_proxy_async_smem();
    }
    tc_fence_before();
    named_bar_sync(kBarQ, kSoft + 32);  // (a wait: keeps the roles in step after a wait has run out)

    // ---- draft visibility, when this part holds draft keys: per draft key
    // dk, the packed rows r = t * group + h of the tokens t that see it.  Up to
    // 32 rows it is built at once, while the part's first tiles are still on
    // their way (chain -1%, sparse attention -3%); the 64-row instance, whose
    // hot loop has no registers to spare, loads the parents now and builds the
    // masks before the first draft tile ----
    DraftPre dpre{-1, -1, 0ull, 0ull};
    const bool has_draft = lt1 * TK > g.n_prefix;
    if (warp == 0 && has_draft) dpre = draft_prefetch(p, g.b);
    bool masks_ready = false;
    auto build_masks = [&]() {
      if (warp == 0) {
        uint64_t lo, hi;
        draft_rows(p, dpre, lo, hi);
        if (lane < p.T) rowmask[lane] = lo;
        if (lane + 32 < p.T) rowmask[lane + 32] = hi;
      }
      named_bar_sync(kBarSoft, kSoft);
      if (tid < p.T) {
        uint64_t kmask = 0;
        const int koff = kMod != 0 ? mod_off(p.mod, p.T, g.b, tid, g.L) : 0;
        for (int t = 0; t < p.T; ++t) {
          bool see = (rowmask[t] >> tid) & 1ull;
          if (kMod != 0 && p.mod.window > 0) see = see && mod_off(p.mod, p.T, g.b, t, g.L) - koff < p.mod.window;
          if (see) kmask |= kBlocks ? tok_rows[t] : token_rows(t);
        }
        keymask[tid] = kmask;
      }
      named_bar_sync(kBarSoft, kSoft);
      masks_ready = true;
    };
    if (NR <= 32 && has_draft) build_masks();
    // Score shaping: the rows' slopes and offsets, the first key each token sees,
    // where the part needs them (the previous segment's readers are past its
    // epilogue's barriers)
    bool ahead = true;  // no token sits before the end of the prefix
    if constexpr (kMod != 0) {
      const bool slopes = kMod == 2 && p.mod.slopes != nullptr, edge = lt0 * TK < g.hi;
      // (the masks of the draft keys come later, behind a barrier of their own)
      if (kBlocks && (edge || has_draft) && tid < p.T) tok_rows[tid] = token_rows(tid);
      if (slopes && tid < 64) {
        const int t = (base + tid) / group, hq = g.hkv * group + (base + tid) % group;
        mod_row[tid] = tid < R ? make_float2(mod_slope(p.mod, hq), (float)mod_off(p.mod, p.T, g.b, t, g.L))
                                 : make_float2(0.f, 0.f);
      }
      if (edge && tid < p.T)
        mod_first[tid] = mod_first_slot(p.mod, g.b, mod_off(p.mod, p.T, g.b, tid, g.L), g.L) - g.base;
      if (slopes || edge) ahead = !bar_red_or(kBarSoft, kSoft, slopes && tid < R && mod_row[tid].y < 0.f);
    }

    float mu[NW];  // reference max per row, log2 units
#pragma unroll
    for (int r = 0; r < NW; ++r) mu[r] = -INFINITY;
    // (kRegL) sums over this thread's keys of P (the fp32 weights, which the
    // bf16 hi + lo parts the PV MMA multiplies carry to ~2^-16)
    float lsum[kRegL ? NW : 1];
#pragma unroll
    for (int r = 0; r < (kRegL ? NW : 1); ++r) lsum[r] = 0.f;

    for (int lt = lt0; lt < lt1; ++lt, ++it, ++jt) {
      const int b = jt & 1;
      const int st = it % NS;
      const uint32_t tS = tO + (2 + b) * NC + r_wg;
      const int tile = kMod == 2 ? tile_of<true>(p, lt, lt0, lt1) : lt;
      const int key = tile * TK + ktid;
      const bool draft_tile = tile * TK + TK > g.n_prefix;
      const bool masked = draft_tile || (kMod != 0 && tile * TK < g.hi);
      if (NR > 32 && draft_tile && !masks_ready) build_masks();
      uint64_t km = ~0ull;  // rows that see this key
      if (masked) {
        if (key >= g.nkeys) km = 0;
        else if (key >= g.n_prefix) km = keymask[key - g.n_prefix];
        else if (kMod != 0 && key < g.hi) {
          km = 0;
          for (int t = 0; t < p.T; ++t)
            if (key >= mod_first[t]) km |= kBlocks ? tok_rows[t] : token_rows(t);
        }
      }
      const uint64_t km_all = km;
      if constexpr (WG > 1) km >>= r_wg;
      float koff = 0.f;  // the key's position relative to L
      const bool behind = kMod == 2 && !draft_tile && ahead;
      if constexpr (kMod == 2) {
        koff = (float)(key - g.n_prefix);
        if (p.mod.slopes != nullptr && key >= g.n_prefix && key < g.nkeys)
          koff = (float)mod_off(p.mod, p.T, g.b, key - g.n_prefix, g.L);
      }
      wait_ok(s_full + b, (uint32_t)(jt >> 1) & 1u);
      // PV of tile jt-2 (same o_done barrier): waiting for every PV in order,
      // two tiles late, keeps each barrier at most one phase ahead of its waiter
      if (jt >= 2) wait_ok(o_done + b, (uint32_t)((jt - 2) >> 1) & 1u);
      tc_fence_after();
      float x[NW];  // raw scores of this key, -inf where the row does not see it
      auto load_scores = [&]() {
        tmem_ld_f<NW>(tS, x);
        if constexpr (kMod == 2) {
          if (p.mod.softcap > 0.f) cap_scores<NW, false, false>(p.mod, x, km_all == 0ull, false);
          if (p.mod.slopes != nullptr) {
            const float mul = p.mod.softcap > 0.f ? 1.f : p.mod.out_mul;
            if (behind) {
              // every row is past the key: the bias is linear in the key's position
#pragma unroll
              for (int r = 0; r < NW; r += 2) {
                const float4 c = *reinterpret_cast<const float4 *>(mod_row + r_wg + r);
                const float2 y = fma2(make_float2(x[r], x[r + 1]), make_float2(mul, mul),
                                      make_float2(c.x * c.y, c.z * c.w));
                const float2 s2 = fma2(make_float2(c.x, c.z), make_float2(-koff, -koff), y);
                x[r] = s2.x;
                x[r + 1] = s2.y;
              }
            } else {
#pragma unroll
              for (int r = 0; r < NW; ++r) {
                const float2 c = mod_row[r_wg + r];
                x[r] = fmaf(c.x, fabsf(c.y - koff), x[r] * mul);
              }
            }
          }
        }
        if (masked) {
#pragma unroll
          for (int r = 0; r < NW; ++r)
            if (!((km >> r) & 1ull)) x[r] = -INFINITY;
        }
      };
      auto set_reference = [&]() {
        // first tile of this part: the scores of key 0 are the reference; the
        // vote below moves it to the exact maxima only when some score is more
        // than 2^8 above it (or key 0 is hidden from a row)
        // (at the edge of a window key 0 is mostly hidden, the tile's last key is not)
        if (ktid == (kMod != 0 && masked && !draft_tile ? TK - 1 : 0)) {
#pragma unroll
          for (int r = 0; r < NW; ++r) reinterpret_cast<float *>(red + r_wg)[r] = x[r] * cl2;
        }
        named_bar_sync(kBarRed, 128);
#pragma unroll
        for (int r = 0; r < NW; r += 4) {
          const float4 m4 = red[r_wg + (r >> 2)];
          mu[r] = m4.x;
          mu[r + 1] = m4.y;
          mu[r + 2] = m4.z;
          mu[r + 3] = m4.w;
        }
      };
      auto passed_reference = [&]() {
        float dmax = -INFINITY;  // (NaN where a row has seen nothing yet: ignored by fmaxf)
#pragma unroll
        for (int r = 0; r < NW; ++r) dmax = fmaxf(dmax, fmaf(x[r], cl2, -mu[r]));
        return bar_red_or(kBarRed, 128, dmax > 8.f);
      };
      auto move_reference = [&]() {
        // some score passed its reference by more than 2^8: move the references
        // to the exact row maxima seen so far
        WarpScatterMax<NW, 16>::run(x, lane);
        if constexpr (NW >= 32) {
#pragma unroll
          for (int j = 0; j < NW / 32; ++j)
            reinterpret_cast<float *>(red + r_wg)[(j + (NW / 32) * lane) * 4 + wq] = x[j];
        } else {
          if ((lane & (32 / NW - 1)) == 0) reinterpret_cast<float *>(red + r_wg)[(lane / (32 / NW)) * 4 + wq] = x[0];
        }
        named_bar_sync(kBarRed, 128);
        float *alpha = x;  // the scores are reloaded below
#pragma unroll
        for (int r = 0; r < NW; ++r) {
          const float4 m4 = red[r_wg + r];
          const float mnew = fmaxf(mu[r], fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)) * cl2);
          alpha[r] = mu[r] == -INFINITY ? 0.f : ex2_approx(mu[r] - mnew);
          mu[r] = mnew;
        }
        if constexpr (kRegL) {
#pragma unroll
          for (int r = 0; r < NW; ++r) lsum[r] *= alpha[r];
        }
        if (lt != lt0) {
          wait_ok(o_done + (b ^ 1), (uint32_t)((jt - 1) >> 1) & 1u);  // O and l hold every PV up to tile jt-1
          tc_fence_after();
          tmem_scale_cols<NW>(tO + r_wg, x);
          tmem_scale_cols<NW>(tO + NR + r_wg, x);
          if constexpr (!kRegL) {
            tmem_scale_cols<NW>(tL, x);
            tmem_scale_cols<NW>(tL + NR, x);
          }
          tmem_st_wait();
        }
      };
      if constexpr (kMod == 2) {
        // (one copy of the code that shapes the scores)
        bool moved = false;
#pragma unroll 1
        while (true) {
          load_scores();
          if (moved) break;
          if (lt == lt0) set_reference();
          if (!passed_reference()) break;
          move_reference();
          moved = true;
        }
      } else {
        load_scores();
        if (lt == lt0) set_reference();
        if (passed_reference()) {
          move_reference();
          load_scores();
        }
      }
      // P^T row of this key over the K tile of the stage (the S MMA is done with
      // it): chunk cc of the hi part, and of the lo part NR/8 chunks further
      // (64 rows: in the second swizzle atom, 16 KB further)
      uint8_t *pk = stages + st * SM::kStageBytes;
      const int sw = ktid & 7;
      auto put_p = [&](int cw, const uint32_t (&h)[4], const uint32_t (&l)[4]) {
        const int cc = r_wg / 8 + cw;
        *reinterpret_cast<uint4 *>(pk + ktid * 128 + ((cc ^ sw) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        if constexpr (NR <= 32)
          *reinterpret_cast<uint4 *>(pk + ktid * 128 + (((cc + NR / 8) ^ sw) << 4)) = make_uint4(l[0], l[1], l[2], l[3]);
        else
          *reinterpret_cast<uint4 *>(pk + TK * 128 + ktid * 128 + ((cc ^ sw) << 4)) = make_uint4(l[0], l[1], l[2], l[3]);
      };
      if (masked) {
#pragma unroll
        for (int cc = 0; cc < NW / 8; ++cc) {
          uint32_t h[4], l[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 8 * cc + 2 * q;
            // a row that has seen no key yet has mu = -inf and only -inf scores: P = 0
            const float2 e = fma2(make_float2(x[r], x[r + 1]), make_float2(cl2, cl2),
                                  make_float2(mu[r] == -INFINITY ? 0.f : -mu[r],
                                              mu[r + 1] == -INFINITY ? 0.f : -mu[r + 1]));
            const float a = ex2_approx(e.x), bq = ex2_approx(e.y);
            split_bf16x2(a, bq, h[q], l[q]);
            if constexpr (kRegL) {
              const float2 s2 = add2(make_float2(lsum[r], lsum[r + 1]), make_float2(a, bq));
              lsum[r] = s2.x;
              lsum[r + 1] = s2.y;
            }
          }
          put_p(cc, h, l);
        }
        if (kMod != 0 ? (R < 64 ? (km_all & ((1ull << R) - 1ull)) : km_all) == 0ull : (use_tma && key >= g.nkeys)) {
          // rows past the segment end: TMA brought whatever follows; zero V so 0 * V
          // stays 0 (with score shaping: every key that no row sees)
          wait_ok(full + st, (uint32_t)(it / NS) & 1u);
          uint8_t *vt = pk + SM::kVOff;
#pragma unroll
          for (int c0 = 0; c0 < D / 8 / WG; ++c0)
            *reinterpret_cast<uint4 *>(vt + swz<TK>(ktid, wg * (D / 8 / WG) + c0)) = make_uint4(0, 0, 0, 0);
        }
      } else {
        // every row sees every key of a prefix tile, so mu is finite here
#pragma unroll
        for (int cc = 0; cc < NW / 8; ++cc) {
          uint32_t h[4], l[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 8 * cc + 2 * q;
            const float2 e = fma2(make_float2(x[r], x[r + 1]), make_float2(cl2, cl2), make_float2(-mu[r], -mu[r + 1]));
            const float a = ex2_approx(e.x), bq = ex2_approx(e.y);
            split_bf16x2(a, bq, h[q], l[q]);
            if constexpr (kRegL) {
              const float2 s2 = add2(make_float2(lsum[r], lsum[r + 1]), make_float2(a, bq));
              lsum[r] = s2.x;
              lsum[r + 1] = s2.y;
            }
          }
          put_p(cc, h, l);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(p_full + b);
    }

    // ---- epilogue: column d = tid of O / l for every row of this segment part ----
    if (jt >= 2) wait_ok(o_done + (jt & 1), (uint32_t)((jt - 2) >> 1) & 1u);
    wait_ok(o_done + ((jt - 1) & 1), (uint32_t)((jt - 1) >> 1) & 1u);
    tc_fence_after();
    constexpr int CH = NW < 32 ? NW : 32;  // columns per TMEM load
    const size_t slot = (size_t)(s + c);
    // per-row constants, once: thread r (of the warpgroup) takes its row r (l is the same on every
    // lane); its l and reference max are picked out of the register arrays by
    // predicated selects, so the rows are done by the threads in parallel
    float my_l = 0.f, my_mu = 0.f;
    if constexpr (kRegL) {
      // l: this thread's key sums, reduce-scattered over the warp (lane l gets
      // row l, or l / 2 for 16 rows), then the four warps' sums of each row
      WarpScatterSum<NW, 16>::run(lsum, lane);
      if ((lane & (32 / NW - 1)) == 0) reinterpret_cast<float *>(red + r_wg)[(lane / (32 / NW)) * 4 + wq] = lsum[0];
      named_bar_sync(kBarSoft, kSoft);
      if (ktid < NW) {
        const float4 l4 = red[r_wg + ktid];
        my_l = (l4.x + l4.y) + (l4.z + l4.w);
      }
#pragma unroll
      for (int j = 0; j < NW; ++j) my_mu = ktid == j ? mu[j] : my_mu;
    } else {
#pragma unroll
      for (int h = 0; h < NR / CH; ++h) {
        float lv[CH];
        tmem_ld_hilo<CH>(tL + h * CH, NR, lv);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          my_l = tid == h * CH + j ? lv[j] : my_l;
          my_mu = tid == h * CH + j ? mu[h * CH + j] : my_mu;
        }
      }
    }
    if (ktid < NW && r_wg + ktid < R) {
      const int r = r_wg + ktid;
      const int t = (base + r) / group;
      const int hq = g.hkv * group + (base + r) % group;
      const bool seen = kMod != 0 ? mod_row_seen(my_l) : my_l > 0.f;
      const float lse_nat = seen ? (my_mu + __log2f(my_l)) * kLn2 : -INFINITY;
      row_inv[r] = seen ? __fdividef(1.f, my_l) : 0.f;
      if (ok) {
        if (n_parts == 1)
          p.lse[((size_t)g.b * p.Hq + hq) * p.T + t] = lse_nat;
        else
          p.lse_part[slot * p.rows_pad + r] = lse_nat;
      }
    }
    named_bar_sync(kBarSoft, kSoft);
    // column d = tid of O / l for every row, staged row-major in the Q buffer
    // (free: every MMA of this part has completed) and written by bulk copies
    if (n_parts > 1) {
      constexpr int HR = NW / 2;
      if constexpr (NW <= 32) {
        // fp32 part: thread d stores column d of every row straight from TMEM
        // (a warp writes 128 contiguous bytes of a row)
        float *orow = p.o_part + (slot * p.rows_pad + r_wg) * D + ktid;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float ov[HR];
          tmem_ld_hilo<HR>(tO + r_wg + half * HR, NR, ov);
          if (ok && (D == 128 || ktid < D)) {
#pragma unroll
            for (int j = 0; j < HR; j += 4) {
              const float4 inv4 = *reinterpret_cast<const float4 *>(row_inv + r_wg + half * HR + j);
              orow[(half * HR + j + 0) * D] = ov[j] * inv4.x;
              orow[(half * HR + j + 1) * D] = ov[j + 1] * inv4.y;
              orow[(half * HR + j + 2) * D] = ov[j + 2] * inv4.z;
              orow[(half * HR + j + 3) * D] = ov[j + 3] * inv4.w;
            }
          }
        }
        // publish the part (always, also after a failed wait, so the counters
        // return to zero): the block barrier orders every thread's row and lse
        // stores before thread 0's release increment, which is cumulative
        named_bar_sync(kBarSoft, kSoft);
        if (tid == 0 && c != p.test_drop_part)
          red_release_inc_gpu(reinterpret_cast<unsigned *>(&p.merge_cnt[s].x), 2u * n_parts - 1u);
      } else {
        // 64 rows (registers are short): rows staged row-major in the Q buffer,
        // two halves of NR/2 rows written by bulk copies
        float *stage_f = reinterpret_cast<float *>(sQ);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float ov[HR];
          tmem_ld_hilo<HR>(tO + half * HR, NR, ov);
#pragma unroll
          for (int j = 0; j < HR; j += 4) {
            if (D < 128 && tid >= D) break;
            const float4 inv4 = *reinterpret_cast<const float4 *>(row_inv + half * HR + j);
            stage_f[(j + 0) * D + tid] = ov[j] * inv4.x;
            stage_f[(j + 1) * D + tid] = ov[j + 1] * inv4.y;
            stage_f[(j + 2) * D + tid] = ov[j + 2] * inv4.z;
            stage_f[(j + 3) * D + tid] = ov[j + 3] * inv4.w;
          }
          fence_proxy_async_smem();
          named_bar_sync(kBarSoft, kSoft);
          if (tid == 0 && ok) {
            bulk_store_s2g(p.o_part + (slot * p.rows_pad + half * HR) * D, stage_f, (uint32_t)(HR * D * 4));
            bulk_commit();
            bulk_wait_read_all();
          }
          named_bar_sync(kBarSoft, kSoft);
        }
        // publish (always): the block barrier orders every thread's lse stores
        // before thread 0's release, which follows the landing of the bulk rows
        named_bar_sync(kBarSoft, kSoft);
        if (tid == 0) {
          bulk_wait_all();
          if (c != p.test_drop_part)
            red_release_inc_gpu(reinterpret_cast<unsigned *>(&p.merge_cnt[s].x), 2u * n_parts - 1u);
        }
      }
      if (n_split < 2) {
        ms[n_split] = s;
        mslot[n_split] = s + first_cta;
        mnp[n_split] = n_parts;
        mpart[n_split] = c - first_cta;
        ++n_split;
      }
    } else {
      // final bf16 rows: the group rows of one draft token are contiguous in out
      __nv_bfloat16 *stage_b = reinterpret_cast<__nv_bfloat16 *>(sQ);
#pragma unroll
      for (int h = 0; h < NW / CH; ++h) {
        float ov[CH];
        tmem_ld_hilo<CH>(tO + r_wg + h * CH, NR, ov);
#pragma unroll
        for (int j = 0; j < CH; j += 4) {
          if (D < 128 && ktid >= D) break;
          const float4 inv4 = *reinterpret_cast<const float4 *>(row_inv + r_wg + h * CH + j);
          stage_b[(r_wg + h * CH + j + 0) * D + ktid] = __float2bfloat16_rn(ov[j] * inv4.x);
          stage_b[(r_wg + h * CH + j + 1) * D + ktid] = __float2bfloat16_rn(ov[j + 1] * inv4.y);
          stage_b[(r_wg + h * CH + j + 2) * D + ktid] = __float2bfloat16_rn(ov[j + 2] * inv4.z);
          stage_b[(r_wg + h * CH + j + 3) * D + ktid] = __float2bfloat16_rn(ov[j + 3] * inv4.w);
        }
      }
      fence_proxy_async_smem();
      named_bar_sync(kBarSoft, kSoft);
      if (ok && tid < p.T) {
        const int t = tid;
        const int r0 = kBlocks ? max(t * group - base, 0) : t * group;  // its rows of the segment
        const int n = kBlocks ? min((t + 1) * group - base, R) - r0 : group;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                             (((size_t)g.b * p.T + t) * p.Hq + g.hkv * group + (base + r0 - t * group)) * D;
        const __nv_bfloat16 *src = stage_b + (size_t)r0 * D;
        if (kBlocks && n <= 0) {
        } else if (p.out_align16) {
          bulk_store_s2g(dst, src, (uint32_t)(n * D * 2));
          bulk_commit();
          bulk_wait_read_all();
        } else {
          for (int e = 0; e < n * D; ++e) dst[e] = src[e];
        }
      }
      named_bar_sync(kBarSoft, kSoft);
    }
  }
  // the output and part rows written by bulk copies have landed
  bulk_wait_all();

  // ---- merge of the split segments: once every part of a segment has
  // arrived, each of its CTAs merges an equal share of its rows ----
  volatile int *merge_ok = abort_flag + 1;
  for (int k = 0; k < n_split; ++k) {
    const int s = ms[k], np = mnp[k];
    if (tid == 0) *merge_ok = wait_parts_arrived(p, s, np) ? 1 : 0;
    named_bar_sync(kBarSoft, kSoft);  // thread 0's acquire, then the barrier, orders the reads below
    if (*merge_ok) {
      const int seg = kBlocks ? s / p.NRB : s, base = kBlocks ? s % p.NRB * NR : 0;
      const int R = kBlocks ? min(NR, p.R - base) : p.R;
      const int r0 = mpart[k] * R / np, r1 = (mpart[k] + 1) * R / np;
      if (np <= 4)
        merge_rows_warp<8, 4, D>(p, seg / p.Hkv, seg % p.Hkv, base, mslot[k], np, r0, r1, warp, 4 * WG, lane);
      else
        merge_rows_warp<D == 128 ? 32 : 16, 24, D>(p, seg / p.Hkv, seg % p.Hkv, base, mslot[k], np, r0, r1, warp, 4 * WG,
                                                   lane);
    }
    named_bar_sync(kBarSoft, kSoft);
    // leave: np arrivals and np departures wrap the counter back to zero
    if (tid == 0) red_relaxed_inc_gpu(reinterpret_cast<unsigned *>(&p.merge_cnt[s].x), 2u * np - 1u);
  }
  tc_fence_before();
  named_bar_sync(kBarEnd, kSoft + 32);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int D, int NR>
static size_t tck_smem_bytes(const AttnParams &p) {
  using SM = TkSmem<D, NR>;
  const size_t n = 1024 + (size_t)SM::kRopeOff + (size_t)(p.mod.on ? SM::kModBytes : rope_table_bytes(p)) +
                   (size_t)(p.S + 1) * 4;
  const size_t least = D == 64 ? 1024 + SM::kQOff + 16384 : 0;  // what the unused MMA lanes read
  return n > least ? n : least;
}

// A kernel instance with the rotary embedding, one with score shaping and one
// with neither: code that never runs still costs the hot loop registers and
// schedule.

// Launch of one instance.  Each translation unit that includes this file builds
// the instances of the launchers it defines (they take long to compile).
template <int D, int NR, int kTma, bool kRope, int kMod>
static cudaError_t launch_tck_t(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                cudaStream_t stream) {
  const size_t smem = tck_smem_bytes<D, NR>(p);
  auto kern = verify_attn_tck_kernel<D, NR, kTma, kRope, kMod>;
  cudaError_t e = allow_smem(kern);
  if (e != cudaSuccess) return e;
  // cooperative: every CTA is resident, so the wait for a segment's parts ends
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(TkCfg<NR, kTma, kMod>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, tmk, tmv);
}

template <int D, int NR, bool kRope, int kMod>
static cudaError_t launch_tck_nr(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                 cudaStream_t stream) {
  if (p.tma_box == 0) return launch_tck_t<D, NR, 0, kRope, kMod>(p, tmk, tmv, grid, stream);
  if (kMod == 0 || p.tma_box == 64) return launch_tck_t<D, NR, 1, kRope, kMod>(p, tmk, tmv, grid, stream);
  return launch_tck_t<D, NR, kMod == 0 ? 1 : 2, kRope, kMod>(p, tmk, tmv, grid, stream);
}

template <int D, bool kRope, int kMod>
static cudaError_t launch_tck(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                              cudaStream_t stream) {
  return p.rows_pad <= 16   ? launch_tck_nr<D, 16, kRope, kMod>(p, tmk, tmv, grid, stream)
         : p.rows_pad <= 32 ? launch_tck_nr<D, 32, kRope, kMod>(p, tmk, tmv, grid, stream)
                            : launch_tck_nr<D, 64, kRope, kMod>(p, tmk, tmv, grid, stream);
}

}  // namespace va
