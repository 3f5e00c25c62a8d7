// Accumulated attention weight: how much attention the accepted tokens of a
// step gave to every cached key, summed over the query heads of a kv-head and
// added to a running total.  The totals are the signal by which a cache is
// evicted (verify_build_index takes them as its score).
//
// After acceptance and commit, sequence b holds L_b + a keys and its accepted
// rows i < a (query rows path[i]) sit at positions L_b + i, a plain causal
// chain.  With the rows' log-sum-exp known from the verification call,
//   p(h, i, j) = exp(s(q[path[i]][h], k_j) - lse[h][path[i]]),  j <= L_b + i,
//   w[g][j]    = (j < L_b ? decay * w[g][j] : 0) + sum over h of g and i of p.
// With decay 0 the old totals are not read: they may be memory never written.
// No softmax pass and no V: K is read once for every 256 rows of a kv-head (the
// totals too), every total by one thread, in a fixed order (the result does not
// depend on the grid).
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "va_common.cuh"
#include "va_mod.cuh"
#include "va_pipeline.cuh"
#include "va_tcgen05.cuh"
#include "va_weight.h"

namespace va {

// Committed length and accepted tokens of sequence b; false (recorded once)
// when they do not fit the cache or the totals: that sequence is left alone.
__device__ __forceinline__ bool weight_seq(const WeightParams &p, int b, bool record, int &L, int &a) {
  L = __ldg(p.seqlens + b);
  a = p.n_accept != nullptr ? __ldg(p.n_accept + b) : p.T;
  const bool good = L >= 0 && a >= 0 && a <= p.T && L <= min(p.len_cap, p.stride) - a;
  if (!good && record) record_status(p.status, VA_ERR_DEVICE_BOUNDS);
  return good;
}

// Row of slot j of kv-head h (hidden slots may have any page entry: nullptr).
template <typename Tin>
__device__ __forceinline__ const Tin *weight_key(const WeightParams &p, int b, int h, int j, bool record) {
  size_t row;
  if (p.page_table != nullptr) {
    const int page = __ldg(p.page_table + (size_t)b * p.max_pages + (j >> p.page_shift));
    if (page < 0 || page >= p.num_pages) {
      if (record) record_status(p.status, VA_ERR_DEVICE_BOUNDS);
      return nullptr;
    }
    row = ((size_t)page << p.page_shift) + (size_t)(j & ((1 << p.page_shift) - 1));
  } else {
    row = (size_t)b * p.len_cap + j;
  }
  return static_cast<const Tin *>(p.k) + (row * p.Hkv + h) * p.D;
}

// fp32 (D = 64): one thread per key, its row in registers, query rows broadcast
// from shared memory; FMA-bound.
__global__ void __launch_bounds__(128) weight_simt_kernel(const WeightParams p) {
  constexpr int D = 64;
  constexpr int RC = 16;  // query rows staged at once
  __shared__ float4 sq[RC][D / 4];
  __shared__ float slse[RC], sns[RC];
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  int L, a;
  if (!weight_seq(p, b, blockIdx.x == 0 && h == 0 && tid == 0, L, a)) return;
  const int j0 = blockIdx.x * 128;
  if (j0 >= L + a) return;
  const int j = j0 + tid;
  const int group = p.Hq / p.Hkv, R = group * a;
  // the first slot each accepted row sees rises with the row: row 0's decides
  // whether anything of this tile is seen
  const int lo = mod_first_slot(p.mod, b, 0, L);
  const bool live = j < L + a && j >= lo;
  float k[D];
  const float *kr = live ? weight_key<float>(p, b, h, j, true) : nullptr;
#pragma unroll
  for (int i = 0; i < D; ++i) k[i] = 0.f;
  if (kr != nullptr) {
#pragma unroll
    for (int i = 0; i < D; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(kr + i));
      k[i] = v.x, k[i + 1] = v.y, k[i + 2] = v.z, k[i + 3] = v.w;
    }
  }
  float acc = 0.f;
  for (int r0 = 0; r0 < R; r0 += RC) {
    __syncthreads();
    for (int e = tid; e < RC * (D / 4); e += 128) {
      const int r = r0 + e / (D / 4), c = e % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < R) {
        const int i = r / group;
        const int t = p.path != nullptr ? __ldg(p.path + (size_t)b * p.T + i) : i;
        if (t >= 0 && t < p.T) {
          const float *qr = static_cast<const float *>(p.q) + (((size_t)b * p.T + t) * p.Hq + h * group + r % group) * D;
          v = __ldg(reinterpret_cast<const float4 *>(qr) + c);
        }
      }
      sq[e / (D / 4)][c] = v;
    }
    if (tid < RC) {
      const int r = r0 + tid;
      float l = INFINITY, ns = 0.f;  // no such row: exp(s - inf) = 0
      if (r < R) {
        const int i = r / group, hq = h * group + r % group;
        const int t = p.path != nullptr ? __ldg(p.path + (size_t)b * p.T + i) : i;
        if (t >= 0 && t < p.T) {
          l = __ldg(p.lse + ((size_t)b * p.Hq + hq) * p.T + t);
          if (l == -INFINITY) l = INFINITY;  // a row that saw no key
          if (p.mod.slopes != nullptr) ns = -__ldg(p.mod.slopes + hq);
        } else if (blockIdx.x == 0) {
          record_status(p.status, VA_ERR_DEVICE_BOUNDS);
        }
      }
      slse[tid] = l;
      sns[tid] = ns;
    }
    __syncthreads();
    const int rn = min(RC, R - r0);
    for (int r = 0; r < rn; ++r) {
      const int i = (r0 + r) / group;
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < D / 4; ++c) {
        const float4 v = sq[r][c];
        s = fmaf(v.x, k[4 * c], s);
        s = fmaf(v.y, k[4 * c + 1], s);
        s = fmaf(v.z, k[4 * c + 2], s);
        s = fmaf(v.w, k[4 * c + 3], s);
      }
      // natural units: the difference s - lse is small where the weight matters
      const float d = (float)(L + i - j);
      const float x = mod_score(p.mod, s, sns[r], d) - slse[r];
      bool see = kr != nullptr && j <= L + i;
      if (p.mod.window > 0) see = see && (j >= L + i - p.mod.window + 1);
      acc += see ? ex2_approx(x * kModLog2e) : 0.f;
    }
  }
  if (j < L + a) {
    float *w = p.weight + ((size_t)b * p.Hkv + h) * p.stride + j;
    *w = j < L && p.decay != 0.f ? fmaf(p.decay, *w, acc) : acc;
  }
}

// ---------------------------------------------------------------------------
// bf16: the products on the 5th-generation tensor cores, keys on the TMEM lanes
// ---------------------------------------------------------------------------
//   S^T (128 keys x N rows) = K (128 x D) . Q^T      A = K tile, B = Q, both K-major
// A thread owns one key of a tile, so the sum over the rows is the thread's own
// and neither P nor a reduction leaves its registers: per score an FMA, an
// exponential and an add.  K streams through a ring of TMA boxes (or cp.async
// gathers), N is the number of accepted rows rounded up to 32.
//
// Bound by HBM (K once) while a kv-head has few rows: 64 sequences of 2K to 8K
// keys (697 MB) take 123 us on 16-row pages and 110 us on 64-row pages, 5.7 and
// 6.3 TB/s.  With 256 rows a tile's 32,768 exponentials and its MMAs take longer
// than its 32 KB: 8 x 128K keys 68 us, 48 us up to 128 rows.
//
// Roles (11 warps, one CTA per SM, a contiguous share of all 128-key tiles each):
//   warps 0-3 / 4-7  the tiles of even / odd number: S from TMEM, exponentials,
//                    row sum, the total's update; all stage Q and the rows' lse
//                    when a kv-head begins.  More than 160 rows without a cap
//                    or slopes: sixteen warps, two warpgroups to a tile with half of
//                    its rows each (eight left the latency of the exponentials in
//                    the open)
//   warp 8           producer; two of them (8 and 10) for pages below 64 rows and
//                    for gathers: a warp issues a TMA box every ~110 cycles, so the
//                    sixteen of a tile of 16-row pages took one warp longer than
//                    HBM takes for the tile (64 sequences: 150 us with one, 125
//                    with two, 134 with three; boxes of 64 rows 109 against 111 us)
//   warp 9           MMA issuer, owns TMEM (two S buffers)
constexpr int kWtTile = 128;
constexpr int kWtRows = 256;  // rows of one pass (N of the MMA)
constexpr int kWtMaxStages = 6;

struct WtSeg {
  int b, h;
  int L, a;
  int R;       // rows of this pass
  int base;    // slot of the stream's first key, a multiple of the tile
  int lo, hi;  // keys below lo no row sees, from hi (to L) every row does; from base
  int nkeys;   // keys of the stream, from base; 0 = nothing to do
};

__device__ __forceinline__ WtSeg wt_seg(const WeightParams &p, int s, bool record) {
  WtSeg g;
  g.b = s / p.Hkv;
  g.h = s % p.Hkv;
  g.R = g.base = g.lo = g.hi = g.nkeys = 0;
  if (!weight_seq(p, g.b, record, g.L, g.a)) return g;
  const int rows = p.Hq / p.Hkv * g.a - p.row0;
  g.R = max(0, min(rows, kWtRows));
  const bool age = p.row0 == 0 && p.decay != 1.f;  // totals change where no row sees the key, too
  if (g.R == 0) {
    g.nkeys = age ? g.L : 0;
    g.lo = g.hi = g.nkeys;  // nothing to load
    return g;
  }
  const int lo = mod_first_slot(p.mod, g.b, 0, g.L), hi = mod_first_slot(p.mod, g.b, g.a - 1, g.L);
  g.base = age ? 0 : lo & ~(kWtTile - 1);
  g.lo = lo - g.base;
  g.hi = hi - g.base;
  g.nkeys = g.L + g.a - g.base;
  return g;
}

struct WtSmem {  // offsets after the Q rows and the stages
  static constexpr int kBars = 2 * kWtMaxStages + 5;  // full, empty, s_full[2], s_empty[2], drain
  static constexpr int kMisc = (kBars * 8 + 15) & ~15;  // tmem base, abort flag
  static constexpr int kLse = kMisc + 16;              // float [256]: -lse (-inf: no such row)
  static constexpr int kSlope = kLse + kWtRows * 4;    // float [256]: -slope
  static constexpr int kTok = kSlope + kWtRows * 4;    // float [256]: accepted rank of the row
  static constexpr int kPart = kTok + kWtRows * 4;     // float [2][2][128]: the second half's row sums
  static constexpr int kPlan = kPart + 4 * 128 * 4;    // int [S + 1]
};

// kMod: a cap or slopes (a window or a document start needs no code of its own in
// the tiles that every row sees).  kGroups: warpgroups that sum (2, or 4 = two to
// a tile).
template <int D, bool kTma, bool kMod, int kProducers, int kGroups>
__global__ void __launch_bounds__((4 * kGroups + 3) * 32, 1)
    weight_tc_kernel(const WeightParams p, const __grid_constant__ CUtensorMap tmk, int RQ, int NS) {
  constexpr int TK = kWtTile;
  constexpr int kHalves = D / 64;
  constexpr int kStage = kHalves * TK * 128;
  constexpr int kThreads = (4 * kGroups + 3) * 32;
  constexpr int kSoft = 128 * kGroups, kProducer = 4 * kGroups, kMma = kProducer + 1;
  constexpr int kPad = 16 * kGroups;  // S columns: whole 32-column loads of each half
  constexpr int kBarQ = 1, kBarSoft = 2, kBarEnd = 3, kBarPair = 4;  // kBarPair + S buffer
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *sQ = smem;  // [D/64 columns][RQ rows][128 B], 128-byte swizzle
  uint8_t *stages = smem + kHalves * RQ * 128;
  uint8_t *rest = stages + NS * kStage;
  uint64_t *full = reinterpret_cast<uint64_t *>(rest);
  uint64_t *empty = full + kWtMaxStages, *s_full = empty + kWtMaxStages, *s_empty = s_full + 2, *drain = s_full + 4;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rest + WtSmem::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(rest + WtSmem::kMisc + 4);
  float *s_nlse = reinterpret_cast<float *>(rest + WtSmem::kLse);
  float *s_slope = reinterpret_cast<float *>(rest + WtSmem::kSlope);
  float *s_tok = reinterpret_cast<float *>(rest + WtSmem::kTok);
  int *tstart = reinterpret_cast<int *>(rest + WtSmem::kPlan);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.B * p.Hkv;
  const int group = p.Hq / p.Hkv;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, kTma ? kProducers : 32 * kProducers);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, (int)blockIdx.x == p.test_stall ? kNever : 1);
      mbar_init(s_empty + i, 64 * kGroups);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  for (int s = tid; s < S; s += kThreads)
    tstart[s] = (wt_seg(p, s, blockIdx.x == 0 && p.row0 == 0 && s % p.Hkv == 0).nkeys + TK - 1) / TK;
  __syncthreads();
  if (warp == 0) warp_scan_inplace(tstart, S);
  __syncthreads();
  const long long total = tstart[S];
  const int G = (int)min((long long)gridDim.x, total);
  if ((int)blockIdx.x >= G) return;
  const int t0 = (int)(blockIdx.x * total / G), t1 = (int)((blockIdx.x + 1) * total / G);
  int s0 = 0;
  for (int hi = S - 1; s0 < hi;) {
    const int mid = (s0 + hi) >> 1;
    if (tstart[mid + 1] > t0) hi = mid; else s0 = mid + 1;
  }
  bool ok = true;
  auto wait_ok = [&](uint64_t *bar, uint32_t parity) { role_wait(bar, parity, ok, abort_flag, p.wait_ns, p.status); };
  // a tile with keys some row sees (the others only age)
  auto live = [](const WtSeg &g, int lt) { return g.R > 0 && lt * TK + TK > g.lo; };
  // the next stage of the ring and the parity of its pass
  struct Ring {
    int st = 0;
    uint32_t ph = 0;
    __device__ void next(int n) {
      if (++st == n) {
        st = 0;
        ph ^= 1u;
      }
    }
  };

  if (warp == kProducer || warp > kMma) {
    const int pw = warp == kProducer ? 0 : warp - kMma;
    if (pw >= kProducers) return;
    const uint64_t policy = l2_evict_first_policy();
    if (kTma && lane == 0) prefetch_tmap(&tmk);
    Ring r;
    int issued = 0;
    const bool paged = p.page_table != nullptr;
    // page entry of this lane's box of tile lt (TMA): fetched one tile ahead, or
    // its latency would be the time of a tile
    auto box_page = [&](const WtSeg &g, int lt) {
      const int k = lt * TK + lane * p.tma_box;
      if (!paged || lane >= TK / p.tma_box || k >= g.nkeys) return 0;
      return __ldg(p.page_table + (size_t)g.b * p.max_pages + ((g.base + k) >> p.page_shift));
    };
    for (int s = s0; s < S && tstart[s] < t1; ++s) {
      const WtSeg g = wt_seg(p, s, false);
      const int lt0 = max(tstart[s], t0) - tstart[s], lt1 = min(tstart[s + 1], t1) - tstart[s];
      int page_next = kTma && lt0 < lt1 ? box_page(g, lt0) : 0;
      for (int lt = lt0; lt < lt1; ++lt) {
        int page = page_next;
        if (kTma && lt + 1 < lt1) page_next = box_page(g, lt + 1);
        if (!live(g, lt)) continue;
        wait_ok(empty + r.st, r.ph ^ 1u);
        // the gather passes row addresses between the lanes: all of them go on, or none
        if constexpr (!kTma) ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        uint8_t *dst = stages + r.st * kStage;
        const int k0 = lt * TK, slot0 = g.base + k0;
        if constexpr (kTma) {
          const int BR = p.tma_box, nbox = TK / BR;
          const int nb = paged ? min(nbox, (g.nkeys - k0 + BR - 1) / BR) : nbox;
          // two producers take a 128-byte column each (D 64: every other box)
          constexpr bool two = kProducers == 2;
          const int mine = !two ? nb * kHalves : kHalves == 2 ? nb : (nb + 1 - pw) / 2;
          if (lane == 0) mbar_arrive_expect_tx(full + r.st, (uint32_t)(mine * BR * 128));
          __syncwarp();
          if (lane < nb && (kHalves == 2 || !two || (lane & 1) == pw)) {
            const int slot = slot0 + lane * BR;
            int row = g.b * p.len_cap + slot;
            if (paged) {
              if (page < 0 || page >= p.num_pages) {
                if (k0 + (lane + 1) * BR > g.lo) record_status(p.status, VA_ERR_DEVICE_BOUNDS);
                page = 0;
              }
              row = (page << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
            }
#pragma unroll
            for (int i = 0; i < (kHalves == 2 && two ? 1 : kHalves); ++i) {
              const int c = kHalves == 2 && two ? pw : i;
              tma_load_3d(dst + c * TK * 128 + lane * BR * 128, &tmk, c * 64, g.h, row, full + r.st, policy);
            }
          }
        } else {
          // pages below 8 rows: lane l resolves rows l + 32 j, 16-byte copies
          constexpr int CPR = D / 8, RPP = 32 / CPR;
          const int cc = lane % CPR, rsub = lane / CPR;
          for (int j = pw; j < TK / 32; j += kProducers) {
            const int k = k0 + lane + 32 * j;
            const __nv_bfloat16 *row = nullptr;
            if (k < g.nkeys) row = weight_key<__nv_bfloat16>(p, g.b, g.h, g.base + k, k >= g.lo);
#pragma unroll
            for (int i = 0; i < 32 / RPP; ++i) {
              const int rl = i * RPP + rsub;
              const uint64_t a = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(row), rl);
              const void *src = a != 0 ? reinterpret_cast<const uint8_t *>(a) + cc * 16 : p.k;
              cp_async_16(dst + swz<TK>(32 * j + rl, cc), src, a != 0 ? 16u : 0u);
            }
          }
          cp_async_mbar_arrive(full + r.st);
        }
        r.next(NS);
        ++issued;
      }
    }
    // the copies this warp issued land before it leaves (bounded), so that the block
    // cannot end before them
    if constexpr (kTma) {
      for (int j = 0; j < min(issued, NS); ++j) {
        r.st = r.st == 0 ? NS - 1 : r.st - 1;
        if (r.st == NS - 1) r.ph ^= 1u;
        mbar_wait(full + r.st, r.ph, p.wait_ns >> 4);
      }
    } else {
      cp_async_wait_all();
    }
    return;
  }

  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  named_bar_sync(kBarEnd, kSoft + 32);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kMma) {
    Ring r;
    int jt = 0;
    const uint64_t dK0 = umma_sdesc(smem_u32(stages), 16, 1024), dQ0 = umma_sdesc(smem_u32(sQ), 16, 1024);
    for (int s = s0; s < S && tstart[s] < t1; ++s) {
      const WtSeg g = wt_seg(p, s, false);
      const int lt0 = max(tstart[s], t0) - tstart[s], lt1 = min(tstart[s + 1], t1) - tstart[s];
      if (lt0 >= lt1 || !live(g, lt1 - 1)) continue;
      named_bar_sync(kBarQ, kSoft + 32);  // Q of this kv-head is in shared memory
      const uint32_t idesc = umma_idesc(128, (g.R + kPad - 1) & ~(kPad - 1), 0, 0);
      for (int lt = lt0; lt < lt1; ++lt) {
        if (!live(g, lt)) continue;
        const int b = jt & 1;
        wait_ok(full + r.st, r.ph);
        if (jt >= 2) wait_ok(s_empty + b, (uint32_t)((jt >> 1) - 1) & 1u);
        // (after giving up, too: no lane may leave the warp that elects an issuer)
        if constexpr (!kTma) fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t dK = dK0 + (uint64_t)((r.st * kStage) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_ss_warp(tmem + 256 * b, dK + (uint64_t)(((ks >> 2) * (TK * 128) + (ks & 3) * 32) >> 4),
                       dQ0 + (uint64_t)(((ks >> 2) * (RQ * 128) + (ks & 3) * 32) >> 4), idesc, ks > 0 ? 1u : 0u);
        umma_commit_warp(s_full + b);
        umma_commit_warp(empty + r.st);
        __syncwarp();
        r.next(NS);
        ++jt;
      }
    }
    umma_commit_warp(drain);
    mbar_wait(drain, 0u, p.wait_ns);
    tc_fence_before();
    named_bar_sync(kBarEnd, kSoft + 32);
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    return;
  }

  // ============================ sums over the rows ============================
  const int wg = (warp >> 2) / (kGroups / 2);  // S buffer: takes the live tiles jt = wg mod 2
  const int half = kGroups == 4 ? (warp >> 2) & 1 : 0;  // half of the rows
  const int key_l = tid & 127;                 // key of the tile = TMEM lane
  float *s_part = reinterpret_cast<float *>(rest + WtSmem::kPart) + wg * 128 + key_l;
  int jt = 0;
  for (int s = s0; s < S && tstart[s] < t1; ++s) {
    const WtSeg g = wt_seg(p, s, false);
    const int lt0 = max(tstart[s], t0) - tstart[s], lt1 = min(tstart[s + 1], t1) - tstart[s];
    if (lt0 >= lt1) continue;
    const int NP = (g.R + kPad - 1) & ~(kPad - 1);  // columns of S
    const bool any = live(g, lt1 - 1);  // (tiles turn live once)
    if (any) {
      named_bar_sync(kBarSoft, kSoft);  // every MMA that reads Q has completed (all tiles were waited for)
      const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(p.q);
      for (int e = tid; e < NP * (D / 8); e += kSoft) {
        const int r = e / (D / 8), ch = e % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < g.R) {
          const int i = (p.row0 + r) / group;
          const int t = p.path != nullptr ? __ldg(p.path + (size_t)g.b * p.T + i) : i;
          if (t >= 0 && t < p.T)
            v = __ldg(reinterpret_cast<const uint4 *>(
                          qb + (((size_t)g.b * p.T + t) * p.Hq + g.h * group + (p.row0 + r) % group) * D) + ch);
        }
        *reinterpret_cast<uint4 *>(sQ + (ch >> 3) * (RQ * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
      }
      if (tid < NP) {
        float nl = -INFINITY, ns = 0.f;
        const int i = (p.row0 + tid) / group, hq = g.h * group + (p.row0 + tid) % group;
        if (tid < g.R) {
          const int t = p.path != nullptr ? __ldg(p.path + (size_t)g.b * p.T + i) : i;
          if (t >= 0 && t < p.T) {
            const float l = __ldg(p.lse + ((size_t)g.b * p.Hq + hq) * p.T + t);
            nl = l == -INFINITY ? -INFINITY : -l;  // a row that saw no key adds nothing
            if (kMod && p.mod.slopes != nullptr) ns = -__ldg(p.mod.slopes + hq);
          } else {
            record_status(p.status, VA_ERR_DEVICE_BOUNDS);
          }
        }
        s_nlse[tid] = nl;
        s_slope[tid] = ns;
        s_tok[tid] = (float)i;
      }
      fence_proxy_async_smem();
      tc_fence_before();
      named_bar_sync(kBarSoft, kSoft);
      named_bar_sync(kBarQ, kSoft + 32);  // (a wait: keeps the roles in step after a wait has run out)
    }

    float *w = p.weight + ((size_t)g.b * p.Hkv + g.h) * p.stride + g.base;
    const int n_old = g.L - g.base;  // keys of the prefix
    const float window = p.mod.window > 0 ? (float)p.mod.window : INFINITY;
    auto total_of = [&](int key) {
      return (p.row0 > 0 ? key < g.nkeys : key < n_old && p.decay != 0.f) ? w[key] : 0.f;
    };
    // S has been read: the MMA warp may write the buffer again
    auto release = [&]() {
      tc_fence_before();
      mbar_arrive(s_empty + wg);
    };
    bool have_next = false;
    float next_old = 0.f;
    const int NH = kGroups == 4 ? NP / 2 : NP;  // this warpgroup's columns
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256 * wg + half * NH;
    const float *w_nlse = s_nlse + half * NH, *w_slope = s_slope + half * NH, *w_tok = s_tok + half * NH;
    for (int lt = lt0; lt < lt1; ++lt) {
      const int key = lt * TK + key_l;
      if (!live(g, lt)) {
        if ((lt & 1) == wg && half == 0 && key < g.nkeys) w[key] = p.decay != 0.f ? w[key] * p.decay : 0.f;
        continue;
      }
      const int mine = (jt & 1) == wg;
      const uint32_t ph = (uint32_t)(jt >> 1) & 1u;
      ++jt;
      if (!mine) continue;
      // what the total keeps (row0 > 0: a later pass adds to the earlier ones'),
      // loaded while this warpgroup works on its tile before
      const float old = have_next ? next_old : half == 0 ? total_of(key) : 0.f;
      have_next = lt + 2 < lt1;
      next_old = have_next && half == 0 ? total_of(key + 2 * TK) : 0.f;
      const bool masked = lt * TK < g.hi || lt * TK + TK > n_old;
      const float koff = (float)(key - n_old);
      const bool there = key >= g.lo && key < g.nkeys;
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      // adds the terms of 32 rows, S columns c0 ..; `edge`: rows that do not see the key are left out
      auto rows32 = [&](const uint32_t (&u)[32], int c0, auto edge) {
        float x[32];
#pragma unroll
        for (int r = 0; r < 32; ++r) x[r] = __uint_as_float(u[r]);
        if (kMod && p.mod.softcap > 0.f) cap_scores<32, true, true>(p.mod, x, !there, false);
        const float mul = kMod && p.mod.softcap > 0.f ? 1.f : p.mod.out_mul;
        if (kMod && p.mod.slopes != nullptr) {
#pragma unroll
          for (int r = 0; r < 32; r += 2) {
            const float2 ns = *reinterpret_cast<const float2 *>(w_slope + c0 + r);
            const float2 tk = *reinterpret_cast<const float2 *>(w_tok + c0 + r);
            x[r] = fmaf(ns.x, fabsf(tk.x - koff), x[r] * mul);
            x[r + 1] = fmaf(ns.y, fabsf(tk.y - koff), x[r + 1] * mul);
          }
        }
        const float mul2nd = kMod && p.mod.slopes != nullptr ? 1.f : mul;
#pragma unroll
        for (int r = 0; r < 32; r += 4) {
          const float4 nl = *reinterpret_cast<const float4 *>(w_nlse + c0 + r);
          float2 d[2] = {fma2(make_float2(x[r], x[r + 1]), make_float2(mul2nd, mul2nd), make_float2(nl.x, nl.y)),
                         fma2(make_float2(x[r + 2], x[r + 3]), make_float2(mul2nd, mul2nd), make_float2(nl.z, nl.w))};
          if constexpr (decltype(edge)::value) {
            const float4 tk = *reinterpret_cast<const float4 *>(w_tok + c0 + r);
            if (!(there && koff <= tk.x && tk.x - koff < window)) d[0].x = -INFINITY;
            if (!(there && koff <= tk.y && tk.y - koff < window)) d[0].y = -INFINITY;
            if (!(there && koff <= tk.z && tk.z - koff < window)) d[1].x = -INFINITY;
            if (!(there && koff <= tk.w && tk.w - koff < window)) d[1].y = -INFINITY;
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            // natural units so far: s - lse is small, and so exact, where the weight matters
            d[q] = mul2(d[q], make_float2(kModLog2e, kModLog2e));
            acc[q] = add2(acc[q], make_float2(ex2_approx(d[q].x), ex2_approx(d[q].y)));
          }
        }
      };
      wait_ok(s_full + wg, ph);
      tc_fence_after();
      uint32_t ua[32];
      tmem_ld32(tS, ua);
      if (masked || kMod || kGroups == 4) {  // (no registers to load ahead, or warps enough)
        for (int c0 = 0; c0 < NH; c0 += 32) {
          if (c0 > 0) tmem_ld32(tS + c0, ua);
          tmem_ld_wait(ua);
          if (c0 + 32 >= NH) release();
          if (masked) rows32(ua, c0, std::true_type());
          else if constexpr (kMod || kGroups == 4) rows32(ua, c0, std::false_type());
        }
      } else {
        // the next columns are on their way from TMEM while these are summed
        uint32_t ub[32];
        tmem_ld_wait(ua);
        for (int c0 = 0; c0 < NH; c0 += 64) {
          const bool two = c0 + 32 < NH, more = c0 + 64 < NH;
          if (two) tmem_ld32(tS + c0 + 32, ub);
          else release();
          rows32(ua, c0, std::false_type());
          if (!two) break;
          tmem_ld_wait(ub);
          if (more) tmem_ld32(tS + c0 + 64, ua);
          else release();
          rows32(ub, c0 + 32, std::false_type());
          if (more) tmem_ld_wait(ua);
        }
      }
      float sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
      if constexpr (kGroups == 4) {
        // the halves' sums meet in shared memory, in the slot of the tile's parity:
        // the slot is written again two tiles on, after the next barrier
        float *slot = s_part + ((jt >> 1) & 1) * 256;
        if (half == 1) *slot = sum;
        named_bar_sync(kBarPair + wg, 256);
        if (half == 1) continue;
        sum += *slot;
      }
      if (ok && key < g.nkeys) w[key] = p.row0 > 0 ? old + sum : fmaf(p.decay, old, sum);
    }
  }
  tc_fence_before();
  named_bar_sync(kBarEnd, kSoft + 32);
}

template <int D, bool kTma, bool kMod, int kProducers, int kGroups>
static cudaError_t launch_weight_tc(const WeightParams &p, const CUtensorMap &tmk, int grid, cudaStream_t stream) {
  const int rows = p.Hq / p.Hkv * p.T - p.row0;
  const int pad = 16 * kGroups;
  const int RQ = rows >= kWtRows ? kWtRows : (rows + pad - 1) & ~(pad - 1);
  const size_t fixed = 1024 + (size_t)(D / 64) * RQ * 128 + WtSmem::kPlan + (size_t)(p.B * p.Hkv + 1) * 4;
  const size_t stage = (size_t)(D / 64) * kWtTile * 128;
  int NS = (int)((kSmemLimit - fixed) / stage);
  if (NS > kWtMaxStages) NS = kWtMaxStages;
  const size_t smem = fixed + NS * stage;
  auto kern = weight_tc_kernel<D, kTma, kMod, kProducers, kGroups>;
  cudaError_t e = allow_smem(kern);
  if (e != cudaSuccess) return e;
  kern<<<grid, (4 * kGroups + 3) * 32, smem, stream>>>(p, tmk, RQ, NS);
  return cudaGetLastError();
}

template <int D, bool kTma, int kProducers>
static cudaError_t launch_weight_p(const WeightParams &p, const CUtensorMap &tmk, int grid, cudaStream_t stream) {
  // (a cap or slopes leave four warpgroups too few registers: 256 rows capped 138 / 238 us;
  // 142 with the term that the weights' cap has more)
  if (p.mod.on == 2) return launch_weight_tc<D, kTma, true, kProducers, 2>(p, tmk, grid, stream);
  // 8 x 128K keys, one warpgroup a tile against two: 160 rows 50.9 / 51.7 us, 192 rows
  // 57.9 / 52.1, 256 rows 72.8 / 65.7
  return p.Hq / p.Hkv * p.T - p.row0 > 160 ? launch_weight_tc<D, kTma, false, kProducers, 4>(p, tmk, grid, stream)
                                           : launch_weight_tc<D, kTma, false, kProducers, 2>(p, tmk, grid, stream);
}

template <int D>
static cudaError_t launch_weight_bf16(const WeightParams &p, const CUtensorMap &tmk, int grid, cudaStream_t stream) {
  return p.tma_box == 64  ? launch_weight_p<D, true, 1>(p, tmk, grid, stream)
         : p.tma_box > 0  ? launch_weight_p<D, true, 2>(p, tmk, grid, stream)
                          : launch_weight_p<D, false, 2>(p, tmk, grid, stream);
}

// fp32: one thread per key (no TF32).  bf16: one pass of the tensor-core kernel
// for every 256 rows of a kv-head; the later passes add to the totals.
cudaError_t launch_accumulate_weight(const WeightParams &p, const CUtensorMap &tmk, int sms, cudaStream_t stream) {
  const int keys = p.len_cap < p.stride ? p.len_cap : p.stride;
  if (p.dtype == VA_DTYPE_FP32) {
    const dim3 grid((unsigned)((keys + 127) / 128), (unsigned)p.Hkv, (unsigned)p.B);
    weight_simt_kernel<<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
  }
  const long long tiles = (long long)p.B * p.Hkv * ((keys + kWtTile - 1) / kWtTile);
  const int grid = (int)(tiles < sms ? tiles : sms);
  WeightParams q = p;
  for (q.row0 = 0; q.row0 < p.Hq / p.Hkv * p.T; q.row0 += kWtRows) {
    const cudaError_t e = p.D == 64 ? launch_weight_bf16<64>(q, tmk, grid, stream)
                                    : launch_weight_bf16<128>(q, tmk, grid, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace va
