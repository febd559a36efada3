// Attention weight of cached tokens, many queries: the sums of key_weights.cu on the tensor cores.
//
// One CTA per SM loops over items (sequence, KV head, 256 keys as two tiles), the ones with the most
// queries first, in alternating direction round by round. The K tiles stay in shared memory while the
// group's query rows stream by, R of them a step (R = G floor(128 / G), row u the query u / G of the
// step and head u mod G, which is how one TMA box of G heads x R / G queries lands). Two tiles share a
// step's rows: with one, the rows (32 KB of L2 for every 2^21 multiply-adds) take 6.4 TB/s.
//   warp 0      TMA producer: K tiles (page by page, eight lanes) into a ring of three, Q tiles
//               into another
//   warp 1      MMA issuer (one thread): S^T = K Q^T of each unit (step, tile) into one of four
//               TMEM buffers; a tile takes part in the steps whose queries can see it
//   warps 2-3   the units' per-column vectors, -lse log2(e) (shared memory, a slot per buffer)
//   warps 4-7, 8-11   a thread owns a key row: it sums 2^(score - lse) over the columns of every
//               other unit; at the end of the item the second warpgroup hands its sums to the
//               first, which writes w_out. Fixed order, no atomics.
// One product per pair of tiles and no P V leaves an exponential per 2 d flops. Two prompts of 2048 and 1536 queries
// over 8.6k tokens, 32 heads over 8: 128 us, 800 TFLOP/s; four of 4096 over 8192 each: 981 us, 1120 TFLOP/s.
// Bound by the chain of a unit (product, TMEM load, exponentials, release): tensor pipe and special function unit are
// both busy 38 % (50 % in the second); wider loads, a third summing warpgroup or pairs of CTAs that share the
// rows by multicast (137 us) do not shorten it.
// Every wait is bounded, as in the other tensor-core kernels.
#include "device_common.cuh"
#include "ops_internal.h"
#include "score_shape.cuh"
#include "sm100_primitives.cuh"

#include <math_constants.h>

#include <algorithm>

namespace fattn {
namespace {

using namespace sm100;

constexpr int BT = 128;
constexpr int kGroups = 2;      // summing warpgroups
constexpr int kThreads = 128 * (1 + kGroups);
constexpr uint32_t kTmemCols = 512;
constexpr int kBufs = 4;        // S^T buffers of 128 columns
constexpr int kQStages = 3, kKStages = 3;
constexpr uint64_t kDrainLimitNs = 200000000ull;
enum : int { kShapeCap = 1, kShapeBias = 2 };

// barriers
enum : int {
  kKFull = 0, kKEmpty = kKStages, kQFull = 2 * kKStages, kQEmpty = kQFull + kQStages, kSFull = kQEmpty + kQStages, kSFree = kSFull + kBufs,
  kSumFull = kSFree + kBufs, kSumFree = kSumFull + 1, kMmaDone = kSumFree + 1,
  kBarStall = kMmaDone + 1, kNumBars = kBarStall + 1
};

template <int D>
struct KwTcLayout {
  static constexpr int kTile = BT * D * 2;
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kKStages * kTile;
  static constexpr int kOffVec = kOffQ + kQStages * kTile;     // [kBufs][2][128] -lse log2(e), -slope log2(e)
  static constexpr int kOffCol = kOffVec + kBufs * 2 * BT * 4; // [128] query of a column, u / G
  static constexpr int kOffSum = kOffCol + BT * 4;             // [kGroups - 1][2][128] the other warpgroups' sums
  static constexpr int kOffBar = kOffSum + (kGroups - 1) * 2 * BT * 4;
  static constexpr int kOffHolder = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffHolder + 8;
  static constexpr int kUsed = kOffAbort + 8 + 1024;           // + slack to align the base to 1024 B
  // at least 117 KB, so that a second CTA (which would block in tcgen05.alloc) never shares the SM
  static constexpr int kBytes = kUsed > 117 * 1024 ? kUsed : 117 * 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kDrainLimitNs) break;
  }
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, int* status,
                                          uint64_t limit_ns) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort, status, limit_ns);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

struct KwItem {
  int b, hkv, key0, n, m, q0, off;  // n keys, m queries (first row q0, first position off) of the sequence
  int i0, steps;                    // queries from i0 on, in steps of `per`
  int f0, e0, f1, e1;               // tile t takes part in steps [f_t, e_t)
  bool valid;                       // the sequence's lengths are consistent
  __device__ __forceinline__ bool takes(int t, int s) const { return t ? s >= f1 && s < e1 : s >= f0 && s < e0; }
  // units in the issuer's order (steps, tile 0 before tile 1): first those of tile 0 alone, then of both, then of tile 1
  // alone (a later tile's queries neither start nor end before an earlier one's)
  __device__ __forceinline__ int alone0() const { return e1 > f1 ? min(f1, e0) - f0 : e0 - f0; }
  __device__ __forceinline__ int both() const { return e0 > f0 && e1 > f1 ? 2 * max(e0 - f1, 0) : 0; }
  __device__ __forceinline__ int start1() const { return e0 > f0 ? max(f1, e0) : f1; }  // first step of tile 1 alone
  __device__ __forceinline__ int units() const { return alone0() + both() + max(e1 - start1(), 0); }
  __device__ __forceinline__ void unit(int j, int& s, int& t) const {
    const int a = alone0(), b = both();
    t = j < a ? 0 : j < a + b ? (j - a) & 1 : 1;
    s = j < a ? f0 + j : j < a + b ? f1 + ((j - a) >> 1) : start1() + (j - a - b);
  }
};

// k-th item of this CTA, or -1 past the end.
__device__ __forceinline__ int kw_index(int k, int total) {
  const int G = (int)gridDim.x;
  const int idx = k * G + ((k & 1) ? (G - 1 - (int)blockIdx.x) : (int)blockIdx.x);
  return idx < total ? idx : -1;
}

__device__ __forceinline__ KwItem kw_item(const KeyWeightsParams& p, int it, int per) {
  KwItem x;
  const int heads = p.B * p.Hkv;
  const int kt = it / heads, bh = it - kt * heads;
  x.b = bh / p.Hkv;
  x.hkv = bh - x.b * p.Hkv;
  x.key0 = kt * p.tiles * BT;
  x.n = __ldg(p.seqlens_k + x.b);
  x.q0 = __ldg(p.cu_seqlens + x.b);
  const int q1 = __ldg(p.cu_seqlens + x.b + 1);
  x.m = q1 - x.q0;
  x.valid = x.n >= 0 && x.n <= p.max_pages * p.page_size && x.q0 >= 0 && x.m >= 0 && q1 <= p.total_q && x.m <= x.n && x.m <= p.max_q;
  x.off = x.n - x.m;
  x.i0 = x.steps = x.f0 = x.e0 = x.f1 = x.e1 = 0;
  if (!x.valid || x.key0 >= x.n) return x;
  // queries [lo, hi) that can see a key of [a, a + 128)
  auto range = [&](int a, int& lo, int& hi) {
    lo = hi = 0;
    if (a >= x.n) return;
    const int last = min(a + BT, x.n) - 1;
    long long e = x.m;
    if (p.causal) lo = max(0, a - x.off);
    if (p.shape.window > 0) {
      e = min(e, (long long)last + p.shape.window - x.off);
      if (!p.causal) lo = (int)max(0ll, (long long)a - x.off - p.shape.window + 1);
    }
    hi = (int)max(e, (long long)lo);
  };
  int l0, h0, l1, h1;
  range(x.key0, l0, h0);
  l1 = h1 = 0;
  if (p.tiles > 1) range(x.key0 + BT, l1, h1);
  x.i0 = h0 > l0 ? l0 : l1;   // (l0 <= l1)
  if (h0 > l0) {
    x.f0 = (l0 - x.i0) / per;
    x.e0 = (h0 - x.i0 + per - 1) / per;
  }
  if (h1 > l1) {
    x.f1 = (l1 - x.i0) / per;
    x.e1 = (h1 - x.i0 + per - 1) / per;
  }
  x.steps = max(x.e0, x.e1);
  return x;
}

// Four consecutive floats of shared memory as two packed pairs.
__device__ __forceinline__ void lds_pairs(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}

// A thread's sum of 2^(score + nl) over columns [va, vb) of 128 (its key's row of S^T); nl, the slopes and the
// columns' queries in shared memory. Without cap or bias and nothing hidden a column goes straight from
// TMEM to its sum (four prompts of 4096 queries over 8192 tokens, 8 KV heads: 1053 us with the scores kept in
// between, 977 so; 64 or 128 columns a load and a third warpgroup change nothing). The cap is a polynomial while no
// |u| of the thread's 32 columns exceeds its range (fattn_internal.h), which takes half of the special
// function unit's work away.
template <int kShape>
__device__ __forceinline__ float sum_columns(const KeyWeightsParams& p, uint32_t s_col, uint32_t nl, uint32_t slope,
                                             uint32_t query, float dist, int va, int vb) {
  const ScoreShape& sh = p.shape;
  const uint64_t mul = f2_pack(sh.sl2, sh.sl2), dist2 = f2_pack(dist, dist);
  const bool edge = __any_sync(0xffffffffu, va > 0 || vb < BT);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
  // columns c .. c + 3: nl, less the bias if there is one, as two pairs
  auto offsets = [&](int c, uint64_t (&l)[2]) {
    lds_pairs(nl + c * 4, l[0], l[1]);
    if constexpr (kShape & kShapeBias) {  // nl - slope |pos - key|
      uint64_t q[2], sl[2];
      lds_pairs(query + c * 4, q[0], q[1]);
      lds_pairs(slope + c * 4, sl[0], sl[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) l[i] = f2_fma(sl[i], f2_add(q[i], dist2) & 0x7fffffff7fffffffull, l[i]);
    }
  };
  auto add = [&](int i, float y0, float y1) { acc[i & 3] = f2_add(acc[i & 3], f2_pack(ex2(y0), ex2(y1))); };
  if (kShape == 0 && !edge) {
#pragma unroll 1
    for (int c = 0; c < BT; c += 32) {
      uint32_t u[32];
      tmem_ld32(s_col + c, u);
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        uint64_t l[2];
        offsets(c + e, l);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float y0, y1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(u[e + 2 * i]), __uint_as_float(u[e + 2 * i + 1])), mul, l[i]), y0, y1);
          add((e >> 1) + i, y0, y1);
        }
      }
    }
  } else {
#pragma unroll 1
    for (int c = 0; c < BT; c += 32) {
      uint32_t u[32];
      tmem_ld32(s_col + c, u);
      const int a = max(va - c, 0), z = min(vb - c, 32);
      const uint32_t vis = a < z ? (0xffffffffu << a) & (0xffffffffu >> (32 - z)) : 0u;
      float y[32];
      if constexpr (kShape & kShapeCap) {
        if (edge) {  // hidden columns must not decide between the cap's forms
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((vis >> e) & 1u)) u[e] = 0u;
        }
        float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 32; e += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            m[i] = fmax3(m[i], fabsf(__uint_as_float(u[e + i])), fabsf(__uint_as_float(u[e + 4 + i])));
        capped_scores(sh, u, fmax3(fmaxf(m[0], m[1]), m[2], m[3]), y);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(u[e]);
      }
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        uint64_t l[2];
        offsets(c + e, l);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float& y0 = y[e + 2 * i];
          float& y1 = y[e + 2 * i + 1];
          f2_unpack(kShape & kShapeCap ? f2_add(f2_pack(y0, y1), l[i]) : f2_fma(f2_pack(y0, y1), mul, l[i]), y0, y1);
        }
      }
      if (edge) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!((vis >> e) & 1u)) y[e] = -CUDART_INF_F;
      }
#pragma unroll
      for (int e = 0; e < 32; e += 2) add(e >> 1, y[e], y[e + 1]);
    }
  }
  float s0, s1;
  f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
  return s0 + s1;
}

template <int D, int kShape>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                          const KeyWeightsParams p) {
  using Lay = KwTcLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + Lay::kOffBar + 8 * i; };
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Lay::kOffAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const int per = BT / G;       // queries per step (the launch checks G <= 128)
  const int R = per * G;        // rows per step
  float* col_query = reinterpret_cast<float*>(smem + Lay::kOffCol);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bar(i), ((i >= kSFree && i < kSFree + kBufs) || i == kSumFree) ? 4
                        : i == kSumFull                                        ? 4 * (kGroups - 1)
                        : i >= kSFull && i < kSFull + kBufs                    ? 2   // the product and its vector
                                                                               : 1);
    *abort = 0;
    fence_mbar_init();
  }
  // rows past R of the Q tiles are never copied: zeros, so that their (unused) products are numbers
  for (int idx = threadIdx.x; idx < kQStages * Lay::kTile / 16; idx += kThreads)
    reinterpret_cast<uint4*>(smem + Lay::kOffQ)[idx] = make_uint4(0, 0, 0, 0);
  for (int u = threadIdx.x; u < BT; u += kThreads) col_query[u] = (float)(u / G);
  fence_proxy_async_smem();
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
  }
  if (warp == 1) {
    tmem_alloc(sb + Lay::kOffHolder, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Lay::kOffHolder);
  const int cap_keys = p.max_pages * p.page_size;
  const int total = (cap_keys + p.tiles * BT - 1) / (p.tiles * BT) * p.B * p.Hkv;

  if (warp == 0) {
    // ------------------------------------------------------------ producer (lane i: page i of a K tile)
    if (lane < BT / 16) {
      uint32_t nk = 0, nq = 0;
      const uint64_t pol_k = policy_evict_first(), pol_q = policy_evict_last();
      bool ok = true;
      for (int k = 0, it; ok && (it = kw_index(k, total)) >= 0; ++k) {
        const KwItem x = kw_item(p, it, per);
        const int P = p.page_size, pages = BT / P;
        auto load_k = [&](int t) -> bool {
          const uint32_t kb = nk % kKStages;
          if (!mbar_wait(bar(kKEmpty + kb), ((nk / kKStages) & 1) ^ 1, abort, p.status, p.wait_ns)) return false;
          if (lane == 0) mbar_arrive_expect_tx(bar(kKFull + kb), Lay::kTile);
          if (lane < pages) {
            const int slot = (x.key0 + t * BT) / P + lane;
            int row = p.num_pages * P;   // past the pool: zeros
            if (slot < (x.n + P - 1) / P) {
              const int page = __ldg(p.block_table + (size_t)x.b * p.max_pages + slot);
              if (page >= 0 && page < p.num_pages)
                row = page * P;
              else
                record_status(p.status, kStatusDeviceCheck);
            }
#pragma unroll
            for (int dc = 0; dc < D / 64; ++dc)
              tma_load_3d(sb + Lay::kOffK + kb * Lay::kTile + dc * BT * 128 + lane * P * 128, &tk, bar(kKFull + kb),
                          dc * 64, x.hkv, row, pol_k);
          }
          ++nk;
          return true;
        };
        // The Q tiles are lane 0's alone (the other lanes, which nothing would hold back here, could miss
        // a phase): they go on to the next item's pages, as far as KEmpty lets them.
        auto load_q = [&](int s) -> bool {
          const uint32_t st = nq % kQStages;
          if (!mbar_wait(bar(kQEmpty + st), ((nq / kQStages) & 1) ^ 1, abort, p.status, p.wait_ns)) return false;
          mbar_arrive_expect_tx(bar(kQFull + st), R * D * 2);
#pragma unroll
          for (int dc = 0; dc < D / 64; ++dc)
            tma_load_3d(sb + Lay::kOffQ + st * Lay::kTile + dc * BT * 128, &tq, bar(kQFull + st), dc * 64, x.hkv * G,
                        x.q0 + x.i0 + s * per, pol_q);
          ++nq;
          return true;
        };
        // tile 0, the first step's rows, tile 1 (which waits for the previous item to end), the rest
        if (x.e0 > x.f0 && !load_k(0)) break;
        if (lane == 0 && x.steps > 0 && !load_q(0)) break;
        if (x.e1 > x.f1 && !load_k(1)) break;
        for (int s = 1; ok && lane == 0 && s < x.steps; ++s) ok = load_q(s);
      }
      // no copy may land after the CTA is gone: wait for the last armed phase of each barrier
      for (uint32_t st = 0; st < (uint32_t)kKStages; ++st) {
        const uint32_t c = nk > st ? (nk - st + kKStages - 1) / kKStages : 0;
        if (c) drain(bar(kKFull + st), (c - 1) & 1);
      }
      for (uint32_t st = 0; st < (uint32_t)kQStages; ++st) {
        const uint32_t c = nq > st ? (nq - st + kQStages - 1) / kQStages : 0;
        if (c) drain(bar(kQFull + st), (c - 1) & 1);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id = idesc_bf16_f32(BT, BT, 0);
      constexpr int kAtom = BT * 128 / 16;
      uint32_t nk = 0, nq = 0, n = 0;   // K tiles, steps, units
      bool ok = true;
      for (int k = 0, it; ok && (it = kw_index(k, total)) >= 0; ++k) {
        const KwItem x = kw_item(p, it, per);
        const bool has[2] = {x.e0 > x.f0, x.e1 > x.f1};
        const uint32_t tile0 = nk, tile1 = nk + (has[0] ? 1 : 0);  // this item's tiles in the ring
        for (int s = 0; ok && s < x.steps; ++s, ++nq) {
          const uint32_t st = nq % kQStages;
          if (!mbar_wait(bar(kQFull + st), (nq / kQStages) & 1, abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          const uint64_t b0 = smem_desc_sw128(sb + Lay::kOffQ + st * Lay::kTile, 16, 1024);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!x.takes(t, s)) continue;
            const uint32_t tile = t ? tile1 : tile0, kb = tile % kKStages, buf = n % kBufs;
            // (the tile's first step: later waits return at once, its next phase needs KEmpty below)
            if (!mbar_wait(bar(kKFull + kb), (tile / kKStages) & 1, abort, p.status, p.wait_ns) ||
                !mbar_wait(bar(kSFree + buf), ((n / kBufs) & 1) ^ 1, abort, p.status, p.wait_ns)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t a0 = smem_desc_sw128(sb + Lay::kOffK + kb * Lay::kTile, 16, 1024);
            mma_ss_c<false>(tmem + buf * BT, a0, b0, id);
#pragma unroll
            for (int ks = 1; ks < D / 16; ++ks) {
              const uint64_t o = (uint64_t)((ks >> 2) * kAtom + (ks & 3) * 2);
              mma_ss_c<true>(tmem + buf * BT, a0 + o, b0 + o, id);
            }
            mma_commit(bar(kSFull + buf));
            ++n;
          }
          if (!ok) break;
          mma_commit(bar(kQEmpty + st));
        }
        if (!ok) break;
        if (has[0]) mma_commit(bar(kKEmpty + nk++ % kKStages));
        if (has[1]) mma_commit(bar(kKEmpty + nk++ % kKStages));
      }
      mma_commit(bar(kMmaDone));
      drain(bar(kMmaDone), 0);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ per-column vectors
    // warps 2 and 3 take turns unit by unit; a warp's next step is on its way while it waits for a slot
    int uq[BT / 32];             // this lane's columns u = 32 e + lane: query u / G of the step (-1: none)
    long long ul[BT / 32];       // and lse offset of head u mod G
    float sl[BT / 32];
    uint32_t n = 0;
    bool ok = true;
#pragma unroll
    for (int e = 0; e < BT / 32; ++e) {
      const int u = 32 * e + lane;
      uq[e] = u < R ? u / G : -1;
      ul[e] = (long long)(u % G) * p.lse_head;
    }
    for (int k = 0, it; ok && (it = kw_index(k, total)) >= 0; ++k) {
      const KwItem x = kw_item(p, it, per);
      const float* lse = p.lse + (long long)x.hkv * G * p.lse_head + (long long)x.q0 * p.lse_row;
      float v[BT / 32];
      int loaded = -1;           // the step that v holds
      auto load = [&](int s) {
        loaded = s;
#pragma unroll
        for (int e = 0; e < BT / 32; ++e) {
          const int i = x.i0 + s * per + uq[e];
          v[e] = uq[e] >= 0 && s < x.steps && i < x.m ? __ldg(lse + ul[e] + i * p.lse_row) : -CUDART_INF_F;
        }
      };
      if (kShape & kShapeBias) {
#pragma unroll
        for (int e = 0; e < BT / 32; ++e)
          sl[e] = uq[e] >= 0 ? -__ldg(p.shape.slopes + x.hkv * G + (32 * e + lane) % G) * kLog2e : 0.f;
      }
      const int units = x.units();
      for (int j = (int)((n ^ (uint32_t)warp) & 1u); j < units; j += 2) {
        const uint32_t buf = (n + j) % kBufs, phase = (((n + j) / kBufs) & 1) ^ 1;
        int s, t, s2, t2;
        x.unit(j, s, t);
        if (loaded != s) load(s);
        float w[BT / 32];
#pragma unroll
        for (int e = 0; e < BT / 32; ++e)  // rows past R or the chunk, and rows that saw no key, give nothing; a NaN stays one
          w[e] = v[e] != -CUDART_INF_F ? -v[e] * kLog2e : -CUDART_INF_F;
        x.unit(j + 2, s2, t2);
        load(s2);
        if (!warp_wait(bar(kSFree + buf), phase, abort, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        float* dst = reinterpret_cast<float*>(smem + Lay::kOffVec) + buf * 2 * BT;
#pragma unroll
        for (int e = 0; e < BT / 32; ++e) {
          dst[32 * e + lane] = w[e];
          if (kShape & kShapeBias) dst[BT + 32 * e + lane] = sl[e];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFull + buf));
      }
      n += (uint32_t)units;
    }
  } else {
    // ------------------------------------------------------------ sums (one key of each tile per thread)
    const int wg = (warp - 4) >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const uint32_t s_base = tmem + ((uint32_t)(q4 * 32) << 16);
    float* sums = reinterpret_cast<float*>(smem + Lay::kOffSum);
    uint32_t n = 0, nsum = 0;
    bool ok = true;
    // test hook: a wait that runs out (nothing arrives on the stall barrier)
    if (p.debug_stall && !warp_wait(bar(kBarStall), 0, abort, p.status, p.wait_ns)) ok = false;
    for (int k = 0, it; ok && (it = kw_index(k, total)) >= 0; ++k) {
      const KwItem x = kw_item(p, it, per);
      if (!x.valid) {
        if (it < p.B * p.Hkv && x.hkv == 0 && warp == 4 && lane == 0) record_status(p.status, kStatusDeviceCheck);
        continue;  // the sequence is skipped
      }
      float sum0 = 0.f, sum1 = 0.f;
      const int units = x.units();
      // units n + j with buffer mod kGroups == wg
      for (int j = (int)((uint32_t)(wg - (int)n) % kGroups); j < units; j += kGroups) {
        const uint32_t buf = (n + j) % kBufs, phase = ((n + j) / kBufs) & 1;
        int s, t;
        x.unit(j, s, t);
        if (!warp_wait(bar(kSFull + buf), phase, abort, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        mbar_try_wait(bar(kSFull + buf), phase);  // completed: this lane's own acquire of the vector
        tc_fence_after();
        // columns whose query sees the key: positions [key, key + W) (causal) or (key - W, key + W)
        const int key = x.key0 + t * BT + r;
        const int first = x.i0 + s * per + x.off;              // position of column 0
        int va = 0, vb = min(per, x.m - x.i0 - s * per) * G;
        if (p.causal) va = min(max(key - first, 0), per) * G;
        if (p.shape.window > 0) {
          const long long hi = (long long)key + p.shape.window - first;
          if (hi < per) vb = min(vb, (int)max(hi, 0ll) * G);
          if (!p.causal) va = (int)min(max((long long)key - p.shape.window + 1 - first, 0ll), (long long)per) * G;
        }
        const uint32_t vec = sb + Lay::kOffVec + buf * 2 * BT * 4;
        const float w = sum_columns<kShape>(p, s_base + buf * BT, vec, vec + BT * 4, sb + Lay::kOffCol, (float)(first - key),
                                            va, vb);
        if (t)
          sum1 += w;
        else
          sum0 += w;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFree + buf));
      }
      n += (uint32_t)units;
      if (!ok) break;
      if (x.steps > 0) {  // (a warpgroup that took no unit of the item adds 0)
        if (wg > 0) {
          if (!warp_wait(bar(kSumFree), (nsum & 1) ^ 1, abort, p.status, p.wait_ns)) break;
          sums[(wg - 1) * 2 * BT + r] = sum0;
          sums[(wg - 1) * 2 * BT + BT + r] = sum1;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kSumFull));
        } else {
          if (!warp_wait(bar(kSumFull), nsum & 1, abort, p.status, p.wait_ns)) break;
          mbar_try_wait(bar(kSumFull), nsum & 1);
#pragma unroll
          for (int g = 0; g < kGroups - 1; ++g) {
            sum0 += sums[g * 2 * BT + r];
            sum1 += sums[g * 2 * BT + BT + r];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kSumFree));
        }
        ++nsum;
      }
      if (wg > 0) continue;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = x.key0 + t * BT + r;
        if (t >= p.tiles || key >= cap_keys) continue;
        const size_t at = ((size_t)x.b * p.Hkv + x.hkv) * cap_keys + key;
        float sum = t ? sum1 : sum0;
        if (key < x.n) {
          const int page = x.steps > 0 ? __ldg(p.block_table + (size_t)x.b * p.max_pages + key / p.page_size) : 0;
          if (page < 0 || page >= p.num_pages) sum = 0.f;  // (recorded by the producer)
          p.w_out[at] = p.w_in ? fmaf(p.decay, p.w_in[at], sum) : sum;
        } else if (p.w_out != p.w_in) {
          p.w_out[at] = 0.f;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int kShape>
cudaError_t launch_t(KeyWeightsParams p, const CUtensorMap& tq, const CUtensorMap& tk, int num_sms,
                     cudaStream_t stream) {
  auto kern = key_weights_tc_kernel<D, kShape>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, KwTcLayout<D>::kBytes);
  if (e != cudaSuccess) return e;
  const long long tiles = ((long long)p.max_pages * p.page_size + BT - 1) / BT * p.B * p.Hkv;
  // Two tiles share a step's rows (half the L2 traffic, fewer items to start), one tile balances better:
  // one with fewer than four items of two tiles per SM (two 2048-query prompts over 8.6k tokens, 8 KV heads,
  // 280 items: 130 us with one, 141 us with two; 16 queries over 8 contexts of up to 16k tokens, 4096 items:
  // 121 and 92 us).
  p.tiles = tiles < 8ll * num_sms ? 1 : 2;
  const long long items = p.tiles == 1 ? tiles : ((long long)p.max_pages * p.page_size + 2 * BT - 1) / (2 * BT) * p.B * p.Hkv;
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  kern<<<(int)std::min<long long>(items, num_sms), kThreads, KwTcLayout<D>::kBytes, stream>>>(tq, tk, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_weights_tc(const KeyWeightsParams& p, const CUtensorMap& tq, const CUtensorMap& tk, int num_sms,
                                  cudaStream_t stream) {
  const int shape = (p.shape.cap > 0.f ? kShapeCap : 0) + (p.shape.slopes ? kShapeBias : 0);
  switch (shape + (p.d == 128 ? 4 : 0)) {
    case 0: return launch_t<64, 0>(p, tq, tk, num_sms, stream);
    case 1: return launch_t<64, 1>(p, tq, tk, num_sms, stream);
    case 2: return launch_t<64, 2>(p, tq, tk, num_sms, stream);
    case 3: return launch_t<64, 3>(p, tq, tk, num_sms, stream);
    case 4: return launch_t<128, 0>(p, tq, tk, num_sms, stream);
    case 5: return launch_t<128, 1>(p, tq, tk, num_sms, stream);
    case 6: return launch_t<128, 2>(p, tq, tk, num_sms, stream);
    default: return launch_t<128, 3>(p, tq, tk, num_sms, stream);
  }
}

}  // namespace fattn
