// Attention weight of cached tokens, many queries: the sums of key_weights.cu on the tensor cores.
//
// One CTA per SM loops over items (sequence, KV head, tile of 128 keys), the tiles with the most
// queries first. The K tile stays in shared memory while the group's query rows stream by, R of
// them a step (R = G floor(128 / G), row u the query u / G of the step and head u mod G, which is
// how one TMA box of G heads x R / G queries lands):
//   warp 0      TMA producer: K tile (page by page, eight lanes), Q tiles into a ring of three
//   warp 1      MMA issuer (one thread): S^T = K Q^T into one of four TMEM buffers
//   warp 2      the steps' per-column vectors, -lse log2(e) (shared memory, a slot per buffer)
//   warps 4-7, 8-11   a thread owns a key: it sums 2^(score - lse) over the columns of every other
//               step; at the end of the item the second warpgroup hands its sums to the first,
//               which writes w_out. Fixed order, no atomics.
// One product per pair of tiles and no P V: the exponentials bound it (one per 2 d flops), so
// two warpgroups take turns on four buffers and the tensor core never waits for one of them.
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
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr int kBufs = 4;        // S^T buffers of 128 columns
constexpr int kQStages = 3;
constexpr uint64_t kDrainLimitNs = 200000000ull;
enum : int { kShapeCap = 1, kShapeBias = 2 };

// barriers
enum : int {
  kKFull = 0, kKEmpty = 2, kQFull = 4, kQEmpty = kQFull + kQStages, kSFull = kQEmpty + kQStages, kSFree = kSFull + kBufs,
  kVecFull = kSFree + kBufs, kSumFull = kVecFull + kBufs, kSumFree = kSumFull + 1, kMmaDone = kSumFree + 1,
  kBarStall = kMmaDone + 1, kNumBars = kBarStall + 1
};

template <int D>
struct KwTcLayout {
  static constexpr int kTile = BT * D * 2;
  static constexpr int kOffK = 0;                              // two K tiles
  static constexpr int kOffQ = 2 * kTile;
  static constexpr int kOffVec = kOffQ + kQStages * kTile;     // [kBufs][2][128] -lse log2(e), -slope log2(e)
  static constexpr int kOffCol = kOffVec + kBufs * 2 * BT * 4; // [128] query of a column, u / G
  static constexpr int kOffSum = kOffCol + BT * 4;             // [128] the second warpgroup's sums
  static constexpr int kOffBar = kOffSum + BT * 4;
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
  int i0, steps;                    // queries from i0 on, in steps of R rows
  bool valid;                       // the sequence's lengths are consistent
};

__device__ __forceinline__ KwItem kw_item(const KeyWeightsParams& p, int it, int G, int per) {
  KwItem x;
  const int heads = p.B * p.Hkv;
  const int kt = it / heads, bh = it - kt * heads;
  x.b = bh / p.Hkv;
  x.hkv = bh - x.b * p.Hkv;
  x.key0 = kt * BT;
  x.n = __ldg(p.seqlens_k + x.b);
  x.q0 = __ldg(p.cu_seqlens + x.b);
  const int q1 = __ldg(p.cu_seqlens + x.b + 1);
  x.m = q1 - x.q0;
  x.valid = x.n >= 0 && x.n <= p.max_pages * p.page_size && x.q0 >= 0 && x.m >= 0 && q1 <= p.total_q && x.m <= x.n;
  x.off = x.n - x.m;
  x.steps = x.i0 = 0;
  if (!x.valid || x.key0 >= x.n) return x;
  const int last = min(x.key0 + BT, x.n) - 1;
  long long i1 = x.m;
  if (p.causal) x.i0 = max(0, x.key0 - x.off);
  if (p.shape.window > 0) {
    i1 = min(i1, (long long)last + p.shape.window - x.off);
    if (!p.causal) x.i0 = max(0, x.key0 - x.off - p.shape.window + 1);
  }
  if (i1 > x.i0) x.steps = (int)((i1 - x.i0 + per - 1) / per);
  return x;
}

// A thread's sum of 2^(score + nl) over columns [va, vb) of 128 (its key's row of S^T).
template <int kShape>
__device__ __forceinline__ float sum_columns(const KeyWeightsParams& p, uint32_t s_col, const float* nl, const float* query,
                                             const float* slope, float dist, int va, int vb) {
  const ScoreShape& sh = p.shape;
  const uint64_t mul = f2_pack(sh.sl2, sh.sl2);
  const bool edge = __any_sync(0xffffffffu, va > 0 || vb < BT);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
  for (int c = 0; c < BT / 32; ++c) {
    uint32_t u[32];
    tmem_ld32(s_col + 32 * c, u);
    float y[32];
    if constexpr (kShape & kShapeCap) {
#pragma unroll
      for (int e = 0; e < 32; ++e) y[e] = fmaf(-2.f * sh.cap2, tanh_r(__uint_as_float(u[e]) * sh.capk), sh.cap2);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(u[e]);
    }
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      float4 l = *reinterpret_cast<const float4*>(nl + 32 * c + e);
      if constexpr (kShape & kShapeBias) {
        const float4 qi = *reinterpret_cast<const float4*>(query + 32 * c + e);
        const float4 sl = *reinterpret_cast<const float4*>(slope + 32 * c + e);
        l.x = fmaf(sl.x, fabsf(dist + qi.x), l.x);
        l.y = fmaf(sl.y, fabsf(dist + qi.y), l.y);
        l.z = fmaf(sl.z, fabsf(dist + qi.z), l.z);
        l.w = fmaf(sl.w, fabsf(dist + qi.w), l.w);
      }
      const uint64_t y0 = f2_pack(y[e], y[e + 1]), y1 = f2_pack(y[e + 2], y[e + 3]);
      const uint64_t l0 = f2_pack(l.x, l.y), l1 = f2_pack(l.z, l.w);
      f2_unpack((kShape & kShapeCap) ? f2_add(y0, l0) : f2_fma(y0, mul, l0), y[e], y[e + 1]);
      f2_unpack((kShape & kShapeCap) ? f2_add(y1, l1) : f2_fma(y1, mul, l1), y[e + 2], y[e + 3]);
    }
    if (edge) {
      const int a = max(va - 32 * c, 0), z = min(vb - 32 * c, 32);
      const uint32_t vis = a < z ? (0xffffffffu << a) & (0xffffffffu >> (32 - z)) : 0u;
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (!((vis >> e) & 1u)) y[e] = -CUDART_INF_F;
    }
#pragma unroll
    for (int e = 0; e < 32; e += 2) acc[(e >> 1) & 3] = f2_add(acc[(e >> 1) & 3], f2_pack(ex2(y[e]), ex2(y[e + 1])));
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
      mbar_init(bar(i), ((i >= kSFree && i < kSFree + kBufs) || i == kSumFull || i == kSumFree) ? 4 : 1);
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
  const int total = (cap_keys + BT - 1) / BT * p.B * p.Hkv;

  if (warp == 0) {
    // ------------------------------------------------------------ producer (lane i: page i of a K tile)
    if (lane < BT / 16) {
      uint32_t nk = 0, nq = 0;
      const uint64_t pol_k = policy_evict_first(), pol_q = policy_evict_last();
      bool ok = true;
      for (int it = blockIdx.x; ok && it < total; it += gridDim.x) {
        const KwItem x = kw_item(p, it, G, per);
        if (x.steps == 0) continue;
        const uint32_t kb = nk & 1;
        if (!mbar_wait(bar(kKEmpty + kb), ((nk >> 1) & 1) ^ 1, abort, p.status, p.wait_ns)) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(kKFull + kb), Lay::kTile);
        const int P = p.page_size, pages = BT / P;
        if (lane < pages) {
          const int slot = x.key0 / P + lane;
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
            tma_load_3d(sb + Lay::kOffK + kb * Lay::kTile + dc * BT * 128 + lane * P * 128, &tk, bar(kKFull + kb), dc * 64,
                        x.hkv, row, pol_k);
        }
        ++nk;
        // the Q tiles are lane 0's alone (the other lanes, which nothing would hold back here, could miss
        // a phase): they go on to the next item's pages, as far as KEmpty lets them
        for (int s = 0; lane == 0 && s < x.steps; ++s, ++nq) {
          const uint32_t st = nq % kQStages;
          if (!mbar_wait(bar(kQEmpty + st), ((nq / kQStages) & 1) ^ 1, abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(kQFull + st), R * D * 2);
#pragma unroll
          for (int dc = 0; dc < D / 64; ++dc)
            tma_load_3d(sb + Lay::kOffQ + st * Lay::kTile + dc * BT * 128, &tq, bar(kQFull + st), dc * 64, x.hkv * G,
                        x.q0 + x.i0 + s * per, pol_q);
        }
      }
      // no copy may land after the CTA is gone: wait for the last armed phase of each barrier
      for (uint32_t st = 0; st < 2; ++st) {
        const uint32_t c = (nk + 1 - st) / 2;
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
      uint32_t nk = 0, nq = 0;
      bool ok = true;
      for (int it = blockIdx.x; ok && it < total; it += gridDim.x) {
        const KwItem x = kw_item(p, it, G, per);
        if (x.steps == 0) continue;
        const uint32_t kb = nk & 1;
        if (!mbar_wait(bar(kKFull + kb), (nk >> 1) & 1, abort, p.status, p.wait_ns)) break;
        const uint64_t a0 = smem_desc_sw128(sb + Lay::kOffK + kb * Lay::kTile, 16, 1024);
        for (int s = 0; s < x.steps; ++s, ++nq) {
          const uint32_t st = nq % kQStages, buf = nq % kBufs;
          if (!mbar_wait(bar(kQFull + st), (nq / kQStages) & 1, abort, p.status, p.wait_ns) ||
              !mbar_wait(bar(kSFree + buf), ((nq / kBufs) & 1) ^ 1, abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t b0 = smem_desc_sw128(sb + Lay::kOffQ + st * Lay::kTile, 16, 1024);
          mma_ss_c<false>(tmem + buf * BT, a0, b0, id);
#pragma unroll
          for (int ks = 1; ks < D / 16; ++ks) {
            const uint64_t o = (uint64_t)((ks >> 2) * kAtom + (ks & 3) * 2);
            mma_ss_c<true>(tmem + buf * BT, a0 + o, b0 + o, id);
          }
          mma_commit(bar(kSFull + buf));
          mma_commit(bar(kQEmpty + st));
        }
        if (!ok) break;
        mma_commit(bar(kKEmpty + kb));
        ++nk;
      }
      mma_commit(bar(kMmaDone));
      drain(bar(kMmaDone), 0);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ per-column vectors
    uint32_t nq = 0;
    bool ok = true;
    for (int it = blockIdx.x; ok && it < total; it += gridDim.x) {
      const KwItem x = kw_item(p, it, G, per);
      for (int s = 0; s < x.steps; ++s, ++nq) {
        const uint32_t buf = nq % kBufs;
        float v[BT / 32], sl[BT / 32];
#pragma unroll
        for (int e = 0; e < BT / 32; ++e) {
          const int u = 32 * e + lane, i = x.i0 + s * per + u / G;
          v[e] = -CUDART_INF_F;   // rows past R or past the chunk, and rows that saw no key, give nothing
          if (u < R && i < x.m) {
            const float lse = __ldg(p.lse + (x.hkv * G + u % G) * p.lse_head + (long long)(x.q0 + i) * p.lse_row);
            if (lse > -CUDART_INF_F) v[e] = -lse * kLog2e;
          }
          sl[e] = (kShape & kShapeBias) && u < R ? -__ldg(p.shape.slopes + x.hkv * G + u % G) * kLog2e : 0.f;
        }
        if (!warp_wait(bar(kSFree + buf), ((nq / kBufs) & 1) ^ 1, abort, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        float* dst = reinterpret_cast<float*>(smem + Lay::kOffVec) + buf * 2 * BT;
#pragma unroll
        for (int e = 0; e < BT / 32; ++e) {
          dst[32 * e + lane] = v[e];
          if (kShape & kShapeBias) dst[BT + 32 * e + lane] = sl[e];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kVecFull + buf));
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums (one key per thread)
    const int wg = (warp - 4) >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const uint32_t s_base = tmem + ((uint32_t)(q4 * 32) << 16);
    float* sums = reinterpret_cast<float*>(smem + Lay::kOffSum);
    uint32_t nq = 0, nsum = 0;
    bool ok = true;
    // test hook: a wait that runs out (nothing arrives on the stall barrier)
    if (p.debug_stall && !warp_wait(bar(kBarStall), 0, abort, p.status, p.wait_ns)) ok = false;
    for (int it = blockIdx.x; ok && it < total; it += gridDim.x) {
      const KwItem x = kw_item(p, it, G, per);
      if (!x.valid) {
        if (it < p.B * p.Hkv && x.hkv == 0 && warp == 4 && lane == 0) record_status(p.status, kStatusDeviceCheck);
        continue;  // the sequence is skipped
      }
      const int key = x.key0 + r;
      const size_t at = ((size_t)x.b * p.Hkv + x.hkv) * cap_keys + key;
      float sum = 0.f;
      for (int s = 0; s < x.steps; ++s, ++nq) {
        if ((int)(nq & 1) != wg) continue;
        const uint32_t buf = nq % kBufs;
        if (!warp_wait(bar(kVecFull + buf), (nq / kBufs) & 1, abort, p.status, p.wait_ns) ||
            !warp_wait(bar(kSFull + buf), (nq / kBufs) & 1, abort, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        mbar_try_wait(bar(kVecFull + buf), (nq / kBufs) & 1);  // completed: this lane's own acquire of the vector
        tc_fence_after();
        // columns whose query sees the key: positions [key, key + W) (causal) or (key - W, key + W)
        const int first = x.i0 + s * per + x.off;              // position of column 0
        const int nrows = (int)min((long long)R, ((long long)x.m - x.i0 - (long long)s * per) * G);
        int va = 0, vb = nrows;
        if (p.causal) va = max(va, min(key - first, per) * G);
        if (p.shape.window > 0) {
          const long long hi = (long long)key + p.shape.window - first;
          if (hi < per) vb = min(vb, (int)max(hi, 0ll) * G);
          if (!p.causal) va = max(va, (int)min((long long)key - p.shape.window + 1 - first, (long long)per) * G);
        }
        const float* vec = reinterpret_cast<const float*>(smem + Lay::kOffVec) + buf * 2 * BT;
        sum += sum_columns<kShape>(p, s_base + buf * BT, vec, col_query, vec + BT, (float)(first - key), va, vb);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFree + buf));
      }
      if (!ok) break;
      if (x.steps > 1) {  // both warpgroups took steps of the item
        if (wg == 1) {
          if (!warp_wait(bar(kSumFree), (nsum & 1) ^ 1, abort, p.status, p.wait_ns)) break;
          sums[r] = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kSumFull));
        } else {
          if (!warp_wait(bar(kSumFull), nsum & 1, abort, p.status, p.wait_ns)) break;
          mbar_try_wait(bar(kSumFull), nsum & 1);
          sum += sums[r];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kSumFree));
        }
        ++nsum;
      }
      // the writer: the first warpgroup, or the one that took the item's only step
      const bool writer = x.steps == 1 ? (int)((nq - 1) & 1) == wg : wg == 0;
      if (writer && key < cap_keys) {
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
cudaError_t launch_t(const KeyWeightsParams& p, const CUtensorMap& tq, const CUtensorMap& tk, int num_sms,
                     cudaStream_t stream) {
  auto kern = key_weights_tc_kernel<D, kShape>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, KwTcLayout<D>::kBytes);
  if (e != cudaSuccess) return e;
  const long long items = (long long)((p.max_pages * p.page_size + BT - 1) / BT) * p.B * p.Hkv;
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
