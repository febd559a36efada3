// Eviction: every KV head of every sequence cut down to `keep` tokens — the first `first`, the
// last `recent` and the heaviest of the others — compacted in order.
//
// select_kernel, one block (or a cluster) per (sequence, KV head): the weights of the middle tokens as
// order-preserving 32-bit integers, the threshold by three passes of an 11-bit histogram from the top
// digit down (its first digit tells quarter octaves apart: few lanes of a warp meet in a bin, where the
// 8-bit digit of an exponent brought most of them together), then a scan in index order that counts what is kept and the ties already taken
// (ties go to the lowest index) and places the kept indices and their weights.
// move_kernel copies the kept K and V rows by that list. Into other pages every row is
// independent. In place a row moves to a slot at or below its own, which may hold a row that has
// yet to move: there a block owns one 32-byte column slice of one head's K or V and walks its
// rows in order, a batch in registers at a time, so a slot is read before it is written.
// 8 contexts of 7k to 16k tokens of 8 heads (d = 128) to 4096: the selection 18 us (64 blocks, a block's three
// passes over its 16k weights), the move 40 us (268 MB, 6.7 TB/s).
#include "device_common.cuh"
#include "ops_internal.h"

#include <math_constants.h>

namespace fattn {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;

// Larger float, larger integer; -0 and +0 alike; NaN below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

constexpr int kTile = 16 * kSelThreads;         // 16384 tokens
constexpr int kBins = 2048;
static_assert(kBins == 2 * kSelThreads, "two bins per thread");

// The blocks of a cluster: all of them at the barrier, and a pair of words in another one's shared memory.
template <int C>
__device__ __forceinline__ void cluster_sync() {
  if constexpr (C == 1)
    __syncthreads();
  else
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ int2 read_block(const int* local, int rank) {
  int2 v;
  asm volatile(
      "{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %2, %3;\nld.shared::cluster.v2.s32 {%0, %1}, [a];\n}"
      : "=r"(v.x), "=r"(v.y)
      : "r"(smem_u32(local)), "r"(rank)
      : "memory");
  return v;
}

// C blocks, a cluster, per (sequence, KV head): each takes 1 / C of every tile.
template <int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kSelThreads) select_kernel(const EvictParams p) {
  constexpr int kPer = kTile / kSelThreads / C;   // weights per thread and tile
  __shared__ __align__(8) int s_hists[2][kBins];  // in turn: a block may still read the last pass's of another
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int s_warp[32];
  __shared__ int s_cnt[kPer * 32];   // per 32 consecutive tokens of a tile: kept above the threshold | ties << 16
  __shared__ __align__(8) int s_tile[2];   // of the block's part of the tile
  const int b = blockIdx.y, h = blockIdx.x / C, rank = blockIdx.x % C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = p.max_pages * p.page_size;
  const int out_cap = p.dst_max_pages * p.page_size;
  int n = __ldg(p.seqlens + b);
  if (n < 0 || n > cap) {
    if (h == 0 && rank == 0 && tid == 0) record_status(p.status, kStatusDeviceCheck);
    n = 0;
  }
  const int m = min(n, p.keep);
  if (h == 0 && rank == 0 && tid == 0) p.seqlens_out[b] = m;
  const float* w = p.w_in + ((size_t)b * p.Hkv + h) * cap;
  float* wo = p.w_out + ((size_t)b * p.Hkv + h) * out_cap;
  int* kept = p.kept + ((size_t)b * p.Hkv + h) * p.keep;

  // A tile's weights in registers (token mine + tile + 1024 i + tid in x[i]): the loads are on their way
  // together, and with a single tile (16384 tokens) they are read once for all the passes.
  const int mine = rank * kPer * kSelThreads + tid;
  float x[kPer];
  auto load = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = t0 + i * kSelThreads + mine;
      x[i] = t < n ? w[t] : 0.f;
    }
  };
  if (n <= kTile) load(0);

  // middle tokens [lo, hi): `need` of them are kept
  const int lo = m < n ? p.first : 0, hi = m < n ? n - p.recent : 0;
  const int need = m < n ? m - p.first - p.recent : 0;
  if (tid == 0) {
    s_prefix = 0;
    s_need = need;
  }
  if (need > 0) {
    for (int pass = 0; pass < 3; ++pass) {   // digits of 11, 11 and 10 bits
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 0 ? 32 : pass == 1 ? 21 : 10;
      const uint32_t digits = pass == 2 ? 1023u : 2047u;
      int* s_hist = s_hists[pass & 1];
      s_hist[tid] = s_hist[tid + kSelThreads] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix;
      const int want = s_need;
      for (int t0 = 0; t0 < n; t0 += kTile) {
        if (n > kTile) load(t0);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int t = t0 + i * kSelThreads + mine;
          if (t - tid >= n) break;
          if (t >= lo && t < hi) {
            const uint32_t k = order_key(x[i]);
            if (pass == 0 || (k >> above) == (prefix >> above)) atomicAdd(&s_hist[(k >> shift) & digits], 1);
          }
        }
      }
      cluster_sync<C>();
      // the threshold's digit, found by every block: thread i counts bins 2047 - 2 i and 2046 - 2 i, after all that
      // are higher
      int c0 = 0, c1 = 0;
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const int* pair = s_hist + kBins - 2 - 2 * tid;
        const int2 v = C == 1 ? *reinterpret_cast<const int2*>(pair) : read_block(pair, r);
        c1 += v.x;
        c0 += v.y;
      }
      int v = c0 + c1;
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += a;
      }
      if (lane == 31) s_warp[warp] = v;
      __syncthreads();
      int u = lane < warp ? s_warp[lane] : 0;
      for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
      const int before = u + v - c0 - c1;
      if (before < want && want <= before + c0 + c1) {  // one thread
        const bool first_bin = want <= before + c0;
        s_prefix = prefix | ((uint32_t)(kBins - (first_bin ? 1 : 2) - 2 * tid) << shift);
        s_need = want - before - (first_bin ? 0 : c0);
      }
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  const uint32_t thr = s_prefix;
  const int ties = s_need;   // tokens equal to the threshold that are kept, the lowest indices

  // In index order, tile by tile: counts per 32 tokens, their scan, then every kept token's place.
  // `done` and `tied` count over the tiles before. In place a weight moves to or below its own place,
  // and a tile's are all in registers before any is written.
  int done = 0, tied = 0;
  for (int t0 = 0; t0 < n; t0 += kTile) {
    if (n > kTile) load(t0);
    const int batches = min(kPer, max(0, n - t0 - (mine - tid) + kSelThreads - 1) / kSelThreads);
    uint32_t gts = 0, eqs = 0;   // bit i: this thread's token of batch i
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= batches) {
        if (lane == 0) s_cnt[i * 32 + warp] = 0;
        continue;
      }
      const int t = t0 + i * kSelThreads + mine;
      const bool in = t < n, mid = in && t >= lo && t < hi;
      const uint32_t k = order_key(x[i]);
      const bool gt = in && (!mid || (need > 0 && k > thr)), eq = mid && need > 0 && k == thr;
      gts |= (uint32_t)gt << i;
      eqs |= (uint32_t)eq << i;
      const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
      if (lane == 0) s_cnt[i * 32 + warp] = __popc(bg) | (__popc(be) << 16);
    }
    __syncthreads();
    if (warp == 0) {   // exclusive scan of the 32 kPer counts (the sums stay below 2^15 and 2^16: 16384 tokens)
      int c[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        c[i] = s_cnt[lane * kPer + i];
        sum += c[i];
      }
      int v = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += a;
      }
      if (lane == 31) {
        s_tile[0] = v & 0xffff;
        s_tile[1] = v >> 16;
      }
      v -= sum;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        s_cnt[lane * kPer + i] = v;
        v += c[i];
      }
    }
    cluster_sync<C>();   // (in place: every block's weights of the tile are in registers)
    int done_next = done, tied_next = tied;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const int2 v = C == 1 ? *reinterpret_cast<const int2*>(s_tile) : read_block(s_tile, r);
      done += r < rank ? v.x : 0;
      tied += r < rank ? v.y : 0;
      done_next += v.x;
      tied_next += v.y;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= batches) break;
      const bool gt = (gts >> i) & 1u, eq = (eqs >> i) & 1u;
      const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
      const int before = s_cnt[i * 32 + warp];
      const uint32_t below = (1u << lane) - 1u;
      const int g_before = done + (before & 0xffff) + __popc(bg & below);
      const int e_before = tied + (before >> 16) + __popc(be & below);
      if (gt || (eq && e_before < ties)) {
        const int at = g_before + min(e_before, ties);
        kept[at] = t0 + i * kSelThreads + mine;
        wo[at] = x[i];
      }
    }
    done = done_next;
    tied = tied_next;
    cluster_sync<C>();   // (the counts are read, here and by the other blocks)
  }
  for (int t = m + rank * kSelThreads + tid; t < p.keep; t += C * kSelThreads) kept[t] = -1;
  for (int t = m + rank * kSelThreads + tid; t < out_cap; t += C * kSelThreads) wo[t] = 0.f;
}

// Slot of token t of sequence b, in 16-byte units of head h's row; -1 if its page is not in the pool.
__device__ __forceinline__ long long slot_unit(const EvictParams& p, const int32_t* table, int width, int b, int h, int t) {
  const int page = __ldg(table + (size_t)b * width + t / p.page_size);
  if (page < 0 || page >= p.num_pages) return -1;
  return (((long long)page * p.page_size + t % p.page_size) * p.Hkv + h) * (p.d / 8);
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p) {
  const int bh = blockIdx.y, b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int m = __ldg(p.seqlens_out + b);
  const int U = p.d / 8;                       // 16-byte units per row
  const int* kept = p.kept + (size_t)bh * p.keep;
  const int rows = kMoveThreads / U;           // rows of a block's step, K and V of each
  const int r = threadIdx.x / U, u = threadIdx.x - r * U;
  if (r >= rows) return;
  uint4* kc = static_cast<uint4*>(p.kcache);
  uint4* vc = static_cast<uint4*>(p.vcache);
  // (unsigned: with tables of nearly 2^31 tokens the step past the last row leaves the int range)
  for (unsigned s = blockIdx.x * rows + r; s < (unsigned)m; s += gridDim.x * rows) {
    const long long a = slot_unit(p, p.block_table, p.max_pages, b, h, __ldg(kept + s));
    const long long d = slot_unit(p, p.dst_table, p.dst_max_pages, b, h, (int)s);
    if (a < 0 || d < 0) {
      record_status(p.status, kStatusDeviceCheck);
      continue;
    }
    const uint4 x = kc[a + u], y = vc[a + u];
    kc[d + u] = x;
    vc[d + u] = y;
  }
}

constexpr int kBatch = 8;  // rows per thread of an in-place step

__global__ void __launch_bounds__(kMoveThreads) move_in_place_kernel(const EvictParams p) {
  const int bh = blockIdx.y, b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int m = __ldg(p.seqlens_out + b);
  const int u = (blockIdx.x >> 1) * 2 + (threadIdx.x & 1);   // this thread's 16-byte unit of the row
  const bool live = u < p.d / 8;               // (an odd number of units leaves half a slice)
  uint4* c = static_cast<uint4*>(blockIdx.x & 1 ? p.vcache : p.kcache);
  const int* kept = p.kept + (size_t)bh * p.keep;
  for (int s0 = 0; s0 < m; s0 += kMoveThreads / 2 * kBatch) {
    uint4 x[kBatch];
    long long d[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + i * (kMoveThreads / 2) + (threadIdx.x >> 1);
      d[i] = -1;
      if (live && s < m) {
        const int t = __ldg(kept + s);
        if (t != s) {
          const long long a = slot_unit(p, p.block_table, p.max_pages, b, h, t);
          d[i] = slot_unit(p, p.block_table, p.max_pages, b, h, s);
          if (a < 0 || d[i] < 0) {
            record_status(p.status, kStatusDeviceCheck);
            d[i] = -1;
          } else {
            x[i] = c[a + u];
          }
        }
      }
    }
    __syncthreads();  // the batch is read: its slots, all at or below its sources, may be written
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (d[i] >= 0) c[d[i] + u] = x[i];
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream) {
  // a cluster of four blocks for tables of more than one tile and few heads: the passes' re-reads go four times as fast
  // (8 heads of 131072 tokens, the whole call: 189 us with one block a head, 126 with four); up to a tile the
  // cluster's barriers cost what they bring (64 heads of 16384: 58 and 57 us), and with many heads more (512 heads of
  // 16384: 135 and 173 us)
  if ((long long)p.max_pages * p.page_size > kTile && (long long)p.B * p.Hkv * 4 <= num_sms)
    select_kernel<4><<<dim3(p.Hkv * 4, p.B), kSelThreads, 0, stream>>>(p);
  else
    select_kernel<1><<<dim3(p.Hkv, p.B), kSelThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int heads = p.B * p.Hkv;
  if (p.dst_table == nullptr) {
    move_in_place_kernel<<<dim3(2 * ((p.d / 8 + 1) / 2), heads), kMoveThreads, 0, stream>>>(p);
  } else {
    const int rows = kMoveThreads / (p.d / 8);
    const int steps = (p.keep + rows - 1) / rows;
    const int want = (num_sms * 8 + heads - 1) / heads;   // eight blocks per SM
    move_kernel<<<dim3(steps < want ? steps : want, heads), kMoveThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fattn
