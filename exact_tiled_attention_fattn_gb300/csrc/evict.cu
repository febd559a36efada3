// Eviction: every KV head of every sequence cut down to `keep` tokens — the first `first`, the
// last `recent` and the heaviest of the others — compacted in order.
//
// select_kernel, one block per (sequence, KV head): the weights of the middle tokens as
// order-preserving 32-bit integers, the threshold by four passes of an 8-bit histogram from the top
// digit down, then one walk in index order that counts what is kept and the ties already taken
// (ties go to the lowest index) and writes the kept indices and their weights.
// move_kernel copies the kept K and V rows by that list. Into other pages every row is
// independent. In place a row moves to a slot at or below its own, which may hold a row that has
// yet to move: there a block owns one 16-byte column slice of one head's K or V and walks its
// rows in order, a batch in registers at a time, so a slot is read before it is written.
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

__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictParams p) {
  __shared__ int s_hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int s_warp[32];
  const int b = blockIdx.y, h = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = p.max_pages * p.page_size;
  const int out_cap = p.dst_max_pages * p.page_size;
  int n = __ldg(p.seqlens + b);
  if (n < 0 || n > cap) {
    if (h == 0 && tid == 0) record_status(p.status, kStatusDeviceCheck);
    n = 0;
  }
  const int m = min(n, p.keep);
  if (h == 0 && tid == 0) p.seqlens_out[b] = m;
  const float* w = p.w_in + ((size_t)b * p.Hkv + h) * cap;
  float* wo = p.w_out + ((size_t)b * p.Hkv + h) * out_cap;
  int* kept = p.kept + ((size_t)b * p.Hkv + h) * p.keep;

  // middle tokens [lo, hi): `need` of them are kept
  const int lo = m < n ? p.first : 0, hi = m < n ? n - p.recent : 0;
  const int need = m < n ? m - p.first - p.recent : 0;
  if (tid == 0) {
    s_prefix = 0;
    s_need = need;
  }
  __syncthreads();
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) s_hist[tid] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix;
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t k = order_key(w[t]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (warp == 0) {  // digits from the highest down: lane l holds digits 255 - 8l ... 248 - 8l
        int c[8], sum = 0;
        for (int i = 0; i < 8; ++i) {
          c[i] = s_hist[255 - 8 * lane - i];
          sum += c[i];
        }
        int before = sum;
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += v;
        }
        before -= sum;  // tokens with a higher digit than this lane's
        const int want = s_need;
        __syncwarp();
        for (int i = 0; i < 8; ++i) {
          if (before < want && want <= before + c[i]) {  // one (lane, i): the threshold's digit
            s_prefix = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
            s_need = want - before;
          }
          before += c[i];
        }
      }
      __syncthreads();
    }
  }
  const uint32_t thr = s_prefix;
  const int ties = s_need;   // tokens equal to the threshold that are kept, the lowest indices

  // walk in index order; `done` and `tied` count over the tokens before the batch
  int done = 0, tied = 0;
  for (int t0 = 0; t0 < n; t0 += kSelThreads) {
    const int t = t0 + tid;
    const bool in = t < n, mid = in && t >= lo && t < hi;
    const float x = in ? w[t] : 0.f;
    const uint32_t k = order_key(x);
    const bool gt = in && (!mid || (need > 0 && k > thr)), eq = mid && need > 0 && k == thr;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_warp[warp] = __popc(bg) | (__popc(be) << 16);
    __syncthreads();   // also: every weight of the batch is read before any is written (in place)
    int v = s_warp[lane];
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += a;
    }
    const int all = __shfl_sync(0xffffffffu, v, 31);
    const int prev = warp ? __shfl_sync(0xffffffffu, v, warp - 1) : 0;
    const uint32_t below = (1u << lane) - 1u;
    const int g_before = done + (prev & 0xffff) + __popc(bg & below);
    const int e_before = tied + (prev >> 16) + __popc(be & below);
    if (gt || (eq && e_before < ties)) {
      const int at = g_before + min(e_before, ties);
      kept[at] = t;
      wo[at] = x;
    }
    done += all & 0xffff;
    tied += all >> 16;
    __syncthreads();
  }
  for (int t = m + tid; t < p.keep; t += kSelThreads) kept[t] = -1;
  for (int t = m + tid; t < out_cap; t += kSelThreads) wo[t] = 0.f;
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
  for (int s = blockIdx.x * rows + r; s < m; s += gridDim.x * rows) {
    const long long a = slot_unit(p, p.block_table, p.max_pages, b, h, __ldg(kept + s));
    const long long d = slot_unit(p, p.dst_table, p.dst_max_pages, b, h, s);
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
  const int u = blockIdx.x >> 1;               // this block's 16-byte unit of the row
  uint4* c = static_cast<uint4*>(blockIdx.x & 1 ? p.vcache : p.kcache);
  const int* kept = p.kept + (size_t)bh * p.keep;
  for (int s0 = 0; s0 < m; s0 += kMoveThreads * kBatch) {
    uint4 x[kBatch];
    long long d[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + i * kMoveThreads + threadIdx.x;
      d[i] = -1;
      if (s < m) {
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
  select_kernel<<<dim3(p.Hkv, p.B), kSelThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int heads = p.B * p.Hkv;
  if (p.dst_table == nullptr) {
    move_in_place_kernel<<<dim3(2 * (p.d / 8), heads), kMoveThreads, 0, stream>>>(p);
  } else {
    const int rows = kMoveThreads / (p.d / 8);
    const int steps = (p.keep + rows - 1) / rows;
    const int want = (num_sms * 8 + heads - 1) / heads;   // eight blocks per SM
    move_kernel<<<dim3(steps < want ? steps : want, heads), kMoveThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fattn
