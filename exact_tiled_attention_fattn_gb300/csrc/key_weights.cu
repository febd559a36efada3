// Attention weight that the tokens of a paged cache received:
//   w_out[b, hkv, t] = decay w_in[b, hkv, t] + sum over the group's heads and the chunk's queries of e^{s - lse}
// (s the shaped score, lse the row's logsumexp from the attention call), the statistic by
// which fattn_evict_paged picks the tokens to keep.
//
// The softmax's statistics are known, so one product per pair of tiles is enough and nothing
// is kept per query: S^T = K Q^T with the keys as rows, summed over its columns in fp32
// registers. A block owns 128 keys of one (sequence, KV head) and no other block writes their
// sums: no atomics, the same order of additions every time. Each of the 4 warps holds its 32
// keys as A fragments in registers for the whole walk over the queries, whose rows (all heads
// of the group of a query are contiguous) stream through a two-stage ring in shared memory.
//
// With few query rows (single tokens, short drafts) the walk over the queries is short and K's
// bytes are the bound: stream_kernel.
#include "device_common.cuh"
#include "ops_internal.h"
#include "score_shape.cuh"
#include "sm100_primitives.cuh"

#include <math_constants.h>

namespace fattn {
namespace {

constexpr int kKeys = 128;   // keys per block
constexpr int kQRows = 32;   // query rows (query x head of the group) per step
constexpr int kWarps = 4;

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// C (16 x 8, fp32) += A (16 x 16, bf16, row) B (16 x 8, bf16, col)
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16-byte unit u of row r at u ^ (r & 7): the 8 rows that ldmatrix reads hit 8 bank groups.
template <int D>
__device__ __forceinline__ uint32_t unit_at(int r, int u) {
  return (uint32_t)((r * (D / 8) + (u ^ (r & 7))) * 16);
}

template <int D>
struct KwLayout {
  static constexpr int kK = kKeys * D * 2;
  static constexpr int kQ = kQRows * D * 2;
  static constexpr int kVec = kQRows * 16;   // per query row: -lse log2(e), slope, position, (unused)
  static constexpr int kOffQ = kK;
  static constexpr int kOffVec = kOffQ + 2 * kQ;
  static constexpr int kBytes = kOffVec + 2 * kVec;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) key_weights_kernel(const KeyWeightsParams p) {
  using Lay = KwLayout<D>;
  constexpr int U = D / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_row[kKeys];  // each key's first element in the cache, -1: none
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y, hkv = blockIdx.x % p.Hkv;  // heads first: the blocks that run together read whole rows
  const int n = __ldg(p.seqlens_k + b);
  const int key0 = blockIdx.x / p.Hkv * kKeys;
  const int cap = p.max_pages * p.page_size;
  const int q0 = __ldg(p.cu_seqlens + b), q1 = __ldg(p.cu_seqlens + b + 1), m = q1 - q0;
  if (n < 0 || n > cap || q0 < 0 || m < 0 || q1 > p.total_q || m > n || m > p.max_q) {
    if (key0 == 0 && hkv == 0 && threadIdx.x == 0) record_status(p.status, kStatusDeviceCheck);
    return;  // the sequence is skipped
  }
  const size_t w_row = ((size_t)b * p.Hkv + hkv) * cap;
  if (p.w_out != p.w_in) {  // slots past the sequence
    for (int t = max(key0, n) + threadIdx.x; t < min(key0 + kKeys, cap); t += kWarps * 32) p.w_out[w_row + t] = 0.f;
  }
  if (key0 >= n) return;
  const int nkeys = min(kKeys, n - key0), off = n - m;
  const int G = p.Hq / p.Hkv;

  // queries [i0, i1) that can see one of the block's keys, and their rows i * G + head
  int i0 = 0, i1 = m;
  if (p.causal) i0 = max(0, key0 - off);
  if (p.shape.window > 0) {
    i1 = (int)min((long long)m, (long long)key0 + nkeys - 1 + p.shape.window - off);
    if (!p.causal) i0 = (int)max(0ll, (long long)key0 - off - p.shape.window + 1);
  }
  const long long u0 = (long long)i0 * G, u1 = (long long)max(i0, i1) * G;
  const int steps = (int)((u1 - u0 + kQRows - 1) / kQRows);

  // ---- K rows of the block
  if (threadIdx.x < kKeys) {
    long long row = -1;
    if ((int)threadIdx.x < nkeys && steps > 0) {
      const int t = key0 + threadIdx.x;
      const int page = __ldg(p.block_table + (size_t)b * p.max_pages + t / p.page_size);
      if (page >= 0 && page < p.num_pages)
        row = (((long long)page * p.page_size + t % p.page_size) * p.Hkv + hkv) * D;
      else
        record_status(p.status, kStatusDeviceCheck);
    }
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(p.kcache);
  const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(p.q);
  for (int idx = threadIdx.x; idx < kKeys * U; idx += kWarps * 32) {
    const int r = idx / U, u = idx % U;
    const long long row = s_row[r];
    cp16(sb + unit_at<D>(r, u), kc + (row < 0 ? 0 : row + u * 8), row < 0 ? 0 : 16);
  }
  auto load_q = [&](int s) {
    const uint32_t dst = sb + Lay::kOffQ + (s & 1) * Lay::kQ;
    for (int idx = threadIdx.x; idx < kQRows * U; idx += kWarps * 32) {
      const int r = idx / U, u = idx % U;
      const long long w = u0 + (long long)s * kQRows + r;
      const bool ok = w < u1;
      const long long i = ok ? w / G : 0, h = ok ? w - i * G : 0;
      cp16(dst + unit_at<D>(r, u), qg + ((q0 + i) * p.Hq + (long long)hkv * G + h) * D + u * 8, ok ? 16 : 0);
    }
    if (threadIdx.x < kQRows) {
      const long long w = u0 + (long long)s * kQRows + threadIdx.x;
      float4 v = make_float4(-CUDART_INF_F, 0.f, 0.f, 0.f);
      if (w < u1) {
        const long long i = w / G;
        const int h = hkv * G + (int)(w - i * G);
        const float lse = __ldg(p.lse + h * p.lse_head + (q0 + i) * p.lse_row);
        // a row that saw no key (lse = -inf) gives no weight; a NaN stays one
        if (lse != -CUDART_INF_F) v.x = -lse * kLog2e;
        if (p.shape.slopes) v.y = -__ldg(p.shape.slopes + h) * kLog2e;
        v.z = __int_as_float((int)i + off);
      }
      *reinterpret_cast<float4*>(smem + Lay::kOffVec + (s & 1) * Lay::kVec + threadIdx.x * 16) = v;
    }
  };
  if (steps > 0) load_q(0);
  cp_commit();
  cp_wait<0>();
  __syncthreads();

  // ---- this warp's 32 keys as A fragments
  uint32_t ka[2][D / 16][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      ldsm4(sb + unit_at<D>(warp * 32 + mt * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, kk * 2 + (lane >> 4)), ka[mt][kk]);

  const float sl2 = p.scale * kLog2e;
  const int g = lane >> 2;
  const int kg = key0 + warp * 32 + g;        // this thread's keys: kg, + 8, + 16, + 24
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < steps; ++s) {
    if (s + 1 < steps) load_q(s + 1);
    cp_commit();
    const uint32_t qb = sb + Lay::kOffQ + (s & 1) * Lay::kQ;
    const float4* vec = reinterpret_cast<const float4*>(smem + Lay::kOffVec + (s & 1) * Lay::kVec);
#pragma unroll
    for (int nt = 0; nt < kQRows / 16; ++nt) {
      float c[2][2][4] = {};
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t bq[4];
        ldsm4(qb + unit_at<D>(nt * 16 + (lane & 7) + (lane >> 4) * 8, kk * 2 + ((lane >> 3) & 1)), bq);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          mma(c[mt][0], ka[mt][kk], bq[0], bq[1]);
          mma(c[mt][1], ka[mt][kk], bq[2], bq[3]);
        }
      }
      if (p.shape.cap > 0.f) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int n8 = 0; n8 < 2; ++n8) cap_in_place(p.shape, c[mt][n8]);
      }
#pragma unroll
      for (int n8 = 0; n8 < 2; ++n8)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 v = vec[nt * 16 + n8 * 8 + (lane & 3) * 2 + e];
          const int pos = __float_as_int(v.z);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int dist = pos - (kg + mt * 16 + hf * 8);
              const float x = c[mt][n8][hf * 2 + e];
              float y = p.shape.cap > 0.f ? x : x * sl2;
              y = fmaf(v.y, fabsf((float)dist), y);
              bool see = !p.causal || dist >= 0;
              if (p.shape.window > 0) see = see && abs(dist) < p.shape.window;
              const float w = ex2(y + v.x);
              acc[mt * 2 + hf] += see ? w : 0.f;
            }
        }
    }
    cp_wait<0>();
    __syncthreads();  // the next stage has landed, this one is read
  }
  // the four lanes of a key hold different queries
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 1);
    acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 2);
    const int r = warp * 32 + g + (i >> 1) * 16 + (i & 1) * 8;
    if ((lane & 3) == 0 && r < nkeys) {
      const size_t at = w_row + key0 + r;
      const float sum = s_row[r] >= 0 ? acc[i] : 0.f;
      p.w_out[at] = p.w_in ? fmaf(p.decay, p.w_in[at], sum) : sum;
    }
  }
}

// ------------------------------------------------------------------ few query rows
// At most 8 NT rows (queries x heads of the group): they are B fragments in registers, and a warp on its
// own streams 16-key chunks (part of one page: page_size is a multiple of 16) through a ring of TMA
// boxes, d / 64 per chunk. With cp.async by 16 bytes and Q fragments read per chunk the walk took 420
// instructions a chunk and was bound by them (55 us where K's bytes take 30), with one 256-byte bulk
// copy per key by the copies' number (48 us). Single tokens of 8 contexts of 7k to 16k tokens, 32 heads over 8,
// d = 128: 39 us, 5.3 TB/s.
constexpr int kChunk = 16;      // keys per warp and stage
constexpr int kStages = 3;
constexpr int kBlocksPerSm = 4;
constexpr uint64_t kDrainLimitNs = 200000000ull;

template <int D>
struct StreamLayout {
  static constexpr int kStage = kChunk * D * 2;    // 64-column halves of 16 rows x 128 bytes, 128-byte swizzle
  static constexpr int kOffBar = kWarps * kStages * kStage;
  static constexpr int kOffAbort = kOffBar + kWarps * (kStages + 1) * 8;   // (and a barrier that nothing arrives on: test hook)
  static constexpr int kBytes = kOffAbort + kWarps * 8 + 1024;  // + slack to align the base to 1024 B
};

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm) stream_kernel(const __grid_constant__ CUtensorMap tk, const KeyWeightsParams p, int segment) {
  using Lay = StreamLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = sb + warp * kStages * Lay::kStage, bars = sb + Lay::kOffBar + warp * (kStages + 1) * 8;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Lay::kOffAbort + warp * 8);
  if (lane == 0) {
    for (int i = 0; i <= kStages; ++i) sm100::mbar_init(bars + 8 * i, 1);
    *abort = 0;
    sm100::fence_mbar_init();
  }
  __syncwarp();
  // heads first: the blocks that run together read whole rows of the cache
  const int b = blockIdx.y, hkv = blockIdx.x % p.Hkv, key0 = blockIdx.x / p.Hkv * segment;
  const int cap = p.max_pages * p.page_size, G = p.Hq / p.Hkv;
  const int n = __ldg(p.seqlens_k + b);
  const int q0 = __ldg(p.cu_seqlens + b), q1 = __ldg(p.cu_seqlens + b + 1), m = q1 - q0;
  if (n < 0 || n > cap || q0 < 0 || m < 0 || q1 > p.total_q || m > n || m > p.max_q) {
    if (key0 == 0 && hkv == 0 && threadIdx.x == 0) record_status(p.status, kStatusDeviceCheck);
    return;  // the sequence is skipped
  }
  const size_t w_row = ((size_t)b * p.Hkv + hkv) * cap;
  if (p.w_out != p.w_in) {  // slots past the sequence
    for (int t = max(key0, n) + threadIdx.x; t < (int)min((long long)key0 + segment, (long long)cap); t += kWarps * 32) p.w_out[w_row + t] = 0.f;
  }
  if (key0 >= n) return;
  const int end = (int)min((long long)key0 + segment, (long long)n), off = n - m, rows = m * G;
  const int32_t* table = p.block_table + (size_t)b * p.max_pages;

  // Chunk c of this warp: keys key0 + 16 (4 c + warp) ..., in the pool's rows find(c) ... (-1: no such page)
  const int chunks = (end - key0 + kChunk - 1) / kChunk;
  const int mine = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;
  auto first_key = [&](int c) -> int { return key0 + kChunk * (kWarps * c + warp); };
  auto find = [&](int c) -> int {
    if (c >= mine) return -1;
    const int t = first_key(c), slot = t / p.page_size;
    const int page = __ldg(table + slot);
    if (page < 0 || page >= p.num_pages) {
      record_status(p.status, kStatusDeviceCheck);
      return -1;
    }
    return page * p.page_size + (t - slot * p.page_size);
  };
  uint32_t have = 0;   // bit c mod 32: chunk c is in the cache
  const uint64_t pol = sm100::policy_evict_first();
  auto issue = [&](int c, int row) {
    const uint32_t st = (uint32_t)c % kStages, bar = bars + 8 * st;
    have = (have & ~(1u << (c & 31))) | ((row >= 0 ? 1u : 0u) << (c & 31));
    if (lane == 0) {
      sm100::mbar_arrive_expect_tx(bar, row >= 0 ? Lay::kStage : 0);
      if (row >= 0) {
#pragma unroll
        for (int dc = 0; dc < D / 64; ++dc)
          sm100::tma_load_3d(ring + st * Lay::kStage + dc * kChunk * 128, &tk, bar, dc * 64, hkv, row, pol);
      }
    }
  };
  int row[kStages + 1];
#pragma unroll
  for (int c = 0; c <= kStages; ++c) row[c] = find(c);   // (one ahead of the copies from here on)
#pragma unroll
  for (int c = 0; c < kStages; ++c)
    if (c < mine) issue(c, row[c]);
  int next = row[kStages];

  // ---- the query rows as B fragments, and their columns' vectors
  const int g = lane >> 2;
  uint32_t qb[NT][D / 16][2];
  float nl[NT][2], slope[NT][2];
  int pos[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + g, i = r / G;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        static_cast<const __nv_bfloat16*>(p.q) + ((long long)(q0 + i) * p.Hq + hkv * G + (r - i * G)) * D + (lane & 3) * 2);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qb[nt][kk][0] = r < rows ? __ldg(src + kk * 8) : 0u;
      qb[nt][kk][1] = r < rows ? __ldg(src + kk * 8 + 4) : 0u;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int u = 8 * nt + (lane & 3) * 2 + e, iu = u / G, h = hkv * G + u - iu * G;
      nl[nt][e] = -CUDART_INF_F;
      slope[nt][e] = 0.f;
      pos[nt][e] = iu + off;
      if (u < rows) {
        const float lse = __ldg(p.lse + h * p.lse_head + (long long)(q0 + iu) * p.lse_row);
        if (lse != -CUDART_INF_F) nl[nt][e] = -lse * kLog2e;   // a row that saw no key gives no weight; a NaN stays one
        if (p.shape.slopes) slope[nt][e] = -__ldg(p.shape.slopes + h) * kLog2e;
      }
    }
  }

  const ScoreShape& sh = p.shape;
  // whether a key of the sequence can be hidden from a query (one query sees all that come before it)
  const bool partial = (p.causal && m > 1) || sh.window > 0;
  int c = 0;
  // test hook: a wait that runs out, with the first copies on their way
  bool stalled = false;
  if (p.debug_stall) {
    if (lane == 0) stalled = !sm100::mbar_wait(bars + 8 * kStages, 0, abort, p.status, p.wait_ns);
    stalled = __any_sync(0xffffffffu, stalled);
  }
  for (; c < mine && !stalled; ++c) {
    const int kt = first_key(c), key = kt + g + 8 * (lane & 1);   // (what lanes 0 and 1 of a quad write)
    float w_in = 0.f;
    if (p.w_in && (lane & 3) < 2 && key < end) w_in = __ldg(p.w_in + w_row + key);
    const uint32_t st = (uint32_t)c % kStages;
    bool ok = true;
    if (lane == 0) ok = sm100::mbar_wait(bars + 8 * st, (c / kStages) & 1, abort, p.status, p.wait_ns);
    if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
    sm100::mbar_try_wait(bars + 8 * st, (c / kStages) & 1);  // completed: this lane's own acquire
    const uint32_t kb = ring + st * Lay::kStage + ((lane & 7) + ((lane >> 3) & 1) * 8) * 128;
    float s[NT][4] = {};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t ka[4];
      ldsm4(kb + (kk >> 2) * kChunk * 128 + (((((kk & 3) * 2) + (lane >> 4)) ^ (lane & 7)) << 4), ka);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma(s[nt], ka, qb[nt][kk][0], qb[nt][kk][1]);
    }
    __syncwarp();   // the stage is read: it may take the chunk kStages on
    if (c + kStages < mine) issue(c + kStages, next);
    next = find(c + kStages + 1);
    if (sh.cap > 0.f) cap_in_place(sh, *reinterpret_cast<float(*)[NT * 4]>(&s[0][0]));
    float acc[2] = {0.f, 0.f};   // keys kt + g and kt + g + 8
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int dist = pos[nt][e] - (kt + g + hf * 8);
          const float x = s[nt][hf * 2 + e];
          float y;
          if (sh.cap > 0.f)
            y = x + nl[nt][e];
          else
            y = fmaf(x, sh.sl2, nl[nt][e]);
          if (sh.slopes) y = fmaf(slope[nt][e], fabsf((float)dist), y);
          if (partial && ((p.causal && dist < 0) || (sh.window > 0 && abs(dist) >= sh.window))) y = -CUDART_INF_F;
          acc[hf] += ex2(y);
        }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {   // the four lanes of a key hold different rows
      acc[hf] += __shfl_xor_sync(0xffffffffu, acc[hf], 1);
      acc[hf] += __shfl_xor_sync(0xffffffffu, acc[hf], 2);
    }
    if ((lane & 3) < 2 && key < end) {
      const float sum = (have >> (c & 31)) & 1u ? acc[lane & 1] : 0.f;
      p.w_out[w_row + key] = p.w_in ? fmaf(p.decay, w_in, sum) : sum;
    }
  }
  // after a wait that ran out: no copy may land once the block is gone
  for (int d = c; d < min(c + kStages, mine); ++d) {
    const uint64_t t0 = sm100::globaltimer_ns();
    while (!sm100::mbar_try_wait(bars + 8 * (d % kStages), (d / kStages) & 1))
      if (sm100::globaltimer_ns() - t0 > kDrainLimitNs) break;
  }
}

template <int D, int NT>
cudaError_t launch_stream(const KeyWeightsParams& p, const CUtensorMap& tk, int num_sms, cudaStream_t stream) {
  auto kern = stream_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, StreamLayout<D>::kBytes);
  if (e != cudaSuccess) return e;
  // two rounds of blocks if every table were full: a block's start (lengths, table, first copies) is paid
  // seldom, and ragged lengths still spread (8 contexts of 7k to 16k tokens, 8 KV heads: 43.7 us with one round,
  // 45.7 with two; 16 of 3000 tokens, 31.2 and 27.3)
  const long long keys = (long long)p.max_pages * p.page_size;
  const long long share = (keys * p.B * p.Hkv + (long long)num_sms * kBlocksPerSm - 1) / ((long long)num_sms * kBlocksPerSm);
  const int segment = (int)((share < keys ? (share + 1) / 2 : keys) + kWarps * kChunk - 1) / (kWarps * kChunk) * (kWarps * kChunk);
  const dim3 grid((unsigned)((keys + segment - 1) / segment * p.Hkv), p.B);
  kern<<<grid, kWarps * 32, StreamLayout<D>::kBytes, stream>>>(tk, p, segment);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_kw(const KeyWeightsParams& p, cudaStream_t stream) {
  auto kern = key_weights_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, KwLayout<D>::kBytes);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.max_pages * p.page_size + kKeys - 1) / kKeys * p.Hkv, p.B);
  kern<<<grid, kWarps * 32, KwLayout<D>::kBytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsParams& p, cudaStream_t stream) {
  return p.d == 128 ? launch_kw<128>(p, stream) : launch_kw<64>(p, stream);
}

cudaError_t launch_key_weights_stream(const KeyWeightsParams& p, const CUtensorMap& tk, int max_rows, int num_sms,
                                      cudaStream_t stream) {
  if (max_rows <= 8)
    return p.d == 128 ? launch_stream<128, 1>(p, tk, num_sms, stream) : launch_stream<64, 1>(p, tk, num_sms, stream);
  if (max_rows <= 16)
    return p.d == 128 ? launch_stream<128, 2>(p, tk, num_sms, stream) : launch_stream<64, 2>(p, tk, num_sms, stream);
  return p.d == 128 ? launch_stream<128, 4>(p, tk, num_sms, stream) : launch_stream<64, 4>(p, tk, num_sms, stream);
}

}  // namespace fattn
