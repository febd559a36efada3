// Tensor-core attention backward for sm_103a ("The backward pass recomputes
// instead of reading", FlashAttention explained): P is rebuilt tile by tile
// from the saved logsumexp, never read from HBM, and
//   D = rowsum(dO o O),  dV += P^T dO,  dP = dO V^T,  dS = P o (dP - D),
//   dQ += scale dS K,    dK += scale dS^T Q     (S = scale Q K^T).
//
// Two launches on the caller's stream, in this order:
//   bwd_dq_kernel<d>       items (sequence, query head, 128-query tile i); an
//                          item walks the key tiles j (causal: j <= i):
//                            S = Q K_j^T, dP = dO V_j^T, dS (bf16, in two
//                            TMEM buffers of its own), dQ += dS K_j.
//                          Its otherwise idle warps 2-3 form D and
//                          -lse * log2(e) of each item's rows ahead of the
//                          element-wise warps, into a workspace padded to whole
//                          128-row tiles (pad: D = 0, -lse log2(e) = -inf, so
//                          padded rows get P = 0); then
//                          P = 2^(S log2(e) scale - lse log2(e)) is one FMA and
//                          one exponential per element. An item's dQ is written
//                          after the next item's first key tile, while that
//                          item's next S and dP run.
//   bwd_dkdv_kernel<d>     one CTA per SM over items (sequence, KV head, 128-key
//                          tile j); an item walks the query tiles i of every
//                          query head sharing the KV head (causal: i >= j) and
//                          accumulates dV and dK in TMEM:
//                            S^T = K Q_i^T, dP^T = V dO_i^T (TMEM, fp32),
//                            P^T (bf16, over S^T), dV += P^T dO_i,
//                            dS^T (bf16, over dP^T), dK += dS^T Q_i;
//                          the next S^T follows dV when its Q/dO stage has
//                          landed (it overwrites only P^T, which dV reads); it
//                          reads the two workspace vectors of every query tile.
//                          dV is written while the item's last dK product
//                          runs, then dK (d = 128: staged in shared memory and
//                          stored by TMA, 32 rows x 64 columns per warp).
// In both passes an item's resident tiles (K_j, V_j; Q_i, dO_i) are released as
// soon as the last product that reads them completes, so the next item's load
// overlaps the item's last products.
// dQ is computed in its own pass (recomputing S and dP) instead of being
// accumulated with atomics from the dK/dV pass: at d = 128 the dK/dV pass
// already uses all 512 TMEM columns (S^T, dP^T, dV, dK).
//
// Roles (384 threads): warp 0 TMA producer, warp 1 MMA issuer (one thread), in
// the dQ pass warps 2-3 the per-row vectors, warps 4-7 and 8-11 the element-wise work: a thread owns one TMEM lane (tile
// row), warpgroup g columns [64 g, 64 g + 64) of it. In the dK/dV pass each
// warpgroup packs its bf16 P^T or dS^T into the first 32 columns of its own 64,
// so the two never touch each other's columns and the MMA reads its TMEM
// operand from the two halves; the dQ pass writes dS to columns 384-511.
// Shaped variants (fattn_ops.h): P is rebuilt from the shaped score and dS gets the
// cap's derivative; the dQ pass walks the key tiles of its rows' ranges, the dK/dV pass the
// query tiles that see its keys (ranges turned over by the dQ pass's warp 3), per KV head or
// per query head (bwd_per_head). Bound by the element-wise warps: the cap's polynomial and
// derivative are ten packed operations a pair of scores. Packed documents of 540 to 1260 rows,
// B=4 H=32 N=4096 d=128: 677 us, capped 954 (the whole triangle 1595 and 2255; plain 1606); with scores that
// now and then pass 0.6 of the cap (four of their deviations) 1105. P and dS are rounded to bf16, the type of the other
// operand of their products (0.0024 off in relative norm; the rounding of the results alone 0.0017).
// Every pipeline wait is bounded as in the forward kernel: a wait past its
// limit records FATTN_ERR_TIMEOUT, every role stops, copies and MMAs are
// drained and TMEM is freed.
#include "device_common.cuh"
#include "fattn_internal.h"
#include "score_shape.cuh"
#include "sm100_primitives.cuh"

#include <math_constants.h>

#include <algorithm>
#include <type_traits>

namespace fattn {
namespace {

using namespace sm100;

constexpr int BT = 128;          // rows of every tile (query rows or keys)
constexpr int kThreads = 384;   // warps 0-3 control, 4-7 and 8-11 element-wise
constexpr int kEwArrivals = 8;  // element-wise warps arriving on a barrier
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kDrainLimitNs = 200000000ull;
// TMEM columns (both passes): S or S^T at 0 (P / P^T in bf16 over its first 64
// columns), dP or dP^T at 128 (dS in bf16 over its first 64), accumulators at 256.
constexpr uint32_t kColS = 0, kColDP = 128, kColAcc = 256;

__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
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

// ------------------------------------------------------------------ per-row vectors
// One warp forms D = rowsum(dO o O) and -lse * log2(e) for 32 consecutive query rows
// i0 .. i0 + 31 of one (sequence, head) and writes both into the workspace: lane u
// reads row u's lse (one 128-byte read per warp), the warp walks the 32 rows of O and
// dO (each a contiguous d-long row; kRowsPerWarp rows with their loads in flight
// together, each lane d / 32 elements of both), reduces each row's dot product with
// shuffles and keeps row u's in lane u, and writes the two vectors with one 128-byte
// store each. Rows past N (the padding up to Npad) get -inf and 0, so their P is 0.
constexpr int kRowsPerWarp = 8;

template <int D>
__device__ __forceinline__ void row_vectors(const BwdParams& p, int b, int h, int i0, int lane) {
  constexpr int E = D / 32;  // elements per lane: 4 (8 bytes) or 2 (4 bytes)
  using Vec = typename std::conditional<E == 4, uint2, uint32_t>::type;
  const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(p.o);
  const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(p.dout);
  const int bh = b * p.Hq + h;
  const int i = i0 + lane;                        // this lane's row of the block
  const float lse = i < p.N ? __ldg(p.lse + (size_t)bh * p.N + i) : -CUDART_INF_F;
  const int nrows = min(32, p.N - i0);            // rows of the block inside the sequence (may be <= 0)
  float mine = 0.f;
  for (int u0 = 0; u0 < nrows; u0 += kRowsPerWarp) {
    Vec a[kRowsPerWarp], d[kRowsPerWarp];
#pragma unroll
    for (int u = 0; u < kRowsPerWarp; ++u) {
      if (u0 + u < nrows) {
        const size_t off = (((size_t)b * p.N + i0 + u0 + u) * p.Hq + h) * D + lane * E;
        a[u] = __ldg(reinterpret_cast<const Vec*>(o + off));
        d[u] = __ldg(reinterpret_cast<const Vec*>(g + off));
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsPerWarp; ++u) {
      if (u0 + u >= nrows) break;
      const uint32_t* aw = reinterpret_cast<const uint32_t*>(&a[u]);
      const uint32_t* dw = reinterpret_cast<const uint32_t*>(&d[u]);
      float dsum = 0.f;
#pragma unroll
      for (int w = 0; w < E / 2; ++w) {
        dsum = fmaf(bf16_lo(aw[w]), bf16_lo(dw[w]), dsum);
        dsum = fmaf(bf16_hi(aw[w]), bf16_hi(dw[w]), dsum);
      }
#pragma unroll
      for (int sft = 16; sft > 0; sft >>= 1) dsum += __shfl_xor_sync(0xffffffffu, dsum, sft);
      if (lane == u0 + u) mine = dsum;
    }
  }
  // a row with no visible key (lse = -inf), and a padding row, get P = 0
  p.ws_nl2[(size_t)bh * p.Npad + i] = (lse > -CUDART_INF_F && lse < CUDART_INF_F) ? -lse * kLog2e : -CUDART_INF_F;
  p.ws_d[(size_t)bh * p.Npad + i] = i < p.N ? mine : 0.f;
}

// The same for the shaped passes, whose items may be short (a document's few key tiles leave the two
// warps 15k cycles for their 128 rows, where 8 rows at a time with five shuffles each took 20k): 16-byte
// loads, D / 8 lanes a row, half of the 32 rows on their way together, and the lanes' partial sums of all
// rows reduced by exchanging halves (D / 8 - 1 shuffles for D / 8 sums).
template <int D>
__device__ __forceinline__ void row_vectors_wide(const BwdParams& p, int b, int h, int i0, int lane) {
  constexpr int L = D / 8, R = 32 / L;            // lanes per row, rows per load; L loads cover the block
  const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(p.o);
  const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(p.dout);
  const int bh = b * p.Hq + h;
  const int mine = i0 + (lane % L) * R + lane / L;  // the row whose sum this lane ends with
  const float lse = mine < p.N ? __ldg(p.lse + (size_t)bh * p.N + mine) : -CUDART_INF_F;
  float sum[L];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint4 a[L / 2], d[L / 2];
#pragma unroll
    for (int t = 0; t < L / 2; ++t) {
      const int i = i0 + (half * (L / 2) + t) * R + lane / L;
      a[t] = d[t] = make_uint4(0, 0, 0, 0);
      if (i < p.N) {
        const size_t off = (((size_t)b * p.N + i) * p.Hq + h) * D + (lane % L) * 8;
        a[t] = __ldg(reinterpret_cast<const uint4*>(o + off));
        d[t] = __ldg(reinterpret_cast<const uint4*>(g + off));
      }
    }
#pragma unroll
    for (int t = 0; t < L / 2; ++t) {
      float s0 = bf16_lo(a[t].x) * bf16_lo(d[t].x), s1 = bf16_hi(a[t].x) * bf16_hi(d[t].x);
      s0 = fmaf(bf16_lo(a[t].y), bf16_lo(d[t].y), s0);
      s1 = fmaf(bf16_hi(a[t].y), bf16_hi(d[t].y), s1);
      s0 = fmaf(bf16_lo(a[t].z), bf16_lo(d[t].z), s0);
      s1 = fmaf(bf16_hi(a[t].z), bf16_hi(d[t].z), s1);
      s0 = fmaf(bf16_lo(a[t].w), bf16_lo(d[t].w), s0);
      s1 = fmaf(bf16_hi(a[t].w), bf16_hi(d[t].w), s1);
      sum[half * (L / 2) + t] = s0 + s1;
    }
  }
#pragma unroll
  for (int step = L / 2; step > 0; step /= 2) {   // lanes with bit `step` keep the upper half of the sums
    const bool up = lane & step;
#pragma unroll
    for (int t = 0; t < step; ++t) {
      const float keep = up ? sum[t + step] : sum[t], send = up ? sum[t] : sum[t + step];
      sum[t] = keep + __shfl_xor_sync(0xffffffffu, send, step);
    }
  }
  p.ws_nl2[(size_t)bh * p.Npad + mine] = (lse > -CUDART_INF_F && lse < CUDART_INF_F) ? -lse * kLog2e : -CUDART_INF_F;
  p.ws_d[(size_t)bh * p.Npad + mine] = mine < p.N ? sum[0] : 0.f;
}

// Bounded wait until a shared-memory counter reaches `target` (abort and time limit as
// in the mbarrier waits).
__device__ __forceinline__ bool count_wait(volatile int* c, int target, volatile int* abort, int* status,
                                           uint64_t limit_ns) {
  if (*c >= target) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    __nanosleep(256);
    if (*c >= target) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      record_status(status, 5 /* timeout */);
      *abort = 1;
      return false;
    }
  }
}

// ------------------------------------------------------------------ work order
// Items (head, tile) are taken in groups of heads whose items fill about four
// rounds of the grid (measured on the causal MHA workload, B=4 H=32 N=4096: 1.74 ms
// for the whole backward call against 1.96 with two rounds, 1.86 with one, 1.81 with
// three or five, 1.84 with six, 1.75 with eight; on the 32k-token GQA one 23.9 against
// 24.0 ms); inside a group the items go heaviest tile first (all heads
// of the group at one tile index, then the next), and the grid walks the list in
// alternating direction round by round ("snake"), so the tiles the CTAs stream
// (Q and dO in the dK/dV pass, K and V in the dQ pass) belong to a few heads at
// a time and are shared through L2. `unit` keeps GQA groups whole.
struct BwdSchedule {
  int tiles, heads, group, total;
};
__device__ __forceinline__ BwdSchedule make_bwd_schedule(int heads, int tiles, int unit) {
  BwdSchedule s;
  s.tiles = tiles;
  s.heads = heads;
  int grp = (4 * (int)gridDim.x + tiles - 1) / tiles;
  grp = ((grp + unit - 1) / unit) * unit;
  s.group = grp < heads ? grp : heads;
  s.total = heads * tiles;
  return s;
}
__device__ __forceinline__ int bwd_item_index(const BwdSchedule& s, int k) {
  const int G = (int)gridDim.x;
  const int idx = k * G + ((k & 1) ? (G - 1 - (int)blockIdx.x) : (int)blockIdx.x);
  return idx < s.total ? idx : -1;
}
// head and rank (0 = heaviest) of item it
__device__ __forceinline__ void bwd_decode(const BwdSchedule& s, int it, int& head, int& rank) {
  const int per_group = s.group * s.tiles;
  const int g = it / per_group;
  const int rem = it - g * per_group;
  const int gh = min(s.group, s.heads - g * s.group);
  rank = rem / gh;
  head = g * s.group + (rem - rank * gh);
}

// ------------------------------------------------------------------ shared helpers
template <int D>
struct BwdTiles {
  static constexpr int kTile = BT * D * 2;   // one 128-row bf16 tile (D / 64 swizzled 64-column halves)
  static constexpr int kAtom = BT * 128 / 16;  // 16-byte units between the 64-column halves
};

// K-major x K-major product D[tmem] = A B^T over the head dimension (128 x 128 x D).
template <int D>
__device__ __forceinline__ void issue_kk(uint32_t d_tmem, uint64_t a0, uint64_t b0) {
  constexpr uint32_t id = idesc_bf16_f32(BT, BT, 0);
  mma_ss_c<false>(d_tmem, a0, b0, id);
#pragma unroll
  for (int ks = 1; ks < D / 16; ++ks) {
    const uint64_t o = (uint64_t)((ks >> 2) * BwdTiles<D>::kAtom + (ks & 3) * 2);
    mma_ss_c<true>(d_tmem, a0 + o, b0 + o, id);
  }
}
// D[tmem] (+)= A[tmem] B over 128 rows of B (B MN-major: the head dimension contiguous);
// A (bf16) in the two warpgroups' packed halves, columns [0, 32) and [64, 96).
template <int D>
__device__ __forceinline__ void issue_tn(uint32_t d_tmem, uint32_t a_tmem, uint64_t b0, bool acc) {
  constexpr uint32_t id = idesc_bf16_f32(BT, D, 1);
  mma_ts(d_tmem, a_tmem, b0, id, acc ? 1u : 0u);
#pragma unroll
  for (int ks = 1; ks < BT / 16; ++ks)  // keys 64 g + 16 k' live at column 64 g + 8 k'
    mma_ts_acc(d_tmem, a_tmem + (ks >> 2) * 64 + (ks & 3) * 8, b0 + (uint64_t)(ks * 16 * 128 / 16), id);
}

// The same product with A packed contiguously: keys 16 k live at columns [8 k, 8 k + 8).
template <int D>
__device__ __forceinline__ void issue_tn_packed(uint32_t d_tmem, uint32_t a_tmem, uint64_t b0, bool acc) {
  constexpr uint32_t id = idesc_bf16_f32(BT, D, 1);
  mma_ts(d_tmem, a_tmem, b0, id, acc ? 1u : 0u);
#pragma unroll
  for (int ks = 1; ks < BT / 16; ++ks)
    mma_ts_acc(d_tmem, a_tmem + ks * 8, b0 + (uint64_t)(ks * 16 * 128 / 16), id);
}

// Load 128-row tile (rows r0.., head h) of a [rows, H, D] tensor map into dst.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int h, int r0,
                                          uint64_t pol) {
#pragma unroll
  for (int dc = 0; dc < D / 64; ++dc) tma_load_3d(dst + dc * BT * 128, map, bar, dc * 64, h, r0, pol);
}

// Write one accumulator row (D fp32 TMEM columns) times `mul` as bf16.
template <int D>
__device__ __forceinline__ void store_row(uint32_t t_col, float mul, __nv_bfloat16* dst, bool live) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t u[32];
    tmem_ld32(t_col + 32 * c, u);
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(__uint_as_float(u[2 * e]) * mul, __uint_as_float(u[2 * e + 1]) * mul);
    if (live) {
      uint4* q = reinterpret_cast<uint4*>(dst + 32 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
    }
  }
}

// The same in fp32.
template <int D>
__device__ __forceinline__ void store_row_f32(uint32_t t_col, float mul, float* dst, bool live) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t u[32];
    tmem_ld32(t_col + 32 * c, u);
    if (live) {
      float4* q = reinterpret_cast<float4*>(dst + 32 * c);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        q[e] = make_float4(__uint_as_float(u[4 * e]) * mul, __uint_as_float(u[4 * e + 1]) * mul,
                           __uint_as_float(u[4 * e + 2]) * mul, __uint_as_float(u[4 * e + 3]) * mul);
    }
  }
}

// dS = P o (dP - Dvec) over this warpgroup's 64 columns (pv[c] is column
// 64 g + c), written as bf16 over the first 32 of them, 32 columns at a time:
// pass q reads dP columns [32q, 32q + 32) and then writes packed columns
// [16q, 16q + 16), all of which the same or an earlier pass has already read.
template <bool kVecD>
__device__ __forceinline__ void write_ds(uint32_t dp_col, const float (&pv)[64], const float* dvec, float dval) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t a[32];
    tmem_ld32(dp_col + 32 * q, a);
    float dd[32];
    if (kVecD) {  // D of each column (shared memory, 16-byte aligned)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 v = reinterpret_cast<const float4*>(dvec + 32 * q)[e];
        dd[4 * e] = v.x;
        dd[4 * e + 1] = v.y;
        dd[4 * e + 2] = v.z;
        dd[4 * e + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) dd[e] = dval;
    }
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int c = 32 * q + 2 * e;
      w[e] = pack_bf16x2(pv[c] * (__uint_as_float(a[2 * e]) - dd[2 * e]),
                         pv[c + 1] * (__uint_as_float(a[2 * e + 1]) - dd[2 * e + 1]));
    }
    tmem_st16(dp_col + 16 * q, w);
  }
}

// ------------------------------------------------------------------ shaped scores
// Variants of both kernels: kPlain, or what the shaped scores get (key ranges and the window always).
// kShapeFar: a cap above 128, under which cap (1 - 2 r), off by 2^-22 of the cap, is not as good as the fp32 sum of
// a small product next to a large one. (A kernel of its own: under a run-time switch the others lose 2 to 3 %.)
enum : int { kPlain = -1, kShapeCap = 1, kShapeBias = 2, kShapeFar = 4 };
// Key tiles [top - n, top) that the rows of query tile i see, n >= 1: a tile whose rows see no
// key visits one tile with everything masked (its dQ is the zero that this gives).
__device__ __forceinline__ void shaped_key_tiles(const BwdParams& p, int b, int i, int nt, int& top, int& n) {
  const int first = i * BT, last = min(first + BT, p.N) - 1;
  const int lo = shape_lo(p.shape, (long long)b * p.N + first, first);
  const int hi = shape_hi(p.shape, (long long)b * p.N + last, last, p.N, p.causal);
  const int t0 = min(lo / BT, nt - 1);
  top = lo < hi ? (hi + BT - 1) / BT : t0 + 1;
  n = max(top - t0, 1);
}
// The ranges seen from the keys: the queries that see key j are [qa_j, qb_j), as the bounds are
// monotone: qa_j the first row whose end is above j, qb_j the first whose begin is. The dQ pass's
// warps 2-3 write them for the dK/dV pass, 32 rows a warp at a time: row i is qa of the keys
// [end_{i-1}, end_i) and qb of the keys [begin_{i-1}, begin_i), row N that of the rest, and the
// whole warp writes each row's keys. (Searching them per key and item in the dK/dV pass took 2 to 3 us
// at the start of every item: packed documents, B=4 H=32 N=4096, 966 us for the whole call.)
__device__ __forceinline__ void write_key_ranges(const BwdParams& p, int worker, int workers, int lane) {
  const int blocks = (p.N + 1 + 31) / 32;  // rows 0 .. N of a sequence
  for (int w = worker; w < p.B * blocks; w += workers) {
    const int b = w / blocks, i = (w - b * blocks) * 32 + lane;
    const long long row0 = (long long)b * p.N;
    auto begin = [&](int r) { return r < 0 ? 0 : r >= p.N ? p.Npad : min(shape_lo(p.shape, row0 + r, r), p.N); };
    auto end = [&](int r) {
      return r < 0 ? 0 : r >= p.N ? p.Npad : shape_hi(p.shape, row0 + r, r, p.N, p.causal);
    };
    int a0 = 0, a1 = 0, b0 = 0, b1 = 0;      // this lane's keys: qa = i for [a0, a1), qb = i for [b0, b1)
    if (i <= p.N) {
      a0 = end(i - 1);
      a1 = end(i);
      b0 = begin(i - 1);
      b1 = begin(i);
      // ranges that decrease cannot be turned over: the gradients of the keys concerned would be wrong
      if (a0 > a1 || b0 > b1) record_status(p.status, kStatusDeviceCheck);
    }
    int2* out = p.ws_keys + (size_t)b * p.Npad;
    for (int l = 0; l < 32; ++l) {
      const int r = (w - b * blocks) * 32 + l;
      const int x0 = __shfl_sync(0xffffffffu, a0, l), x1 = __shfl_sync(0xffffffffu, a1, l);
      const int y0 = __shfl_sync(0xffffffffu, b0, l), y1 = __shfl_sync(0xffffffffu, b1, l);
      for (int k = x0 + lane; k < x1; k += 32) out[k].x = r;
      for (int k = y0 + lane; k < y1; k += 32) out[k].y = r;
    }
  }
}
// Query tiles [i0, i0 + n) that see a key of key tile j, n >= 1 (a key tile that no row sees
// visits one with everything masked: its dK and dV are the zeros that this gives).
__device__ __forceinline__ void shaped_query_tiles(const BwdParams& p, int b, int j, int nt, int& i0, int& n) {
  const int2* keys = p.ws_keys + (size_t)b * p.Npad;
  const int first = __ldg(&keys[j * BT].x), last = __ldg(&keys[min((j + 1) * BT, p.N) - 1].y);
  // (clamped, so that even a workspace the dQ pass did not finish keeps the tiles inside the sequence)
  i0 = max(min(first / BT, nt - 1), 0);
  n = max(min(last / BT + (last % BT != 0), nt) - i0, 1);
}

// One thread's 32 columns of raw products u: pv = P o f with P = 2^(score + nl) and f the factor that
// the cap puts on dS (1 - tanh^2), and P itself as bf16 pairs into pk (kPack). Column c lies at
// distance |dist + step c| and is visible iff va <= c < vb; nl is its row's -lse log2(e), per column
// (kCols, nlv) or one for all.
template <int kShape, bool kCols, bool kPack>
__device__ __forceinline__ void shaped_p32(const BwdParams& p, float slope2, uint32_t (&u)[32], float dist, float step,
                                           int va, int vb, const float* nlv, float nl, float* pv, uint32_t* pk) {
  const ScoreShape& sh = p.shape;
  const bool edge = !__all_sync(0xffffffffu, va <= 0 && vb >= 32);
  const uint32_t vis = vb <= 0 || va >= 32 || va >= vb
                           ? 0u
                           : (0xffffffffu << max(va, 0)) & (0xffffffffu >> (32 - min(vb, 32)));
  constexpr bool cap = kShape & kShapeCap, bias = kShape & kShapeBias;
  float y[32], f[32];
  if constexpr (cap) {
    if (edge) {  // hidden keys must not decide between the two forms of the cap
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (!((vis >> c) & 1u)) u[c] = 0u;
    }
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = fmax3(fabsf(__uint_as_float(u[i])), fabsf(__uint_as_float(u[i + 4])), fabsf(__uint_as_float(u[i + 8])));
#pragma unroll
    for (int c = 12; c < 28; c += 8)
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = fmax3(a[i], fabsf(__uint_as_float(u[c + i])), fabsf(__uint_as_float(u[c + 4 + i])));
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = fmaxf(a[i], fabsf(__uint_as_float(u[28 + i])));
    const float amax = fmax3(fmaxf(a[0], a[1]), a[2], a[3]);
    if (amax <= sh.poly_limit) {  // by row of the tile; the cap as a polynomial (fattn_internal.h)
      const uint64_t c0 = f2_bits(sh.poly[0]), c1 = f2_bits(sh.poly[1]),
                     c2 = f2_bits(sh.poly[2]), c3 = f2_bits(sh.poly[3]),
                     c4 = f2_bits(sh.poly[4]), one = f2_pack(1.f, 1.f), nic2 = f2_pack(sh.nicap2, sh.nicap2);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const uint64_t x = f2_pack(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), v = f2_mul(x, x);
        const uint64_t t = f2_mul(x, f2_fma(f2_fma(f2_fma(f2_fma(c4, v, c3), v, c2), v, c1), v, c0));
        f2_unpack(t, y[c], y[c + 1]);
        f2_unpack(f2_fma(f2_mul(t, t), nic2, one), f[c], f[c + 1]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float z = __uint_as_float(u[c]) * sh.capk, r = tanh_r(fabsf(z));  // r <= 1/2: 4 r (1 - r) keeps its digits
        y[c] = copysignf(fmaf(-2.f * sh.cap2, r, sh.cap2), z);
        f[c] = 4.f * r * (1.f - r);
      }
      if constexpr (kShape & kShapeFar) {  // products in the polynomial's range keep it
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float y0, y1;
          f2_unpack(capped_pair(sh, __uint_as_float(u[c]), __uint_as_float(u[c + 1])), y0, y1);
          if (fabsf(__uint_as_float(u[c])) <= sh.poly_limit) y[c] = y0;
          if (fabsf(__uint_as_float(u[c + 1])) <= sh.poly_limit) y[c + 1] = y1;
        }
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < 32; ++c) y[c] = __uint_as_float(u[c]);
  }
  // y (times the scale without a cap) + bias + nl
  const uint64_t mul = f2_pack(sh.sl2, sh.sl2);
#pragma unroll
  for (int c4 = 0; c4 < 32; c4 += 4) {
    float4 l = kCols ? *reinterpret_cast<const float4*>(nlv + c4) : make_float4(nl, nl, nl, nl);
    if constexpr (bias) {
      l.x = fmaf(slope2, fabsf(fmaf(step, (float)c4, dist)), l.x);
      l.y = fmaf(slope2, fabsf(fmaf(step, (float)(c4 + 1), dist)), l.y);
      l.z = fmaf(slope2, fabsf(fmaf(step, (float)(c4 + 2), dist)), l.z);
      l.w = fmaf(slope2, fabsf(fmaf(step, (float)(c4 + 3), dist)), l.w);
    }
    const uint64_t y0 = f2_pack(y[c4], y[c4 + 1]), y1 = f2_pack(y[c4 + 2], y[c4 + 3]);
    const uint64_t l0 = f2_pack(l.x, l.y), l1 = f2_pack(l.z, l.w);
    f2_unpack(cap ? f2_add(y0, l0) : f2_fma(y0, mul, l0), y[c4], y[c4 + 1]);
    f2_unpack(cap ? f2_add(y1, l1) : f2_fma(y1, mul, l1), y[c4 + 2], y[c4 + 3]);
  }
  if (edge) {
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!((vis >> c) & 1u)) y[c] = -CUDART_INF_F;
  }
#pragma unroll
  for (int c = 0; c < 32; ++c) pv[c] = ex2(y[c]);
  if constexpr (kPack) {
#pragma unroll
    for (int c = 0; c < 32; c += 2) pk[c / 2] = pack_bf16x2(pv[c], pv[c + 1]);
  }
  if constexpr (cap) {
#pragma unroll
    for (int c = 0; c < 32; c += 2)
      f2_unpack(f2_mul(f2_pack(pv[c], pv[c + 1]), f2_pack(f[c], f[c + 1])), pv[c], pv[c + 1]);
  }
}

// 64 consecutive fp32 TMEM columns of this lane.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  uint32_t (&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(&r[0]);
  uint32_t (&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(&r[32]);
  tmem_ld32(taddr, lo);
  tmem_ld32(taddr + 32, hi);
}

// ------------------------------------------------------------------ dK, dV pass
template <int D>
struct DkdvLayout {
  static constexpr int kTile = BwdTiles<D>::kTile;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kTile;
  static constexpr int kOffRing = 2 * kTile;      // stage s: Q_i, dO_i, -lse log2(e) [128], D[128]
  static constexpr int kStage = 2 * kTile + 1024;
  static constexpr int kStages = 2;
  // d = 128: each element-wise warp stages 32 rows x 64 columns of dV, then of dK (bf16,
  // 128-byte swizzle) in a 4 KB slot of its own and stores them with one TMA box each
  static constexpr bool kStoreTma = D == 128;
  static constexpr int kOutSlot = 32 * 128;
  static constexpr int kOffOut = kOffRing + kStages * kStage;
  static constexpr int kEnd = kOffOut + (kStoreTma ? 8 * kOutSlot : 0);
  // barriers, the TMEM address and the abort flag (8-byte words) sit in whichever end of
  // the 1 KB alignment slack has room for them: before the aligned base if the slack
  // there is at least kSmallBytes, else after kEnd (where 1 KB minus that slack remains)
  static constexpr int kNumBars = 14;
  static constexpr int kBarStall = kNumBars;      // test hook: a barrier no role arrives on
  static constexpr int kOffHolder = (kNumBars + 1) * 8;  // from the start of the small words
  static constexpr int kOffAbort = kOffHolder + 8;
  static constexpr int kSmallBytes = kOffAbort + 8;
  static_assert(2 * kSmallBytes <= 1024, "small words in the slack");
  // + slack to align the base to 1024 B; at least 117 KB so that a second CTA
  // (which would wait in tcgen05.alloc for all 512 columns) never shares the SM
  static constexpr int kUsed = kEnd + 1024;
  static constexpr int kBytes = kUsed > 117 * 1024 ? kUsed : 117 * 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};
enum : int {
  kKvFull = 0, kKvEmpty = 1, kQdFull = 2, kQdEmpty = 4, kSFull = 6, kDpFull = 7, kPFull = 8, kDsFull = 9,
  kAccFull = 10, kAccEmpty = 11, kMmaDone = 12, kDvFull = 13
};

// kPerHead (shaped only): an item is a query head's share of dK and dV, written in fp32 to p.ws_part for
// sum_heads_kernel to add over the group; else the group's heads follow one another in an item.
template <int D, int kShape, bool kPerHead>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_dkdv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                    const __grid_constant__ CUtensorMap tdk, const __grid_constant__ CUtensorMap tdv,
                    const BwdParams p) {
  using Lay = DkdvLayout<D>;
  constexpr bool kShaped = kShape != kPlain;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  uint8_t* small = smem - smem_raw >= Lay::kSmallBytes ? smem_raw : smem + Lay::kEnd;
  const uint32_t ssb = smem_u32(small);
  auto bar = [&](int i) -> uint32_t { return ssb + 8 * i; };
  volatile int* abort = reinterpret_cast<volatile int*>(small + Lay::kOffAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Lay::kNumBars; ++i)
      mbar_init(bar(i), (i == kPFull || i == kDsFull || i == kAccEmpty) ? kEwArrivals : 1);
    mbar_init(bar(Lay::kBarStall), 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
    tma_prefetch_desc(&tdo);
    if constexpr (Lay::kStoreTma) {
      tma_prefetch_desc(&tdk);
      tma_prefetch_desc(&tdv);
    }
  }
  if (warp == 1) {
    tmem_alloc(ssb + Lay::kOffHolder, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(small + Lay::kOffHolder);

  const int nt = (p.N + BT - 1) / BT;
  const int G = kPerHead ? 1 : p.Hq / p.Hkv;
  const BwdSchedule sch = make_bwd_schedule(p.B * (kPerHead ? p.Hq : p.Hkv), nt, 1);
  // item: (sequence, KV head, or query head with kPerHead, key tile j); rank 0 = j 0, the most query tiles under the causal rule
  auto item = [&](int it, int& b, int& hkv, int& j) {
    int head;
    bwd_decode(sch, it, head, j);
    b = head / (kPerHead ? p.Hq : p.Hkv);
    hkv = head - b * (kPerHead ? p.Hq : p.Hkv);
  };
  // query tiles [i0, i0 + ni) of an item
  auto tiles = [&](int b, int j, int& i0, int& ni) {
    if constexpr (kShaped) {
      shaped_query_tiles(p, b, j, nt, i0, ni);
    } else {
      i0 = p.causal ? j : 0;
      ni = nt - i0;
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t nkv = 0, nqd = 0;
      const uint64_t pol_kv = policy_evict_first(), pol_q = policy_evict_last();
      bool ok = true;
      for (int kk = 0, it; ok && (it = bwd_item_index(sch, kk)) >= 0; ++kk) {
        int b, hkv, j;
        item(it, b, hkv, j);
        if (!mbar_wait(bar(kKvEmpty), (nkv & 1) ^ 1, abort, p.status, p.wait_ns)) break;
        mbar_arrive_expect_tx(bar(kKvFull), 2 * Lay::kTile);
        const int kv_head = kPerHead ? hkv / (p.Hq / p.Hkv) : hkv;
        load_tile<D>(sb + Lay::kOffK, &tk, bar(kKvFull), kv_head, b * p.N + j * BT, pol_kv);
        load_tile<D>(sb + Lay::kOffV, &tv, bar(kKvFull), kv_head, b * p.N + j * BT, pol_kv);
        ++nkv;
        int i0, ni;
        tiles(b, j, i0, ni);
        for (int t = 0; t < G * ni; ++t) {
          const int h = hkv * G + t / ni, i = i0 + t % ni;
          const uint32_t st = nqd & 1, base = sb + Lay::kOffRing + st * Lay::kStage;
          if (!mbar_wait(bar(kQdEmpty + st), ((nqd >> 1) & 1) ^ 1, abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(kQdFull + st), 2 * Lay::kTile + 1024);
          load_tile<D>(base, &tq, bar(kQdFull + st), h, b * p.N + i * BT, pol_q);
          load_tile<D>(base + Lay::kTile, &tdo, bar(kQdFull + st), h, b * p.N + i * BT, pol_q);
          const size_t vrow = (size_t)(b * p.Hq + h) * p.Npad + (size_t)i * BT;
          bulk_load(base + 2 * Lay::kTile, p.ws_nl2 + vrow, 512, bar(kQdFull + st));
          bulk_load(base + 2 * Lay::kTile + 512, p.ws_d + vrow, 512, bar(kQdFull + st));
          ++nqd;
        }
      }
      if (nkv) mbar_drain(bar(kKvFull), (nkv - 1) & 1);
      for (uint32_t st = 0; st < 2; ++st) {
        const uint32_t c = (nqd + 1 - st) / 2;
        if (c) mbar_drain(bar(kQdFull + st), (c - 1) & 1);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t nkv = 0, nqd = 0, np = 0, nds = 0, nacc = 0;
      const uint64_t kd = smem_desc_sw128(sb + Lay::kOffK, 16, 1024);
      const uint64_t vd = smem_desc_sw128(sb + Lay::kOffV, 16, 1024);
      const uint32_t tS = tmem + kColS, tDP = tmem + kColDP, tDV = tmem + kColAcc, tDK = tmem + kColAcc + D;
      bool ok = true;
      for (int kk = 0, it; ok && (it = bwd_item_index(sch, kk)) >= 0; ++kk) {
        int b, hkv, j;
        item(it, b, hkv, j);
        int i0, ni;
        tiles(b, j, i0, ni);
        const int steps = G * ni;
        if (!mbar_wait(bar(kKvFull), nkv & 1, abort, p.status, p.wait_ns)) break;
        ++nkv;
        tc_fence_after();
        bool s_issued = false;  // S^T of step t already issued (early, in step t - 1)
        for (int t = 0; t < steps; ++t) {
          const uint32_t st = nqd & 1, base = sb + Lay::kOffRing + st * Lay::kStage;
          const uint64_t dok = smem_desc_sw128(base + Lay::kTile, 16, 1024);
          const uint64_t qmn = smem_desc_sw128(base, BT * 128, 1024);
          const uint64_t domn = smem_desc_sw128(base + Lay::kTile, BT * 128, 1024);
          if (!s_issued) {
            if (!mbar_wait(bar(kQdFull + st), (nqd >> 1) & 1, abort, p.status, p.wait_ns)) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_kk<D>(tS, kd, smem_desc_sw128(base, 16, 1024));  // S^T = K Q^T
            mma_commit(bar(kSFull));
          }
          issue_kk<D>(tDP, vd, dok);  // dP^T = V dO^T (dS^T of the previous step was read by its dK product)
          mma_commit(bar(kDpFull));
          // the item's last product that reads K_j or V_j: the next item's tiles may load
          // as soon as it completes, while this item's last dV and dK run
          if (t + 1 == steps) mma_commit(bar(kKvEmpty));
          if (t == 0 && !mbar_wait(bar(kAccEmpty), (nacc & 1) ^ 1, abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          if (!mbar_wait(bar(kPFull), np & 1, abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          ++np;
          tc_fence_after();
          issue_tn<D>(tDV, tS, domn, t > 0);  // dV += P^T dO
          if (t + 1 == steps) mma_commit(bar(kDvFull));  // the item's dV is complete
          // The next S^T may follow right away if its Q stage has landed: it overwrites
          // P^T, which only the dV product just issued reads (the element-wise warps keep
          // P^T in registers for dS^T), and runs while they compute dS^T. Otherwise it
          // waits until after dK, as the stage may still be loading.
          s_issued = false;
          if (t + 1 < steps) {
            const uint32_t n1 = nqd + 1;
            if (mbar_try_wait(bar(kQdFull + (n1 & 1)), (n1 >> 1) & 1)) {
              tc_fence_after();
              issue_kk<D>(tS, kd, smem_desc_sw128(sb + Lay::kOffRing + (n1 & 1) * Lay::kStage, 16, 1024));
              mma_commit(bar(kSFull));
              s_issued = true;
            }
          }
          if (!mbar_wait(bar(kDsFull), nds & 1, abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          ++nds;
          tc_fence_after();
          issue_tn<D>(tDK, tDP, qmn, t > 0);  // dK += dS^T Q
          mma_commit(bar(kQdEmpty + st));
          ++nqd;
        }
        if (!ok) break;
        if (steps == 0) mma_commit(bar(kKvEmpty));
        mma_commit(bar(kAccFull));
        ++nacc;
      }
      mma_commit(bar(kMmaDone));
      mbar_drain(bar(kMmaDone), 0);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ element-wise (one key row per thread)
    const int q4 = warp & 3, wg = (warp - 4) >> 2;
    const int r = q4 * 32 + lane;                    // key row within the tile
    const int cb = 64 * wg;                          // this warpgroup's query columns
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t s_col = tmem + lane_off + kColS + cb, dp_col = tmem + lane_off + kColDP + cb;
    const uint32_t acc_col = tmem + lane_off + kColAcc;  // dV, then dK at + D
    // this warp's output slot (d = 128): row `lane` at 128 lane, 16-byte chunk c at
    // c ^ (lane mod 8), the 128-byte swizzle of the dK and dV tensor maps
    uint8_t* slot = smem + Lay::kOffOut + (warp - 4) * Lay::kOutSlot;
    const uint32_t slot_s = sb + Lay::kOffOut + (warp - 4) * Lay::kOutSlot;
    // 64 accumulator columns of this thread's row, times mul, in bf16 into the slot, then
    // one TMA store of the warp's 32 x 64 box at (column c0, head h, row row0)
    auto stage_out = [&](uint32_t t_col, float mul, const CUtensorMap* map, int c0, int h, int row0) {
      if (lane == 0) bulk_wait_read_all();  // the slot's previous store has read it
      __syncwarp();
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {
        uint32_t u[32];
        tmem_ld32(t_col + 32 * c2, u);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16x2(__uint_as_float(u[8 * e + 2 * i]) * mul, __uint_as_float(u[8 * e + 2 * i + 1]) * mul);
          const int chunk = 4 * c2 + e;
          *reinterpret_cast<uint4*>(slot + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(map, slot_s, c0, h, row0);
        bulk_commit_group();
      }
    };
    const float sl2 = p.scale * kLog2e;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    uint32_t nqd = 0, ns = 0, ndp = 0, nacc = 0;
    bool ok = true;
    // test hook: a wait that runs out (nothing arrives on the stall barrier), after which
    // every role stops, drains and frees TMEM; the outputs stay unwritten
    if (p.debug_stall && !warp_wait(bar(Lay::kBarStall), 0, abort, p.status, p.wait_ns)) ok = false;
    for (int kk = 0, it; ok && (it = bwd_item_index(sch, kk)) >= 0; ++kk) {
      int b, hkv, j;
      item(it, b, hkv, j);
      int i0, ni;
      tiles(b, j, i0, ni);
      // shaped: the queries [qa, qb) that see this thread's key (none for a key past the sequence)
      int qa = 0, qb = 0;
      if constexpr (kShaped) {
        const int key = j * BT + r;
        if (key < p.N) {
          const int2 q = __ldg(p.ws_keys + (size_t)b * p.Npad + key);
          qa = q.x;
          qb = q.y;
        }
      }
      for (int t = 0; t < G * ni; ++t) {
        const int i = i0 + t % ni;
        const uint32_t st = nqd & 1;
        const float* vec = reinterpret_cast<const float*>(smem + Lay::kOffRing + st * Lay::kStage + 2 * Lay::kTile);
        if (!warp_wait(bar(kSFull), ns & 1, abort, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        ++ns;
        // the stage's vectors arrived with its tiles, which S^T has consumed
        mbar_try_wait(bar(kQdFull + st), (nqd >> 1) & 1);
        tc_fence_after();
        float pv[64];
        if constexpr (kShaped) {
          const float slope2 = (kShape & kShapeBias) ? -__ldg(p.shape.slopes + hkv * G + t / ni) * kLog2e : 0.f;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[16];  // P^T in bf16 over the first 32 of this warpgroup's S^T columns, 16 at a time
            uint32_t u[32];
            tmem_ld32(s_col + 32 * q, u);
            const int i32 = i * BT + cb + 32 * q;  // query of the first column
            shaped_p32<kShape, true, true>(p, slope2, u, (float)(i32 - (j * BT + r)), 1.f, qa - i32, qb - i32,
                                   vec + cb + 32 * q, 0.f, pv + 32 * q, pk);
            tmem_st16(s_col + 16 * q, pk);
          }
        } else {
          uint32_t u[64];
          tmem_ld64(s_col, u);
          const bool diag = p.causal && i == j;       // queries before this key are masked
          const float4* nl = reinterpret_cast<const float4*>(vec + cb);  // -lse log2(e) per query column
#pragma unroll
          for (int c4 = 0; c4 < 16; ++c4) {
            const float4 l = nl[c4];
            float x0, x1, x2, x3;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(u[4 * c4]), __uint_as_float(u[4 * c4 + 1])), sl2x2,
                             f2_pack(l.x, l.y)), x0, x1);
            f2_unpack(f2_fma(f2_pack(__uint_as_float(u[4 * c4 + 2]), __uint_as_float(u[4 * c4 + 3])), sl2x2,
                             f2_pack(l.z, l.w)), x2, x3);
            const int c = 4 * c4;
            pv[c] = (diag && cb + c < r) ? 0.f : ex2(x0);
            pv[c + 1] = (diag && cb + c + 1 < r) ? 0.f : ex2(x1);
            pv[c + 2] = (diag && cb + c + 2 < r) ? 0.f : ex2(x2);
            pv[c + 3] = (diag && cb + c + 3 < r) ? 0.f : ex2(x3);
          }
        }
        if constexpr (!kShaped) {
          uint32_t pk[32];  // P^T in bf16 over the first 32 of this warpgroup's S^T columns
#pragma unroll
          for (int c = 0; c < 32; ++c) pk[c] = pack_bf16x2(pv[2 * c], pv[2 * c + 1]);
          tmem_st32(s_col, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull));
        if (!warp_wait(bar(kDpFull), ndp & 1, abort, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        ++ndp;
        tc_fence_after();
        write_ds<true>(dp_col, pv, vec + BT + cb, 0.f);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kDsFull));
        ++nqd;
      }
      if (!ok) break;
      // epilogue, one key row per thread, warpgroup g columns [g D / 2, (g + 1) D / 2) of it:
      // dV as soon as the item's last dV product has completed (while its last dK product
      // runs), then scale * dK; at d = 128 through the warp's slot and a TMA store when
      // all 32 of the warp's key rows lie in the sequence
      if (!warp_wait(bar(kDvFull), nacc & 1, abort, p.status, p.wait_ns)) break;
      tc_fence_after();
      const int key = j * BT + r;
      const bool live = key < p.N;
      const size_t off = (((size_t)b * p.N + (live ? key : 0)) * (kPerHead ? p.Hq : p.Hkv) + hkv) * D + wg * (D / 2);
      const int wkey0 = j * BT + q4 * 32;  // the warp's first key row
      const bool staged = Lay::kStoreTma && wkey0 + 32 <= p.N;
      if constexpr (kPerHead)
        store_row_f32<D / 2>(acc_col + wg * (D / 2), 1.f, p.ws_part + off, live);
      else if (staged)
        stage_out(acc_col + wg * (D / 2), 1.f, &tdv, wg * (D / 2), hkv, b * p.N + wkey0);
      else
        store_row<D / 2>(acc_col + wg * (D / 2), 1.f, static_cast<__nv_bfloat16*>(p.dv) + off, live);
      if (!warp_wait(bar(kAccFull), nacc & 1, abort, p.status, p.wait_ns)) break;
      ++nacc;
      tc_fence_after();
      if constexpr (kPerHead)
        store_row_f32<D / 2>(acc_col + D + wg * (D / 2), p.scale, p.ws_part + (size_t)p.B * p.N * p.Hq * D + off, live);
      else if (staged)
        stage_out(acc_col + D + wg * (D / 2), p.scale, &tdk, wg * (D / 2), hkv, b * p.N + wkey0);
      else
        store_row<D / 2>(acc_col + D + wg * (D / 2), p.scale, static_cast<__nv_bfloat16*>(p.dk) + off, live);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kAccEmpty));
    }
    // the TMA stores complete before the CTA (and its slots) goes away
    if (Lay::kStoreTma && lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ dQ pass
template <int D>
struct DqLayout {
  static constexpr int kTile = BwdTiles<D>::kTile;
  static constexpr int kOffQ = 0;
  static constexpr int kOffDO = kTile;
  // K_j lives in stage j % 3 of the K ring (read by S_j and dQ += dS_j K_j), V_j in
  // stage j % 2 of the V ring (read by dP_j alone, so it is released two products sooner)
  static constexpr int kKStages = 3, kVStages = 2;
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + kKStages * kTile;
  static constexpr int kOffBar = kOffV + kVStages * kTile;
  static constexpr int kNumBars = 21;
  static constexpr int kBarStall = kNumBars;      // test hook: a barrier no role arrives on
  static constexpr int kOffHolder = kOffBar + (kNumBars + 1) * 8;
  static constexpr int kOffAbort = kOffHolder + 8;
  // three counters: items whose per-row vectors warp 2 (rows 0-63) and warp 3 (rows 64-127)
  // have put into the workspace, and items the element-wise warps have started
  static constexpr int kOffCounts = kOffAbort + 8;
  // + slack to align the base to 1024 B; at least 117 KB so that a second CTA
  // (which would wait in tcgen05.alloc for all 512 columns) never shares the SM
  static constexpr int kUsed = kOffCounts + 16 + 1024;
  static constexpr int kBytes = kUsed > 117 * 1024 ? kUsed : 117 * 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};
enum : int {
  kQFull = 0, kQEmpty = 1, kQKvFull = 2, kKEmpty = 5, kVEmpty = 10, kQSFull = 12,
  kQDpFull = 14, kQDpFree = 15, kQDsFull = 16, kQAccFull = 18, kQAccEmpty = 19, kQMmaDone = 20
};
// dQ pass: dS of key tile n goes to TMEM columns [kColDs + 64 (n & 1), +64) (bf16 pairs;
// warpgroup g writes the 32 columns of its keys at + 32 g), so dP of the next tile can be
// written while dS of this one still feeds dQ += dS K.
constexpr uint32_t kColDs = 384;

template <int D, int kShape>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_dq_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                  const BwdParams p) {
  using Lay = DqLayout<D>;
  constexpr bool kShaped = kShape != kPlain;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + Lay::kOffBar + 8 * i; };
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Lay::kOffAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // warps 2 and 3: items whose vectors of their rows are in the workspace (one count each, as one
  // warp may be an item ahead of the other); element-wise warps: items started
  volatile int* halves_done = reinterpret_cast<volatile int*>(smem + Lay::kOffCounts);
  volatile int* items_started = halves_done + 2;
  if (threadIdx.x == 0) {
    for (int i = 0; i < Lay::kNumBars; ++i)
      mbar_init(bar(i), (i == kQDpFree || i == kQDsFull || i == kQDsFull + 1 || i == kQAccEmpty) ? kEwArrivals : 1);
    mbar_init(bar(Lay::kBarStall), 1);
    *abort = 0;
    halves_done[0] = halves_done[1] = 0;
    *items_started = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
    tma_prefetch_desc(&tdo);
  }
  if (warp == 1) {
    tmem_alloc(sb + Lay::kOffHolder, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Lay::kOffHolder);

  const int nt = (p.N + BT - 1) / BT;
  const int G = p.Hq / p.Hkv;
  const BwdSchedule sch = make_bwd_schedule(p.B * p.Hq, nt, G);
  // item: (sequence, query head, query tile i); rank 0 = the last tile, the most key tiles under the causal rule
  auto item = [&](int it, int& b, int& h, int& i) {
    int head, rank;
    bwd_decode(sch, it, head, rank);
    i = nt - 1 - rank;
    b = head / p.Hq;
    h = head - b * p.Hq;
  };
  // key tiles [top - jn, top) of an item, from the highest down
  auto tiles = [&](int b, int i, int& top, int& jn) {
    if constexpr (kShaped)
      shaped_key_tiles(p, b, i, nt, top, jn);
    else
      top = jn = p.causal ? i + 1 : nt;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t nq = 0, nk = 0, nv = 0;
      const uint64_t pol_q = policy_evict_first(), pol_kv = policy_evict_last();
      bool ok = true;
      for (int kk = 0, it; ok && (it = bwd_item_index(sch, kk)) >= 0; ++kk) {
        int b, h, i;
        item(it, b, h, i);
        int top, jn;
        tiles(b, i, top, jn);
        const int hkv = h / G;
        for (int j = 0; j < jn; ++j) {
          // K_j (stage j mod 3) and V_j (stage j mod 2) land on one barrier, QKvFull j mod 2:
          // the MMA issuer waits once for both (S_j comes before dP_j). Two slots suffice:
          // step j + 2 is armed only after V_j's stage is free, i.e. after dP_j, which the
          // issuer started after its wait for step j.
          const uint32_t ks = nk % 3, vs = nv & 1;
          if (!mbar_wait(bar(kKEmpty + ks), ((nk / 3) & 1) ^ 1, abort, p.status, p.wait_ns) ||
              !mbar_wait(bar(kVEmpty + vs), ((nv >> 1) & 1) ^ 1, abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(kQKvFull + vs), 2 * Lay::kTile);
          const int kt = top - 1 - j;  // key tiles from the diagonal down
          load_tile<D>(sb + Lay::kOffK + ks * Lay::kTile, &tk, bar(kQKvFull + vs), hkv, b * p.N + kt * BT, pol_kv);
          load_tile<D>(sb + Lay::kOffV + vs * Lay::kTile, &tv, bar(kQKvFull + vs), hkv, b * p.N + kt * BT, pol_kv);
          ++nk;
          ++nv;
          if (j == 0) {  // Q and dO after the first K and V, whose stages are free a tile earlier
            if (!mbar_wait(bar(kQEmpty), (nq & 1) ^ 1, abort, p.status, p.wait_ns)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(bar(kQFull), 2 * Lay::kTile);
            load_tile<D>(sb + Lay::kOffQ, &tq, bar(kQFull), h, b * p.N + i * BT, pol_q);
            load_tile<D>(sb + Lay::kOffDO, &tdo, bar(kQFull), h, b * p.N + i * BT, pol_q);
            ++nq;
          }
        }
      }
      // wait for the last load into each buffer before the CTA may exit
      if (nq) mbar_drain(bar(kQFull), (nq - 1) & 1);
      for (uint32_t st = 0; st < 2; ++st) {
        const uint32_t c = (nv + 1 - st) / 2;  // steps armed on slot st
        if (c) mbar_drain(bar(kQKvFull + st), (c - 1) & 1);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // per key tile j: S_j = Q K_j^T and dP_j = dO V_j^T; S_{j+1} and dP_{j+1} as soon
    // as the element-wise warps have read S_j and dP_j (one signal for both), then
    // dQ += dS_j K_j once dS_j is written. dS alternates between two TMEM
    // buffers: dS_{n+2} is written only after dP_{n+2} completes, which was issued
    // after dQ += dS_n K_n, so that product has finished reading buffer n & 1.
    if (lane == 0) {
      // n counts key tiles over all items: K_n in K stage n % 3, V_n in V stage n % 2
      uint32_t nq = 0, n = 0, ndpf = 0, nacc = 0;
      const uint64_t qd = smem_desc_sw128(sb + Lay::kOffQ, 16, 1024);
      const uint64_t dod = smem_desc_sw128(sb + Lay::kOffDO, 16, 1024);
      const uint32_t tS = tmem + kColS, tDP = tmem + kColDP, tDQ = tmem + kColAcc;
      bool ok = true;
      auto k_addr = [&](uint32_t t) -> uint32_t { return sb + Lay::kOffK + (t % 3) * Lay::kTile; };
      auto v_addr = [&](uint32_t t) -> uint32_t { return sb + Lay::kOffV + (t & 1) * Lay::kTile; };
      // S_t = Q K_t^T
      auto issue_s = [&](uint32_t t) -> bool {  // K_t and V_t have landed after this wait
        if (!mbar_wait(bar(kQKvFull + (t & 1)), (t >> 1) & 1, abort, p.status, p.wait_ns)) return false;
        tc_fence_after();
        issue_kk<D>(tS, qd, smem_desc_sw128(k_addr(t), 16, 1024));
        mma_commit(bar(kQSFull));
        return true;
      };
      // dP_t = dO V_t^T, then V_t's stage is free
      auto issue_dp = [&](uint32_t t) -> bool {  // after issue_s(t), whose wait covers V_t
        tc_fence_after();
        issue_kk<D>(tDP, dod, smem_desc_sw128(v_addr(t), 16, 1024));
        mma_commit(bar(kQDpFull));
        mma_commit(bar(kVEmpty + (t & 1)));
        return true;
      };
      for (int kk = 0, it; ok && (it = bwd_item_index(sch, kk)) >= 0; ++kk) {
        int b, h, i;
        item(it, b, h, i);
        int top, jn;
        tiles(b, i, top, jn);
        if (!mbar_wait(bar(kQFull), nq & 1, abort, p.status, p.wait_ns)) break;
        ++nq;
        if (!issue_s(n) || !issue_dp(n)) break;
        // Q and dO are read by the item's S and dP products alone: once the last of them
        // completes, the next item's tiles may load while this item's last dQ runs
        if (jn == 1) mma_commit(bar(kQEmpty));
        for (int j = 0; j < jn; ++j, ++n) {
          if (j + 1 < jn) {  // S_n and dP_n both read: the next two products may overwrite them
            if (!mbar_wait(bar(kQDpFree), ndpf & 1, abort, p.status, p.wait_ns) || !issue_s(n + 1) ||
                !issue_dp(n + 1)) {
              ok = false;
              break;
            }
            ++ndpf;
            if (j + 2 == jn) mma_commit(bar(kQEmpty));
          }
          if (j == 0 && !mbar_wait(bar(kQAccEmpty), (nacc & 1) ^ 1, abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          // dS alternates between two barriers as between its buffers: S and dP of tile n + 1 are
          // issued before this wait, so the element-wise warps may finish dS_{n+1} before a
          // late issuer looks at dS_n; on one barrier that phase would be gone (a wait by
          // parity cannot tell two completed phases from none) and the pass would stop
          if (!mbar_wait(bar(kQDsFull + (n & 1)), (n >> 1) & 1, abort, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          issue_tn_packed<D>(tDQ, tmem + kColDs + 64 * (n & 1), smem_desc_sw128(k_addr(n), BT * 128, 1024), j > 0);
          mma_commit(bar(kKEmpty + n % 3));  // dQ += dS_n K_n
        }
        if (!ok) break;
        // the item's last S and dP were read before its last dS was written
        if (!mbar_wait(bar(kQDpFree), ndpf & 1, abort, p.status, p.wait_ns)) break;
        ++ndpf;
        mma_commit(bar(kQAccFull));
        ++nacc;
      }
      mma_commit(bar(kQMmaDone));
      mbar_drain(bar(kQMmaDone), 0);
    }
  } else if (warp == 2 || warp == 3) {
    // ------------------------------------------------------------ per-row vectors
    // For this CTA's items in order, D and -lse log2(e) of the tile's 128 rows into the
    // workspace (warp 2 rows 0-63, warp 3 rows 64-127), at most three items ahead of the
    // element-wise warps; they read the vectors back once the warp's count shows them
    // written, and the dK/dV pass (launched after this one) reads them all.
    if constexpr (kShaped) {
      if (warp == 3) write_key_ranges(p, blockIdx.x, gridDim.x, lane);
    }
    for (int kk = 0, it; (it = bwd_item_index(sch, kk)) >= 0; ++kk) {
      if (!count_wait(items_started, kk - 2, abort, p.status, p.wait_ns)) break;
      int b, h, i;
      item(it, b, h, i);
#pragma unroll 1
      for (int blk = 0; blk < 2; ++blk) {
        const int r0 = i * BT + 64 * (warp - 2) + 32 * blk;
        if constexpr (kShaped)
          row_vectors_wide<D>(p, b, h, r0, lane);
        else
          row_vectors<D>(p, b, h, r0, lane);
      }
      __threadfence_block();  // the stores above before the count that announces them
      __syncwarp();
      if (lane == 0) halves_done[warp - 2] = kk + 1;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ element-wise (one query row per thread)
    const int q4 = warp & 3, wg = (warp - 4) >> 2;
    const int r = q4 * 32 + lane;
    const int cb = 64 * wg;                          // this warpgroup's key columns
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t s_col = tmem + lane_off + kColS + cb, dp_col = tmem + lane_off + kColDP + cb;
    const uint32_t dq_col = tmem + lane_off + kColAcc, ds_col = tmem + lane_off + kColDs + 32 * wg;
    const float sl2 = p.scale * kLog2e;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    uint32_t ns = 0, ndp = 0, nacc = 0;
    bool ok = true;
    // The epilogue of an item (dQ in bf16, warpgroup g columns [g D / 2, (g + 1) D / 2) of
    // the row) runs after the first key tile of the next item, so that it overlaps that
    // item's next S and dP products instead of holding up its first ones.
    int pend = -1, pb = 0, ph = 0;  // query tile of the item whose epilogue is pending (-1: none)
    auto epilogue = [&]() -> bool {
      if (!warp_wait(bar(kQAccFull), nacc & 1, abort, p.status, p.wait_ns)) return false;
      ++nacc;
      tc_fence_after();
      const int prow = pend * BT + r;
      const bool live = prow < p.N;
      const size_t off = (((size_t)pb * p.N + (live ? prow : 0)) * p.Hq + ph) * D + wg * (D / 2);
      store_row<D / 2>(dq_col + wg * (D / 2), p.scale, static_cast<__nv_bfloat16*>(p.dq) + off, live);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQAccEmpty));
      pend = -1;
      return true;
    };
    // test hook: a wait that runs out (nothing arrives on the stall barrier), after which
    // every role stops, drains and frees TMEM; the outputs stay unwritten
    if (p.debug_stall && !warp_wait(bar(Lay::kBarStall), 0, abort, p.status, p.wait_ns)) ok = false;
    for (int kk = 0, it; ok && (it = bwd_item_index(sch, kk)) >= 0; ++kk) {
      int b, h, i;
      item(it, b, h, i);
      int top, jn;
      tiles(b, i, top, jn);
      const int qrow = i * BT + r;
      // shaped: the keys [klo, khi) that this thread's query sees
      int klo = 0, khi = 0;
      if constexpr (kShaped) {
        if (qrow < p.N) {
          klo = shape_lo(p.shape, (long long)b * p.N + qrow, qrow);
          khi = shape_hi(p.shape, (long long)b * p.N + qrow, qrow, p.N, p.causal);
        }
      }
      const size_t vrow = (size_t)(b * p.Hq + h) * p.Npad + qrow;
      if (warp == 4 && lane == 0) atomicAdd(const_cast<int*>(items_started), 1);
      // the vectors of this warp's rows are in the workspace
      if (!count_wait(halves_done + (q4 >> 1), kk + 1, abort, p.status, p.wait_ns)) break;
      __threadfence_block();
      const float nl2 = p.ws_nl2[vrow], dval = p.ws_d[vrow];
      const uint64_t nl2x2 = f2_pack(nl2, nl2);
      for (int j = 0; j < jn; ++j) {
        if (!warp_wait(bar(kQSFull), ns & 1, abort, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        ++ns;
        tc_fence_after();
        float pv[64];
        if constexpr (kShaped) {
          const float slope2 = (kShape & kShapeBias) ? -__ldg(p.shape.slopes + h) * kLog2e : 0.f;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t u[32];
            tmem_ld32(s_col + 32 * q, u);
            const int kb = (top - 1 - j) * BT + cb + 32 * q;  // key of the first column
            shaped_p32<kShape, false, false>(p, slope2, u, (float)(qrow - kb), -1.f, klo - kb, khi - kb, nullptr, nl2, pv + 32 * q,
                                     nullptr);
          }
        } else {
          uint32_t u[64];
          tmem_ld64(s_col, u);
          // visible keys of this tile: column c < lim
          const int lim = min(p.causal ? qrow + 1 : p.N, p.N) - (top - 1 - j) * BT - cb;  // key tile top - 1 - j
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), sl2x2, nl2x2), x0, x1);
            pv[c] = c < lim ? ex2(x0) : 0.f;
            pv[c + 1] = c + 1 < lim ? ex2(x1) : 0.f;
          }
        }
        if (!warp_wait(bar(kQDpFull), ndp & 1, abort, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        {
          uint32_t a[64];
          tmem_ld64(dp_col, a);
          tc_fence_before();
          __syncwarp();
          // S and dP may be overwritten by the next tile's products (one signal for both: one
          // wait fewer for the MMA issuer)
          if (lane == 0) mbar_arrive(bar(kQDpFree));
          // dS = P o (dP - D) as bf16 pairs
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            w[e] = pack_bf16x2(pv[2 * e] * (__uint_as_float(a[2 * e]) - dval),
                               pv[2 * e + 1] * (__uint_as_float(a[2 * e + 1]) - dval));
          tmem_st32(ds_col + 64 * (ndp & 1), w);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kQDsFull + (ndp & 1)));
        ++ndp;
        // the previous item's dQ: its accumulator is free for this item's first dQ product
        if (j == 0 && pend >= 0 && !epilogue()) {
          ok = false;
          break;
        }
      }
      if (!ok) break;
      pend = i;
      pb = b;
      ph = h;
    }
    if (ok && pend >= 0) epilogue();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// dV (blockIdx.y 0) and dK (1) of the KV heads: the sums, in order, of their query heads' fp32 shares. A thread takes 4
// columns of a (row, KV head); bound by the shares' bytes.
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) sum_heads_kernel(const BwdParams p) {
  const int lanes = p.d / 4, G = p.Hq / p.Hkv;
  const long long at = (long long)blockIdx.x * (kSumThreads / lanes) + threadIdx.x / lanes;  // row * Hkv + KV head
  if (at >= (long long)p.B * p.N * p.Hkv) return;
  const int c = (threadIdx.x % lanes) * 4;
  const float4* src = reinterpret_cast<const float4*>(p.ws_part + (blockIdx.y ? (size_t)p.B * p.N * p.Hq * p.d : 0) +
                                                      (size_t)at * G * p.d + c);
  float4 sum = __ldg(src);
#pragma unroll 4
  for (int g = 1; g < G; ++g) {
    const float4 v = __ldg(src + (size_t)g * lanes);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  uint2 o;
  o.x = pack_bf16x2(sum.x, sum.y);
  o.y = pack_bf16x2(sum.z, sum.w);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(blockIdx.y ? p.dk : p.dv) + (size_t)at * p.d + c) = o;
}

template <int D, int kShape, bool kPerHead>
cudaError_t launch_dkdv(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const CUtensorMap& tdo, const CUtensorMap& tdk, const CUtensorMap& tdv, int num_sms,
                        cudaStream_t stream) {
  const int nt = (p.N + BT - 1) / BT;
  auto kern = bwd_dkdv_kernel<D, kShape, kPerHead>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, DkdvLayout<D>::kBytes);
  if (e != cudaSuccess) return e;
  const long long items = (long long)p.B * (kPerHead ? p.Hq : p.Hkv) * nt;
  const int grid = (int)std::min<long long>(items, num_sms);
  kern<<<grid, kThreads, DkdvLayout<D>::kBytes, stream>>>(tq, tk, tv, tdo, tdk, tdv, p);
  e = cudaGetLastError();
  if (!kPerHead || e != cudaSuccess) return e;
  const int rows = kSumThreads / (D / 4);
  sum_heads_kernel<<<dim3((unsigned)(((long long)p.B * p.N * p.Hkv + rows - 1) / rows), 2), kSumThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int kShape>
cudaError_t launch_bwd_t(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                         const CUtensorMap& tdo, const CUtensorMap& tdk, const CUtensorMap& tdv, int num_sms,
                         cudaStream_t stream) {
  const int nt = (p.N + BT - 1) / BT;
  cudaError_t e;
  {  // dQ, and the two per-row vectors the dK/dV pass reads
    auto kern = bwd_dq_kernel<D, kShape>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, DqLayout<D>::kBytes);
    if (e != cudaSuccess) return e;
    const long long items = (long long)p.B * p.Hq * nt;
    const int grid = (int)std::min<long long>(items, num_sms);
    kern<<<grid, kThreads, DqLayout<D>::kBytes, stream>>>(tq, tk, tv, tdo, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if constexpr (kShape != kPlain) {
    if (p.ws_part) return launch_dkdv<D, kShape, true>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream);
  }
  return launch_dkdv<D, kShape, false>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream);
}

template <int D>
cudaError_t launch_bwd_d(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                         const CUtensorMap& tdo, const CUtensorMap& tdk, const CUtensorMap& tdv, int num_sms,
                         cudaStream_t stream) {
  if (!p.shaped) return launch_bwd_t<D, kPlain>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream);
  const bool cap = p.shape.cap > 0.f, bias = p.shape.slopes != nullptr;
  if (p.shape.cap > 128.f)
    return bias ? launch_bwd_t<D, kShapeCap + kShapeBias + kShapeFar>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream)
                : launch_bwd_t<D, kShapeCap + kShapeFar>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream);
  if (cap && bias) return launch_bwd_t<D, kShapeCap + kShapeBias>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream);
  if (cap) return launch_bwd_t<D, kShapeCap>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream);
  if (bias) return launch_bwd_t<D, kShapeBias>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream);
  return launch_bwd_t<D, 0>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream);
}

}  // namespace

cudaError_t launch_backward(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const CUtensorMap& tdo, const CUtensorMap& tdk, const CUtensorMap& tdv, int num_sms,
                            cudaStream_t stream) {
  return p.d == 128 ? launch_bwd_d<128>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream)
                    : launch_bwd_d<64>(p, tq, tk, tv, tdo, tdk, tdv, num_sms, stream);
}

}  // namespace fattn
