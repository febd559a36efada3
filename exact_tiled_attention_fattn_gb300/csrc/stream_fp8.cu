// Attention of few query rows over the 8-bit paged cache (single tokens, and chunks of a few queries), split along the
// keys, the splits joined in the same launch.
//
// Bound by the cache's bytes where a KV head has few rows: 8 contexts to 32k tokens, 32 heads over 8 of 128, 409 MB, in 77 us
// (5.3 TB/s; 6.4 in the stream itself, the rest is launch, first lookups and the joining), four times the tokens in 262 us
// (6.2 TB/s). By the latency of a step with more (24 rows, 4 contexts to 12k, capped: 78 MB in 41 us, 8 warps an SM): the
// registers hold a warp's O^T, 32 a tile of 8 rows.
// A warp streams tokens 16 at a time straight from global memory into registers: the codes are laid out as the tensor-core
// fragments want them, so that shared memory, shuffles of the cache and transposes are not needed. The next step's K is
// loaded while this one's softmax and V are worked on, its V brought to the L2 cache. (Through shared memory by
// cp.async, three stages, 16 warps an SM: 91 us for the first case above.) Both products are taken transposed, with tokens
// (K) and head elements (V) as the 16 rows of mma.sync m16n8k16 and up to 8 query rows as its columns, which is what a group
// of heads gives. (tcgen05.mma takes the same transposed products, tokens or head elements as M = 128 and N = 16 or more query
// rows, with O^T in tensor memory; its operands come from shared memory, where the codes would have to be written as fp16
// first. That way is not tried.)
//   S^T = K Q^T   lane (g, c) holds tokens g and g + 8: 16 consecutive codes of each are the A fragments of four steps, if
//                 the head's elements are taken in the order in which they lie there (Q^T is permuted alike);
//   O^T = V^T P^T lane (g, c) holds the codes 16 g .. 16 g + 15 of tokens 2c, 2c + 1, 2c + 8 and 2c + 9: pairs of tokens
//                 are put side by side by byte permutations; P^T comes out of S^T by one 8x8 transpose (movmatrix).
// Codes become fp16 by one conversion a pair, exactly. Q is brought to fp16 by a power of two per row that puts its largest
// element in [2^14, 2^15): bf16 values of up to 2^28 below it stay exact, smaller ones are off by 2^-39 of the largest.
// The scales: a page's K scale goes into the factor of its scores; its V scale into the exponent, p' = 2^(score + log2 vscale
// - m), with m the running maximum of just that sum, so that P (fp16, 2^-11 of it) is largest where it weighs most; the
// softmax's sum takes p' / vscale in 32 bits. m is raised lazily, when a score exceeds it by 2^8, which is seen by a vote.
#include "device_common.cuh"
#include "fattn_internal.h"
#include "ops_internal.h"
#include "score_shape.cuh"

#include <cuda_fp16.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>

namespace fattn {
namespace {

// Warps of a CTA, two CTAs an SM: what the registers of one to four tiles of 8 query rows leave.
template <int NT>
constexpr int kWarps = NT <= 2 ? 6 : 4;
// Chunks of 16 tokens that a warp works on together.
template <int NT>
constexpr int kTogether = NT == 1 ? 2 : 1;
constexpr int kTurn = kStreamTurn, kPieces = kStreamPieces;
constexpr int kMostCluster = kStreamMostCluster;   // CTAs of a cluster
constexpr int kChunk = 16;       // tokens of a step
constexpr int kZeros = -2;       // page of tokens whose K and V are zeros
constexpr float kNone = -3.0e38f;  // no maximum yet: finite, so that hidden scores give 2^(-inf) = 0 against it
constexpr float kLazy = 8.f;     // log2 units that scores may exceed the running maximum by

__device__ __forceinline__ uint4 ldg16(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ldg8(const void* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}
// The low and the high two of four codes as fp16 pairs (exact).
__device__ __forceinline__ void cvt4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// D(16x8, f32) += A(16x16, f16, row) * B(16x8, f16, col)
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// This CTA's rank in its cluster; a float4 and a float of the CTA of rank r, at the shared-memory address that `p` has here.
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_address(const void* p, int r) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(r));
  return a;
}
__device__ __forceinline__ float4 peer_float4(const float* p, int r) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(peer_address(p, r)) : "memory");
  return v;
}
__device__ __forceinline__ float peer_float(const float* p, int r) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_address(p, r)) : "memory");
  return v;
}

// u / d by a multiplication with m = ceil(2^42 / d), for u d < 2^42 (a division by a run-time number takes some 40 cycles
// a piece's first and last steps wait for).
__device__ __forceinline__ int quotient(int u, unsigned long long m) { return (int)(((unsigned long long)(unsigned)u * m) >> 42); }

// The rows of a group: row r is query i = r / G of the sequence, head r % G of the KV head's group. The tokens that they
// can see are counted without those between the sinks and the window's first page: from cut on token v is v + gap.
struct Group {
  int b, r0, rows;    // sequence; first row, rows of this group
  int q0;             // packed row of the sequence's query 0
  int off, L;         // position of query 0, context tokens
  int lo, hi;         // keys that some row sees beside its sinks
  int cut, gap;
  int chunks;         // steps of 16 tokens; at least 1 where there are rows (they are written, whatever they see)
};

// The v-th group of rows: sequence v / nsub, rows from (v % nsub) R on; inconsistent lengths: no rows.
template <int R>
__device__ __forceinline__ Group describe(const StreamFp8Params& p, int v, bool tell) {
  const int cap = p.max_pages << p.page_shift;
  Group x;
  x.b = p.subs == 1 ? v : quotient(v, p.by_subs);
  x.r0 = (v - x.b * p.subs) * R;
  x.L = __ldg(p.seqlens_k + x.b);
  x.q0 = x.b;
  int lq = 1;
  bool bad;
  if (p.cu_seqlens) {
    x.q0 = __ldg(p.cu_seqlens + x.b);
    lq = __ldg(p.cu_seqlens + x.b + 1) - x.q0;
    bad = x.q0 < 0 || lq < 0 || lq > p.rows - x.q0 || lq > p.max_q || x.L < lq || x.L > cap;
    if (bad) lq = 0;
  } else {
    bad = x.L < 0 || x.L > cap;
    x.L = min(max(x.L, 0), cap);
  }
  if (bad && tell && x.r0 == 0) record_status(p.status, kStatusDeviceCheck);
  x.rows = min(R, lq * p.group - x.r0);
  x.chunks = 0;
  if (x.rows <= 0) return x;
  x.off = x.L - lq;
  const int W = p.shape.window, at0 = x.off + quotient(x.r0, p.by_group), at1 = x.off + quotient(x.r0 + x.rows - 1, p.by_group);
  x.lo = W > 0 ? max(at0 - W + 1, 0) : 0;
  x.hi = p.causal ? at1 + 1 : W > 0 && W < x.L - at1 ? at1 + W : x.L;
  const int first = x.lo >> p.page_shift;
  x.cut = min(p.shape.sinks > 0 ? ((p.shape.sinks - 1) >> p.page_shift) + 1 : 0, first) << p.page_shift;
  x.gap = (first << p.page_shift) - x.cut;
  const int n = max(x.hi, shape_sinks(p.shape, at1, x.L, p.causal)) - x.gap;
  x.chunks = max((n + kChunk - 1) / kChunk, 1);
  return x;
}

__device__ __forceinline__ void store_row(const StreamFp8Params& p, int row, int head, int d, int col, const float4& v, float lse) {
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + ((size_t)row * p.Hq + head) * d + col) =
      make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  if (p.lse && col == 0) p.lse[head * p.lse_head + row * p.lse_row] = lse;
}

// What a row sees: keys [lo, hi) and [0, sk); pos its position.
struct Sight {
  int lo, hi, sk, pos;
  __device__ __forceinline__ bool sees(int t) const { return (t >= lo && t < hi) || t < sk; }
};
// A group's rows, kept out of registers: they are looked at where a chunk holds tokens that not every row sees.
template <int D, int R>
struct Shared {
  uint2 q[R / 8][D / 16][32];   // Q^T's fragments
  Sight rows[R], all, any;      // of each row, what all of them see, and what at least one does
  float slope[R], fac[R];
  float lse[R];                 // of a cluster's piece
};

// Raw codes of 16 tokens: K of tokens g, g + 8 and V of tokens 2c, 2c + 1, 2c + 8, 2c + 9.
template <int D>
struct KCodes {
  uint32_t w[2][D / 16];
};
template <int D>
struct VCodes {
  uint32_t w[4][D / 32];
};
// What a warp knows of 32 chunks, one per lane: the chunk's page (-1: none, its tokens are hidden; kZeros: a chunk of queries
// met a table entry outside the pool, whose tokens are zeros, as for the prefill) and first row in the pool, and its page's
// scales. It is asked for in two trips, each many steps before it is used: the table's entry, then the scales.
struct Meta {
  int page, row;
  float ks, vs;
};

template <int D, int NT, bool kScores>
__device__ __forceinline__ void stream_piece(const StreamFp8Params& p, float* scratch, Shared<D, 8 * NT>& sh, const Group& x,
                                             int hkv, int chunk0, int nchunks, int piece, bool alone) {
  constexpr int W = kWarps<NT>, Y = kTogether<NT>, kBatch = 32 / Y;   // steps that a warp looks ahead for at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int G = p.group;
  // (the last step's second chunk may not exist)
  const int nsteps = (nchunks + Y - 1) / Y, n_mine = warp < nsteps ? (nsteps - warp + W - 1) / W : 0;
  const int32_t* table = p.block_table + (size_t)x.b * p.max_pages;
  const size_t token_bytes = (size_t)p.Hkv * D;
  const uint8_t* kc = static_cast<const uint8_t*>(p.kcache) + (size_t)hkv * D + 16 * c + g * token_bytes;
  const uint8_t* vc = static_cast<const uint8_t*>(p.vcache) + (size_t)hkv * D + (D / 8) * g + 2 * c * token_bytes;
  // chunk y of this warp's step i: its number in the piece, and its tokens from this one on
  auto number = [&](int i, int y) -> int { return Y * (warp + i * W) + y; };
  auto token = [&](int i, int y) -> int {
    const int v = (chunk0 + number(i, y)) * kChunk;
    return v >= x.cut ? v + x.gap : v;
  };
  auto look = [&](Meta& m, int i0) {
    const int i = i0 + lane / Y, y = lane % Y, t = token(i, y);
    // (a group that sees nothing: one chunk, all hidden, past the sequence's end)
    m.page = i < n_mine && number(i, y) < nchunks && t < x.L ? __ldg(table + (t >> p.page_shift)) : -1;
  };
  auto scales = [&](Meta& m, int i0) {
    const int i = i0 + lane / Y, y = lane % Y, t = token(i, y);
    if (m.page < 0 || m.page >= p.num_pages) {
      const bool mine = i < n_mine && number(i, y) < nchunks && t < x.L;
      if (mine) record_status(p.status, kStatusDeviceCheck);
      m.page = mine && p.cu_seqlens ? kZeros : -1;
    }
    const size_t at = (size_t)max(m.page, 0) * p.Hkv + hkv;
    m.row = m.page < 0 ? 0 : (m.page << p.page_shift) + (t & ((1 << p.page_shift) - 1));
    m.ks = __ldg(p.kscale + at);
    m.vs = __ldg(p.vscale + at);
  };
  auto load_k = [&](KCodes<D>& k, int row) {
    const uint8_t* src = kc + (size_t)row * token_bytes;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        const uint4 a = ldg16(src + 8 * t * token_bytes + 64 * u);
        k.w[t][4 * u] = a.x, k.w[t][4 * u + 1] = a.y, k.w[t][4 * u + 2] = a.z, k.w[t][4 * u + 3] = a.w;
      }
  };
  auto load_v = [&](VCodes<D>& v, int row) {
    const uint8_t* src = vc + (size_t)row * token_bytes;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint8_t* at = src + ((t & 1) + 8 * (t >> 1)) * token_bytes;
      if constexpr (D == 128) {
        const uint4 a = ldg16(at);
        v.w[t][0] = a.x, v.w[t][1] = a.y, v.w[t][2] = a.z, v.w[t][3] = a.w;
      } else {
        const uint2 a = ldg8(at);
        v.w[t][0] = a.x, v.w[t][1] = a.y;
      }
    }
  };
  // V's rows of step i on their way to the L2 cache, a row a lane: its loads, for which registers are free only later, then
  // wait for the cache and not for memory (8 contexts to 32k: 80 -> 77.5 us; two and more steps ahead, or K as well, is
  // slower: 80 to 84)
  const uint8_t* line = static_cast<const uint8_t*>(p.vcache) + (size_t)(lane & 15) * token_bytes + (size_t)hkv * D;
  auto prefetch_v = [&](const int (&row)[Y]) {
    if (Y == 2 || lane < 16)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(line + (size_t)(lane < 16 ? row[0] : row[Y - 1]) * token_bytes));
  };
  // the first step's codes are on their way while Q is brought to fp16 (a chunk without a page reads the pool's first)
  Meta meta, ahead{-1, 0, 1.f, 1.f};
  look(meta, 0);
  look(ahead, kBatch);
  scales(meta, 0);
  KCodes<D> kw[Y];
  VCodes<D> vw[Y];
#pragma unroll
  for (int y = 0; y < Y; ++y) {
    const int row = __shfl_sync(0xffffffffu, meta.row, y);
    load_k(kw[y], row);
    load_v(vw[y], row);
  }

  if (threadIdx.x < 8 * NT) {
    const int r = x.r0 + min((int)threadIdx.x, x.rows - 1), query = quotient(r, p.by_group);
    const int W0 = p.shape.window;
    auto sight = [&](int at) -> Sight {
      return {W0 > 0 ? max(at - W0 + 1, 0) : 0, p.causal ? at + 1 : W0 > 0 && W0 < x.L - at ? at + W0 : x.L,
              shape_sinks(p.shape, at, x.L, p.causal), at};
    };
    sh.rows[threadIdx.x] = sight(x.off + query);
    sh.slope[threadIdx.x] = kScores && p.shape.slopes ? -__ldg(p.shape.slopes + hkv * G + r - query * G) * kLog2e : 0.f;
    if (threadIdx.x == 0) {
      const Sight a = sight(x.off + quotient(x.r0, p.by_group)), e = sight(x.off + quotient(x.r0 + x.rows - 1, p.by_group));
      sh.all = {e.lo, a.hi, a.sk, 0};
      sh.any = {a.lo, e.hi, e.sk, 0};
    }
  }
  // Q^T, a tile of 8 rows a warp: columns are rows g; and the factors of its rows' scores
  if (warp >= W - NT) {
    const int n = W - 1 - warp, r = x.r0 + min(8 * n + g, x.rows - 1), query = quotient(r, p.by_group);
    const bool live = 8 * n + g < x.rows;
    float f[D / 4], m = 0.f;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) +
                               ((size_t)(x.q0 + query) * p.Hq + hkv * G + r - query * G) * D;
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 a = live ? __ldg(reinterpret_cast<const uint4*>(src + 64 * u + 16 * c + 8 * i)) : make_uint4(0, 0, 0, 0);
        const uint32_t y[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[16 * u + 8 * i + 2 * k] = bf16_lo(y[k]), f[16 * u + 8 * i + 2 * k + 1] = bf16_hi(y[k]);
          m = fmax3(m, fabsf(bf16_lo(y[k])), fabsf(bf16_hi(y[k])));
        }
      }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    int up = m > 0.f ? 14 - ((int)(__float_as_uint(m) >> 23) - 127) : 0;   // (subnormal rows: as far as floats go)
    up = min(max(up, -126), 126);
    const float mul = __uint_as_float((uint32_t)(up + 127) << 23), back = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sh.q[n][4 * u + j][lane] = make_uint2(pack_f16x2(f[16 * u + 4 * j] * mul, f[16 * u + 4 * j + 1] * mul),
                                              pack_f16x2(f[16 * u + 4 * j + 2] * mul, f[16 * u + 4 * j + 3] * mul));
    if (c == 0) sh.fac[8 * n + g] = back * (kScores && p.shape.cap > 0.f ? 1.f : p.scale * kLog2e);
  }
  __syncthreads();
  float fac[NT][2], o[NT][D / 16][4];
  float m[NT][2], limit[NT][2], l[NT][2];   // limit: m + kLazy once there is a maximum
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      fac[n][z] = sh.fac[8 * n + 2 * c + z];
      m[n][z] = limit[n][z] = kNone;
      l[n][z] = 0.f;
    }
  }

  float lv_of = 0.f, iv_of = 1.f;
  for (int i = 0; i < n_mine; ++i) {
    if (i % kBatch == 0) {
      if (i > 0) {
        meta = ahead;
        look(ahead, i + kBatch);
      }
      // log2 and the reciprocal of V's scale; a power of two has both exactly (2^127 by the division)
      const uint32_t b = __float_as_uint(meta.vs);
      if (meta.page < 0) meta.ks = 1.f;
      lv_of = meta.page < 0 ? 0.f : (b & 0x7fffffu) == 0 ? (float)((int)(b >> 23) - 127) : log2f(meta.vs);
      iv_of = meta.page < 0 ? 1.f : (b & 0x7fffffu) == 0 && b < 254u << 23 ? __uint_as_float((254u << 23) - b) : 1.f / meta.vs;
    } else if (i % kBatch == kBatch / 2) {
      scales(ahead, i + kBatch / 2);
    }
    float s[Y][NT][4], ivs[Y];
    const bool last = i + 1 == n_mine, wrap = i % kBatch == kBatch - 1;
#pragma unroll
    for (int y = 0; y < Y; ++y)
#pragma unroll
      for (int n = 0; n < NT; ++n) s[y][n][0] = s[y][n][1] = s[y][n][2] = s[y][n][3] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint2 b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) b[n] = sh.q[n][j][lane];
#pragma unroll
      for (int y = 0; y < Y; ++y) {
        uint32_t a0, a1, a2, a3;
        cvt4(kw[y].w[0][j], a0, a2);
        cvt4(kw[y].w[1][j], a1, a3);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(s[y][n], a0, a1, a2, a3, b[n].x, b[n].y);
      }
    }
    int next[Y];   // the next step's rows: its keys take the registers
#pragma unroll
    for (int y = 0; y < Y; ++y) {
      next[y] = __shfl_sync(0xffffffffu, wrap ? ahead.row : meta.row, ((i + 1) % kBatch) * Y + y);
      if (!last) load_k(kw[y], next[y]);
    }
    if (!last) prefetch_v(next);
#pragma unroll
    for (int y = 0; y < Y; ++y) {
      const int from = (i % kBatch) * Y + y;
      const int page = __shfl_sync(0xffffffffu, meta.page, from);
      const bool none = page < 0;
      const float ks = __shfl_sync(0xffffffffu, meta.ks, from), lv = __shfl_sync(0xffffffffu, lv_of, from);
      ivs[y] = __shfl_sync(0xffffffffu, iv_of, from);
      const int t0 = token(i, y);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float (&u)[4] = s[y][n];
        const float f0 = fac[n][0] * ks, f1 = fac[n][1] * ks;
        if constexpr (kScores) {
          u[0] *= f0, u[1] *= f1, u[2] *= f0, u[3] *= f1;
          if (p.shape.cap > 0.f) cap_in_place(p.shape, u);
          if (p.shape.slopes) {
            const int t = t0 + g, r = 8 * n + 2 * c;
            const float away0 = (float)(sh.rows[r].pos - t), away1 = (float)(sh.rows[r + 1].pos - t);
            const float slope0 = sh.slope[r], slope1 = sh.slope[r + 1];
            u[0] = fmaf(slope0, fabsf(away0), u[0]);
            u[1] = fmaf(slope1, fabsf(away1), u[1]);
            u[2] = fmaf(slope0, fabsf(away0 - 8.f), u[2]);
            u[3] = fmaf(slope1, fabsf(away1 - 8.f), u[3]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) u[k] += lv;
        } else {
          u[0] = fmaf(u[0], f0, lv), u[1] = fmaf(u[1], f1, lv);
          u[2] = fmaf(u[2], f0, lv), u[3] = fmaf(u[3], f1, lv);
        }
      }
      // hidden tokens: -inf, and V codes that mean nothing must not meet a weight of 0
      if (none || !((t0 >= sh.all.lo && t0 + kChunk <= sh.all.hi) || t0 + kChunk <= sh.all.sk)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = 8 * n + 2 * c + (k & 1), t = t0 + g + 8 * (k >> 1);
            if (page == kZeros) s[y][n][k] = sh.slope[r] * fabsf((float)(sh.rows[r].pos - t));   // (a score of 0, biased)
            if (page == -1 || !sh.rows[r].sees(t)) s[y][n][k] = -CUDART_INF_F;
          }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (none || !sh.any.sees(t0 + 2 * c + (k & 1) + 8 * (k >> 1))) {
#pragma unroll
            for (int e = 0; e < D / 32; ++e) vw[y].w[k][e] = 0;
          }
      }
    }
    auto top_of = [&](int n, int z) -> float {
      return Y == 2 ? fmaxf(fmax3(s[0][n][z], s[0][n][2 + z], s[Y - 1][n][z]), s[Y - 1][n][2 + z]) : fmaxf(s[0][n][z], s[0][n][2 + z]);
    };
    bool more = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) more |= top_of(n, 0) > limit[n][0] || top_of(n, 1) > limit[n][1];
    if (__any_sync(0xffffffffu, more)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float mx = top_of(n, z);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float top = fmaxf(m[n][z], mx), a = ex2(m[n][z] - top);
          m[n][z] = top;
          limit[n][z] = top + kLazy;
          l[n][z] *= a;
#pragma unroll
          for (int e = 0; e < D / 16; ++e) o[n][e][z] *= a, o[n][e][2 + z] *= a;
        }
    }
    uint32_t pt[Y][NT][2];
#pragma unroll
    for (int y = 0; y < Y; ++y)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float (&u)[4] = s[y][n];
        const float p0 = ex2(u[0] - m[n][0]), p1 = ex2(u[1] - m[n][1]), p2 = ex2(u[2] - m[n][0]), p3 = ex2(u[3] - m[n][1]);
        l[n][0] = fmaf(p0 + p2, ivs[y], l[n][0]);
        l[n][1] = fmaf(p1 + p3, ivs[y], l[n][1]);
        pt[y][n][0] = transpose8x8(pack_f16x2(p0, p1));
        pt[y][n][1] = transpose8x8(pack_f16x2(p2, p3));
      }
#pragma unroll
    for (int y = 0; y < Y; ++y)
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint32_t sel = z ? 0x7362 : 0x5140;    // codes 2z, 2z + 1 of two tokens, token by token
          uint32_t a0, a1, a2, a3;
          cvt4(__byte_perm(vw[y].w[0][e], vw[y].w[1][e], sel), a0, a1);
          cvt4(__byte_perm(vw[y].w[2][e], vw[y].w[3][e], sel), a2, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(o[n][2 * e + z], a0, a1, a2, a3, pt[y][n][0], pt[y][n][1]);
        }
    if (!last) {
#pragma unroll
      for (int y = 0; y < Y; ++y) load_v(vw[y], next[y]);
    }
  }

  // ---- the warps' states joined: scratch[w] = { m[R], l[R], O[R][D] }
  constexpr int R = 8 * NT, kWs = R * (D + 2);
  {
    float* ws = scratch + warp * kWs;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = 8 * n + 2 * c + y;
        float t = l[n][y];
        t += __shfl_xor_sync(0xffffffffu, t, 4);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        if (g == 0) ws[r] = m[n][y], ws[R + r] = t;
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
          *reinterpret_cast<float2*>(ws + 2 * R + r * D + (D / 8) * g + 2 * e) = make_float2(o[n][e][y], o[n][e][2 + y]);
      }
  }
  __syncthreads();
  constexpr int C4 = D / 4;
  for (int idx = threadIdx.x; idx < x.rows * C4; idx += W * 32) {
    const int r = idx / C4, col = (idx - r * C4) * 4;
    float top = kNone;
#pragma unroll
    for (int u = 0; u < W; ++u) top = fmaxf(top, scratch[u * kWs + r]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < W; ++u) {
      const float f = ex2(scratch[u * kWs + r] - top);
      const float4 a = *reinterpret_cast<const float4*>(scratch + u * kWs + 2 * R + r * D + col);
      acc.x = fmaf(f, a.x, acc.x), acc.y = fmaf(f, a.y, acc.y);
      acc.z = fmaf(f, a.z, acc.z), acc.w = fmaf(f, a.w, acc.w);
      sum = fmaf(f, scratch[u * kWs + R + r], sum);
    }
    // (a NaN sum stays one; no key seen: 0 and -inf)
    const float inv = sum == 0.f ? 0.f : 1.f / sum, lse = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * kLn2;
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
    const int query = quotient(x.r0 + r, p.by_group), head = hkv * G + x.r0 + r - query * G;
    const size_t out = (size_t)(x.q0 + query) * p.Hq + head;
    if (alone) {
      store_row(p, x.q0 + query, head, D, col, acc, lse);
    } else if (p.cluster > 1) {                        // (in place of the first warp's, which this thread alone has read)
      *reinterpret_cast<float4*>(scratch + 2 * R + r * D + col) = acc;
      if (col == 0) sh.lse[r] = lse;
    } else {
      *reinterpret_cast<float4*>(p.o_part + (out * p.num_splits + piece) * D + col) = acc;
      if (col == 0) p.lse_part[out * p.num_splits + piece] = lse;
    }
  }
}

// The group's rows from their pieces: lse = ln sum_s e^{lse_s}, O = sum_s e^{lse_s - lse} O_s. kRound pieces of all of a
// thread's rows are loaded together (they cost a trip to the L2 cache each otherwise).
template <int D, int NT>
__device__ __forceinline__ void join_pieces(const StreamFp8Params& p, const Group& x, int hkv, int pieces) {
  constexpr int C4 = D / 4, kPer = kWarps<NT> * 32 / C4, kRows = (8 * NT + kPer - 1) / kPer, kRound = 24 / kRows;
  const int col = threadIdx.x % C4 * 4;
  size_t prow[kRows];
  int query[kRows], head[kRows];
  float4 acc[kRows];
  float sum[kRows], top[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = x.r0 + min((int)threadIdx.x / C4 + k * kPer, x.rows - 1);
    query[k] = quotient(r, p.by_group);
    head[k] = hkv * p.group + r - query[k] * p.group;
    prow[k] = ((size_t)(x.q0 + query[k]) * p.Hq + head[k]) * p.num_splits;
    acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    sum[k] = 0.f;
    top[k] = kNone;
  }
  for (int s0 = 0; s0 < pieces; s0 += kRound) {
    float ls[kRows][kRound];
    float4 a[kRows][kRound];
#pragma unroll
    for (int k = 0; k < kRows; ++k)
#pragma unroll
      for (int s = 0; s < kRound; ++s) {
        const size_t at = prow[k] + min(s0 + s, pieces - 1);
        ls[k][s] = __ldcg(p.lse_part + at);
        a[k][s] = __ldcg(reinterpret_cast<const float4*>(p.o_part + at * D + col));
      }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      float mx = top[k];
#pragma unroll
      for (int s = 0; s < kRound; ++s) {
        ls[k][s] = s0 + s < pieces ? ls[k][s] * kLog2e : -CUDART_INF_F;
        mx = fmaxf(mx, ls[k][s]);
      }
      const float keep = ex2(top[k] - mx);
      top[k] = mx;
      acc[k].x *= keep, acc[k].y *= keep, acc[k].z *= keep, acc[k].w *= keep, sum[k] *= keep;
#pragma unroll
      for (int s = 0; s < kRound; ++s) {
        const float f = ex2(ls[k][s] - mx);
        acc[k].x = fmaf(f, a[k][s].x, acc[k].x), acc[k].y = fmaf(f, a[k][s].y, acc[k].y);
        acc[k].z = fmaf(f, a[k][s].z, acc[k].z), acc[k].w = fmaf(f, a[k][s].w, acc[k].w);
        sum[k] += f;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if ((int)threadIdx.x / C4 + k * kPer >= x.rows) continue;
    const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
    acc[k].x *= inv, acc[k].y *= inv, acc[k].z *= inv, acc[k].w *= inv;
    store_row(p, x.q0 + query[k], head[k], D, col, acc[k], sum[k] == 0.f ? -CUDART_INF_F : (top[k] + log2f(sum[k])) * kLn2);
  }
}

// The group's rows from the pieces of its cluster's CTAs, which share the rows out. A CTA leaves when all have read.
template <int D, int NT>
__device__ __forceinline__ void join_cluster(const StreamFp8Params& p, float* scratch, const Shared<D, 8 * NT>& sh, const Group& x,
                                             int hkv, int rank) {
  constexpr int C4 = D / 4, T = kWarps<NT> * 32, R = 8 * NT;
  cluster_sync();
  for (int idx = rank * T + threadIdx.x; idx < x.rows * C4; idx += p.cluster * T) {
    const int r = idx / C4, col = (idx - r * C4) * 4;
    float ls[kMostCluster];
    float4 a[kMostCluster];
    float top = kNone;
#pragma unroll
    for (int s = 0; s < kMostCluster; ++s)
      if (s < p.cluster) {
        ls[s] = peer_float(sh.lse + r, s) * kLog2e;
        a[s] = peer_float4(scratch + 2 * R + r * D + col, s);
        top = fmaxf(top, ls[s]);
      }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < kMostCluster; ++s)
      if (s < p.cluster) {
        const float f = ex2(ls[s] - top);
        acc.x = fmaf(f, a[s].x, acc.x), acc.y = fmaf(f, a[s].y, acc.y);
        acc.z = fmaf(f, a[s].z, acc.z), acc.w = fmaf(f, a[s].w, acc.w);
        sum += f;
      }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
    const int query = quotient(x.r0 + r, p.by_group), head = hkv * p.group + x.r0 + r - query * p.group;
    store_row(p, x.q0 + query, head, D, col, acc, sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * kLn2);
  }
  cluster_sync();
}

// Where the groups are short, or few and not long, a cluster of CTAs (or one) takes each (stream_fp8_cluster), their pieces joined
// through its shared memory, with neither counters to clear nor partials in global memory. Else:
// the groups' steps in one line, group of rows after group of rows, cut into equal shares, one for Hkv CTAs, which take a KV
// head each: every SM streams the same number of bytes whatever the sequences' lengths are, and the heads of a page, side
// by side in memory, are read at about the same time (reading the pages of 8 heads of 128 alone: 58.5 us for 393 MB so,
// 64 to 66 with head after head). A share is long enough that no group is cut into more than num_splits pieces. A group that lies
// in one share is written at once; else its pieces' partials are joined by the CTA that finishes the last of them.
template <int D, int NT, bool kScores>
__global__ void __launch_bounds__(kWarps<NT> * 32, 2) stream_fp8_kernel(const StreamFp8Params p) {
  constexpr int R = 8 * NT, W = kWarps<NT>, Y = kTogether<NT>, T = W * 32;
  extern __shared__ __align__(16) float scratch[];     // kScratch<D, NT> bytes
  __shared__ Shared<D, R> sh;
  __shared__ Group s_x;
  __shared__ int s_sum[W], s_most[W], s_begin, s_v, s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.cluster > 0) {
    const int rank = p.cluster > 1 ? cluster_rank() : 0, at = blockIdx.x / p.cluster, v = at / p.Hkv, hkv = at - v * p.Hkv;
    const Group x = describe<R>(p, v, hkv == 0 && rank == 0 && threadIdx.x == 0);
    if (x.chunks == 0) {   // (as all of the cluster; it stays for the others should the lengths change under the kernel)
      if (p.cluster > 1) cluster_sync(), cluster_sync();
      return;
    }
    const int share = (x.chunks + p.cluster - 1) / p.cluster, from = min(rank * share, x.chunks);
    stream_piece<D, NT, kScores>(p, scratch, sh, x, hkv, from, min(share, x.chunks - from), 0, p.cluster == 1);
    if (p.cluster > 1) join_cluster<D, NT>(p, scratch, sh, x, hkv, rank);
    return;
  }
  const int V = p.B * p.subs;                          // groups of rows
  // a thread's groups of rows, and the steps before them (the host has made sure that all of them are an int)
  const int per = (V + T - 1) / T;
  const int mine0 = min((int)threadIdx.x * per, V), mine1 = min(mine0 + per, V);
  int sum = 0, most = 0;
  Group x;
  for (int v = mine0; v < mine1; ++v) {
    x = describe<R>(p, v, blockIdx.x == 0);
    sum += x.chunks > 0 ? kTurn + x.chunks : 0;
    most = max(most, x.chunks);
  }
  int before = sum;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, m);
    if (lane >= m) before += y;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) s_sum[warp] = before, s_most[warp] = most;
  before -= sum;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
    most = max(most, s_most[w]);
  }
  const unsigned splits = min(p.num_splits, kPieces);
  const unsigned block = blockIdx.x / p.Hkv, blocks = gridDim.x / p.Hkv;
  const int hkv = blockIdx.x - block * p.Hkv;
  unsigned share = ((unsigned)total + blocks - 1) / blocks;
  share = max(share, ((unsigned)most + splits - 2) / (splits - 1));
  share = max(share, (unsigned)(Y * W));               // (a step for every warp)
  if ((unsigned long long)share * block >= total) return;
  int at = (int)(share * block);                       // in steps
  const int stop = (int)min((unsigned long long)share * (block + 1ull), (unsigned long long)total);
  if (at >= before && at < before + sum) {
    int y = before;
    for (int v = mine0; v < mine1; ++v) {
      if (per > 1) x = describe<R>(p, v, false);
      const int n = x.chunks > 0 ? kTurn + x.chunks : 0;
      if (at < y + n) {
        s_v = v;
        s_begin = y;
        s_x = x;
        break;
      }
      y += n;
    }
  }
  __syncthreads();
  int v = s_v, begin = s_begin;                        // the group, and where it begins in the line
  x = s_x;
  for (;;) {
    const int zero = begin + kTurn;                    // of its first chunk
    const int from = max(at, zero), to = min(stop, zero + x.chunks);
    if (from < to) {
      const int c0 = (unsigned)zero / share, c1 = (unsigned)(zero + x.chunks - 1) / share;
      const int pieces = c1 - c0 + 1;
      stream_piece<D, NT, kScores>(p, scratch, sh, x, hkv, from - zero, to - from, (int)block - c0, pieces == 1);
      if (pieces > 1) {
        __syncthreads();                               // the partial is written
        if (threadIdx.x == 0) {
          __threadfence();
          s_last = atomicAdd(p.counters + v * p.Hkv + hkv, 1) == pieces - 1;
          __threadfence();
        }
        __syncthreads();
        if (s_last) join_pieces<D, NT>(p, x, hkv, pieces);
      }
      __syncthreads();                                 // the scratch is read
    }
    begin = zero + x.chunks;
    if (begin >= stop) break;
    do {
      if (++v >= V) return;                            // (only if the lengths change under the kernel)
      x = describe<R>(p, v, false);
    } while (x.chunks == 0);
  }
}

template <int D, int NT>
constexpr int kScratch = kWarps<NT> * 8 * NT * (D + 2) * 4;

// CTAs that a cluster of this kernel may have on the current device: 16 where the GPU has room for one (8 is what every
// launch may have; a part of a GPU, or a context held to a few SMs, may have room for fewer). Asked for once per device.
template <int D, int NT, bool kScores>
int most_cluster() {
  static std::atomic<int> known[128];
  int dev = 0, most = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev >= 0 && dev < 128 && (most = known[dev].load(std::memory_order_relaxed)) > 0) return most;
  auto kern = stream_fp8_kernel<D, NT, kScores>;
  // (an answer of no, which is no error of this call, does not stay behind; what was there before does)
  auto yes = [](cudaError_t e) -> bool { return e == cudaSuccess || (cudaGetLastError(), false); };
  const bool wide = yes(cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
  for (most = wide ? kStreamMostCluster : 8; most > 1; most /= 2) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(most);
    c.blockDim = dim3(kWarps<NT> * 32);
    c.dynamicSmemBytes = kScratch<D, NT>;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim = {(unsigned)most, 1, 1};
    c.attrs = &a;
    c.numAttrs = 1;
    int room = 0;
    if (yes(cudaOccupancyMaxActiveClusters(&room, kern, &c)) && room > 0) break;
  }
  if (dev >= 0 && dev < 128) known[dev].store(most, std::memory_order_relaxed);
  return most;
}

template <int D, int NT, bool kScores>
cudaError_t launch_t(const StreamFp8Params& p0, cudaStream_t stream) {
  const int sms = num_sms_current();
  if (sms <= 0) return cudaErrorInvalidValue;
  StreamFp8Params p = p0;
  auto kern = stream_fp8_kernel<D, NT, kScores>;
  if (kScratch<D, NT> > 40 * 1024) {   // (without asking, 48 KB with the static part)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kScratch<D, NT>);
    if (e != cudaSuccess) return e;
  }
  p.cluster = stream_fp8_cluster(p, kWarps<NT> * kTogether<NT>, sms, most_cluster<D, NT, kScores>());
  const long long groups = (long long)p.B * p.subs * p.Hkv;
  if (p.cluster > 0) {
    if (p.cluster > 8) {               // (8 is what every launch may have)
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(groups * p.cluster));
    c.blockDim = dim3(kWarps<NT> * 32);
    c.dynamicSmemBytes = kScratch<D, NT>;
    c.stream = stream;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim = {(unsigned)p.cluster, 1, 1};
    c.attrs = &a;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kern, p);
  }
  const cudaError_t e = cudaMemsetAsync(p.counters, 0, (size_t)groups * sizeof(int), stream);
  if (e != cudaSuccess) return e;
  const long long blocks = std::min<long long>((long long)p.B * p.subs * p.num_splits, std::max(2 * sms / p.Hkv, 1));
  kern<<<(int)(blocks * p.Hkv), kWarps<NT> * 32, kScratch<D, NT>, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int NT>
cudaError_t launch_n(const StreamFp8Params& p, cudaStream_t stream) {
  return p.shape.cap > 0.f || p.shape.slopes ? launch_t<D, NT, true>(p, stream) : launch_t<D, NT, false>(p, stream);
}

template <int D>
cudaError_t launch_d(const StreamFp8Params& p, cudaStream_t stream) {
  switch (stream_fp8_rows((long long)p.max_q * p.group)) {
    case 8: return launch_n<D, 1>(p, stream);
    case 16: return launch_n<D, 2>(p, stream);
    case 24: return launch_n<D, 3>(p, stream);
    default: return launch_n<D, 4>(p, stream);
  }
}

}  // namespace

cudaError_t launch_stream_fp8(const StreamFp8Params& p0, cudaStream_t stream) {
  StreamFp8Params p = p0;
  p.group = p.Hq / p.Hkv;
  p.subs = (int)(stream_fp8_groups(p.B, p.Hkv, (long long)p.max_q * p.group) / ((long long)p.B * p.Hkv));
  p.by_group = ((1ull << 42) + p.group - 1) / p.group;
  p.by_subs = ((1ull << 42) + p.subs - 1) / p.subs;
  p.page_shift = p.page_size == 16 ? 4 : p.page_size == 32 ? 5 : p.page_size == 64 ? 6 : 7;
  return p.d == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace fattn
