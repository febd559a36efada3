// Attention of few query rows over the 8-bit paged cache (single tokens, and chunks of a few queries), split along the
// keys, the splits joined in the same launch.
//
// Bound by the cache's bytes. A warp streams tokens 16 at a time straight from global memory into registers: the codes are
// laid out as the tensor-core fragments want them, so that shared memory, shuffles of the cache and transposes are not
// needed, and the registers of the next 16 tokens are in flight while these are worked on. Both products are taken
// transposed, with tokens (K) and head elements (V) as the 16 rows of mma.sync m16n8k16 and up to 8 query rows as its columns, which is
// what a group of heads gives:
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

namespace fattn {
namespace {

constexpr int kWarps = 4;
constexpr int kChunk = 16;       // tokens of a step
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

// The rows of a group: row r is query i = r / G of the sequence, head r % G of the KV head's group.
struct Group {
  int b, hkv;
  int r0, rows;       // first row, rows of this group
  int q0;             // packed row of the sequence's query 0
  int off, L;         // position of query 0, context tokens
  int lo, hi;         // keys that some row sees beside its sinks
};

__device__ __forceinline__ void store_row(const StreamFp8Params& p, int row, int head, int d, int col, const float4& v, float lse) {
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + ((size_t)row * p.Hq + head) * d + col) =
      make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  if (p.lse && col == 0) p.lse[head * p.lse_head + row * p.lse_row] = lse;
}

// Raw codes of 16 tokens: K of tokens g, g + 8 and V of tokens 2c, 2c + 1, 2c + 8, 2c + 9.
template <int D>
struct Codes {
  uint32_t k[2][D / 16], v[4][D / 32];
};
// What a warp knows of 32 chunks ahead, one per lane: the chunk's first row in the pool (-1: none) and its page's scales.
struct Meta {
  int row;
  float ks, vs;
};

template <int D, int NT, bool kScores>
__device__ __forceinline__ void stream_split(const StreamFp8Params& p, float* scratch, const Group& x, int split, int v0,
                                             int v1, int cut, int gap, bool alone) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int G = p.Hq / p.Hkv;
  const int nchunks = (v1 - v0 + kChunk - 1) / kChunk;
  const int n_mine = warp < nchunks ? (nchunks - warp + kWarps - 1) / kWarps : 0;
  const int32_t* table = p.block_table + (size_t)x.b * p.max_pages;
  const size_t token_bytes = (size_t)p.Hkv * D;
  const uint8_t* kc = static_cast<const uint8_t*>(p.kcache) + (size_t)x.hkv * D;
  const uint8_t* vc = static_cast<const uint8_t*>(p.vcache) + (size_t)x.hkv * D;
  const int P = p.page_size;
  // chunk i of this warp: tokens from this one on (v0 is a multiple of 16, pages are as well)
  auto token = [&](int i) -> int {
    const int v = v0 + (warp + i * kWarps) * kChunk;
    return v >= cut ? v + gap : v;
  };
  auto look = [&](int i0) -> Meta {
    Meta m{-1, 1.f, 1.f};
    if (i0 + lane < n_mine) {
      const int t = token(i0 + lane), pi = t / P;
      const int page = __ldg(table + pi);
      if (page >= 0 && page < p.num_pages) {
        m.row = page * P + (t - pi * P);
        m.ks = __ldg(p.kscale + (size_t)page * p.Hkv + x.hkv);
        m.vs = __ldg(p.vscale + (size_t)page * p.Hkv + x.hkv);
      } else {
        record_status(p.status, kStatusDeviceCheck);
      }
    }
    return m;
  };
  auto load_k = [&](Codes<D>& w, int row) {
    const uint8_t* src = kc + (size_t)max(row, 0) * token_bytes + 16 * c;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        const uint4 a = ldg16(src + (size_t)(g + 8 * t) * token_bytes + 64 * u);
        w.k[t][4 * u] = a.x, w.k[t][4 * u + 1] = a.y, w.k[t][4 * u + 2] = a.z, w.k[t][4 * u + 3] = a.w;
      }
  };
  auto load_v = [&](Codes<D>& w, int row) {
    const uint8_t* src = vc + (size_t)max(row, 0) * token_bytes + (D / 8) * g;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint8_t* at = src + (size_t)(2 * c + (t & 1) + 8 * (t >> 1)) * token_bytes;
      if constexpr (D == 128) {
        const uint4 a = ldg16(at);
        w.v[t][0] = a.x, w.v[t][1] = a.y, w.v[t][2] = a.z, w.v[t][3] = a.w;
      } else {
        const uint2 a = ldg8(at);
        w.v[t][0] = a.x, w.v[t][1] = a.y;
      }
    }
  };

  // the first chunks' codes are on their way while Q is brought to fp16
  Meta meta = look(0), ahead = look(32);
  Codes<D> w[2];
  const int row_0 = __shfl_sync(0xffffffffu, meta.row, 0), row_1 = __shfl_sync(0xffffffffu, meta.row, 1);
  if (n_mine > 0) load_k(w[0], row_0), load_v(w[0], row_0);
  if (n_mine > 1) load_k(w[1], row_1), load_v(w[1], row_1);

  // Q^T: columns are rows g of each tile of 8; and the factors of the lane's two score columns 2c, 2c + 1
  uint32_t q[NT][D / 16][2];
  float fac[NT][2], slope[NT][2];
  int lo[NT][2], hi[NT][2], sk[NT][2], pos[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = x.r0 + 8 * n + g;
    const bool live = 8 * n + g < x.rows;
    float f[D / 4];
    float m = 0.f;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) +
                               ((size_t)(x.q0 + (live ? r / G : 0)) * p.Hq + x.hkv * G + (live ? r % G : 0)) * D;
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
      for (int j = 0; j < 4; ++j) {
        q[n][4 * u + j][0] = pack_f16x2(f[16 * u + 4 * j] * mul, f[16 * u + 4 * j + 1] * mul);
        q[n][4 * u + j][1] = pack_f16x2(f[16 * u + 4 * j + 2] * mul, f[16 * u + 4 * j + 3] * mul);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = 2 * c + i;
      fac[n][i] = __shfl_sync(0xffffffffu, back, col * 4) * (kScores && p.shape.cap > 0.f ? 1.f : p.scale * kLog2e);
      const int rr = x.r0 + min(8 * n + col, x.rows - 1);
      const int at = x.off + rr / G;
      pos[n][i] = at;
      lo[n][i] = p.shape.window > 0 ? max(at - p.shape.window + 1, 0) : 0;
      hi[n][i] = p.causal ? at + 1 : p.shape.window > 0 && p.shape.window < x.L - at ? at + p.shape.window : x.L;
      sk[n][i] = shape_sinks(p.shape, at, x.L, p.causal);
      slope[n][i] = kScores && p.shape.slopes ? -__ldg(p.shape.slopes + x.hkv * G + rr % G) * kLog2e : 0.f;
    }
  }
  // tokens that every row of the group sees: [all_lo, all_hi) and [0, all_sk)
  const int at0 = x.off + x.r0 / G, at1 = x.off + (x.r0 + x.rows - 1) / G;
  const int all_lo = p.shape.window > 0 ? max(at1 - p.shape.window + 1, 0) : 0;
  const int all_hi = p.causal ? at0 + 1 : p.shape.window > 0 && p.shape.window < x.L - at0 ? at0 + p.shape.window : x.L;
  const int all_sk = shape_sinks(p.shape, at0, x.L, p.causal);
  const int any_sk = shape_sinks(p.shape, at1, x.L, p.causal);

  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    m[n][0] = m[n][1] = -CUDART_INF_F;
    l[n][0] = l[n][1] = 0.f;
  }

  auto step = [&](int i, Codes<D>& cur) {
    const int row = __shfl_sync(0xffffffffu, meta.row, i & 31);
    const float ks = __shfl_sync(0xffffffffu, meta.ks, i & 31), vs = __shfl_sync(0xffffffffu, meta.vs, i & 31);
    const int t0 = token(i);
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t a0, a1, a2, a3;
      cvt4(cur.k[0][j], a0, a2);
      cvt4(cur.k[1][j], a1, a3);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(s[n], a0, a1, a2, a3, q[n][j][0], q[n][j][1]);
    }
    // chunk i + 2 takes the registers
    const bool more_chunks = i + 2 < n_mine;
    const int next_row = __shfl_sync(0xffffffffu, ((i + 2) & 31) < 2 ? ahead.row : meta.row, (i + 2) & 31);
    if (more_chunks) load_k(cur, next_row);
    // the page's scales; log2 of a power of two is exact
    const uint32_t vb = __float_as_uint(vs);
    const float lv = (vb & 0x7fffffu) == 0 ? (float)((int)(vb >> 23) - 127) : log2f(vs);
    const float ivs = (vb & 0x7fffffu) == 0 ? __uint_as_float((254u << 23) - vb) : 1.f / vs;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float f0 = fac[n][0] * ks, f1 = fac[n][1] * ks;
      s[n][0] *= f0, s[n][1] *= f1, s[n][2] *= f0, s[n][3] *= f1;
      if constexpr (kScores) {
        if (p.shape.cap > 0.f) cap_in_place(p.shape, s[n]);
        if (p.shape.slopes) {
          const int t = t0 + g;
          s[n][0] = fmaf(slope[n][0], fabsf((float)(pos[n][0] - t)), s[n][0]);
          s[n][1] = fmaf(slope[n][1], fabsf((float)(pos[n][1] - t)), s[n][1]);
          s[n][2] = fmaf(slope[n][0], fabsf((float)(pos[n][0] - t - 8)), s[n][2]);
          s[n][3] = fmaf(slope[n][1], fabsf((float)(pos[n][1] - t - 8)), s[n][3]);
        }
      }
    }
    // hidden tokens: -inf, and V codes that mean nothing must not meet a weight of 0
    if (row < 0 || !((t0 >= all_lo && t0 + kChunk <= all_hi) || t0 + kChunk <= all_sk)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = t0 + g + 8 * (k >> 1), y = k & 1;
          if (row < 0 || !((t >= lo[n][y] && t < hi[n][y]) || t < sk[n][y])) s[n][k] = -CUDART_INF_F;
        }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = t0 + 2 * c + (k & 1) + 8 * (k >> 1);
        if (row < 0 || !((t >= x.lo && t < x.hi) || t < any_sk)) {
#pragma unroll
          for (int e = 0; e < D / 32; ++e) cur.v[k][e] = 0;
        }
      }
    }
    bool more = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[n][k] += lv;
      more |= fmaxf(s[n][0], s[n][2]) > m[n][0] + kLazy || fmaxf(s[n][1], s[n][3]) > m[n][1] + kLazy;
    }
    if (__any_sync(0xffffffffu, more)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float mx = fmaxf(s[n][y], s[n][2 + y]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float next = fmaxf(m[n][y], mx);
          const float a = next == -CUDART_INF_F ? 1.f : ex2(m[n][y] - next);
          m[n][y] = next;
          l[n][y] *= a;
#pragma unroll
          for (int e = 0; e < D / 16; ++e) o[n][e][y] *= a, o[n][e][2 + y] *= a;
        }
    }
    uint32_t pt[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float b0 = m[n][0] == -CUDART_INF_F ? 0.f : m[n][0], b1 = m[n][1] == -CUDART_INF_F ? 0.f : m[n][1];
      const float p0 = ex2(s[n][0] - b0), p1 = ex2(s[n][1] - b1), p2 = ex2(s[n][2] - b0), p3 = ex2(s[n][3] - b1);
      l[n][0] = fmaf(p0 + p2, ivs, l[n][0]);
      l[n][1] = fmaf(p1 + p3, ivs, l[n][1]);
      pt[n][0] = transpose8x8(pack_f16x2(p0, p1));
      pt[n][1] = transpose8x8(pack_f16x2(p2, p3));
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t sel = y ? 0x7362 : 0x5140;    // codes 2y, 2y + 1 of two tokens, token by token
        uint32_t a0, a1, a2, a3;
        cvt4(__byte_perm(cur.v[0][e], cur.v[1][e], sel), a0, a1);
        cvt4(__byte_perm(cur.v[2][e], cur.v[3][e], sel), a2, a3);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(o[n][2 * e + y], a0, a1, a2, a3, pt[n][0], pt[n][1]);
      }
    }
    if (more_chunks) load_v(cur, next_row);
  };
  for (int i = 0; i < n_mine; i += 2) {
    if ((i & 31) == 0 && i > 0) {
      meta = ahead;
      ahead = look(i + 32);
    }
    step(i, w[0]);
    if (i + 1 < n_mine) step(i + 1, w[1]);
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
  for (int idx = threadIdx.x; idx < x.rows * C4; idx += kWarps * 32) {
    const int r = idx / C4, col = (idx - r * C4) * 4;
    float top = -CUDART_INF_F;
#pragma unroll
    for (int u = 0; u < kWarps; ++u) top = fmaxf(top, scratch[u * kWs + r]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    if (top != -CUDART_INF_F) {
#pragma unroll
      for (int u = 0; u < kWarps; ++u) {
        const float f = ex2(scratch[u * kWs + r] - top);
        const float4 a = *reinterpret_cast<const float4*>(scratch + u * kWs + 2 * R + r * D + col);
        acc.x = fmaf(f, a.x, acc.x), acc.y = fmaf(f, a.y, acc.y);
        acc.z = fmaf(f, a.z, acc.z), acc.w = fmaf(f, a.w, acc.w);
        sum = fmaf(f, scratch[u * kWs + R + r], sum);
      }
    }
    // (a NaN sum stays one; no key seen: 0 and -inf)
    const float inv = sum == 0.f ? 0.f : 1.f / sum, lse = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * kLn2;
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
    const int rr = x.r0 + r;
    const size_t out = (size_t)(x.q0 + rr / G) * p.Hq + x.hkv * G + rr % G;
    if (alone) {
      store_row(p, x.q0 + rr / G, x.hkv * G + rr % G, D, col, acc, lse);
    } else {
      *reinterpret_cast<float4*>(p.o_part + (out * p.num_splits + split) * D + col) = acc;
      if (col == 0) p.lse_part[out * p.num_splits + split] = lse;
    }
  }
}

// The group's rows from their non-empty splits: lse = ln sum_s e^{lse_s}, O = sum_s e^{lse_s - lse} O_s.
template <int D>
__device__ __forceinline__ void merge_group(const StreamFp8Params& p, const Group& x, int nvalid) {
  constexpr int C4 = D / 4;
  const int G = p.Hq / p.Hkv;
  for (int idx = threadIdx.x; idx < x.rows * C4; idx += kWarps * 32) {
    const int r = x.r0 + idx / C4, col = (idx % C4) * 4;
    const size_t prow = ((size_t)(x.q0 + r / G) * p.Hq + x.hkv * G + r % G) * p.num_splits;
    float top = -CUDART_INF_F;
    for (int s = 0; s < nvalid; ++s) top = fmaxf(top, __ldcg(p.lse_part + prow + s));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll 4
    for (int s = 0; s < nvalid; ++s) {
      const float ls = __ldcg(p.lse_part + prow + s);
      const float f = ls == -CUDART_INF_F ? 0.f : ex2((ls - top) * kLog2e);
      const float4 a = __ldcg(reinterpret_cast<const float4*>(p.o_part + (prow + s) * D + col));
      acc.x = fmaf(f, a.x, acc.x), acc.y = fmaf(f, a.y, acc.y), acc.z = fmaf(f, a.z, acc.z), acc.w = fmaf(f, a.w, acc.w);
      sum += f;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
    store_row(p, x.q0 + r / G, x.hkv * G + r % G, D, col, acc, sum == 0.f ? -CUDART_INF_F : top + logf(sum));
  }
}

// Persistent grid over items (group of rows, split) from a counter, highest split first, as in decode.cu; the groups of one
// KV head follow each other, so that their reads of it meet in the L2 cache. The CTA that finishes the last non-empty split
// of a group joins them.
template <int D, int NT, bool kScores>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 3 : 2) stream_fp8_kernel(const StreamFp8Params p) {
  __shared__ __align__(16) float scratch[kWarps * 8 * NT * (D + 2)];
  __shared__ int s_item, s_last;
  const int G = p.Hq / p.Hkv, P = p.page_size;
  const int R = 8 * NT;
  const int nsub = (int)(((long long)p.max_q * G + R - 1) / R);
  const int groups = p.B * p.Hkv * nsub, total = p.num_splits * groups;
  const int cap = p.max_pages * P;
  // pages that a group's rows can see, which the splits share
  const long long width = (p.causal ? 1ll : 2ll) * p.shape.window + (R - 1) / G + 1;
  int seen = p.max_pages;
  if (p.shape.window > 0)
    seen = (int)min((long long)seen, (width + P - 2) / P + 1 + sink_blocks(p.shape.sinks, P));
  const long long span = (long long)((seen + p.num_splits - 1) / p.num_splits) * P;
  for (;;) {
    if (threadIdx.x == 0) s_item = atomicAdd(p.counters, 1);
    __syncthreads();
    const int item = s_item;
    __syncthreads();
    if (item < 0 || item >= total) break;
    const int split = p.num_splits - 1 - item / groups;
    const int gi = item % groups;
    Group x;
    const int sub = gi % nsub;
    x.hkv = gi / nsub % p.Hkv;
    x.b = gi / nsub / p.Hkv;
    x.L = __ldg(p.seqlens_k + x.b);
    int lq = 1;
    if (p.cu_seqlens) {
      x.q0 = __ldg(p.cu_seqlens + x.b);
      lq = __ldg(p.cu_seqlens + x.b + 1) - x.q0;
      if (x.q0 < 0 || lq < 0 || lq > p.rows - x.q0 || lq > p.max_q || x.L < lq || x.L > cap) {
        if (threadIdx.x == 0 && split == 0) record_status(p.status, kStatusDeviceCheck);
        continue;
      }
    } else {
      x.q0 = x.b;
      if (x.L < 0 || x.L > cap) {
        if (threadIdx.x == 0 && split == 0) record_status(p.status, kStatusDeviceCheck);
        x.L = x.L < 0 ? 0 : cap;
      }
    }
    x.r0 = sub * R;
    x.rows = min(R, lq * G - x.r0);
    if (x.rows <= 0) continue;
    x.off = x.L - lq;
    const int at0 = x.off + x.r0 / G, at1 = x.off + (x.r0 + x.rows - 1) / G;
    x.lo = p.shape.window > 0 ? max(at0 - p.shape.window + 1, 0) : 0;
    x.hi = p.causal ? at1 + 1 : p.shape.window > 0 && p.shape.window < x.L - at1 ? at1 + p.shape.window : x.L;
    // the tokens of the group, counted without those between the sinks and the window's first page: from cut on token v is
    // v + gap
    const int first = x.lo / P * P, sinks = shape_sinks(p.shape, at1, x.L, p.causal);
    const int cut = min(sink_blocks(p.shape.sinks, P), first / P) * P, gap = first - cut;
    const int n = max(x.hi, sinks) - gap;
    const int nvalid = (int)((n + span - 1) / span);
    const long long v0 = (long long)split * span;
    if (v0 >= n) {   // nothing here; rows that see no token at all are written by split 0
      if (split == 0) merge_group<D>(p, x, 0);
      continue;
    }
    stream_split<D, NT, kScores>(p, scratch, x, split, (int)v0, (int)min((long long)n, v0 + span), cut, gap, nvalid == 1);
    if (nvalid > 1) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) s_last = atomicAdd(p.counters + 1 + gi, 1) == nvalid - 1;
      __syncthreads();
      if (s_last) {
        __threadfence();
        merge_group<D>(p, x, nvalid);
      }
    }
    __syncthreads();   // the scratch is read
  }
}

template <int D, int NT, bool kScores>
cudaError_t launch_t(const StreamFp8Params& p, cudaStream_t stream) {
  auto kern = stream_fp8_kernel<D, NT, kScores>;
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kWarps * 32, 0);
  if (e != cudaSuccess) return e;
  const int sms = num_sms_current();
  if (sms <= 0 || per_sm <= 0) return cudaErrorInvalidValue;
  const int G = p.Hq / p.Hkv;
  const long long groups = stream_fp8_groups(p.B, p.Hkv, (long long)p.max_q * G), items = groups * p.num_splits;
  e = cudaMemsetAsync(p.counters, 0, (size_t)(1 + groups) * sizeof(int), stream);
  if (e != cudaSuccess) return e;
  kern<<<(int)std::min<long long>(items, (long long)sms * per_sm), kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const StreamFp8Params& p, cudaStream_t stream) {
  const bool scores = p.shape.cap > 0.f || p.shape.slopes;
  if ((long long)p.max_q * (p.Hq / p.Hkv) <= 8) return scores ? launch_t<D, 1, true>(p, stream) : launch_t<D, 1, false>(p, stream);
  return scores ? launch_t<D, 2, true>(p, stream) : launch_t<D, 2, false>(p, stream);
}

}  // namespace

cudaError_t launch_stream_fp8(const StreamFp8Params& p, cudaStream_t stream) {
  return p.d == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace fattn
