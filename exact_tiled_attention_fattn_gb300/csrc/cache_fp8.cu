// The 8-bit paged cache: E4M3 codes [pages, page_size, Hkv, d] for K and for V, and one fp32 scale per page and KV head of
// each, value = scale * code. Two kernels: new tokens rotated, quantized and put into their pages, and visible pages
// expanded to bf16 for the tensor-core prefill.
//
// Scales are powers of two where this file writes them. A code is a floating-point number, so a scale only shifts its
// range: a power of two costs no precision (the largest magnitude of a page lies in (224, 448] code units), makes code *
// scale exact in bf16, and lets a page that outgrows its scale be re-scaled exactly except for codes that become subnormal.
#include "device_common.cuh"
#include "fattn_internal.h"
#include "ops_internal.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

namespace fattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;            // rows that a lane has in flight
constexpr int kMinScaleExp = -100;   // the scale of a page of zeros

// The least power of two s with a <= 448 s (448 = 1.75 * 2^8), a >= 0 finite.
__device__ __forceinline__ float pow2_scale(float a) {
  const int e = (int)((__float_as_uint(a) + 0x1fffffu) >> 23) - 127 - 8;   // mantissas above 1.75 carry into the exponent
  return __uint_as_float((uint32_t)(max(e, kMinScaleExp) + 127) << 23);
}

__device__ __forceinline__ uint32_t codes4(const float (&y)[4]) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3) << 16;
}
__device__ __forceinline__ float2 values2(uint32_t codes) {   // of the low two codes, exact
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
  return __half22float2(__half2(h));
}

// ------------------------------------------------------------------ append
// Two kinds of blocks in one launch. A block of K and V takes one page of one sequence, as far as the call's new tokens
// reach into it, and a share of the KV heads: a head of a page is worked on by this block alone, so its scale and the old
// codes change without atomics on global memory. It forms the magnitudes (shared-memory maxima), the scales, re-scales old
// codes of pages that outgrew theirs, and reads K and V again (from the caches) to make them codes. A block of q takes a
// few rows with all their heads. The rows' angles are formed once in a block's shared memory (as in rope.cu, 64-bit fixed
// point): with q's heads shared out over the pages' blocks, angles were half of the work. A lane has eight elements of a
// row, both halves of its four pairs among them, so that D / 8 lanes take a row and a warp two or four rows at a time.
// Bound by the chain lookup - load - maximum - load - store of a block for prompts (6.7k tokens, 32 + 8 heads of 128, 150 MB
// by the formula: 34 us, 22 at the copy rate; q in the pages' blocks: 85), as for single tokens (64 of them: 6.4 us).
//
// kFast: 8-byte aligned rows and heads, and pairs that never split a lane's elements; else element by element.
struct Eight {
  float x[8];
};

// Where a lane's elements lie: two quads. A turned head in halves: the low and the high elements of four pairs; else eight
// in a row.
struct Quads {
  int a, b;
};
template <bool kInter>
__device__ __forceinline__ Quads quads_of(int sl, int rot, bool turned) {
  const int lanes = rot >> 3;
  if (!kInter && turned && sl < lanes) return {4 * sl, 4 * sl + (rot >> 1)};
  return {8 * sl, 8 * sl + 4};   // (the lanes before have 8 elements each as well, whatever their order)
}

// (cos, sin) of a lane's four pairs.
struct Turn {
  float c[4], s[4];
};
__device__ __forceinline__ Turn load_turn(const float2* cs, int sl, int rot) {
  Turn t;
  if (sl < (rot >> 3)) {
    const float4* c4 = reinterpret_cast<const float4*>(cs + 4 * sl);
    const float4 a = c4[0], b = c4[1];
    t.c[0] = a.x, t.s[0] = a.y, t.c[1] = a.z, t.s[1] = a.w, t.c[2] = b.x, t.s[2] = b.y, t.c[3] = b.z, t.s[3] = b.w;
  } else {   // (not used: products by 1 and 0 would make NaN of infinities)
    t.c[0] = t.c[1] = t.c[2] = t.c[3] = 1.f;
    t.s[0] = t.s[1] = t.s[2] = t.s[3] = 0.f;
  }
  return t;
}

// The lane's elements of a row, as they lie in memory (kFast) and as numbers.
struct Raw {
  uint2 a, b;
};
template <bool kFast>
__device__ __forceinline__ Raw load_raw(const __nv_bfloat16* p, const Quads& at) {
  if constexpr (kFast) return {__ldg(reinterpret_cast<const uint2*>(p + at.a)), __ldg(reinterpret_cast<const uint2*>(p + at.b))};
  Raw r;
  const __nv_bfloat16* q = p + at.a;                  // (eight in a row)
  auto two = [&](int k) -> uint32_t {
    return (uint32_t)__bfloat16_as_ushort(q[k]) | (uint32_t)__bfloat16_as_ushort(q[k + 1]) << 16;
  };
  r.a = make_uint2(two(0), two(2));
  r.b = make_uint2(two(4), two(6));
  return r;
}
__device__ __forceinline__ Eight numbers(const Raw& w) {
  return {{bf16_lo(w.a.x), bf16_hi(w.a.x), bf16_lo(w.a.y), bf16_hi(w.a.y), bf16_lo(w.b.x), bf16_hi(w.b.x), bf16_lo(w.b.y),
           bf16_hi(w.b.y)}};
}
// Turned; cs: the row's table (element by element where pairs may split a lane's elements).
template <bool kFast, bool kInter>
__device__ __forceinline__ void turn_eight(Eight& r, const Turn& t, const __nv_bfloat16* p, int sl, int rot, const float2* cs) {
  if constexpr (kFast) {
    if (sl >= (rot >> 3)) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float& lo = kInter ? r.x[2 * k] : r.x[k];
      float& hi = kInter ? r.x[2 * k + 1] : r.x[4 + k];
      const float a = lo, b = hi;
      lo = a * t.c[k] - b * t.s[k];
      hi = b * t.c[k] + a * t.s[k];
    }
  } else {
    const int half = rot >> 1;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = 8 * sl + k;
      if (e >= rot) break;
      const bool low = kInter ? !(e & 1) : e < half;
      const float2 w = cs[kInter ? e >> 1 : low ? e : e - half];
      const float o = __bfloat162float(p[kInter ? e ^ 1 : low ? e + half : e - half]);
      r.x[k] = low ? r.x[k] * w.x - o * w.y : r.x[k] * w.x + o * w.y;
    }
  }
}

constexpr float kMaxFloat = 3.4028235e38f;
// The largest finite magnitude (infinities and NaN do not decide a scale); `inf`: there is an infinity.
__device__ __forceinline__ float magnitude(const Eight& r, bool& inf) {
  float a = fmax3(fmax3(fabsf(r.x[0]), fabsf(r.x[1]), fabsf(r.x[2])), fmax3(fabsf(r.x[3]), fabsf(r.x[4]), fabsf(r.x[5])),
                  fmaxf(fabsf(r.x[6]), fabsf(r.x[7])));   // (a maximum leaves NaN out)
  if (a > kMaxFloat) {
    inf = true;
    a = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) a = fabsf(r.x[k]) <= kMaxFloat ? fmaxf(a, fabsf(r.x[k])) : a;
  }
  return a == a ? a : 0.f;
}

// Frequencies as fractions of a turn, 2^-64, by the block's last threads (the first ones look for sequences meanwhile).
__device__ __forceinline__ void frequencies(const AppendFp8Params& p, unsigned long long* freq) {
  const int i = kThreads - 1 - (int)threadIdx.x;
  if (i < p.rot >> 1) {
    double turns = __ldg(p.inv_freq + i) * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= floor(turns);
    freq[i] = (unsigned long long)(turns * 18446744073709551616.0);
  }
}
// The rows' tables: pos_of(r) is row r's position.
template <typename Pos>
__device__ __forceinline__ void angles(const AppendFp8Params& p, float2* cs, const unsigned long long* freq, int rows, Pos pos_of) {
  const int half = p.rot >> 1, pitch = (half + 1) & ~1;
  for (int x = threadIdx.x; x < rows * half; x += kThreads) {
    const int r = (int)(((unsigned long long)(unsigned)x * p.by_half) >> 42), i = x - r * half;
    cs[r * pitch + i] = turn_of((long long)(freq[i] * (unsigned long long)pos_of(r)), p.amplitude);
  }
}

struct AppendShared {
  unsigned long long freq[64];
  uint32_t max[2 * kAppendMaxHeads];     // magnitudes (bits) of the block's KV heads: K, then V
  float scale[2 * kAppendMaxHeads], ratio[2 * kAppendMaxHeads];
  int inf[2 * kAppendMaxHeads];
  int b[kAppendRows], t[kAppendRows];    // of q's rows: sequence and token, -1: none
};

// q's rows [row0, row0 + n) with all heads.
template <int D, bool kFast, bool kInter>
__device__ __forceinline__ void append_q(const AppendFp8Params& p, float2* cs, AppendShared& sh, int row0, int n) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;   // lanes of a row, rows of a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / kLanes, sl = lane % kLanes;
  if (threadIdx.x < kAppendRows) sh.b[threadIdx.x] = -1;
  frequencies(p, sh.freq);
  __syncthreads();
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const int c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1);
    if (c0 < 0 || c1 < c0 || c1 > p.rows) continue;   // (recorded by the pages' blocks)
    for (int r = 0; r < n; ++r)
      if (row0 + r >= c0 && row0 + r < c1) sh.b[r] = b;
  }
  __syncthreads();
  if ((int)threadIdx.x < n) {
    int t = -1;
    const int b = sh.b[threadIdx.x];
    if (b >= 0) {
      const long long y = (long long)__ldg(p.seqlens_k + b) - __ldg(p.cu_seqlens + b + 1) + row0 + threadIdx.x;
      if (y >= 0 && y < (long long)p.max_pages << p.page_shift) {
        const int page = __ldg(p.block_table + (size_t)b * p.max_pages + (y >> p.page_shift));
        if (page >= 0 && page < p.num_pages) t = (int)y;
      }
    }
    sh.t[threadIdx.x] = t;
  }
  __syncthreads();
  const int half = p.rot >> 1, pitch = (half + 1) & ~1;
  angles(p, cs, sh.freq, n, [&](int r) -> long long {
    return p.positions ? (long long)__ldg(p.positions + row0 + r) : (long long)max(sh.t[r], 0);
  });
  __syncthreads();
  // a warp: kPer rows and a share of the heads
  const int trips = (n + kPer - 1) / kPer, parts = max(1, kWarps / trips);
  const Quads at = quads_of<kInter>(sl, kFast ? p.rot : 0, true);
  for (int it = warp; it < trips * parts; it += kWarps) {
    const int part = it / trips, r = (it - part * trips) * kPer + sub;
    if (r >= n || sh.t[r] < 0) continue;
    const Turn turn = kFast ? load_turn(cs + r * pitch, sl, p.rot) : Turn{};
    // (pointers that step: a 64-bit product a head is half of what a head costs beside its numbers)
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q.in) + (long long)(row0 + r) * p.q.in_row + part * p.q.in_head;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.q.out) + (long long)(row0 + r) * p.q.out_row + part * p.q.out_head;
    const long long in_step = parts * p.q.in_head, out_step = parts * p.q.out_head;
    for (int h0 = part; h0 < p.q.heads; h0 += kBatch * parts) {
      Raw w[kBatch];                                  // in flight together
      const __nv_bfloat16* from = src;
#pragma unroll
      for (int i = 0; i < kBatch; ++i, src += in_step)
        if (h0 + i * parts < p.q.heads) w[i] = load_raw<kFast>(src, at);
#pragma unroll
      for (int i = 0; i < kBatch; ++i, out += out_step, from += in_step) {
        if (h0 + i * parts >= p.q.heads) break;
        Eight x = numbers(w[i]);
        turn_eight<kFast, kInter>(x, turn, from, sl, p.rot, cs + r * pitch);
        if constexpr (kFast) {
          *reinterpret_cast<uint2*>(out + at.a) = make_uint2(pack_bf16x2(x.x[0], x.x[1]), pack_bf16x2(x.x[2], x.x[3]));
          *reinterpret_cast<uint2*>(out + at.b) = make_uint2(pack_bf16x2(x.x[4], x.x[5]), pack_bf16x2(x.x[6], x.x[7]));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) out[8 * sl + e] = __float2bfloat16_rn(x.x[e]);
        }
      }
    }
  }
}

// K and V of page `id` (of the sequence that it belongs to), share y of ny of the KV heads.
template <int D, bool kFast, bool kInter>
__device__ __forceinline__ void append_kv(const AppendFp8Params& p, float2* cs, AppendShared& sh, int id, int y, int ny) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / kLanes, sl = lane % kLanes;
  const int shift = p.page_shift, P = 1 << shift;
  // sequence b has the blocks from cu[b] / P + 2 b on (it touches at most Lq / P + 2 pages)
  if (threadIdx.x == 0) sh.b[0] = -1;
  frequencies(p, sh.freq);
  __syncthreads();
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const int c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1);
    if (c0 < 0 || c1 < c0 || c1 > p.rows) {
      if (id == 0) record_status(p.status, kStatusDeviceCheck);
    } else if (id >= (c0 >> shift) + 2 * b && id < (c1 >> shift) + 2 * (b + 1)) {
      sh.b[0] = b;
    }
  }
  __syncthreads();
  const int b = sh.b[0];
  if (b < 0) return;
  const int c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1);
  const int end = __ldg(p.seqlens_k + b);             // tokens [start, end) are new
  const long long start = (long long)end - (c1 - c0), cap = (long long)p.max_pages << shift;
  const int local = id - ((c0 >> shift) + 2 * b);
  if (local == 0 && y == 0 && threadIdx.x == 0 && c1 > c0 && (start < 0 || end > cap))
    record_status(p.status, kStatusDeviceCheck);      // rows outside the table are skipped
  const long long first = max(start, 0ll);
  const long long pi = (first >> shift) + local;
  const long long t0 = max(first, pi << shift), t1 = min(min((long long)end, cap), (pi + 1) << shift);
  if (t0 >= t1) return;
  const int page = __ldg(p.block_table + (size_t)b * p.max_pages + pi);
  if (page < 0 || page >= p.num_pages) {
    if (y == 0 && threadIdx.x == 0) record_status(p.status, kStatusDeviceCheck);
    return;
  }
  const int n = (int)(t1 - t0), slot0 = (int)(t0 - (pi << shift));
  const int row0 = c0 + (int)(t0 - start);            // packed row of token t0
  const int kv0 = p.k.heads * y / ny, nkv = p.k.heads * (y + 1) / ny - kv0, units = 2 * nkv;
  float old_scale = 0.f;                              // of thread u's unit
  if ((int)threadIdx.x < units) {
    sh.max[threadIdx.x] = 0;
    sh.inf[threadIdx.x] = 0;
    const int h = kv0 + ((int)threadIdx.x < nkv ? threadIdx.x : threadIdx.x - nkv);
    if (slot0 > 0) old_scale = ((int)threadIdx.x < nkv ? p.kscale : p.vscale)[(size_t)page * p.k.heads + h];
  }
  angles(p, cs, sh.freq, n, [&](int r) -> long long {
    return p.positions ? (long long)__ldg(p.positions + row0 + r) : t0 + r;
  });
  __syncthreads();

  // Units: a head of K (u < nkv) or V; an item is a unit and a share of the page's rows, kPer at a time.
  const int half = p.rot >> 1, pitch = (half + 1) & ~1;
  const int trips = (n + kPer - 1) / kPer, shares = min(trips, (2 * kWarps + units - 1) / units);
  const Quads plain_at = {8 * sl, 8 * sl + 4}, turned_at = quads_of<kInter>(sl, kFast ? p.rot : 0, true);
  auto source = [&](int u) -> const __nv_bfloat16* {
    const RopeTensor& t = u < nkv ? p.k : p.v;
    return static_cast<const __nv_bfloat16*>(t.in) + (long long)row0 * t.in_row + (kv0 + (u < nkv ? u : u - nkv)) * t.in_head;
  };
  // trips [k0, k1) of unit u, kBatch of them in flight together; use(row, values) for each
  auto walk = [&](int u, int k0, int k1, auto use) {
    const bool key = u < nkv;
    const __nv_bfloat16* src = source(u);
    const long long row = key ? p.k.in_row : p.v.in_row;
    const Quads at = key ? turned_at : plain_at;
    const __nv_bfloat16 *last = src + (n - 1) * row, *next = src + (k0 * kPer + sub) * row;   // (stepping: see the rows of q)
    const long long step = kPer * row;
    for (int k = k0; k < k1; k += kBatch) {
      Raw w[kBatch];
      const __nv_bfloat16* from = next;
#pragma unroll
      for (int i = 0; i < kBatch; ++i, next += step)
        if (k + i < k1) w[i] = load_raw<kFast>((k + i) * kPer + sub < n ? next : last, at);
#pragma unroll
      for (int i = 0; i < kBatch; ++i, from += step) {
        if (k + i >= k1) break;
        const int r = min((k + i) * kPer + sub, n - 1);
        Eight x = numbers(w[i]);
        if (key)
          turn_eight<kFast, kInter>(x, kFast ? load_turn(cs + r * pitch, sl, p.rot) : Turn{}, (k + i) * kPer + sub < n ? from : last, sl,
                                    p.rot, cs + r * pitch);
        use((k + i) * kPer + sub, x);
      }
    }
  };
  for (int it = warp; it < units * shares; it += kWarps) {
    const int share = it / units, u = it - share * units;
    float a = 0.f;
    bool inf = false;
    walk(u, trips * share / shares, trips * (share + 1) / shares, [&](int, const Eight& x) { a = fmaxf(a, magnitude(x, inf)); });
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(a));   // (not negative: ordered as integers)
    if (lane == 0) atomicMax(&sh.max[u], top);
    if (inf) sh.inf[u] = 1;
  }
  __syncthreads();
  if ((int)threadIdx.x < units) {
    const float need = pow2_scale(__uint_as_float(sh.max[threadIdx.x]));
    const float s = slot0 > 0 ? fmaxf(old_scale, need) : need;
    sh.scale[threadIdx.x] = s;
    sh.ratio[threadIdx.x] = slot0 > 0 && s > old_scale ? old_scale / s : 1.f;
    const int h = kv0 + ((int)threadIdx.x < nkv ? threadIdx.x : threadIdx.x - nkv);
    ((int)threadIdx.x < nkv ? p.kscale : p.vscale)[(size_t)page * p.k.heads + h] = s;
  }
  __syncthreads();
  auto slot = [&](int u, int s) -> uint8_t* {         // the head's codes of slot s
    const int h = kv0 + (u < nkv ? u : u - nkv);
    return static_cast<uint8_t*>(u < nkv ? p.k.out : p.v.out) + ((((size_t)page << shift) + s) * p.k.heads + h) * D;
  };
  // the other slots of pages that outgrew their scale: RN(code * old / new)
  for (int u = 0; u < units && slot0 > 0; ++u) {
    const float ratio = sh.ratio[u];
    if (ratio == 1.f) continue;
    for (int s = warp * kPer + sub; s < P; s += kWarps * kPer) {
      if (s >= slot0 && s < slot0 + n) continue;
      uint2* c = reinterpret_cast<uint2*>(slot(u, s) + 8 * sl);
      uint2 w = *c;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t& x = k ? w.y : w.x;
        const float2 a = values2(x), z = values2(x >> 16);
        x = codes4({a.x * ratio, a.y * ratio, z.x * ratio, z.y * ratio});
      }
      *c = w;
    }
  }
  for (int it = warp; it < units * shares; it += kWarps) {
    const int share = it / units, u = it - share * units;
    const Quads at = u < nkv ? turned_at : plain_at;
    const float s = sh.scale[u];
    const uint32_t bits = __float_as_uint(s);
    // (old scales may be others, or 2^127, whose reciprocal has no such form)
    const bool pow2 = (bits & 0x7fffffu) == 0 && bits < 254u << 23, inf = sh.inf[u] != 0;
    const float inv = __uint_as_float((254u << 23) - bits);            // 1 / s
    uint8_t* base = slot(u, slot0);
    walk(u, trips * share / shares, trips * (share + 1) / shares, [&](int r, const Eight& x) {
      float y[8];
      if (pow2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x.x[e] * inv;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x.x[e] / s;
      }
      if (inf) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (fabsf(x.x[e]) > kMaxFloat) y[e] = __int_as_float(0x7fffffff);   // (the conversion would take 448)
      }
      if (r < n) {
        uint8_t* dst = base + (unsigned)r * (unsigned)(p.k.heads * D);   // (a page's bytes are an int)
        *reinterpret_cast<uint32_t*>(dst + at.a) = codes4({y[0], y[1], y[2], y[3]});
        *reinterpret_cast<uint32_t*>(dst + at.b) = codes4({y[4], y[5], y[6], y[7]});
      }
    });
  }
}

template <int D, bool kFast, bool kInter>
__global__ void __launch_bounds__(kThreads, 4) append_fp8_kernel(const AppendFp8Params p) {
  extern __shared__ __align__(16) float2 cs[];        // [rows][rot / 2], padded to whole 16 bytes a row
  __shared__ AppendShared sh;
  const int kv_blocks = p.pages * p.head_shares;
  if ((int)blockIdx.x < kv_blocks) {
    const int id = blockIdx.x / p.head_shares;
    append_kv<D, kFast, kInter>(p, cs, sh, id, blockIdx.x - id * p.head_shares, p.head_shares);
  } else {
    const int row0 = ((int)blockIdx.x - kv_blocks) * p.q_rows;
    append_q<D, kFast, kInter>(p, cs, sh, row0, min(p.q_rows, p.rows - row0));
  }
}

template <int D, bool kFast>
cudaError_t launch_append_t(const AppendFp8Params& p, unsigned grid, size_t smem, cudaStream_t stream) {
  auto kern = p.interleaved ? append_fp8_kernel<D, kFast, true> : append_fp8_kernel<D, kFast, false>;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

bool quads(const RopeTensor& t, bool out) {
  uintptr_t b = reinterpret_cast<uintptr_t>(t.in) | (uintptr_t)(t.in_row * 2) | (uintptr_t)(t.in_head * 2);
  if (out) b |= reinterpret_cast<uintptr_t>(t.out) | (uintptr_t)(t.out_row * 2) | (uintptr_t)(t.out_head * 2);
  return t.heads == 0 || (b & 7) == 0;
}

// ------------------------------------------------------------------ expand
// One page of one sequence a block: code * scale in bf16 (exact for scales that are powers of two, else one rounding), the
// slots past the sequence's end zero, as the prefill multiplies them by weights of 0. The page of the copy is
// b * max_pages + page, which is also what the copy's block table gets. Pages that the prefill does not read are left out:
// those between the sinks' last 128-key tile and the first tile of the first query's window. Bound by the bytes (one read,
// two written a value): 28k tokens of 8 heads of 128, K and V, 172 MB, in 32 us.
template <int D>
__global__ void __launch_bounds__(kThreads) expand_fp8_kernel(const ExpandFp8Params p) {
  const int b = blockIdx.x / p.max_pages, pi = blockIdx.x - b * p.max_pages, P = p.page_size;
  const int c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1), L = __ldg(p.seqlens_k + b);
  // (the prefill skips sequences with inconsistent lengths and records them)
  if (c0 < 0 || c1 <= c0 || c1 > p.total_q || L < c1 - c0 || L > (long long)p.max_pages * P) return;
  const int t0 = pi * P;
  if (t0 >= L) return;
  if (p.window > 0) {
    const int lo = max(L - (c1 - c0) - p.window + 1, 0) / 128 * 128;
    if (t0 + P <= lo && t0 >= sink_blocks(p.sinks, 128) * 128) return;
  }
  const int copy = b * p.max_pages + pi;
  int page = __ldg(p.block_table + copy);
  if (threadIdx.x == 0) p.table[copy] = copy;
  const bool bad = page < 0 || page >= p.num_pages;
  if (bad) {
    if (threadIdx.x == 0) record_status(p.status, kStatusDeviceCheck);
    page = 0;
  }
  const int per_slot = p.Hkv * (D / 16), total = P * per_slot;   // 16 codes a step
  const int live = bad ? 0 : min(P, L - t0) * per_slot;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const uint4* src = static_cast<const uint4*>(which ? p.vcache : p.kcache) + (size_t)page * total;
    const float* sc = (which ? p.vscale : p.kscale) + (size_t)page * p.Hkv;
    uint4* dst = static_cast<uint4*>(which ? p.vout : p.kout) + (size_t)copy * total * 2;
    for (int i = threadIdx.x; i < total; i += kThreads) {
      uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (i < live) {
        const uint4 w = __ldg(src + i);
        const float s = __ldg(sc + i % per_slot / (D / 16));
        const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 a = values2(c[k]), z = values2(c[k] >> 16);
          o[2 * k] = pack_bf16x2(a.x * s, a.y * s);
          o[2 * k + 1] = pack_bf16x2(z.x * s, z.y * s);
        }
      }
      dst[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

}  // namespace

cudaError_t launch_append_fp8(const AppendFp8Params& p0, int num_sms, cudaStream_t stream) {
  AppendFp8Params p = p0;
  p.page_shift = p.page_size == 16 ? 4 : p.page_size == 32 ? 5 : p.page_size == 64 ? 6 : 7;
  p.pages = p.rows / p.page_size + 2 * p.B;            // blocks of all sequences (some have nothing to do)
  // KV heads shared out over blocks where the pages are fewer than two blocks an SM (one where a page gets a token or two:
  // 64 single tokens 6.4 us, 7.2 with two; prompts 34 with two, 38 with one and with three), one a block at least, and
  // never more than a block has room for; q: as many rows a block as leave four blocks an SM
  const int pages = std::max(1, std::min(p.pages, p.rows));
  p.head_shares = std::min(p.k.heads, ((p.rows > 2 * pages ? 2 : 1) * num_sms + pages - 1) / pages);
  p.head_shares = std::max(p.head_shares, (p.k.heads + kAppendMaxHeads - 1) / kAppendMaxHeads);
  p.q_rows = std::max(1, std::min(kAppendRows, p.rows / (4 * num_sms)));
  const int half = p.rot / 2, pitch = (half + 1) & ~1;
  p.by_half = half ? ((1ull << 42) + half - 1) / half : 0;
  const size_t smem = (size_t)std::max(std::min(p.page_size, p.rows), p.q_rows) * pitch * sizeof(float2);
  const bool fast = quads(p.q, true) && quads(p.k, false) && quads(p.v, false) && p.rot % 8 == 0;
  const long long grid = (long long)p.pages * p.head_shares + (p.q.heads ? (p.rows + p.q_rows - 1) / p.q_rows : 0);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (p.d == 128)
    return fast ? launch_append_t<128, true>(p, (unsigned)grid, smem, stream) : launch_append_t<128, false>(p, (unsigned)grid, smem, stream);
  return fast ? launch_append_t<64, true>(p, (unsigned)grid, smem, stream) : launch_append_t<64, false>(p, (unsigned)grid, smem, stream);
}

cudaError_t launch_expand_fp8(const ExpandFp8Params& p, cudaStream_t stream) {
  const unsigned grid = (unsigned)p.B * p.max_pages;   // (slots of the copy are an int)
  if (p.d == 128)
    expand_fp8_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  else
    expand_fp8_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fattn
