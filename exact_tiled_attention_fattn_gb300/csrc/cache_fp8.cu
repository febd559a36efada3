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
// A block takes one page of one sequence, as far as the call's new tokens reach into it, and a share of the heads: KV head h
// of a page is worked on by this block alone, so its scale and the old codes change without atomics on global memory. The
// rows' angles are formed once in shared memory (as in rope.cu, 64-bit fixed point); a warp then takes a row of one head at
// a time, four elements a lane, the other halves of its pairs from the lane that has them. Per page: the magnitudes of K
// and V (shared-memory maxima), q rotated meanwhile, the scales, old codes of pages that outgrew theirs, and K and V
// again (from the L1 cache) into codes. Bound by the bytes of q, k and v for prompts, by the chain of loads for single tokens.
//
// kFast: 8-byte aligned rows and heads, and pairs that never split a lane's four elements; else element by element.
struct Row4 {
  float x[4];
};

template <bool kFast>
__device__ __forceinline__ Row4 load4(const __nv_bfloat16* p, int e) {
  Row4 r;
  if constexpr (kFast) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p + e));
    r.x[0] = bf16_lo(w.x), r.x[1] = bf16_hi(w.x), r.x[2] = bf16_lo(w.y), r.x[3] = bf16_hi(w.y);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.x[i] = __bfloat162float(p[e + i]);
  }
  return r;
}

// The lane's four elements e .. e + 3 of a row turned by the row's (cos, sin) table.
template <bool kFast, bool kInter>
__device__ __forceinline__ void turn4(Row4& r, const __nv_bfloat16* p, int e, int rot, const float2* cs, int lane) {
  const int half = rot >> 1;
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      if (e + i >= rot) break;       // (rot is even: pairs are whole)
      const float2 w = cs[(e + i) >> 1];
      const float a = r.x[i], b = r.x[i + 1];
      r.x[i] = a * w.x - b * w.y;
      r.x[i + 1] = b * w.x + a * w.y;
    }
  } else if constexpr (kFast) {
    const bool low = e < half;
    const int other = lane + (low ? half : -half) / 4;
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(0xffffffffu, r.x[i], other & 31);
    if (e < rot) {
      const float4* c4 = reinterpret_cast<const float4*>(cs + (low ? e : e - half));
      const float4 w0 = c4[0], w1 = c4[1];
      const float c[4] = {w0.x, w0.z, w1.x, w1.z}, s[4] = {w0.y, w0.w, w1.y, w1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) r.x[i] = low ? r.x[i] * c[i] - o[i] * s[i] : r.x[i] * c[i] + o[i] * s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e + i >= rot) break;
      const bool low = e + i < half;
      const float2 w = cs[low ? e + i : e + i - half];
      const float o = __bfloat162float(p[low ? e + i + half : e + i - half]);
      r.x[i] = low ? r.x[i] * w.x - o * w.y : r.x[i] * w.x + o * w.y;
    }
  }
}

__device__ __forceinline__ float magnitude(float x) {   // infinities and NaN do not decide a scale
  const float a = fabsf(x);
  return a <= 3.4028235e38f ? a : 0.f;
}

template <int D, bool kFast, bool kInter>
__global__ void __launch_bounds__(kThreads) append_fp8_kernel(const AppendFp8Params p) {
  extern __shared__ __align__(16) float2 s_cs[];      // [rows][rot / 2], padded to whole 16 bytes a row
  __shared__ uint32_t s_max[2 * kAppendMaxHeads];     // magnitudes (bits) of the block's KV heads: K, then V
  __shared__ float s_scale[2 * kAppendMaxHeads], s_ratio[2 * kAppendMaxHeads];
  __shared__ int s_b;
  constexpr int kLanes = D / 4;                       // lanes of a row
  constexpr int kPer = 32 / kLanes;                   // rows a warp takes at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = p.page_size;

  // the block's sequence: sequence b has the blocks from cu[b] / P + 2 b on (it touches at most Lq / P + 2 pages)
  if (threadIdx.x == 0) s_b = -1;
  __syncthreads();
  const int id = blockIdx.x;
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const int c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1);
    if (c0 < 0 || c1 < c0 || c1 > p.rows) {
      if (id == 0) record_status(p.status, kStatusDeviceCheck);
    } else if (id >= c0 / P + 2 * b && id < c1 / P + 2 * (b + 1)) {
      s_b = b;
    }
  }
  __syncthreads();
  const int b = s_b;
  if (b < 0) return;
  const int c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1);
  const int end = __ldg(p.seqlens_k + b);             // tokens [start, end) are new
  const long long start = (long long)end - (c1 - c0), cap = (long long)p.max_pages * P;
  const int local = id - (c0 / P + 2 * b);
  if (local == 0 && blockIdx.y == 0 && threadIdx.x == 0 && c1 > c0 && (start < 0 || end > cap))
    record_status(p.status, kStatusDeviceCheck);      // rows outside the table are skipped
  const long long first = max(start, 0ll);
  const long long pi = first / P + local;
  const long long t0 = max(first, pi * P), t1 = min(min((long long)end, cap), (pi + 1) * P);
  if (t0 >= t1) return;
  const int page = __ldg(p.block_table + (size_t)b * p.max_pages + pi);
  if (page < 0 || page >= p.num_pages) {
    if (blockIdx.y == 0 && threadIdx.x == 0) record_status(p.status, kStatusDeviceCheck);
    return;
  }
  const int n = (int)(t1 - t0), slot0 = (int)(t0 - pi * P);
  const int row0 = c0 + (int)(t0 - start);            // packed row of token t0
  const int half = p.rot >> 1, pitch = (half + 1) & ~1;
  // the block's heads
  const int kv0 = (int)((long long)p.k.heads * blockIdx.y / gridDim.y), kv1 = (int)((long long)p.k.heads * (blockIdx.y + 1) / gridDim.y);
  const int q0 = (int)((long long)p.q.heads * blockIdx.y / gridDim.y), q1 = (int)((long long)p.q.heads * (blockIdx.y + 1) / gridDim.y);
  const int nkv = kv1 - kv0, nq = q1 - q0;
  float old_scale = 0.f;                              // of thread u < 2 nkv's unit
  if ((int)threadIdx.x < 2 * nkv) {
    s_max[threadIdx.x] = 0;
    const int h = kv0 + ((int)threadIdx.x < nkv ? threadIdx.x : threadIdx.x - nkv);
    if (slot0 > 0) old_scale = ((int)threadIdx.x < nkv ? p.kscale : p.vscale)[(size_t)page * p.k.heads + h];
  }
  for (int i = threadIdx.x; i < half; i += kThreads) {
    double turns = __ldg(p.inv_freq + i) * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= floor(turns);
    const unsigned long long f = (unsigned long long)(turns * 18446744073709551616.0);
    for (int r = 0; r < n; ++r) {
      const long long pos = p.positions ? (long long)__ldg(p.positions + row0 + r) : t0 + r;
      s_cs[r * pitch + i] = turn_of((long long)(f * (unsigned long long)pos), p.amplitude);
    }
  }
  __syncthreads();

  const int sub = lane / kLanes, e = (lane % kLanes) * 4;
  const int units = 2 * nkv * n;                      // (head of K or V, row), rows innermost
  auto unit = [&](int idx, int& u, int& r) -> const __nv_bfloat16* {
    u = idx / n;
    r = idx - u * n;
    const RopeTensor& t = u < nkv ? p.k : p.v;
    const int h = kv0 + (u < nkv ? u : u - nkv);
    return static_cast<const __nv_bfloat16*>(t.in) + (long long)(row0 + r) * t.in_row + h * t.in_head;
  };
  // the four elements of unit idx that the lane has, rotated (K) or as they are (V); all lanes of the warp call it
  auto value = [&](int idx, int& u, int& r) -> Row4 {
    const __nv_bfloat16* src = unit(idx, u, r);
    Row4 x = load4<kFast>(src, e);
    const bool key = u < nkv;
    if (__any_sync(0xffffffffu, key)) {
      Row4 y = x;
      turn4<kFast, kInter>(y, src, e, p.rot, s_cs + r * pitch, lane);
      if (key) x = y;
    }
    return x;
  };
  for (int i = warp * kPer + sub; i - sub < units; i += kWarps * kPer) {
    int u, r;
    const bool live = i < units;
    const Row4 x = value(live ? i : units - 1, u, r);
    float a = fmaxf(fmaxf(magnitude(x.x[0]), magnitude(x.x[1])), fmaxf(magnitude(x.x[2]), magnitude(x.x[3])));
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
    if (live && e == 0) atomicMax(&s_max[u], __float_as_uint(a));
  }
  // q meanwhile, heads innermost
  for (int i = warp * kPer + sub; i - sub < nq * n; i += kWarps * kPer) {
    const bool live = i < nq * n;
    const int j = live ? i : 0, r = j / nq, h = q0 + (j - r * nq);
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q.in) + (long long)(row0 + r) * p.q.in_row + h * p.q.in_head;
    Row4 x = load4<kFast>(src, e);
    turn4<kFast, kInter>(x, src, e, p.rot, s_cs + r * pitch, lane);
    if (live) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q.out) + (long long)(row0 + r) * p.q.out_row + h * p.q.out_head + e;
      if constexpr (kFast) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x.x[0], x.x[1]), pack_bf16x2(x.x[2], x.x[3]));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[k] = __float2bfloat16_rn(x.x[k]);
      }
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < 2 * nkv) {
    const float need = pow2_scale(__uint_as_float(s_max[threadIdx.x]));
    const float s = slot0 > 0 ? fmaxf(old_scale, need) : need;
    s_scale[threadIdx.x] = s;
    s_ratio[threadIdx.x] = slot0 > 0 && s > old_scale ? old_scale / s : 1.f;
    const int h = kv0 + ((int)threadIdx.x < nkv ? threadIdx.x : threadIdx.x - nkv);
    ((int)threadIdx.x < nkv ? p.kscale : p.vscale)[(size_t)page * p.k.heads + h] = s;
  }
  __syncthreads();
  auto slot = [&](int u, int s) -> uint32_t* {        // four codes of slot s
    const int h = kv0 + (u < nkv ? u : u - nkv);
    uint8_t* base = static_cast<uint8_t*>(u < nkv ? p.k.out : p.v.out);
    return reinterpret_cast<uint32_t*>(base + (((size_t)page * P + s) * p.k.heads + h) * D + e);
  };
  // the other slots of pages that outgrew their scale: RN(code * old / new)
  for (int u = 0; u < 2 * nkv && slot0 > 0; ++u) {
    const float ratio = s_ratio[u];
    if (ratio == 1.f) continue;
    for (int s = warp * kPer + sub; s < P; s += kWarps * kPer) {
      if (s >= slot0 && s < slot0 + n) continue;
      uint32_t* c = slot(u, s);
      const uint32_t w = *c;
      const float2 a = values2(w), z = values2(w >> 16);
      *c = codes4({a.x * ratio, a.y * ratio, z.x * ratio, z.y * ratio});
    }
  }
  for (int i = warp * kPer + sub; i - sub < units; i += kWarps * kPer) {
    int u, r;
    const bool live = i < units;
    const Row4 x = value(live ? i : units - 1, u, r);
    const float s = s_scale[u];
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = fabsf(x.x[k]) <= 3.4028235e38f ? x.x[k] / s : __int_as_float(0x7fffffff);
    if (live) *slot(u, slot0 + r) = codes4(y);
  }
}

template <int D, bool kFast>
cudaError_t launch_append_t(const AppendFp8Params& p, dim3 grid, size_t smem, cudaStream_t stream) {
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
// two written a value): 2 x 16384 tokens of 8 heads of 128, K and V, in about 35 us.
template <int D>
__global__ void __launch_bounds__(kThreads) expand_fp8_kernel(const ExpandFp8Params p) {
  const int b = blockIdx.y, pi = blockIdx.x, P = p.page_size;
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

cudaError_t launch_append_fp8(const AppendFp8Params& p, int num_sms, cudaStream_t stream) {
  const int ids = p.rows / p.page_size + 2 * p.B;      // blocks of all sequences (some have nothing to do)
  // heads shared out over blocks where pages alone are fewer than four blocks an SM, one KV head a block at least, and never
  // more KV heads a block than it has room for
  const int pages = std::max(1, std::min(ids, p.rows));
  int ny = std::min(p.k.heads, (4 * num_sms + pages - 1) / pages);
  ny = std::max(ny, (p.k.heads + kAppendMaxHeads - 1) / kAppendMaxHeads);
  const int half = p.rot / 2, pitch = (half + 1) & ~1;
  const size_t smem = (size_t)std::min(p.page_size, p.rows) * pitch * sizeof(float2);
  const bool fast = quads(p.q, true) && quads(p.k, false) && quads(p.v, false) && p.rot % (p.interleaved ? 4 : 8) == 0;
  const dim3 grid(ids, ny);
  if (p.d == 128) return fast ? launch_append_t<128, true>(p, grid, smem, stream) : launch_append_t<128, false>(p, grid, smem, stream);
  return fast ? launch_append_t<64, true>(p, grid, smem, stream) : launch_append_t<64, false>(p, grid, smem, stream);
}

cudaError_t launch_expand_fp8(const ExpandFp8Params& p, cudaStream_t stream) {
  const dim3 grid(p.max_pages, p.B);
  if (p.d == 128)
    expand_fp8_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  else
    expand_fp8_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fattn
