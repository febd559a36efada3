// Rotary positions: a streaming pass over q and k (and, in the serving form, v),
// each element read and written once.
//
// A block takes kRows consecutive tokens. Their angles are the same for every
// head, so the block forms the kRows x rot / 2 (cos, sin) pairs once in shared
// memory and then walks the tokens' heads in 16-byte units.
//
// An angle is position * frequency modulo one turn. In fp32 the product loses a
// radian's worth of digits near position 10^7 and 10^-2 near 10^5, so the frequency is
// held as a 64-bit fraction of a turn: the product with the integer position wraps
// modulo 2^64, which is the reduction, exactly, and its top 32 bits are the angle.
#include "device_common.cuh"
#include "fattn_internal.h"
#include "ops_internal.h"

namespace fattn {
namespace {

constexpr int kRopeThreads = 256;

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};

// V elements moved together: one 16-byte access, or (narrow form) element by element, as
// an odd stride puts a pair anywhere.
template <typename T, int V, bool kWide>
struct alignas(kWide ? 16 : sizeof(T)) Unit {
  T e[V];
};

// kWide: 16-byte units (every pointer, stride and segment a multiple of 16 bytes), else
// one element (half layout) or one pair (interleaved) at a time.
template <typename T, bool kInter, bool kAppend, bool kWide>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int rows_per_block) {
  extern __shared__ float2 s_cs[];  // [rows_per_block][rot / 2]
  __shared__ long long s_dst[8];    // serving form: each row's first element in the caches, -1: skipped
  __shared__ int s_b[8];
  constexpr int V = kWide ? Elem<T>::kVec : 1;
  // elements of one rotated unit: two units V apart by rot / 2, or one unit of pairs
  constexpr int VI = kWide ? Elem<T>::kVec : 2;
  const int half = p.rot >> 1;
  const int row0 = blockIdx.x * rows_per_block;
  const int nrows = min(rows_per_block, p.rows - row0);

  if constexpr (kAppend) {
    // the sequence that each row belongs to: every thread tests its own sequences
    if (threadIdx.x < 8) {
      s_b[threadIdx.x] = -1;
      s_dst[threadIdx.x] = -1;
    }
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += kRopeThreads) {
      const int c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1);
      for (int r = 0; r < nrows; ++r)
        if (row0 + r >= c0 && row0 + r < c1) s_b[r] = b;
    }
    __syncthreads();
  }
  for (int idx = threadIdx.x; idx < nrows * half || (kAppend && idx < nrows); idx += kRopeThreads) {
    if constexpr (kAppend) {
      if (idx < nrows && s_b[idx] >= 0) {
        const int b = s_b[idx];
        const long long t = (long long)__ldg(p.seqlens_k + b) - __ldg(p.cu_seqlens + b + 1) + row0 + idx;
        bool ok = t >= 0 && t < (long long)p.max_pages * p.page_size;
        if (ok) {
          const int page = __ldg(p.block_table + (size_t)b * p.max_pages + t / p.page_size);
          ok = page >= 0 && page < p.num_pages;
          if (ok) s_dst[idx] = ((long long)page * p.page_size + t % p.page_size) * p.k.heads * p.d;
        }
        if (!ok) record_status(p.status, kStatusDeviceCheck);
      }
    }
    if (idx < nrows * half) {
      const int r = idx / half, i = idx - r * half;
      long long pos;
      if (p.positions) {
        pos = __ldg(p.positions + row0 + r);
      } else if constexpr (kAppend) {
        const int b = s_b[r];
        pos = b < 0 ? 0 : (long long)__ldg(p.seqlens_k + b) - __ldg(p.cu_seqlens + b + 1) + row0 + r;
      } else {
        pos = (row0 + r) % p.period;
      }
      double turns = __ldg(p.inv_freq + i) * 0.15915494309189533577;  // 1 / (2 pi)
      turns -= floor(turns);
      const unsigned long long f = (unsigned long long)(turns * 18446744073709551616.0);
      const long long a = (long long)(f * (unsigned long long)pos);   // turns * 2^64, wrapped
      float sn, cs;
      sincospif((float)(int)(a >> 32) * (1.f / 2147483648.f), &sn, &cs);
      s_cs[idx] = make_float2(cs * p.amplitude, (p.inverse ? -sn : sn) * p.amplitude);
    }
  }
  __syncthreads();

  const int nrot = kInter ? p.rot / VI : half / V;          // rotated units per head
  const int nu = nrot + (p.d - p.rot) / V;                  // and copied ones
  const int heads = p.q.heads + p.k.heads + (kAppend ? p.v.heads : 0);
  const int total = nrows * heads * nu;
  for (int u = threadIdx.x; u < total; u += kRopeThreads) {
    const int rh = u / nu, c = u - rh * nu;
    const int r = rh / heads;
    int h = rh - r * heads;
    const RopeTensor* t = &p.q;
    bool turn = true;
    bool cache = false;
    if (h >= p.q.heads) {
      h -= p.q.heads;
      t = &p.k;
      cache = kAppend;
      if (kAppend && h >= p.k.heads) {
        h -= p.k.heads;
        t = &p.v;
        turn = false;
      }
    }
    if (kAppend && s_dst[r] < 0) continue;
    const long long row = row0 + r;
    const T* src = static_cast<const T*>(t->in) + row * t->in_row + h * t->in_head;
    T* dst = static_cast<T*>(t->out) + (cache ? s_dst[r] : row * t->out_row) + h * t->out_head;
    if (c < nrot) {
      if constexpr (kInter) {
        using U = Unit<T, VI, kWide>;
        U x = *reinterpret_cast<const U*>(src + c * VI);
        if (turn) {
#pragma unroll
          for (int e = 0; e < VI; e += 2) {
            const float2 w = s_cs[r * half + (c * VI + e) / 2];
            const float a = Elem<T>::get(x.e[e]), b = Elem<T>::get(x.e[e + 1]);
            x.e[e] = Elem<T>::put(a * w.x - b * w.y);
            x.e[e + 1] = Elem<T>::put(b * w.x + a * w.y);
          }
        }
        *reinterpret_cast<U*>(dst + c * VI) = x;
      } else {
        using U = Unit<T, V, kWide>;
        U x = *reinterpret_cast<const U*>(src + c * V), y = *reinterpret_cast<const U*>(src + half + c * V);
        if (turn) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 w = s_cs[r * half + c * V + e];
            const float a = Elem<T>::get(x.e[e]), b = Elem<T>::get(y.e[e]);
            x.e[e] = Elem<T>::put(a * w.x - b * w.y);
            y.e[e] = Elem<T>::put(b * w.x + a * w.y);
          }
        }
        *reinterpret_cast<U*>(dst + c * V) = x;
        *reinterpret_cast<U*>(dst + half + c * V) = y;
      }
    } else {
      using U = Unit<T, V, kWide>;
      const int o = p.rot + (c - nrot) * V;
      *reinterpret_cast<U*>(dst + o) = *reinterpret_cast<const U*>(src + o);
    }
  }
}

// Whether 16-byte units fit the tensor's pointers and strides (el = bytes per element).
bool wide_ok(const RopeTensor& t, int el) {
  if (t.heads == 0) return true;
  const long long b = reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out);
  return ((b | (t.in_row * el) | (t.in_head * el) | (t.out_row * el) | (t.out_head * el)) & 15) == 0;
}

template <typename T, bool kInter, bool kAppend>
cudaError_t launch_rope_t(const RopeParams& p, cudaStream_t stream) {
  constexpr int el = sizeof(T);
  const int seg = kInter ? p.rot : p.rot / 2;   // contiguous rotated elements
  const bool wide = wide_ok(p.q, el) && wide_ok(p.k, el) && wide_ok(p.v, el) && (seg * el) % 16 == 0 &&
                    ((p.d - p.rot) * el) % 16 == 0;
  const int rows_per_block = 1;
  const int grid = (p.rows + rows_per_block - 1) / rows_per_block;
  const size_t smem = (size_t)rows_per_block * (p.rot / 2) * sizeof(float2);
  if (wide)
    rope_kernel<T, kInter, kAppend, true><<<grid, kRopeThreads, smem, stream>>>(p, rows_per_block);
  else
    rope_kernel<T, kInter, kAppend, false><<<grid, kRopeThreads, smem, stream>>>(p, rows_per_block);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool bf16, bool interleaved, bool append, cudaStream_t stream) {
  using B = __nv_bfloat16;
  if (append) return interleaved ? launch_rope_t<B, true, true>(p, stream) : launch_rope_t<B, false, true>(p, stream);
  if (bf16) return interleaved ? launch_rope_t<B, true, false>(p, stream) : launch_rope_t<B, false, false>(p, stream);
  return interleaved ? launch_rope_t<float, true, false>(p, stream) : launch_rope_t<float, false, false>(p, stream);
}

}  // namespace fattn
