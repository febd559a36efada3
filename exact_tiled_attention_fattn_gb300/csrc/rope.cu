// Rotary positions: a streaming pass over q and k (and, in the serving form, v),
// each element read and written once.
//
// A block takes a few consecutive tokens. Their angles are the same for every
// head, so the block forms the rows x rot / 2 (cos, sin) pairs once in shared
// memory and then walks the tokens' heads in units of two 16-byte accesses, the first
// ones loaded before the angles. About four units per thread (16384 tokens of 32 + 8 heads
// of 128, bf16, 336 MB: 58 us back to back, with one unit 66, with two loaded ahead 66, with four 94:
// the registers cost more blocks than the loads bring).
//
// An angle is position * frequency modulo one turn. In fp32 the product loses a
// radian's worth of digits near position 10^7 and 10^-2 near 10^5, so the frequency is
// held as a 64-bit fraction of a turn: the product with the integer position wraps
// modulo 2^64, which is the reduction, exactly, and its top 32 bits are the angle. sincospif gets what is left of it after
// the nearest quarter turn (fp32 q and k: 4e-8 off in the mean square, 5.5e-8 with the angle rounded to 24 bits as a whole).
#include "device_common.cuh"
#include "fattn_internal.h"
#include "ops_internal.h"

#include <algorithm>

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

constexpr int kMaxRows = 8;   // tokens per block
constexpr int kUnits = 4;     // aimed at per thread

// u / d for u d < 2^42 by a multiplication: m = ceil(2^42 / d).
struct Divisor {
  unsigned long long m;
  int d;
  __host__ __device__ explicit Divisor(int d_) : m(((1ull << 42) + d_ - 1) / d_), d(d_) {}
  __device__ __forceinline__ int div(int u) const { return (int)(((unsigned long long)(unsigned)u * m) >> 42); }
};

// kWide: 16-byte units (every pointer, stride and segment a multiple of 16 bytes), else
// one element (half layout) or one pair (interleaved) at a time.
// fp32: held to the 32 registers of eight blocks per SM (0: not held; interleaved, 16384 tokens of 32 + 8 heads of 128: 107 us, with
// 40 registers 117).
template <typename T, bool kInter, bool kAppend, bool kWide>
__global__ void __launch_bounds__(kRopeThreads, sizeof(T) == 4 ? 8 : 0) rope_kernel(const RopeParams p, int rows_per_block, const Divisor by_units,
                                                            const Divisor by_heads) {
  extern __shared__ __align__(16) float2 s_cs[];   // [rows_per_block][rot / 2], a row's pairs in the order of cs_at
  __shared__ long long s_dst[kMaxRows];            // serving form: each row's first element in the caches, -1: skipped
  __shared__ int s_b[kMaxRows];
  constexpr int V = kWide ? Elem<T>::kVec : 1;     // elements of an access
  constexpr int kPairs = kInter ? (kWide ? V / 2 : 1) : V;  // pairs of a unit: two accesses rot / 2 apart, or one of pairs
  constexpr int VI = kWide ? V : 2;                // elements of an interleaved unit
  using U = Unit<T, kInter ? VI : V, kWide>;
  using UC = Unit<T, V, kWide>;
  const int half = p.rot >> 1;
  const int nrot = half / kPairs;                  // rotated units per head
  const int row0 = blockIdx.x * rows_per_block;
  const int nrows = min(rows_per_block, p.rows - row0);
  // place of pair i of a row: the units' first two pairs side by side, then their next two, ..., so that
  // neighbouring lanes (neighbouring units) read neighbouring 16 bytes
  auto cs_at = [&](int unit, int e) -> int { return kPairs > 1 ? ((e >> 1) * nrot + unit) * 2 + (e & 1) : unit; };

  if constexpr (kAppend) {
    // the sequence that each row belongs to: every thread tests its own sequences
    if (threadIdx.x < kMaxRows) {
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
    if ((int)threadIdx.x < nrows && s_b[threadIdx.x] >= 0) {
      const int b = s_b[threadIdx.x];
      const long long t = (long long)__ldg(p.seqlens_k + b) - __ldg(p.cu_seqlens + b + 1) + row0 + threadIdx.x;
      bool ok = t >= 0 && t < (long long)p.max_pages * p.page_size;
      if (ok) {
        const int page = __ldg(p.block_table + (size_t)b * p.max_pages + t / p.page_size);
        ok = page >= 0 && page < p.num_pages;
        if (ok) s_dst[threadIdx.x] = ((long long)page * p.page_size + t % p.page_size) * p.k.heads * p.d;
      }
      if (!ok) record_status(p.status, kStatusDeviceCheck);
    }
  }

  // units per head, the copied ones last: two accesses half of the rest apart where that is possible, as the
  // rotated ones are
  const int rest = p.d - p.rot;
  const int apart = !kInter && rest % (2 * V) == 0 ? rest / 2 : 0;
  const int nu = nrot + (apart ? apart : rest) / V;
  const int heads = p.q.heads + p.k.heads + (kAppend ? p.v.heads : 0);
  const int total = nrows * heads * nu;
  struct Place {
    const T* src;
    T* dst;
    int r, c;       // row of the block, unit of the head (>= nrot: copied)
    bool turn, live;
  };
  auto place = [&](int u) -> Place {
    Place x;
    x.live = u < total;
    u = x.live ? u : 0;    // (addresses of a unit that exists; it is not accessed)
    const int rh = by_units.div(u);
    x.c = u - rh * nu;
    x.r = by_heads.div(rh);
    int h = rh - x.r * heads;
    const RopeTensor* t = &p.q;
    x.turn = x.c < nrot;
    bool cache = false;
    if (h >= p.q.heads) {
      h -= p.q.heads;
      t = &p.k;
      cache = kAppend;
      if (kAppend && h >= p.k.heads) {
        h -= p.k.heads;
        t = &p.v;
        x.turn = false;
      }
    }
    if (kAppend && s_dst[x.r] < 0) x.live = false;
    const long long row = row0 + x.r;
    x.src = static_cast<const T*>(t->in) + row * t->in_row + h * t->in_head;
    x.dst = static_cast<T*>(t->out) + (cache ? s_dst[x.r] : row * t->out_row) + h * t->out_head;
    return x;
  };
  auto fetch = [&](const Place& x, U& a, U& b) {
    if (!x.live) return;
    if (x.c < nrot) {
      a = *reinterpret_cast<const U*>(x.src + x.c * (kInter ? VI : V));
      if constexpr (!kInter) b = *reinterpret_cast<const U*>(x.src + half + x.c * V);
    } else {
      const T* src = x.src + p.rot + (x.c - nrot) * V;
      const UC y = *reinterpret_cast<const UC*>(src);
#pragma unroll
      for (int e = 0; e < V; ++e) a.e[e] = y.e[e];
      if constexpr (!kInter) {
        if (apart) b = *reinterpret_cast<const U*>(src + apart);
      }
    }
  };
  auto finish = [&](const Place& x, U& a, U& b) {
    if (!x.live) return;
    if (x.c >= nrot) {
      UC y;
#pragma unroll
      for (int e = 0; e < V; ++e) y.e[e] = a.e[e];
      T* dst = x.dst + p.rot + (x.c - nrot) * V;
      *reinterpret_cast<UC*>(dst) = y;
      if constexpr (!kInter) {
        if (apart) *reinterpret_cast<U*>(dst + apart) = b;
      }
      return;
    }
    if (x.turn) {
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const float2 w = s_cs[x.r * half + cs_at(x.c, e)];
        T& ta = kInter ? a.e[2 * e] : a.e[e];
        T& tb = kInter ? a.e[2 * e + 1] : b.e[e];
        const float fa = Elem<T>::get(ta), fb = Elem<T>::get(tb);
        ta = Elem<T>::put(fa * w.x - fb * w.y);
        tb = Elem<T>::put(fb * w.x + fa * w.y);
      }
    }
    *reinterpret_cast<U*>(x.dst + x.c * (kInter ? VI : V)) = a;
    if constexpr (!kInter) *reinterpret_cast<U*>(x.dst + half + x.c * V) = b;
  };
  if (kAppend) __syncthreads();   // s_dst
  U a, b;
  Place x = place(threadIdx.x);
  fetch(x, a, b);

  // a thread's pairs, and for each of them the block's rows (the frequency is converted once)
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    double turns = __ldg(p.inv_freq + i) * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= floor(turns);
    const unsigned long long f = (unsigned long long)(turns * 18446744073709551616.0);
    const int at = cs_at(i / kPairs, i % kPairs);
    for (int r = 0; r < nrows; ++r) {
      long long pos;
      if (p.positions) {
        pos = __ldg(p.positions + row0 + r);
      } else if constexpr (kAppend) {
        const int sb = s_b[r];
        pos = sb < 0 ? 0 : (long long)__ldg(p.seqlens_k + sb) - __ldg(p.cu_seqlens + sb + 1) + row0 + r;
      } else {
        pos = (row0 + r) % p.period;
      }
      const float2 w = turn_of((long long)(f * (unsigned long long)pos), p.amplitude);
      s_cs[r * half + at] = make_float2(w.x, p.inverse ? -w.y : w.y);
    }
  }
  __syncthreads();

  for (int u = threadIdx.x;;) {
    finish(x, a, b);
    u += kRopeThreads;
    if (u >= total) break;
    x = place(u);
    fetch(x, a, b);
  }
}

// Whether 16-byte units fit the tensor's pointers and strides (el = bytes per element).
bool wide_ok(const RopeTensor& t, int el) {
  if (t.heads == 0) return true;
  const long long b = reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out);
  return ((b | (t.in_row * el) | (t.in_head * el) | (t.out_row * el) | (t.out_head * el)) & 15) == 0;
}

template <typename T, bool kInter, bool kAppend>
cudaError_t launch_rope_t(const RopeParams& p, int num_sms, cudaStream_t stream) {
  constexpr int el = sizeof(T);
  const int seg = kInter ? p.rot : p.rot / 2;   // contiguous rotated elements
  const bool wide = wide_ok(p.q, el) && wide_ok(p.k, el) && wide_ok(p.v, el) && (seg * el) % 16 == 0 &&
                    ((p.d - p.rot) * el) % 16 == 0;
  const int vec = wide ? 16 / el : 1, pairs = kInter ? (wide ? vec / 2 : 1) : vec;
  const int heads = p.q.heads + p.k.heads + (kAppend ? p.v.heads : 0);
  const int rest = p.d - p.rot;
  const int units = p.rot / 2 / pairs + (!kInter && rest % (2 * vec) == 0 ? rest / 2 : rest) / vec;  // (as the kernel counts)
  // kUnits per thread where there are rows enough for eight blocks per SM, one row at the least (short calls:
  // the more blocks the shorter)
  long long rows = ((long long)kUnits * kRopeThreads + (long long)heads * units - 1) / ((long long)heads * units);
  rows = std::min<long long>({rows, kMaxRows, std::max<long long>(1, p.rows / (num_sms * 8ll))});
  const int rows_per_block = (int)rows;
  const int grid = (int)(((long long)p.rows + rows - 1) / rows);
  const size_t smem = (size_t)rows_per_block * (p.rot / 2) * sizeof(float2);
  const Divisor by_units(units), by_heads(heads);
  if (wide)
    rope_kernel<T, kInter, kAppend, true><<<grid, kRopeThreads, smem, stream>>>(p, rows_per_block, by_units, by_heads);
  else
    rope_kernel<T, kInter, kAppend, false><<<grid, kRopeThreads, smem, stream>>>(p, rows_per_block, by_units, by_heads);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool bf16, bool interleaved, bool append, int num_sms, cudaStream_t stream) {
  using B = __nv_bfloat16;
  if (append)
    return interleaved ? launch_rope_t<B, true, true>(p, num_sms, stream) : launch_rope_t<B, false, true>(p, num_sms, stream);
  if (bf16)
    return interleaved ? launch_rope_t<B, true, false>(p, num_sms, stream)
                       : launch_rope_t<B, false, false>(p, num_sms, stream);
  return interleaved ? launch_rope_t<float, true, false>(p, num_sms, stream)
                     : launch_rope_t<float, false, false>(p, num_sms, stream);
}

}  // namespace fattn
