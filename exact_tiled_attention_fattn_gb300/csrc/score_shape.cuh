// Score shapes shared by the shaped prefill, backward, decode and key-weight kernels:
//   s = scale q.k,  s = cap tanh(s / cap),  s -= slope_h |pos - j|
// in log2 units, and the key range [lo, hi) that a query row sees.
#pragma once

#include "device_common.cuh"
#include "fattn_internal.h"

namespace fattn {

// Hardware reciprocal (MUFU); rcp(inf) = 0.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(z) = 1 - 2 r with r = 1 / (1 + e^{2z}): one exponential and one reciprocal. Its derivative is
// 1 - tanh^2 = 4 r (1 - r), which for z >= 0 keeps its relative precision where tanh saturates.
// k2z = 2 z log2(e).
__device__ __forceinline__ float tanh_r(float k2z) { return rcp_approx(1.f + ex2(k2z)); }

// The capped score of the raw product u as cap (1 - 2 r), log2 units. It is off by 2^-22 of the cap: as good as the score
// itself where |z| is above 0.5 or so, and of no use where the cap is much larger than the score (a cap of 10^6 would
// move it by 0.1). There it is the polynomial, relative 1e-7 whatever the cap is.
__device__ __forceinline__ float capped_far(const ScoreShape& s, float u) {
  return fmaf(-2.f * s.cap2, tanh_r(u * s.capk), s.cap2);
}
// A pair of capped scores, both |u| <= poly_limit: three packed FMAs and products a score, no special function.
__device__ __forceinline__ uint64_t capped_pair(const ScoreShape& s, float u0, float u1) {
  const uint64_t u2 = f2_pack(u0, u1), w2 = f2_mul(u2, u2);
  uint64_t q = f2_bits(s.poly[4]);
#pragma unroll
  for (int i = 3; i >= 0; --i) q = f2_fma(q, w2, f2_bits(s.poly[i]));
  return f2_mul(u2, q);
}
// The scores of 32 raw products of a thread, m the largest of their magnitudes.
__device__ __forceinline__ void capped_scores(const ScoreShape& s, const uint32_t (&u)[32], float m, float (&y)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) f2_unpack(capped_pair(s, __uint_as_float(u[i]), __uint_as_float(u[i + 1])), y[i], y[i + 1]);
  if (!(m <= s.poly_limit)) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (fabsf(__uint_as_float(u[i])) > s.poly_limit) y[i] = capped_far(s, __uint_as_float(u[i]));
  }
}
// n (even) raw products of each thread of a warp replaced by their capped scores (in place: with 16 of them, in the key
// weights of 32 rows, copies spill, 68 and 74 us).
template <int n>
__device__ __forceinline__ void cap_in_place(const ScoreShape& s, float (&x)[n]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < n; i += 2) m = fmax3(m, fabsf(x[i]), fabsf(x[i + 1]));
  if (__all_sync(0xffffffffu, m <= s.poly_limit)) {
#pragma unroll
    for (int i = 0; i < n; i += 2) f2_unpack(capped_pair(s, x[i], x[i + 1]), x[i], x[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < n; i += 2) {
      float y0, y1;
      f2_unpack(capped_pair(s, x[i], x[i + 1]), y0, y1);
      x[i] = fabsf(x[i]) <= s.poly_limit ? y0 : capped_far(s, x[i]);
      x[i + 1] = fabsf(x[i + 1]) <= s.poly_limit ? y1 : capped_far(s, x[i + 1]);
    }
  }
}

// Keys that the query at position pos (key coordinates; row = its index in the packed rows) sees.
// Both bounds are non-decreasing over the rows of a sequence (the ranges are required to be).
__device__ __forceinline__ int shape_lo(const ScoreShape& s, long long row, int pos) {
  int lo = 0;
  if (s.window > 0) lo = max(lo, pos - s.window + 1);
  if (s.key_begin) lo = max(lo, __ldg(s.key_begin + row));
  return lo;
}
__device__ __forceinline__ int shape_hi(const ScoreShape& s, long long row, int pos, int Lk, bool causal) {
  int hi = Lk;
  if (causal)
    hi = min(hi, pos + 1);
  else if (s.window > 0 && s.window < Lk - pos)
    hi = pos + s.window;
  if (s.key_end) hi = min(hi, max(__ldg(s.key_end + row), 0));  // (any int32: differences of bounds stay in 32 bits)
  return hi;
}

}  // namespace fattn
