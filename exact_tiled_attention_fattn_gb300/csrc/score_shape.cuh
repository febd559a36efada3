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

// tanh(z) = 1 - 2 r with r = 1 / (1 + e^{2z}): one exponential and one reciprocal. The absolute
// error is a few 2^-24 (what counts: the capped score is cap tanh(z), an exponent), where the
// hardware tanh's 2^-11 would move a score under a cap of 50 by 0.02. Its derivative is
// 1 - tanh^2 = 4 r (1 - r), which keeps its relative precision where tanh saturates.
// k2z = 2 z log2(e).
__device__ __forceinline__ float tanh_r(float k2z) { return rcp_approx(1.f + ex2(k2z)); }

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
  if (s.key_end) hi = min(hi, __ldg(s.key_end + row));
  return hi;
}

}  // namespace fattn
