// Entry points of include/fattn_ops.h: argument checks and dispatch.
#include "fattn_ops.h"
#include "fattn_internal.h"
#include "ops_internal.h"

#include <cmath>

using namespace fattn;

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Checks that fattn_rope and fattn_rope_append_paged share.
static fattn_status check_rotary(const double* inv_freq, int rows, int Hq, int Hk, int d, int rotary_dim,
                                 float amplitude) {
  if (rows < 0 || Hq < 0 || Hk < 0 || d <= 0 || rotary_dim < 0 || rotary_dim > d || (rotary_dim & 1))
    return FATTN_ERR_INVALID_ARG;
  if (!std::isfinite(amplitude)) return FATTN_ERR_INVALID_ARG;
  if (rows > 0 && rotary_dim > 0 && (!inv_freq || misaligned(inv_freq, 8))) return FATTN_ERR_INVALID_ARG;
  if (d > 1024 || (long long)Hq + Hk > 4096) return FATTN_ERR_UNSUPPORTED;
  return FATTN_OK;
}

extern "C" fattn_status fattn_rope(const void* q, void* q_out, const void* k, void* k_out, const int32_t* positions,
                                   int period, const double* inv_freq, int rows, int Hq, int Hk, int d,
                                   int rotary_dim, long long q_row, long long q_head, long long qo_row,
                                   long long qo_head, long long k_row, long long k_head, long long ko_row,
                                   long long ko_head, int interleaved, int inverse, float amplitude, fattn_dtype dtype,
                                   cudaStream_t stream) {
  const fattn_status st = check_rotary(inv_freq, rows, Hq, Hk, d, rotary_dim, amplitude);
  if (st != FATTN_OK) return st;
  if (dtype != FATTN_BF16 && dtype != FATTN_FP32) return FATTN_ERR_INVALID_ARG;
  if ((k == nullptr) != (k_out == nullptr) || (Hk > 0) != (k != nullptr)) {
    if (rows > 0) return FATTN_ERR_INVALID_ARG;
  }
  if (q_row < 0 || q_head < 0 || qo_row < 0 || qo_head < 0 || k_row < 0 || k_head < 0 || ko_row < 0 || ko_head < 0)
    return FATTN_ERR_INVALID_ARG;
  if (rows == 0) return FATTN_OK;
  const uintptr_t el = dtype == FATTN_BF16 ? 2 : 4;
  if (Hq <= 0 || !q || !q_out || misaligned(q, el) || misaligned(q_out, el) || misaligned(k, el) ||
      misaligned(k_out, el) || misaligned(positions, 4) || (!positions && period <= 0))
    return FATTN_ERR_INVALID_ARG;
  RopeParams p{};
  p.q = {q, q_out, Hq, q_row, q_head, qo_row, qo_head};
  p.k = {k, k_out, Hk, k_row, k_head, ko_row, ko_head};
  p.positions = positions; p.inv_freq = inv_freq; p.period = period;
  p.rows = rows; p.d = d; p.rot = rotary_dim; p.inverse = inverse ? 1 : 0; p.amplitude = amplitude;
  const int sms = num_sms_current();
  if (sms <= 0) return FATTN_ERR_CUDA;
  return launch_rope(p, dtype == FATTN_BF16, interleaved != 0, false, sms, stream) == cudaSuccess ? FATTN_OK
                                                                                                 : FATTN_ERR_CUDA;
}

extern "C" fattn_status fattn_rope_append_paged(const void* q, void* q_out, const void* k, const void* v, void* kcache,
                                                void* vcache, const int32_t* block_table, const int32_t* seqlens_k,
                                                const int32_t* cu_seqlens_q, const int32_t* positions,
                                                const double* inv_freq, int B, int total_q, int Hq, int Hkv, int d,
                                                int rotary_dim, int page_size, int max_pages_per_seq, int num_pages,
                                                long long q_row, long long q_head, long long k_row, long long k_head,
                                                long long v_row, long long v_head, int interleaved, float amplitude,
                                                cudaStream_t stream) {
  const fattn_status st = check_rotary(inv_freq, total_q, q ? Hq : 0, Hkv, d, rotary_dim, amplitude);
  if (st != FATTN_OK) return st;
  if (B < 0 || Hkv <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0) return FATTN_ERR_INVALID_ARG;
  if (q_row < 0 || q_head < 0 || k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0) return FATTN_ERR_INVALID_ARG;
  if ((long long)max_pages_per_seq * page_size > 0x7fffffffLL) return FATTN_ERR_UNSUPPORTED;
  if (B == 0 || total_q == 0) return FATTN_OK;
  if ((q != nullptr) != (q_out != nullptr) || (q && Hq <= 0)) return FATTN_ERR_INVALID_ARG;
  if (!k || !v || !kcache || !vcache || !block_table || !seqlens_k || !cu_seqlens_q) return FATTN_ERR_INVALID_ARG;
  if (misaligned(q, 2) || misaligned(q_out, 2) || misaligned(k, 2) || misaligned(v, 2) || misaligned(kcache, 2) ||
      misaligned(vcache, 2) || misaligned(block_table, 4) || misaligned(seqlens_k, 4) || misaligned(cu_seqlens_q, 4) ||
      misaligned(positions, 4))
    return FATTN_ERR_INVALID_ARG;
  int err = 0;
  RopeParams p{};
  p.q = {q, q_out, q ? Hq : 0, q_row, q_head, (long long)Hq * d, d};
  p.k = {k, kcache, Hkv, k_row, k_head, (long long)Hkv * d, d};
  p.v = {v, vcache, Hkv, v_row, v_head, (long long)Hkv * d, d};
  p.positions = positions; p.inv_freq = inv_freq; p.period = 1;
  p.rows = total_q; p.d = d; p.rot = rotary_dim; p.amplitude = amplitude;
  p.cu_seqlens = cu_seqlens_q; p.seqlens_k = seqlens_k; p.block_table = block_table;
  p.B = B; p.page_size = page_size; p.max_pages = max_pages_per_seq; p.num_pages = num_pages;
  p.status = status_ptr(&err);
  if (err) return FATTN_ERR_CUDA;
  const int sms = num_sms_current();
  if (sms <= 0) return FATTN_ERR_CUDA;
  return launch_rope(p, true, interleaved != 0, true, sms, stream) == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

// The cap as a polynomial: tanh(z) = z (c0 + c1 z^2 + ... + c4 z^8) on |z| <= z_max, folded into powers of u =
// z softcap / scale. Fewer terms on a shorter range where the last coefficient would not be an ordinary float (at d = 128
// and its usual scale with caps above 3000): the Taylor terms 1, -1/3, 2/15 on |z| <= 0.08 (off by 17/315 z^6, 1.4e-8;
// caps to some 10^7), or the first alone on |z| <= 1e-4 (z^2 / 3, 3e-9): with such caps that holds every score of use. (With a
// scale / softcap above 10^4 and a cap above 1, scores past the short range are off by 2^-22 of the cap.) Caps below 1e-15
// go without: 1 / cap^2 has to be a float, and 2^-22 of such a cap is nothing.
static void fold_cap(float scale, float softcap, const double (&c)[5], double z_max, ScoreShape* out) {
  out->poly_limit = -1.f;
  if (!(softcap >= 1e-15f)) return;
  const double k = (double)scale / softcap, k2 = k * k, s = (double)scale * 1.4426950408889634;
  const double taylor[3] = {1.0, -1.0 / 3.0, 2.0 / 15.0}, third = std::fabs(s) * k2 * k2, fifth = third * k2 * k2;
  const int terms = fifth > 1e-36 && fifth < 1e38 ? 5 : third > 1e-36 && third < 1e38 ? 3 : 1;
  double pw = s;
  for (int i = 0; i < 5; ++i, pw *= k2) {
    const float a = i >= terms ? 0.f : (float)((terms == 5 ? c[i] : taylor[i]) * pw);
    out->poly[i] = make_float2(a, a);
  }
  const double limit = (terms == 5 ? z_max : terms == 3 ? 0.08 : 1e-4) / std::fabs(k);   // (scale 0: infinite)
  out->poly_limit = (float)(limit < 1e18 ? limit : 1e18);   // (its square is a float)
}

// A score shape's own checks; fills *out. `scale` is the call's, `keys` the most that a sequence has: a window of that
// many hides nothing, nor does one whose sinks reach it, and the kernels' sums of positions, windows and sinks stay small
// without them.
static fattn_status check_shape(float scale, float softcap, const float* slopes, int window, int sinks, bool causal,
                                const int32_t* key_begin, const int32_t* key_end, long long keys, ScoreShape* out) {
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0 || sinks < 0)
    return FATTN_ERR_INVALID_ARG;
  // the cap's argument 2 log2(e) scale / softcap must be a number
  if (softcap > 0.f && !std::isfinite(2.f * 1.4426951f * scale / softcap)) return FATTN_ERR_INVALID_ARG;
  if (misaligned(slopes, 4) || misaligned(key_begin, 4) || misaligned(key_end, 4)) return FATTN_ERR_INVALID_ARG;
  if (sinks > 0 && (key_begin || key_end)) return FATTN_ERR_UNSUPPORTED;
  if (window >= keys || (sinks > 0 && sinks >= (causal ? keys - window : keys))) window = 0;
  if (window == 0) sinks = 0;
  // a cap of 2^100 moves no score up to 2^88 in 32 bits (tanh z is z within z^3 / 3), and above that, as without it, the
  // largest score takes all the weight
  if (softcap >= 0x1p100f) softcap = 0.f;
  *out = {softcap, slopes, window, key_begin, key_end, 0.f, 0.f, 0.f, 0.f, {}, -1.f, -1.f, sinks};
  out->sl2 = scale * 1.4426950408889634f;
  out->cap2 = softcap * 1.4426950408889634f;
  out->capk = softcap > 0.f ? 2.f * out->sl2 / softcap : 0.f;
  out->nicap2 = softcap > 0.f ? -1.f / (out->cap2 * out->cap2) : 0.f;
  // the cap on |z| <= 0.6, within 8e-8 of itself (interpolation in Chebyshev nodes), about what its rounding takes:
  // the logsumexp keeps its 32 bits (up to 0.75 the same degree is 3e-6 off near 0)
  const double c[5] = {0.999999926, -0.3333230204, 0.1331006443, -0.05209665341, 0.0154687513};
  fold_cap(scale, softcap, c, 0.6, out);
  const double k = (double)scale / (softcap > 0.f ? softcap : 1.0);
  // 2 log2(e) softcap tanh(k u) <= 96
  const double ratio = 48.0 / (1.4426950408889634 * softcap);
  if (softcap > 0.f && std::fabs(k) > 0.0)
    out->bound_limit = ratio >= 1.0 ? INFINITY : (float)(std::atanh(ratio) / std::fabs(k));
  return FATTN_OK;
}

// fattn_fwd_shaped and fattn_fwd_sinks.
static fattn_status fwd_shaped_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                                    int Hkv, int N, int d, int causal, float scale, float softcap, const float* slopes,
                                    int window, int sinks, const int32_t* key_begin, const int32_t* key_end,
                                    cudaStream_t stream) {
  if (B < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || d <= 0) return FATTN_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return FATTN_OK;
  if (!q || !k || !v || !o || Hq % Hkv != 0) return FATTN_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) || misaligned(lse, 4))
    return FATTN_ERR_INVALID_ARG;
  PrefillParams p{};
  const fattn_status st = check_shape(scale, softcap, slopes, window, sinks, causal != 0, key_begin, key_end, N, &p.shape);
  if (st != FATTN_OK) return st;
  if (d != 64 && d != 128) return FATTN_ERR_UNSUPPORTED;
  const long long rows = (long long)B * N;
  const long long pairs = ((long long)N + 255) / 256;  // work items per (sequence, head)
  if (rows > 0x7fffffffLL || (long long)B * Hq > 0x7fffffffLL / pairs) return FATTN_ERR_UNSUPPORTED;
  int err = 0;
  p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.N = N; p.d = d; p.total_rows = (int)rows;
  p.causal = causal ? 1 : 0; p.scale = scale;
  p.mask_heads = 1;
  p.shaped = 1;
  p.splits = 1;
  p.status = status_ptr(&err);
  if (err) return FATTN_ERR_CUDA;
  current_waits(&p.wait_ns, &p.debug_stall);
  CUtensorMap tq, tk, tv, to;
  if (!encode_rows_map(&tq, q, p.total_rows, Hq, d, 128) || !encode_rows_map(&tk, k, p.total_rows, Hkv, d, 128) ||
      !encode_rows_map(&tv, v, p.total_rows, Hkv, d, 128) || !encode_rows_map(&to, o, p.total_rows, Hq, d, 32))
    return FATTN_ERR_CUDA;
  const int sms = num_sms_current();
  if (sms <= 0) return FATTN_ERR_CUDA;
  return launch_prefill_tc(p, tq, tk, tv, to, sms, stream) == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

extern "C" fattn_status fattn_fwd_shaped(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                                         int Hkv, int N, int d, int causal, float scale, float softcap,
                                         const float* slopes, int window, const int32_t* key_begin,
                                         const int32_t* key_end, cudaStream_t stream) {
  return fwd_shaped_impl(q, k, v, o, lse, B, Hq, Hkv, N, d, causal, scale, softcap, slopes, window, 0, key_begin, key_end,
                         stream);
}

extern "C" fattn_status fattn_fwd_sinks(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                                        int Hkv, int N, int d, int causal, float scale, float softcap,
                                        const float* slopes, int window, int sinks, cudaStream_t stream) {
  return fwd_shaped_impl(q, k, v, o, lse, B, Hq, Hkv, N, d, causal, scale, softcap, slopes, window, sinks, nullptr,
                         nullptr, stream);
}

extern "C" size_t fattn_fwd_paged_shaped_workspace_size(int total_q, int Hq, int d, int num_splits) {
  if (total_q <= 0 || Hq <= 0 || d <= 0 || num_splits <= 1) return 0;
  const size_t rows = (size_t)total_q * Hq * num_splits;
  return (rows * 4 + 255) / 256 * 256 + (rows * d * 4 + 255) / 256 * 256;
}

extern "C" fattn_status fattn_fwd_paged_shaped(const void* q, const void* kcache, const void* vcache,
                                               const int32_t* block_table, const int32_t* seqlens_k,
                                               const int32_t* cu_seqlens_q, void* o, float* lse, int B, int Hq, int Hkv,
                                               int d, int page_size, int max_pages_per_seq, int num_pages, int total_q,
                                               int max_seqlen_q, int causal, float scale, float softcap,
                                               const float* slopes, int window, const int32_t* key_begin,
                                               const int32_t* key_end, int num_splits, void* workspace,
                                               size_t workspace_bytes, cudaStream_t stream) {
  ScoreShape shape{};
  const fattn_status st = check_shape(scale, softcap, slopes, window, 0, causal != 0, key_begin, key_end,
                                      (long long)max_pages_per_seq * page_size, &shape);
  if (st != FATTN_OK) return st;
  if (num_splits < 1) return FATTN_ERR_INVALID_ARG;
  return fwd_paged_impl(q, kcache, vcache, block_table, seqlens_k, cu_seqlens_q, o, lse, B, Hq, Hkv, d, page_size,
                        max_pages_per_seq, num_pages, total_q, max_seqlen_q, causal, scale, &shape, num_splits, workspace,
                        workspace_bytes, stream);
}

extern "C" fattn_status fattn_fwd_paged_sinks(const void* q, const void* kcache, const void* vcache,
                                              const int32_t* block_table, const int32_t* seqlens_k,
                                              const int32_t* cu_seqlens_q, void* o, float* lse, int B, int Hq, int Hkv,
                                              int d, int page_size, int max_pages_per_seq, int num_pages, int total_q,
                                              int max_seqlen_q, int causal, float scale, float softcap,
                                              const float* slopes, int window, int sinks, int num_splits, void* workspace,
                                              size_t workspace_bytes, cudaStream_t stream) {
  ScoreShape shape{};
  const fattn_status st = check_shape(scale, softcap, slopes, window, sinks, causal != 0, nullptr, nullptr,
                                      (long long)max_pages_per_seq * page_size, &shape);
  if (st != FATTN_OK) return st;
  if (num_splits < 1) return FATTN_ERR_INVALID_ARG;
  return fwd_paged_impl(q, kcache, vcache, block_table, seqlens_k, cu_seqlens_q, o, lse, B, Hq, Hkv, d, page_size,
                        max_pages_per_seq, num_pages, total_q, max_seqlen_q, causal, scale, &shape, num_splits, workspace,
                        workspace_bytes, stream);
}

extern "C" size_t fattn_bwd_shaped_workspace_size(int B, int Hq, int Hkv, int N, int d) {
  const size_t vectors = fattn_bwd_workspace_size(B, Hq, N);
  if (vectors == 0 || Hkv <= 0 || d <= 0) return 0;
  const size_t npad = ((size_t)N + 127) / 128 * 128;
  const size_t shares = bwd_shares(B, Hq, Hkv, N) ? 2 * (size_t)B * N * Hq * d * sizeof(float) : 0;
  return vectors + ((size_t)B * npad * 8 + 255) / 256 * 256 + (shares + 255) / 256 * 256;
}

extern "C" fattn_status fattn_bwd_shaped(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                         const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N,
                                         int d, int causal, float scale, float softcap, const float* slopes, int window,
                                         const int32_t* key_begin, const int32_t* key_end, void* workspace,
                                         size_t workspace_bytes, cudaStream_t stream) {
  ScoreShape shape{};
  const fattn_status st = check_shape(scale, softcap, slopes, window, 0, causal != 0, key_begin, key_end, N, &shape);
  if (st != FATTN_OK) return st;
  return bwd_impl(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, &shape, workspace,
                  workspace_bytes, stream);
}

extern "C" size_t fattn_bwd_sinks_workspace_size(int B, int Hq, int Hkv, int N, int d, int causal, int window, int sinks) {
  const size_t base = fattn_bwd_shaped_workspace_size(B, Hq, Hkv, N, d);
  // (what check_shape makes of a window that hides nothing)
  if (base == 0 || window <= 0 || sinks <= 0 || window >= N || sinks >= (causal ? N - window : N)) return base;
  const int pieces = bwd_sink_pieces(N, causal, window, sinks);
  if (pieces == 1) return base;
  const size_t rows = (size_t)B * sink_blocks(sinks, 128) * 128 * (bwd_shares(B, Hq, Hkv, N) ? Hq : Hkv);
  return base + (2 * pieces * rows * d * sizeof(float) + 255) / 256 * 256;
}

extern "C" fattn_status fattn_bwd_sinks(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                        const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N,
                                        int d, int causal, float scale, float softcap, const float* slopes, int window,
                                        int sinks, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  ScoreShape shape{};
  const fattn_status st =
      check_shape(scale, softcap, slopes, window, sinks, causal != 0, nullptr, nullptr, N, &shape);
  if (st != FATTN_OK) return st;
  return bwd_impl(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, &shape, workspace,
                  workspace_bytes, stream);
}

extern "C" fattn_status fattn_bwd_strided(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                          const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N,
                                          int d, int causal, float scale, int shaped, float softcap, const float* slopes,
                                          int window, int sinks, const int32_t* key_begin, const int32_t* key_end,
                                          long long o_batch, long long o_row, long long o_head, void* workspace,
                                          size_t workspace_bytes, cudaStream_t stream) {
  const long long strides[3] = {o_batch, o_row, o_head};
  ScoreShape shape{};
  if (shaped) {
    const fattn_status st =
        check_shape(scale, softcap, slopes, window, sinks, causal != 0, key_begin, key_end, N, &shape);
    if (st != FATTN_OK) return st;
  } else if (softcap != 0.f || slopes || window != 0 || sinks != 0 || key_begin || key_end) {
    return FATTN_ERR_INVALID_ARG;
  }
  return bwd_impl(q, k, v, o, lse, dout, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, shaped ? &shape : nullptr, workspace,
                  workspace_bytes, stream, strides);
}

extern "C" fattn_status fattn_decode_paged_shaped(const void* q, const void* kcache, const void* vcache,
                                                  const int32_t* block_table, const int32_t* seqlens, int num_splits,
                                                  void* o, float* lse, int B, int Hq, int Hkv, int d, int page_size,
                                                  int max_pages_per_seq, int num_pages, float scale, float softcap,
                                                  const float* slopes, int window, void* workspace,
                                                  size_t workspace_bytes, cudaStream_t stream) {
  return fattn_decode_paged_sinks(q, kcache, vcache, block_table, seqlens, num_splits, o, lse, B, Hq, Hkv, d, page_size,
                                  max_pages_per_seq, num_pages, scale, softcap, slopes, window, 0, workspace,
                                  workspace_bytes, stream);
}

extern "C" fattn_status fattn_decode_paged_sinks(const void* q, const void* kcache, const void* vcache,
                                                 const int32_t* block_table, const int32_t* seqlens, int num_splits,
                                                 void* o, float* lse, int B, int Hq, int Hkv, int d, int page_size,
                                                 int max_pages_per_seq, int num_pages, float scale, float softcap,
                                                 const float* slopes, int window, int sinks, void* workspace,
                                                 size_t workspace_bytes, cudaStream_t stream) {
  ScoreShape shape{};
  const fattn_status st = check_shape(scale, softcap, slopes, window, sinks, true, nullptr, nullptr,
                                      (long long)max_pages_per_seq * page_size, &shape);
  if (st != FATTN_OK) return st;
  return decode_paged_impl(q, kcache, vcache, block_table, seqlens, num_splits, o, lse, B, Hq, Hkv, d, page_size,
                           max_pages_per_seq, num_pages, scale, &shape, workspace, workspace_bytes, stream);
}

extern "C" fattn_status fattn_key_weights_paged(const void* q, const void* kcache, const int32_t* block_table,
                                                const int32_t* seqlens_k, const int32_t* cu_seqlens_q, const float* lse,
                                                long long lse_head, long long lse_row, const float* weights_in,
                                                float* weights_out, int B, int Hq, int Hkv, int d, int page_size,
                                                int max_pages_per_seq, int num_pages, int total_q, int max_seqlen_q,
                                                int causal, float scale, float softcap, const float* slopes, int window,
                                                float decay, cudaStream_t stream) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || total_q < 0 || max_seqlen_q < 0 || page_size <= 0 ||
      max_pages_per_seq <= 0 || num_pages <= 0 || lse_head < 0 || lse_row < 0)
    return FATTN_ERR_INVALID_ARG;
  KeyWeightsParams p{};
  const fattn_status st =
      check_shape(scale, softcap, slopes, window, 0, causal != 0, nullptr, nullptr, (long long)max_pages_per_seq * page_size,
                  &p.shape);
  if (st != FATTN_OK) return st;
  // every weight is an fp32 output: within 1.3e-8, on a shorter range
  const double c[5] = {0.9999999868, -0.3333306794, 0.133247505, -0.05298423883, 0.01713134443};
  fold_cap(scale, softcap, c, 0.5, &p.shape);
  if (Hq % Hkv != 0 || !std::isfinite(decay)) return FATTN_ERR_INVALID_ARG;
  if (B == 0) return FATTN_OK;
  if (!kcache || !block_table || !seqlens_k || !cu_seqlens_q || !weights_out) return FATTN_ERR_INVALID_ARG;
  if (total_q > 0 && (!q || !lse)) return FATTN_ERR_INVALID_ARG;  // no queries: the weights decay
  if (misaligned(q, 16) || misaligned(kcache, 16) || misaligned(block_table, 4) || misaligned(seqlens_k, 4) ||
      misaligned(cu_seqlens_q, 4) || misaligned(lse, 4) || misaligned(weights_in, 4) || misaligned(weights_out, 4))
    return FATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FATTN_ERR_UNSUPPORTED;
  if ((long long)max_pages_per_seq * page_size > 0x7fffffffLL - 1024 || B > 65535 || Hkv > 65535 ||
      ((long long)max_pages_per_seq * page_size / 128 + 1) * Hkv > 0x7fffffffLL)
    return FATTN_ERR_UNSUPPORTED;
  int err = 0;
  p.q = q; p.kcache = kcache; p.block_table = block_table; p.seqlens_k = seqlens_k; p.cu_seqlens = cu_seqlens_q;
  p.lse = lse; p.lse_head = lse_head; p.lse_row = lse_row; p.w_in = weights_in; p.w_out = weights_out;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.d = d; p.page_size = page_size; p.max_pages = max_pages_per_seq;
  p.num_pages = num_pages; p.total_q = total_q; p.max_q = max_seqlen_q;
  p.causal = causal ? 1 : 0; p.scale = scale; p.decay = decay;
  p.status = status_ptr(&err);
  if (err) return FATTN_ERR_CUDA;
  current_waits(&p.wait_ns, &p.debug_stall);
  const int G = Hq / Hkv;
  const long long rows = (long long)max_seqlen_q * G;
  // up to 32 query rows K's bytes bound the sums (stream kernel); above, the tensor-core kernel, and the
  // mma.sync one for page sizes and groups that TMA boxes do not take (d = 128, 128 rows over 8k tokens: 13 and
  // 15 us; 64 rows over 4 sequences of 2k: 19 and 17 us; 128 rows: 18 and 23 us; 2048-query prompts: 130
  // and 697 us)
  const bool tc = rows > 32 && total_q > 0 && G <= 128 &&
                  (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128) &&
                  (long long)(num_pages + 1) * page_size <= 0x7fffffffLL &&
                  ((long long)max_pages_per_seq * page_size + 127) / 128 * B * Hkv <= 0x7fffffffLL;
  const int sms = num_sms_current();
  if (sms <= 0) return FATTN_ERR_CUDA;
  CUtensorMap tq, tk;
  if (rows <= 32 && page_size % 16 == 0 && (long long)num_pages * page_size <= 0x7fffffffLL) {
    if (!encode_rows_map(&tk, kcache, num_pages * page_size, Hkv, d, 16)) return FATTN_ERR_CUDA;
    return launch_key_weights_stream(p, tk, (int)rows, sms, stream) == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
  }
  if (!tc) return launch_key_weights(p, stream) == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
  if (!encode_rows_map(&tq, q, total_q, Hq, d, 128 / G, G) ||
      !encode_rows_map(&tk, kcache, num_pages * page_size, Hkv, d, page_size))
    return FATTN_ERR_CUDA;
  return launch_key_weights_tc(p, tq, tk, sms, stream) == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

extern "C" fattn_status fattn_evict_paged(void* kcache, void* vcache, const int32_t* block_table,
                                          const int32_t* seqlens, const float* weights_in, const int32_t* dst_table,
                                          int32_t* seqlens_out, float* weights_out, int32_t* kept, int B, int Hkv, int d,
                                          int page_size, int max_pages_per_seq, int num_pages, int dst_max_pages,
                                          int keep, int recent, int first, cudaStream_t stream) {
  if (B < 0 || Hkv <= 0 || d <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0 || dst_max_pages <= 0 ||
      keep <= 0 || recent < 0 || first < 0 || (long long)first + recent > keep)
    return FATTN_ERR_INVALID_ARG;
  if (!dst_table && dst_max_pages != max_pages_per_seq) return FATTN_ERR_INVALID_ARG;
  const long long cap = (long long)max_pages_per_seq * page_size, dst_cap = (long long)dst_max_pages * page_size;
  if (dst_cap < (keep < cap ? keep : cap)) return FATTN_ERR_INVALID_ARG;  // the kept tokens would not fit
  if (B == 0) return FATTN_OK;
  if (!kcache || !vcache || !block_table || !seqlens || !weights_in || !seqlens_out || !weights_out || !kept)
    return FATTN_ERR_INVALID_ARG;
  if (misaligned(kcache, 16) || misaligned(vcache, 16) || misaligned(block_table, 4) || misaligned(seqlens, 4) ||
      misaligned(weights_in, 4) || misaligned(dst_table, 4) || misaligned(seqlens_out, 4) ||
      misaligned(weights_out, 4) || misaligned(kept, 4))
    return FATTN_ERR_INVALID_ARG;
  // every block of a sequence reads its old length; weights in place keep their row length
  if (seqlens_out == seqlens || (weights_out == weights_in && dst_max_pages != max_pages_per_seq))
    return FATTN_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > 1024) return FATTN_ERR_UNSUPPORTED;
  if (cap > 0x7fffffffLL - 32768 || dst_cap > 0x7fffffffLL - 4096 || keep > 0x7fffffff - 4096 ||
      (long long)B * Hkv > 65535)
    return FATTN_ERR_UNSUPPORTED;
  int err = 0;
  EvictParams p{};
  p.kcache = kcache; p.vcache = vcache; p.block_table = block_table; p.seqlens = seqlens; p.w_in = weights_in;
  p.dst_table = dst_table; p.seqlens_out = seqlens_out; p.w_out = weights_out; p.kept = kept;
  p.B = B; p.Hkv = Hkv; p.d = d; p.page_size = page_size; p.max_pages = max_pages_per_seq; p.num_pages = num_pages;
  p.dst_max_pages = dst_max_pages; p.keep = keep; p.first = first; p.recent = recent;
  p.status = status_ptr(&err);
  if (err) return FATTN_ERR_CUDA;
  const int sms = num_sms_current();
  if (sms <= 0) return FATTN_ERR_CUDA;
  return launch_evict(p, sms, stream) == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

static size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// An 8-bit cache's own arguments.
static fattn_status check_cache_fp8(const void* kcache, const void* vcache, const float* kscale, const float* vscale,
                                    const int32_t* block_table, const int32_t* seqlens, int d, int page_size,
                                    int max_pages_per_seq, int num_pages) {
  if (!kcache || !vcache || !kscale || !vscale || !block_table || !seqlens) return FATTN_ERR_INVALID_ARG;
  if (misaligned(kcache, 16) || misaligned(vcache, 16) || misaligned(kscale, 4) || misaligned(vscale, 4) ||
      misaligned(block_table, 4) || misaligned(seqlens, 4))
    return FATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FATTN_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return FATTN_ERR_UNSUPPORTED;
  if ((long long)max_pages_per_seq * page_size > 0x7fffffffLL - 1024 || (long long)num_pages * page_size > 0x7fffffffLL)
    return FATTN_ERR_UNSUPPORTED;
  return FATTN_OK;
}

extern "C" fattn_status fattn_rope_append_paged_fp8(const void* q, void* q_out, const void* k, const void* v, void* kcache,
                                                    void* vcache, float* kscale, float* vscale, const int32_t* block_table,
                                                    const int32_t* seqlens_k, const int32_t* cu_seqlens_q,
                                                    const int32_t* positions, const double* inv_freq, int B, int total_q,
                                                    int Hq, int Hkv, int d, int rotary_dim, int page_size,
                                                    int max_pages_per_seq, int num_pages, long long q_row, long long q_head,
                                                    long long k_row, long long k_head, long long v_row, long long v_head,
                                                    int interleaved, float amplitude, cudaStream_t stream) {
  fattn_status st = check_rotary(inv_freq, total_q, q ? Hq : 0, Hkv, d, rotary_dim, amplitude);
  if (st != FATTN_OK) return st;
  if (B < 0 || Hkv <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0) return FATTN_ERR_INVALID_ARG;
  if (q_row < 0 || q_head < 0 || k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0) return FATTN_ERR_INVALID_ARG;
  if (B == 0 || total_q == 0) return FATTN_OK;
  if ((q != nullptr) != (q_out != nullptr) || (q && Hq <= 0) || !k || !v || !cu_seqlens_q) return FATTN_ERR_INVALID_ARG;
  if (misaligned(q, 2) || misaligned(q_out, 2) || misaligned(k, 2) || misaligned(v, 2) || misaligned(cu_seqlens_q, 4) ||
      misaligned(positions, 4))
    return FATTN_ERR_INVALID_ARG;
  st = check_cache_fp8(kcache, vcache, kscale, vscale, block_table, seqlens_k, d, page_size, max_pages_per_seq, num_pages);
  if (st != FATTN_OK) return st;
  if (total_q / page_size + 2ll * B > 0x7fffffffLL) return FATTN_ERR_UNSUPPORTED;
  int err = 0;
  AppendFp8Params p{};
  p.q = {q, q_out, q ? Hq : 0, q_row, q_head, (long long)Hq * d, d};
  p.k = {k, kcache, Hkv, k_row, k_head, 0, 0};
  p.v = {v, vcache, Hkv, v_row, v_head, 0, 0};
  p.kscale = kscale; p.vscale = vscale; p.positions = positions; p.inv_freq = inv_freq;
  p.cu_seqlens = cu_seqlens_q; p.seqlens_k = seqlens_k; p.block_table = block_table;
  p.rows = total_q; p.B = B; p.d = d; p.rot = rotary_dim; p.interleaved = interleaved != 0;
  p.page_size = page_size; p.max_pages = max_pages_per_seq; p.num_pages = num_pages; p.amplitude = amplitude;
  p.status = status_ptr(&err);
  if (err) return FATTN_ERR_CUDA;
  const int sms = num_sms_current();
  if (sms <= 0) return FATTN_ERR_CUDA;
  return launch_append_fp8(p, sms, stream) == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

// The streaming kernel counts the steps (16 tokens of a group of rows) of all sequences in an int.
static bool countable_steps(int B, int Hkv, long long rows, int max_pages, int page_size) {
  const long long steps = (long long)max_pages * page_size / 16 + 64;   // (and the turns between them)
  return stream_fp8_groups(B, Hkv, rows) <= 0x7fffffffLL / steps;
}

// Workspace of the streaming kernel: partial logsumexps and outputs of `rows` query rows, then its counters.
struct StreamWorkspace {
  size_t o, counters, bytes;
};
static StreamWorkspace stream_workspace(long long rows, int Hq, int d, int num_splits, long long groups) {
  const size_t n = (size_t)rows * Hq * num_splits;
  StreamWorkspace w;
  w.o = round256(n * 4);
  w.counters = w.o + round256(n * d * 4);
  w.bytes = w.counters + round256((size_t)(1 + groups) * 4);
  return w;
}

extern "C" fattn_status fattn_decode_paged_fp8(const void* q, const void* kcache, const void* vcache, const float* kscale,
                                               const float* vscale, const int32_t* block_table, const int32_t* seqlens,
                                               int num_splits, void* o, float* lse, int B, int Hq, int Hkv, int d,
                                               int page_size, int max_pages_per_seq, int num_pages, float scale,
                                               float softcap, const float* slopes, int window, int sinks, void* workspace,
                                               size_t workspace_bytes, cudaStream_t stream) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0 ||
      num_splits <= 0)
    return FATTN_ERR_INVALID_ARG;
  StreamFp8Params p{};
  fattn_status st = check_shape(scale, softcap, slopes, window, sinks, true, nullptr, nullptr,
                                (long long)max_pages_per_seq * page_size, &p.shape);
  if (st != FATTN_OK) return st;
  if (B == 0) return FATTN_OK;
  if (!q || !o || Hq % Hkv != 0 || misaligned(q, 16) || misaligned(o, 16) || misaligned(lse, 4)) return FATTN_ERR_INVALID_ARG;
  st = check_cache_fp8(kcache, vcache, kscale, vscale, block_table, seqlens, d, page_size, max_pages_per_seq, num_pages);
  if (st != FATTN_OK) return st;
  if ((long long)B * Hq * num_splits > 0x7fffffffLL / 512 ||
      !countable_steps(B, Hkv, Hq / Hkv, max_pages_per_seq, page_size))
    return FATTN_ERR_UNSUPPORTED;
  const StreamWorkspace w = stream_workspace(B, Hq, d, num_splits, (long long)B * Hq);
  if (!workspace || workspace_bytes < w.bytes || misaligned(workspace, 256)) return FATTN_ERR_WORKSPACE;
  int err = 0;
  p.q = q; p.kcache = kcache; p.vcache = vcache; p.kscale = kscale; p.vscale = vscale; p.block_table = block_table;
  p.seqlens_k = seqlens; p.o = o; p.lse = lse; p.lse_head = 1; p.lse_row = Hq;
  p.lse_part = static_cast<float*>(workspace);
  p.o_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.o);
  p.counters = reinterpret_cast<int*>(static_cast<char*>(workspace) + w.counters);
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.d = d; p.page_size = page_size; p.max_pages = max_pages_per_seq;
  p.num_pages = num_pages; p.num_splits = num_splits; p.rows = B; p.max_q = 1; p.causal = 1; p.scale = scale;
  p.status = status_ptr(&err);
  if (err) return FATTN_ERR_CUDA;
  return launch_stream_fp8(p, stream) == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

// Workspace of the chunks' call: the streaming kernel's, or the pages' copies in bf16, their table and the prefill's splits.
struct ChunkWorkspace {
  bool stream;
  StreamWorkspace s;
  size_t v, table, splits, bytes;
};
static ChunkWorkspace chunk_workspace(int B, int Hq, int Hkv, int d, int page_size, int max_pages, int total_q, int max_q,
                                      int num_splits) {
  ChunkWorkspace w{};
  const long long rows = (long long)max_q * (Hq / Hkv);
  w.stream = streams_fp8(max_q, Hq / Hkv);
  if (w.stream) {
    w.s = stream_workspace(total_q, Hq, d, num_splits, stream_fp8_groups(B, Hkv, rows));
    w.bytes = w.s.bytes;
    return w;
  }
  const size_t copy = round256((size_t)B * max_pages * page_size * Hkv * d * 2);
  w.v = copy;
  w.table = 2 * copy;
  w.splits = w.table + round256((size_t)B * max_pages * 4);
  w.bytes = w.splits + fattn_fwd_paged_shaped_workspace_size(total_q, Hq, d, num_splits);
  return w;
}

extern "C" size_t fattn_fwd_paged_fp8_workspace_size(int B, int Hq, int Hkv, int d, int page_size, int max_pages_per_seq,
                                                     int total_q, int max_seqlen_q, int num_splits) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || d <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || total_q <= 0 ||
      max_seqlen_q <= 0 || num_splits <= 0)
    return 0;
  return chunk_workspace(B, Hq, Hkv, d, page_size, max_pages_per_seq, total_q, max_seqlen_q, num_splits).bytes;
}

extern "C" fattn_status fattn_fwd_paged_fp8(const void* q, const void* kcache, const void* vcache, const float* kscale,
                                            const float* vscale, const int32_t* block_table, const int32_t* seqlens_k,
                                            const int32_t* cu_seqlens_q, void* o, float* lse, int B, int Hq, int Hkv, int d,
                                            int page_size, int max_pages_per_seq, int num_pages, int total_q,
                                            int max_seqlen_q, int causal, float scale, float softcap, const float* slopes,
                                            int window, int sinks, int num_splits, void* workspace, size_t workspace_bytes,
                                            cudaStream_t stream) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0 || total_q < 0 ||
      max_seqlen_q < 0 || num_splits <= 0)
    return FATTN_ERR_INVALID_ARG;
  StreamFp8Params p{};
  fattn_status st = check_shape(scale, softcap, slopes, window, sinks, causal != 0, nullptr, nullptr,
                                (long long)max_pages_per_seq * page_size, &p.shape);
  if (st != FATTN_OK) return st;
  if (B == 0 || total_q == 0 || max_seqlen_q == 0) return FATTN_OK;
  if (!q || !o || !cu_seqlens_q || Hq % Hkv != 0 || misaligned(q, 16) || misaligned(o, 16) || misaligned(lse, 4) ||
      misaligned(cu_seqlens_q, 4))
    return FATTN_ERR_INVALID_ARG;
  st = check_cache_fp8(kcache, vcache, kscale, vscale, block_table, seqlens_k, d, page_size, max_pages_per_seq, num_pages);
  if (st != FATTN_OK) return st;
  const long long rows = (long long)max_seqlen_q * (Hq / Hkv);
  if (rows > 0x7fffffffLL || (long long)total_q * Hq > 0x7fffffffLL / num_splits) return FATTN_ERR_UNSUPPORTED;
  if (streams_fp8(max_seqlen_q, Hq / Hkv)) {
    if (stream_fp8_groups(B, Hkv, rows) > 0x3fffffffLL / num_splits ||
        !countable_steps(B, Hkv, rows, max_pages_per_seq, page_size))
      return FATTN_ERR_UNSUPPORTED;
  } else {   // the copy's slots, and what the prefill and its joining refuse, before the copy is launched
    const long long pairs = ((long long)max_seqlen_q + 255) / 256;
    if (((long long)B * max_pages_per_seq + 1) * page_size > 0x7fffffffLL || (long long)B * Hq > 0x7fffffffLL / pairs / num_splits ||
        (num_splits > 1 && (B > 65535 || (long long)max_seqlen_q * Hq > 0x7fffffffLL)))
      return FATTN_ERR_UNSUPPORTED;
  }
  const ChunkWorkspace w =
      chunk_workspace(B, Hq, Hkv, d, page_size, max_pages_per_seq, total_q, max_seqlen_q, num_splits);
  if (!workspace || workspace_bytes < w.bytes || misaligned(workspace, 256)) return FATTN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  int err = 0;
  int* status = status_ptr(&err);
  if (err) return FATTN_ERR_CUDA;
  if (w.stream) {
    p.q = q; p.kcache = kcache; p.vcache = vcache; p.kscale = kscale; p.vscale = vscale; p.block_table = block_table;
    p.seqlens_k = seqlens_k; p.cu_seqlens = cu_seqlens_q; p.o = o; p.lse = lse; p.lse_head = total_q; p.lse_row = 1;
    p.lse_part = static_cast<float*>(workspace);
    p.o_part = reinterpret_cast<float*>(ws + w.s.o);
    p.counters = reinterpret_cast<int*>(ws + w.s.counters);
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.d = d; p.page_size = page_size; p.max_pages = max_pages_per_seq;
    p.num_pages = num_pages; p.num_splits = num_splits; p.rows = total_q; p.max_q = max_seqlen_q;
    p.causal = causal ? 1 : 0; p.scale = scale; p.status = status;
    return launch_stream_fp8(p, stream) == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
  }
  ExpandFp8Params e{};
  e.kcache = kcache; e.vcache = vcache; e.kscale = kscale; e.vscale = vscale; e.block_table = block_table;
  e.seqlens_k = seqlens_k; e.cu_seqlens = cu_seqlens_q;
  e.kout = ws; e.vout = ws + w.v; e.table = reinterpret_cast<int32_t*>(ws + w.table);
  e.B = B; e.Hkv = Hkv; e.d = d; e.page_size = page_size; e.max_pages = max_pages_per_seq; e.num_pages = num_pages;
  e.total_q = total_q; e.window = p.shape.window; e.sinks = p.shape.sinks; e.status = status;
  if (launch_expand_fp8(e, stream) != cudaSuccess) return FATTN_ERR_CUDA;
  const bool plain = p.shape.cap == 0.f && !p.shape.slopes && p.shape.window == 0 && num_splits == 1;
  return fwd_paged_impl(q, e.kout, e.vout, e.table, seqlens_k, cu_seqlens_q, o, lse, B, Hq, Hkv, d, page_size,
                        max_pages_per_seq, B * max_pages_per_seq, total_q, max_seqlen_q, causal, scale,
                        plain ? nullptr : &p.shape, num_splits, num_splits > 1 ? ws + w.splits : nullptr,
                        num_splits > 1 ? workspace_bytes - w.splits : 0, stream);
}
