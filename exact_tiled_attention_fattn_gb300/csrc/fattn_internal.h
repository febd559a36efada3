// Internal launchers of libfattn (not part of the ABI). Each returns a
// cudaError_t from the launch; argument checks happen in api.cu before these
// are called.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fattn {

// Device status word codes (match fattn_status).
enum : int { kStatusOk = 0, kStatusTimeout = 5, kStatusDeviceCheck = 6 };

// Limit of one pipeline wait unless a test sets another (fattn_debug_set_wait_limit).
constexpr unsigned long long kDefaultWaitNs = 2000000000ull;

// Shape of the scores (all off when zero): tanh cap, distance bias, window and key ranges.
struct ScoreShape {
  float cap;                // s = cap tanh(s / cap); 0: none
  const float* slopes;      // device [Hq]: s -= slope_h |pos - j|; nullptr: none
  int window;               // |pos - j| < window; 0: none
  const int32_t* key_begin; // device, one per query row, non-decreasing in a sequence: keys
  const int32_t* key_end;   // [begin, end) are visible; nullptr: no bound
  // the scores' constants in log2 units: scale log2(e), cap log2(e), 2 scale log2(e) / cap, and
  // -1 / (cap log2(e))^2
  float sl2, cap2, capk, nicap2;
  // The cap as a polynomial of the raw product u = q.k, for |u| <= poly_limit (below 0: never):
  // log2(e) cap tanh(scale u / cap) = u P(u^2), P's coefficients from the lowest power up.
  float2 poly[5];           // (each twice: the packed FMAs read them as pairs)
  float poly_limit;
  // largest |u| whose cap, taken as a bound of capped scores of either sign, is at most 96 (log2
  // units) above them: exponents against it are those of normal floats
  float bound_limit;
};

// Problem description shared by both prefill kernels.
struct PrefillParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  const int32_t* cu_seqlens;  // device; nullptr = dense
  int B, Hq, Hkv, N, d;       // N = sequence length (dense) / max length (varlen)
  int total_rows;             // rows of the packed [rows, H, d] view (B*N or T)
  int causal;
  float scale;
  int* status;                // device status word
  // block-sparse variant only: uint8 [mask_heads][nb][nb], nb = ceil(N / 128);
  // block (qb, kb) = 0 hides keys [128 kb, 128 kb + 128) from queries [128 qb, 128 qb + 128)
  const uint8_t* block_mask;  // nullptr = dense
  int mask_heads;             // 1 (shared by all heads) or Hq
  // paged variant only (K/V read through a block table; q, o, lse packed as in
  // varlen with cu_seqlens = the chunks' query offsets):
  const int32_t* block_table; // device [B][max_pages]; nullptr = K/V in q's row space
  const int32_t* seqlens_k;   // device [B]: context tokens per sequence (>= its queries)
  int page_size, max_pages, num_pages;
  // masked variant only: additive bf16 mask, entry (b, h, i, j) at
  // mask[b * mask_sb + h * mask_sh + i * mask_ld + j] (strides in elements, multiples of 8)
  const void* mask;           // nullptr = none
  long long mask_sb, mask_sh;
  int mask_ld;
  int mask_v8;                // the mask is 32-byte aligned and its strides are multiples of 16
                              // elements: rows are read with 32-byte loads
  // FP8 variant only: E4M3 q, k and v ([rows, H, d]); scale already holds
  // scale * q_descale * k_descale
  int fp8;
  float v_descale;
  // shaped variant only (dense, or paged with a block table)
  int shaped;
  ScoreShape shape;
  // paged shaped: every query tile's key tiles cut into `splits` runs, each an item of its own; with more than
  // one the partials go to o_part [total_rows, Hq, splits, d] and lse_part [total_rows, Hq, splits]
  int splits;
  float* o_part;
  float* lse_part;
  // bounded pipeline waits: each mbarrier wait gives up after wait_ns; debug_stall != 0
  // (test hook) makes the softmax / element-wise warps first wait on a barrier that no
  // role arrives on, so that the wait runs out and every role takes the abort exit
  unsigned long long wait_ns;
  int debug_stall;
};

// Longest mask row (blocks) the block-sparse kernel holds in shared memory.
constexpr int kSparseMaxBlocks = 2048;

// Tensor-core prefill (bf16 in, fp32 accumulate, bf16 out). Tensor maps are
// encoded by the caller over the packed [rows, H, d] views of q, k and v (128-row
// boxes) and of o (bf16, 32-row boxes: the epilogue's stores).
cudaError_t launch_prefill_tc(const PrefillParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const CUtensorMap& to, int num_sms, cudaStream_t stream);

// Joins the partials of a split paged prefill into p.o and p.lse.
cudaError_t launch_prefill_merge(const PrefillParams& p, cudaStream_t stream);

// CUDA-core fp32 prefill.
cudaError_t launch_prefill_f32(const PrefillParams& p, cudaStream_t stream);

struct DecodeParams {
  const void* q;
  void* o;          // [B, Hq, d] bf16 output
  float* lse;       // [B, Hq] or nullptr
  int* counters;    // workspace: work counter, then one arrival counter per (sequence, KV-head group)
  const void* kcache;
  const void* vcache;
  const int32_t* block_table;
  const int32_t* seqlens;
  float* lse_part;  // [B, Hq, S]
  float* o_part;    // [B, Hq, S, d]
  int B, Hq, Hkv, d, page_size, max_pages_per_seq, num_pages, num_splits;
  float scale;
  int* status;
  int shaped;       // shaped variant: scores formed with `shape` (no key ranges)
  ScoreShape shape;
};

// Split-KV decode with the merge fused in (one launch, after a memset of the counters).
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream);

int num_sms_current();

struct MergeParams {
  const float* o_part;
  const float* lse_part;
  void* o;
  float* lse;
  int B, Hq, S, d;
  int out_bf16;
};

cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream);

// Attention backward (dense [B, N, H, d] bf16, lse [B, Hq, N] fp32 from the forward).
struct BwdParams {
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const void* dout;
  const float* lse;
  void* dq;
  void* dk;
  void* dv;
  float* ws_nl2;              // [B * Hq, Npad]: -lse * log2(e), -inf past N
  float* ws_d;                // [B * Hq, Npad]: rowsum(dO o O), 0 past N
  int2* ws_keys;              // shaped: [B, Npad], the query rows [x, y) that see each key
  float* ws_part;             // shaped, per query head: dV, then dK, [B * N, Hq, d] fp32; else nullptr
  int B, Hq, Hkv, N, d, Npad; // Npad = N rounded up to 128
  int causal;
  float scale;
  int* status;
  int shaped;                 // shaped variant: scores formed with `shape`
  ScoreShape shape;
  // bounded pipeline waits: each mbarrier wait gives up after wait_ns; debug_stall != 0
  // (test hook) makes the softmax / element-wise warps first wait on a barrier that no
  // role arrives on, so that the wait runs out and every role takes the abort exit
  unsigned long long wait_ns;
  int debug_stall;
};

// The shaped backward's dK/dV pass per query head, its fp32 shares added up afterwards, or per KV head, the group's heads
// one after the other in an item. Room for the shares is asked for (bwd_shares) where there are no more (key tile, KV
// head) items than the whole chip has SMs, a constant, as the workspace's size knows no device; bwd_per_head then weighs,
// for the SMs that there are and in steps of 128 queries (about 1.2 us), the longest item or the SMs' mean against the same with single heads, the shares' way through memory and the
// launch that adds them. A key tile is seen from all query tiles, at a mean half of them with causal, from a window's, and
// with key ranges, which the host does not know, from a quarter.
// Whole calls, causal, per KV head and per query head, d = 128 unless said: 997 rows, 8 heads over 2, d = 64 87 and 51 us; 2048
// rows, 32 over 8 188 and 159 us (a window of 512: 97 and 119 us); 8192 rows, 32 over 1, d = 64 4059 and 1533 us; 4096
// rows, 32 over 8 (256 items) 437 and 484 us.
constexpr long long kPerHeadItems = 152;
inline bool bwd_shares(int B, int Hq, int Hkv, int N) {
  return Hq > Hkv && (long long)B * Hkv * (((long long)N + 127) / 128) <= kPerHeadItems;
}
inline bool bwd_per_head(const BwdParams& p, int num_sms) {
  if (!bwd_shares(p.B, p.Hq, p.Hkv, p.N)) return false;
  const double nt = (p.N + 127) / 128, items = p.B * p.Hkv * nt, G = p.Hq / p.Hkv;
  double most = nt, mean = p.causal ? (nt + 1) / 2 : nt;
  if (p.shape.window > 0) {
    const double seen = (p.causal ? 1.0 : 2.0) * p.shape.window / 128 + 1;
    if (seen < most) most = seen;
  }
  if ((p.shape.key_begin || p.shape.key_end) && most > nt / 4) most = nt / 4 > 1 ? nt / 4 : 1;
  if (mean > most) mean = most;
  const double all = items * G * mean / num_sms;
  const double join = 2 + 2.0 * p.B * p.N * p.Hq * p.d * 1.3e-6;   // 8 bytes an element, 5 TB/s
  return (most > all ? most : all) + join < (G * most > all ? G * most : all);
}

// dQ pass (which also writes the workspace's two vectors) and dK/dV pass, in that
// order on `stream`. Tensor maps are over the packed [B * N, H, d] views of q, k, v
// and dout (128-row boxes) and of dk and dv (32-row boxes, for the stores).
cudaError_t launch_backward(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const CUtensorMap& tdo, const CUtensorMap& tdk, const CUtensorMap& tdv, int num_sms,
                            cudaStream_t stream);

}  // namespace fattn
