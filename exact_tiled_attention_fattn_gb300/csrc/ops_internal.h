// Internal launchers behind include/fattn_ops.h (not part of the ABI). Argument
// checks happen in api_ops.cu before these are called.
#pragma once

#include "fattn_ops.h"
#include "fattn_internal.h"

#include <algorithm>
#include <cmath>

namespace fattn {

// One tensor that rotary positions read and write: heads of `heads` x d elements per
// row, strides in elements.
struct RopeTensor {
  const void* in;
  void* out;
  int heads;
  long long in_row, in_head, out_row, out_head;
};

struct RopeParams {
  RopeTensor q, k, v;        // v: serving form only (copied, not rotated); out of k and v = the caches there
  const int32_t* positions;  // nullptr: row % period, or (serving form) the token's index in its sequence
  const double* inv_freq;
  int period, rows, d, rot;
  int inverse;
  float amplitude;
  // serving form (cu_seqlens != nullptr)
  const int32_t* cu_seqlens;
  const int32_t* seqlens_k;
  const int32_t* block_table;
  int B, page_size, max_pages, num_pages;
  int* status;
};

cudaError_t launch_rope(const RopeParams& p, bool bf16, bool interleaved, bool append, int num_sms,
                        cudaStream_t stream);

struct KeyWeightsParams {
  const void* q;              // [total_q, Hq, d] bf16
  const void* kcache;
  const int32_t* block_table;
  const int32_t* seqlens_k;
  const int32_t* cu_seqlens;
  const float* lse;           // of head h, row r at lse[h * lse_head + r * lse_row]
  long long lse_head, lse_row;
  const float* w_in;          // [B, Hkv, max_pages * page_size] or nullptr
  float* w_out;               // likewise; may be w_in
  int B, Hq, Hkv, d, page_size, max_pages, num_pages, total_q;
  int max_q;                  // queries of a sequence at most
  int causal;
  float scale, decay;
  ScoreShape shape;           // no key ranges
  int* status;
  int tiles;                  // tensor-core kernel: 128-key tiles per item, set by its launch
  unsigned long long wait_ns; // tensor-core kernel: limit of a pipeline wait, and the stall flag
  int debug_stall;
};

// mma.sync, any number of queries, page size and group.
cudaError_t launch_key_weights(const KeyWeightsParams& p, cudaStream_t stream);
// At most max_rows <= 32 query rows (queries x heads of a group) per sequence, page_size a multiple of 16;
// tensor map over the key pool with boxes of 16 rows.
cudaError_t launch_key_weights_stream(const KeyWeightsParams& p, const CUtensorMap& tk, int max_rows, int num_sms,
                                      cudaStream_t stream);
// Tensor-core kernel: tensor maps over q (boxes of G heads x 128 / G rows) and the key pool (boxes
// of one page), G = Hq / Hkv <= 128, page_size 16, 32, 64 or 128.
cudaError_t launch_key_weights_tc(const KeyWeightsParams& p, const CUtensorMap& tq, const CUtensorMap& tk, int num_sms,
                                  cudaStream_t stream);

struct EvictParams {
  void* kcache;
  void* vcache;
  const int32_t* block_table;
  const int32_t* seqlens;
  const float* w_in;          // [B, Hkv, max_pages * page_size]
  const int32_t* dst_table;   // nullptr: in place
  int32_t* seqlens_out;
  float* w_out;               // [B, Hkv, dst_max_pages * page_size]
  int32_t* kept;              // [B, Hkv, keep]
  int B, Hkv, d, page_size, max_pages, num_pages, dst_max_pages;
  int keep, first, recent;
  int* status;
};

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream);

// 8-bit paged cache: E4M3 codes [num_pages, page_size, Hkv, d], scales [num_pages, Hkv].
constexpr int kAppendMaxHeads = 64;   // KV heads that a block of the append has room for
constexpr int kAppendRows = 8;        // rows of q that one takes at most

struct AppendFp8Params {
  RopeTensor q, k, v;         // bf16; out of k and v = the code caches
  float* kscale;
  float* vscale;
  const int32_t* positions;   // nullptr: the token's index in its sequence
  const double* inv_freq;
  const int32_t* cu_seqlens;
  const int32_t* seqlens_k;
  const int32_t* block_table;
  int rows, B, d, rot, interleaved, page_size, max_pages, num_pages;
  float amplitude;
  int* status;
  // set by the launch: blocks of pages, shares of the KV heads, rows of a block of q, log2 of the page size, 2^42 / (rot / 2)
  int pages, head_shares, q_rows, page_shift;
  unsigned long long by_half;
};

cudaError_t launch_append_fp8(const AppendFp8Params& p, int num_sms, cudaStream_t stream);

struct ExpandFp8Params {
  const void* kcache;
  const void* vcache;
  const float* kscale;
  const float* vscale;
  const int32_t* block_table;
  const int32_t* seqlens_k;
  const int32_t* cu_seqlens;
  void* kout;                 // bf16 [B * max_pages, page_size, Hkv, d]
  void* vout;
  int32_t* table;             // [B, max_pages], the copy's own
  int B, Hkv, d, page_size, max_pages, num_pages, total_q;
  int window, sinks;
  int* status;
};

// Visible pages of the 8-bit cache as bf16 pages of their own.
cudaError_t launch_expand_fp8(const ExpandFp8Params& p, cudaStream_t stream);

struct StreamFp8Params {
  const void* q;              // [rows, Hq, d] bf16
  const void* kcache;
  const void* vcache;
  const float* kscale;
  const float* vscale;
  const int32_t* block_table;
  const int32_t* seqlens_k;
  const int32_t* cu_seqlens;  // nullptr: one query per sequence
  void* o;
  float* lse;                 // of head h, row r at lse[h * lse_head + r * lse_row]; or nullptr
  long long lse_head, lse_row;
  float* lse_part;            // [rows, Hq, S]
  float* o_part;              // [rows, Hq, S, d]
  int* counters;              // arrivals, one counter per group of rows and KV head
  int B, Hq, Hkv, d, page_size, max_pages, num_pages, num_splits;
  int rows, max_q, causal;
  float scale;
  ScoreShape shape;           // no key ranges
  int* status;
  // set by the launch: heads of a KV head, groups of rows of a sequence, their reciprocals, log2 of the page size
  int group, subs, page_shift;
  int cluster;                // CTAs of a cluster that share a group of rows; 0: the groups' line is shared
  unsigned long long by_group, by_subs;
};

// Rows (queries x heads of a KV head) that a group of the streaming kernel takes, 8 to 32 in steps of 8, equal groups
// of them, and the groups of all sequences and KV heads.
inline int stream_fp8_rows(long long max_rows) {
  const long long groups = (max_rows + 31) / 32;
  return groups <= 1 ? (int)((max_rows + 7) / 8 * 8) : (int)((max_rows + 8 * groups - 1) / (8 * groups) * 8);
}
inline long long stream_fp8_groups(int B, int Hkv, long long max_rows) {
  const int r = stream_fp8_rows(max_rows);
  return (long long)B * Hkv * ((max_rows + r - 1) / r);
}
// What going from one group to the next costs a CTA, in chunks of 16 tokens: it counts in the shares.
constexpr int kStreamTurn = 16;
// Pieces of a group in the line at most: one CTA joins them, a round of loads for some of them (one context of 199k tokens,
// one KV head: 34.9 us, 36.3 in 160 pieces, 41.2 in 304).
constexpr int kStreamPieces = 96;
constexpr int kStreamMostCluster = 16;   // CTAs of a cluster
// CTAs of a cluster for a group of rows, at most `most`; 0: the line of steps for all of them, joined through global memory.
// With M the steps that a group may have, a cluster of c takes ceil(M / c) of them per warp (`step`: chunks that a CTA's warps
// take at a time), two to begin with and one to join, and about as many again for every further round of CTAs (two an SM;
// clusters of 16 find less room); the line takes equal shares (0.85 M for the mean of several sequences), about eight steps for
// the counters and the joining, and a tenth for every piece.
// The line and clusters of 1, 2, 4, 8, 16, d = 128: one context of 2000, 4 KV heads 12.3, 17.5, 12.3, 8.4, 7.2 and 6.3 us, of
// 30000 22.7, 216, 113, 62, 34.6 and 20.4; 8 contexts, 8 heads, to 3000 21.4, 27.2, 17.2 and 13.2, to 32768 77.3, 240, 126, 81.9
// and 81.0; 64 contexts of 1000, 8 heads 39.0, 30.5, 41.7 and 59.5.
inline int stream_fp8_cluster(const StreamFp8Params& p, int step, int sms, int most) {
  if (p.num_splits == 1) return 1;
  const long long groups = (long long)p.B * p.subs * p.Hkv, seqs = (long long)p.B * p.subs;
  long long pages = p.max_pages;
  if (p.shape.window > 0) {   // (without causal on both sides of the queries)
    const long long tokens = (p.causal ? 1ll : 2ll) * p.shape.window + p.max_q;
    pages = std::min<long long>(pages, (tokens + p.page_size - 3) / p.page_size + 1 + sink_blocks(p.shape.sinks, p.page_size));
  }
  const double M = (double)(pages * p.page_size / 16), line_blocks = std::max(2 * sms / p.Hkv, 1);
  const int splits = std::min(p.num_splits, kStreamPieces);
  const double mean = p.B > 1 ? 0.85 : 1.0;
  const double share = std::max({mean * (double)seqs * (M + kStreamTurn) / line_blocks, M / (splits - 1), (double)step});
  double best = share / step + 8.0 + 0.1 * M / share;
  int cluster = 0;
  for (int c = 1; c <= std::min(most, p.num_splits); c *= 2) {
    const int room = c > 8 ? sms : 2 * sms;
    const long long rounds = (groups * c + room - 1) / room;
    const double steps = (rounds == 1 ? 1.0 : 0.95 * (double)rounds) * (std::ceil(M / ((double)c * step)) + 2) + (c > 1 ? 1 : 0);
    if (groups * c <= 0x3fffffff && steps < best) best = steps, cluster = c;
  }
  return cluster;
}
// Whether a chunk goes to the streaming kernel. Its time grows with the rows (2 x 30000 tokens, 8 KV heads of 128: 1.0 us a
// row), the other way's with the query heads, whose tiles have room for 256 queries (44 us for each of a KV head), and the
// copy of the cache (51 us): with 4 heads a KV head 128 rows take 137 and 234 us, 256 rows 258 and 235. A fit to that shape: the
// other way's copy and rounds depend on contexts, sequences and KV heads too, which are not weighed.
inline bool streams_fp8(long long max_q, int group) { return max_q * group <= FATTN_FP8_STREAM_ROWS((long long)group); }
cudaError_t launch_stream_fp8(const StreamFp8Params& p, cudaStream_t stream);

// From api.cu: the device status word of the current device (nullptr and *err != 0 on
// failure), the pipeline waits' limit and stall flag, a bf16 [rows, H, d] tensor map, and the
// calls whose plain and shaped forms differ in `shape` alone (nullptr: plain).
int* status_ptr(int* err);
void current_waits(unsigned long long* wait_ns, int* debug_stall);
bool encode_rows_map(CUtensorMap* map, const void* base, int rows, int H, int d, int box_rows, int box_heads = 1);
fattn_status fwd_paged_impl(const void* q, const void* kcache, const void* vcache, const int32_t* block_table,
                            const int32_t* seqlens_k, const int32_t* cu_seqlens_q, void* o, float* lse, int B, int Hq,
                            int Hkv, int d, int page_size, int max_pages_per_seq, int num_pages, int total_q,
                            int max_seqlen_q, int causal, float scale, const ScoreShape* shape, int num_splits,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream);
fattn_status bwd_impl(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                      void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d, int causal, float scale,
                      const ScoreShape* shape, void* workspace, size_t workspace_bytes, cudaStream_t stream,
                      const long long* o_strides = nullptr);   // batch, row, head; nullptr: packed
fattn_status decode_paged_impl(const void* q, const void* kcache, const void* vcache, const int32_t* block_table,
                               const int32_t* seqlens, int num_splits, void* o, float* lse, int B, int Hq, int Hkv,
                               int d, int page_size, int max_pages_per_seq, int num_pages, float scale,
                               const ScoreShape* shape, void* workspace, size_t workspace_bytes, cudaStream_t stream);

}  // namespace fattn
