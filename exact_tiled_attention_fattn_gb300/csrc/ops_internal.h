// Internal launchers behind include/fattn_ops.h (not part of the ABI). Argument
// checks happen in api_ops.cu before these are called.
#pragma once

#include "fattn_ops.h"
#include "fattn_internal.h"

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
// Whether a chunk goes to the streaming kernel. Its time grows with the rows (2 x 30000 tokens, 8 KV heads of 128: 1.0 us a
// row), the other way's with the query heads, whose tiles have room for 256 queries (44 us for each of a KV head), and the
// copy of the cache (51 us): with 4 heads a KV head 128 rows take 137 and 234 us, 256 rows 258 and 235.
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
                      const ScoreShape* shape, void* workspace, size_t workspace_bytes, cudaStream_t stream);
fattn_status decode_paged_impl(const void* q, const void* kcache, const void* vcache, const int32_t* block_table,
                               const int32_t* seqlens, int num_splits, void* o, float* lse, int B, int Hq, int Hkv,
                               int d, int page_size, int max_pages_per_seq, int num_pages, float scale,
                               const ScoreShape* shape, void* workspace, size_t workspace_bytes, cudaStream_t stream);

}  // namespace fattn
