// Internal launchers behind include/fattn_ops.h (not part of the ABI). Argument
// checks happen in api_ops.cu before these are called.
#pragma once

#include "fattn.h"
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
