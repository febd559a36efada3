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

cudaError_t launch_rope(const RopeParams& p, bool bf16, bool interleaved, bool append, cudaStream_t stream);

// From api.cu: the device status word of the current device (nullptr and *err != 0 on
// failure), the pipeline waits' limit and stall flag, a bf16 [rows, H, d] tensor map, and the
// calls whose plain and shaped forms differ in `shape` alone (nullptr: plain).
int* status_ptr(int* err);
void current_waits(unsigned long long* wait_ns, int* debug_stall);
bool encode_rows_map(CUtensorMap* map, const void* base, int rows, int H, int d, int box_rows);
fattn_status fwd_paged_impl(const void* q, const void* kcache, const void* vcache, const int32_t* block_table,
                            const int32_t* seqlens_k, const int32_t* cu_seqlens_q, void* o, float* lse, int B, int Hq,
                            int Hkv, int d, int page_size, int max_pages_per_seq, int num_pages, int total_q,
                            int max_seqlen_q, int causal, float scale, const ScoreShape* shape, cudaStream_t stream);
fattn_status bwd_impl(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                      void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d, int causal, float scale,
                      const ScoreShape* shape, void* workspace, size_t workspace_bytes, cudaStream_t stream);
fattn_status decode_paged_impl(const void* q, const void* kcache, const void* vcache, const int32_t* block_table,
                               const int32_t* seqlens, int num_splits, void* o, float* lse, int B, int Hq, int Hkv,
                               int d, int page_size, int max_pages_per_seq, int num_pages, float scale,
                               const ScoreShape* shape, void* workspace, size_t workspace_bytes, cudaStream_t stream);

}  // namespace fattn
