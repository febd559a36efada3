// Internal launchers behind include/fattn_ops.h (not part of the ABI). Argument
// checks happen in api_ops.cu before these are called.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

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

// Device status word of the current device (nullptr and *err != 0 on failure).
int* status_ptr(int* err);

}  // namespace fattn
