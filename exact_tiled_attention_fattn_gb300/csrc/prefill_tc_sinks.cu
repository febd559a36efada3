// The tensor-core prefill's variants with sinks, in a translation unit of their own: they are as many as the other shaped
// ones, and compile beside them.
#define FATTN_PREFILL_SINKS
#include "prefill_tc.cu"
