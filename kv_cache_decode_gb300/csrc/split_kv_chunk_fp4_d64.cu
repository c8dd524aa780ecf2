// The fp4 chunk kernel at head_dim 64.
#include "split_kv_chunk_fp4.cuh"

namespace kvd {
KVD_FP4_TABLE(64)
}  // namespace kvd
