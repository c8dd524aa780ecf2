// Attention over listed blocks at head_dim 64.
#include "decode_blocks.cuh"

namespace kvd {
KVD_BLOCKS_LAUNCH(64)
}  // namespace kvd
