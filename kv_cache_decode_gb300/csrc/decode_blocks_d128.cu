// Attention over listed blocks at head_dim 128.
#include "decode_blocks.cuh"

namespace kvd {
KVD_BLOCKS_LAUNCH(128)
}  // namespace kvd
