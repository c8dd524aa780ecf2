// Attention over listed blocks at head_dim 256.
#include "decode_blocks.cuh"

namespace kvd {
KVD_BLOCKS_LAUNCH(256)
}  // namespace kvd
