// Shared host/device declarations of the rotary positions, the rotating appends
// and the fp4 cache: their descriptions and launches.
#pragma once

#include "params.h"

namespace kvd {

// Rotary positions (struct kvd_rope, checked; turns null: no rotation).
struct RopeTable {
    const uint64_t* turns;
    float factor;
    int rotary_dim;
    int interleaved;
};
cudaError_t launch_rope(const RopeTable& rope, const void* x, long long xs, bool in32, void* y, long long ys, bool out32,
                        const int32_t* positions, long long rows, int H, int D, int num_sms, cudaStream_t stream);

// What a rotating append writes: the cache's form and addresses.
enum class CacheForm { kBf16, kInt8, kFp8, kFp4 };
struct AppendTarget {
    void* k;
    void* v;
    float* k_scale;  // 8-bit forms
    float* v_scale;
    CacheForm form;
    int S_max;       // capacity of a sequence
    PagedCache pg;
};
// The new rows of one append (kv_append_rope.cu): strides in elements between tokens' rows.
struct NewRows {
    const void* q;
    void* q_out;
    const void* k;
    const void* v;
    long long qs, qos, ks, vs;
    const int32_t* pos;
    const int32_t* offsets;  // ragged rows [B + 1], or null: T rows to a sequence
    int B, T, Hq, Hkv, D;
    long long rows;
};
cudaError_t launch_append_rope(const AppendTarget& to, const RopeTable& rope, const NewRows& in, int32_t* status,
                               int num_sms, cudaStream_t stream);

// fp4 cache (kv_fp4.cu).
cudaError_t launch_quantize_fp4(const void* src, void* blocks, const int32_t* seq_lens, int B, int S_max, int S_blocks,
                                int len_cap, int Hkv, int D, int num_sms, cudaStream_t stream);
cudaError_t launch_read_fp4(const void* blocks, const PagedCache& pg, int S_blocks, void* out, int S_out,
                            const int32_t* seq_lens, int B, int len_cap, int Hkv, int D, int32_t* status,
                            int num_sms, cudaStream_t stream);
// The attention kernel over an fp4 cache for a pair of `rows` (n_tokens * group) query rows.
const ChunkKernel* fp4_chunk_kernel(int head_dim, bool f32_out, int rows);

}  // namespace kvd
