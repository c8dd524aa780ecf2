// Shared host/device declarations of the page tables, the rotary positions of
// several axes and the attention over selected blocks: parameters and launches.
#pragma once

#include <atomic>

#include "params.h"
#include "rope_fp4.h"

namespace kvd {

// Tokens of a stage of the attention over listed blocks, working warps of a CTA at most, stages of a CTA's ring
// (see BlocksShape).
constexpr int kBlocksStage = 32;
constexpr int blocks_warps(int D) { return D == 256 ? 8 : 4; }
constexpr int blocks_slots(int D) { return (D == 256 ? 192 : 96) * 1024 / (4 * D * kBlocksStage); }
// The attention over listed blocks (decode_blocks.cuh). A pair is a (sequence, query token, KV head).
struct BlocksParams {
    const void* q;            // bf16 [B, T, Hq, D]
    const void* k;            // bf16 cache [B, S_max, Hkv, D], or pool
    const void* v;
    const int32_t* blocks;    // [B, T, Hkv, K], entries outside [0, blocks the token sees) passed over
    const int32_t* seq_lens;
    void* out;                // [B, T, Hq, D] (shards > 1: fp32 [shards, B * T * Hq, D])
    float* lse;               // optional [B, T, Hq] (shards > 1: [shards, B * T * Hq])
    int32_t* status;
    float scale_log2;
    int B, T, Hq, Hkv, G, K, S_max;
    int block_log2, unit_log2;  // tokens of a block, and of a unit: 32 or 16 (the rows of a TMA box)
    int pairs, parts, shards; // CTAs of a pair that join over distributed shared memory, and groups of them over global memory
    int teams, head_warps, head_rows;  // teams of a CTA; warps of a team, which share a pair's query rows; rows of each
    PagedCache pg;
};
// Lets a kernel use so much shared memory and clusters of 16, once a device (a bit of *ready each).
cudaError_t allow_clusters(const void* kernel, int smem_bytes, std::atomic<uint64_t>* ready);
// Clusters of 1, 2, 4, 8 and 16 such CTAs that the current device runs at once (0: it cannot place one of that
// size), asked once a device (known: kMaxDevices of them).
cudaError_t clusters_at_once(const void* kernel, int threads, int smem_bytes, std::atomic<uint64_t>* ready, std::atomic<uint64_t>* known,
                             int (&n)[5]);
cudaError_t blocks_at_once_d64(int (&n)[5]);
cudaError_t blocks_at_once_d128(int (&n)[5]);
cudaError_t blocks_at_once_d256(int (&n)[5]);
cudaError_t launch_decode_blocks_d64(const BlocksParams& p, bool f32_out, cudaStream_t stream);
cudaError_t launch_decode_blocks_d128(const BlocksParams& p, bool f32_out, cudaStream_t stream);
cudaError_t launch_decode_blocks_d256(const BlocksParams& p, bool f32_out, cudaStream_t stream);

// Bounds of the keys of each block of tokens (block_bounds.cu).
struct BoundsParams {
    const void* k;            // bf16 cache or pool
    int8_t* codes;            // [B or pages, blocks of it, Hkv, 2, D]
    float* scales;            // [B or pages, blocks of it, Hkv]
    const int32_t* from_lens; // null: 0
    const int32_t* seq_lens;
    int32_t* status;
    int B, Hkv, D, S_max, block_shift, max_new;
    PagedCache pg;
};
cudaError_t launch_block_bounds(const BoundsParams& p, cudaStream_t stream);

// The blocks of the highest scores (block_select.cu).
struct SelectParams {
    const void* q;            // bf16 [B, T, Hq, D]
    const int8_t* codes;
    const float* scales;
    const int32_t* seq_lens;
    int32_t* blocks;          // out [B, T, Hkv, K]
    int32_t* status;
    uint32_t* keys;           // workspace [B, Hkv, T, max_blocks_scored]
    int B, T, Hq, Hkv, G, D, K, S_max, len_cap, block_shift, n_first, n_last, key_stride;
    int parts;                // CTAs of a (sequence, KV head)
    PagedCache pg;
};
cudaError_t launch_block_select(const SelectParams& p, cudaStream_t stream);
int select_ctas(int D, int G, int T);  // resident CTAs of a multiprocessor

// Page tables from lengths (pages.cu).
struct PagesParams {
    int32_t* table;           // [B, max_blocks]
    int32_t* free_pages;      // [num_pages], a stack
    int32_t* free_count;
    int32_t* seq_lens;
    const int32_t* new_lens;
    int32_t* pos;             // outputs, each optional
    int32_t* offsets;
    int32_t* slots;
    int32_t* positions;
    int32_t* status;
    int B, max_blocks, page_shift, num_pages;
    long long rows;           // length of slots and positions
};
constexpr int kPagesMaxBatch = 8192;  // four integers a sequence in shared memory
cudaError_t launch_pages(const PagesParams& p, cudaStream_t stream);

// Rotary positions of several axes (rope_axes.cu): pair i turns by positions[axes[i]].
struct RopeAxes {
    RopeTable table;
    const uint8_t* axes;          // [rotary_dim / 2]
    const int32_t* positions;     // axis a, row n at a * axis_stride + n
    long long axis_stride;
    int n_axes;
};
cudaError_t launch_rope_axes(const RopeAxes& rope, const void* x, long long xs, bool in32, void* y, long long ys, bool out32,
                             long long rows, int H, int D, int num_sms, cudaStream_t stream);
// Rows to the cache rows `slots` names; `in` as for launch_append_rope, its pos, offsets, B and T not used.
cudaError_t launch_append_axes(const AppendTarget& to, const RopeAxes& rope, const NewRows& in, const int32_t* slots,
                               long long cache_rows, int32_t* status, int num_sms, cudaStream_t stream);

}  // namespace kvd
