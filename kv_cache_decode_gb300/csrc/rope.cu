// Rotary positions: rows [rows, heads, D] turned by their positions (see
// rope.cuh for the phases). One read and one write of every element; bound by memory. A warp takes a
// row, or a share of its heads where there are few rows, with nothing to wait for but its own loads.
#include "../../include/kvdecode.h"
#include "rope.cuh"

namespace kvd {

// Blocks of 4 warps: with 8, 4,099 fp32 rows of 40 x 128 take 33.1 us instead of 30.0, and 65,536 bf16 rows of
// 32 x 128 160.4 instead of 156.0 (1.07 GB: 6.9 TB/s, the copy rate).
constexpr int kRopeWarps = 4;

template <bool IN32, bool OUT32, int DD>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const RopeTable rope, const void* x, long long xs, void* y,
                                                               long long ys, const int32_t* __restrict__ positions,
                                                               long long rows, int parts, int H, int D) {
    extern __shared__ __align__(16) float2 s_cs[];  // [warps][R / 2]
    const long long w = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    const long long row = w / parts;
    if (row >= rows) return;
    RopeWarp<DD> rw;
    rw.init(rope, __ldg(positions + row), D, s_cs + (threadIdx.x >> 5) * (rope.rotary_dim >> 1));
    rw.template heads<IN32, OUT32>(x, (size_t)row * xs, y, (size_t)row * ys, H, (int)(w - row * parts), parts);
}

// Rows of at most 32 units (a warp's step): several rows to a warp. 500,000 bf16 rows of one head of 128 (256 MB) take 57 us,
// by a warp each 219; 200,000 of 4 heads of 64 take 38, by a warp each 88. What is left over the copy's 38 and 30 is in part
// the instructions of the cosines and sines, 64 or 32 a row: shorter ones took 66 to 57, and 40 to 38.
template <bool IN32, bool OUT32, bool ONE>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_rows_kernel(const RopeTable rope, const void* x, long long xs, void* y,
                                                                    long long ys, const int32_t* __restrict__ positions,
                                                                    long long rows, int per_warp, int H, int D) {
    extern __shared__ __align__(16) float2 s_cs[];  // [warps][per_warp][R / 2]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = ((long long)blockIdx.x * kRopeWarps + warp) * per_warp;
    if (row >= rows) return;
    const int n = (int)min((long long)per_warp, rows - row);
    const RopeTokens rt{D, (D + 15) >> 4, rope.rotary_dim, n, rope.interleaved != 0, 0xffffffffu,
                        s_cs + (size_t)warp * per_warp * (rope.rotary_dim >> 1)};
    const long long t = lane < n ? __ldg(positions + row + lane) : 0;
    rt.heads<IN32, OUT32, ONE>(x, (size_t)row * xs, (size_t)xs, y, (size_t)row * ys, (size_t)ys, ONE ? 1 : H, rope, t,
                               [&]() { rt.table(rope, t); });
}

cudaError_t launch_rope(const RopeTable& rope, const void* x, long long xs, bool in32, void* y, long long ys, bool out32,
                        const int32_t* positions, long long rows, int H, int D, int num_sms, cudaStream_t stream) {
    const long long units = (long long)H * ((D + 15) / 16), steps = (units + 31) / 32;
    const int per_warp = rope_tokens(rows, units, 64, num_sms);
    if (per_warp > 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((rows + per_warp * kRopeWarps - 1) / (per_warp * kRopeWarps)), 1, 1);
        cfg.blockDim = dim3(kRopeWarps * 32, 1, 1);
        if (H > 1) cfg.dynamicSmemBytes = (size_t)kRopeWarps * per_warp * (rope.rotary_dim / 2) * sizeof(float2);
        cfg.stream = stream;
#define KVD_ROPE(A, B)                                                                                                 \
    cudaLaunchKernelEx(&cfg, H == 1 ? rope_rows_kernel<A, B, true> : rope_rows_kernel<A, B, false>, rope, x, xs, y, ys, \
                       positions, rows, per_warp, H, D)
        if (in32) return out32 ? KVD_ROPE(true, true) : KVD_ROPE(true, false);
        return out32 ? KVD_ROPE(false, true) : KVD_ROPE(false, false);
#undef KVD_ROPE
    }
    const int parts = rope_parts(rows, steps, num_sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows * parts + kRopeWarps - 1) / kRopeWarps), 1, 1);
    cfg.blockDim = dim3(kRopeWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = (size_t)kRopeWarps * (rope.rotary_dim / 2) * sizeof(float2);
    cfg.stream = stream;
#define KVD_ROPE_D(A, B, DD) cudaLaunchKernelEx(&cfg, rope_kernel<A, B, DD>, rope, x, xs, y, ys, positions, rows, parts, H, D)
#define KVD_ROPE(A, B) \
    (D == 64 ? KVD_ROPE_D(A, B, 64) : D == 128 ? KVD_ROPE_D(A, B, 128) : D == 256 ? KVD_ROPE_D(A, B, 256) : KVD_ROPE_D(A, B, 0))
    if (in32) return out32 ? KVD_ROPE(true, true) : KVD_ROPE(true, false);
    return out32 ? KVD_ROPE(false, true) : KVD_ROPE(false, false);
#undef KVD_ROPE
#undef KVD_ROPE_D
}

}  // namespace kvd
