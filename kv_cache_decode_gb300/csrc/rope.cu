// Rotary positions: rows [rows, heads, D] turned by their positions (see
// rope.cuh for the phases). One read and one write of every element; bound by memory. A block takes a few
// rows: its threads first form the rows' rotary_dim / 2 cosines and sines in
// shared memory, once for all heads, then turn units of 16 columns.
#include <algorithm>

#include "../../include/kvdecode.h"
#include "rope.cuh"

namespace kvd {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;  // rows of a block, at most

template <bool IN32, bool OUT32>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeTable rope, const void* x, long long xs, void* y,
                                                            long long ys, const int32_t* __restrict__ positions,
                                                            long long rows, int rows_per_block, int H, int D) {
    extern __shared__ float2 s_cs[];  // [rows of the block][R / 2]
    const int R = rope.rotary_dim, half = R >> 1, units = (D + 15) >> 4;
    const long long row0 = (long long)blockIdx.x * rows_per_block;
    const int n = (int)min((long long)rows_per_block, rows - row0);
    for (int i = threadIdx.x; i < n * half; i += kRopeThreads) {
        const int r = i / half;
        s_cs[i] = rope_cos_sin(__ldg(positions + row0 + r), __ldg(rope.turns + (i - r * half)), rope.factor);
    }
    __syncthreads();
    const int per_row = H * units;
    for (int i = blockIdx.y * kRopeThreads + threadIdx.x; i < n * per_row; i += gridDim.y * kRopeThreads) {
        const int r = i / per_row, j = i - r * per_row;
        const int h = j / units, u = j - h * units;
        const RopeUnit ru = rope_unit(u, D, R, rope.interleaved);
        const size_t xe = (size_t)(row0 + r) * xs + (size_t)h * D, ye = (size_t)(row0 + r) * ys + (size_t)h * D;
        float a[8], b[8];
        load8<IN32>(x, xe + ru.ca, a);
        if (ru.cb >= 0) load8<IN32>(x, xe + ru.cb, b);
        if (ru.turn) rope_turn(a, b, s_cs + r * half + 8 * u, rope.interleaved);
        store8<OUT32>(y, ye + ru.ca, a);
        if (ru.cb >= 0) store8<OUT32>(y, ye + ru.cb, b);
    }
}

cudaError_t launch_rope(const RopeTable& rope, const void* x, long long xs, bool in32, void* y, long long ys, bool out32,
                        const int32_t* positions, long long rows, int H, int D, int num_sms, cudaStream_t stream) {
    const int rpb = (int)std::max(1LL, std::min((long long)kRopeRows, rows / (4LL * num_sms)));
    const long long bx = (rows + rpb - 1) / rpb;
    // Few rows: several blocks share a row's heads (each forms the cosines anew).
    const long long items = (long long)rpb * H * ((D + 15) / 16);
    const int by = (int)std::max(1LL, std::min((items + kRopeThreads - 1) / kRopeThreads, 2LL * num_sms / bx));
    const dim3 grid((unsigned)bx, (unsigned)by, 1);
    const size_t smem = (size_t)rpb * (rope.rotary_dim / 2) * sizeof(float2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kRopeThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
#define KVD_ROPE(A, B) cudaLaunchKernelEx(&cfg, rope_kernel<A, B>, rope, x, xs, y, ys, positions, rows, rpb, H, D)
    if (in32) return out32 ? KVD_ROPE(true, true) : KVD_ROPE(true, false);
    return out32 ? KVD_ROPE(false, true) : KVD_ROPE(false, false);
#undef KVD_ROPE
}

}  // namespace kvd
