// Bounds of the keys of each block of tokens: for every column the largest and the smallest value over the block's
// tokens, in 8 bits rounded outwards, with one float32 scale a (block, KV head):
//   a = max |k|, scale = a / 127, hi_d = ceil(max_t k_td / scale), lo_d = floor(min_t k_td / scale), in [-127, 127],
// the divisions IEEE float32. For any query, sum_d max(q_d hi_d, q_d lo_d) * scale is then at least q . k_t for
// every token of the block (up to float32's rounding): what block_select.cu scores blocks by. A block with a
// key that is not finite gets the scale NaN and codes 0.
//
// A CTA of four warps takes one KV head of one block, or, of blocks of up to 4,096 values, a warp each: 2 *
// block * D bytes read once, 2 D + 4 written; bound by memory for prompts (80.5 us for 537 MB in blocks of 64,
// the copy rate; in blocks of 16 87, at 64 columns 115), by latency for the few blocks that a step fills (3.3
// us). A thread holds 8 columns' running maxima and minima of its tokens as bf16 pairs (exact), eight loads in
// flight; the divisions are shared out to the lanes that hold the same columns (all of them in each: 83, 106
// and 175 us). Blocks of 16 of 128 columns by whole CTAs: 210.
#include "../../include/kvdecode.h"
#include "blocks.h"
#include "common.cuh"

namespace kvd {

constexpr int kBoundsThreads = 128;

__device__ __forceinline__ uint32_t max_bf16x2_nan(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// WPI: warps of an item, a (block, KV head).
template <int D, int WPI>
__global__ void __launch_bounds__(kBoundsThreads) block_bounds_kernel(const BoundsParams p, unsigned per_seq, unsigned items) {
    constexpr int TPR = D / 8, RPP = 32 * WPI / TPR, IPC = 4 / WPI;  // threads of a row, rows of a pass, items of a CTA
    __shared__ uint4 s_hi[4][TPR], s_lo[4][TPR];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x % (32 * WPI), lane = tid & 31, warp = tid >> 5;  // of the item's
    const unsigned item = blockIdx.x * IPC + threadIdx.x / (32 * WPI);  // (items: below 2^31)
    if (item >= items) return;
    const unsigned rest = item / (unsigned)p.Hkv;
    const int h = (int)(item - rest * p.Hkv), b = (int)(rest / per_seq), i = (int)(rest - b * per_seq);
    const int raw = __ldg(p.seq_lens + b), len = raw < 0 ? 0 : raw > p.S_max ? p.S_max : raw;
    const int raw0 = p.from_lens ? __ldg(p.from_lens + b) : 0, from = raw0 < 0 ? 0 : raw0;
    const int bs = p.block_shift, n_tok = 1 << bs;
    if (i == 0 && h == 0 && tid == 0 && p.status && (raw != len || raw0 != from || (long long)len - from > p.max_new))
        atomicOr(p.status, KVD_STATUS_SEQ_LEN_CLAMPED);
    const int j = (from >> bs) + i;
    if (j >= (len >> bs)) return;  // not full
    // ---- where the block and its bounds lie ----
    const long long tok = (long long)j << bs;
    long long row, block;
    if (p.pg.block_table) {
        const int page = __ldg(p.pg.block_table + (size_t)b * p.pg.max_blocks + (tok >> p.pg.page_shift));
        if ((unsigned)page >= (unsigned)p.pg.num_pages) {
            if (h == 0 && tid == 0 && p.status) atomicOr(p.status, KVD_STATUS_BAD_PAGE);
            return;
        }
        row = ((long long)page << p.pg.page_shift) + (tok & ((1LL << p.pg.page_shift) - 1));
        block = row >> bs;
    } else {
        row = (long long)b * p.S_max + tok;
        block = (long long)b * (p.S_max >> bs) + j;
    }
    // ---- maxima and minima of this thread's columns ----
    const __nv_bfloat16* rows = static_cast<const __nv_bfloat16*>(p.k) + ((size_t)row * p.Hkv + h) * D;
    const uint4* k = reinterpret_cast<const uint4*>(rows) + tid % TPR;
    const size_t step = (size_t)p.Hkv * TPR;  // 16-byte vectors between tokens
    uint32_t hi[4], lo[4];
    const int t0 = tid / TPR;
    for (int t = t0; t < n_tok || t == t0; t += 8 * RPP) {  // eight loads in flight; a thread past the tokens repeats the last
        uint4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __ldg(k + (size_t)min(t + e * RPP, n_tok - 1) * step);
        if (t == t0) {
            hi[0] = lo[0] = v[0].x, hi[1] = lo[1] = v[0].y, hi[2] = lo[2] = v[0].z, hi[3] = lo[3] = v[0].w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) {
                hi[c4] = max_bf16x2_nan(hi[c4], w[c4]);
                lo[c4] = min_bf16x2(lo[c4], w[c4]);
            }
        }
    }
#pragma unroll
    for (int off = TPR; off < 32; off <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = max_bf16x2_nan(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], off));
            lo[e] = min_bf16x2(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], off));
        }
    if constexpr (WPI > 1) {
        if (lane < TPR) {
            s_hi[warp][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            s_lo[warp][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        __syncthreads();
        if (warp != 0) return;
    }
    // ---- the scale and the codes: a lane takes a share of its 8 columns, since all that hold them have the same result ----
    constexpr int SHARES = 32 / TPR, PAIRS = 4 / SHARES;  // lanes of the same columns; pairs of columns of each
    const int share = lane / TPR, c = lane % TPR;
    if constexpr (WPI > 1) {
#pragma unroll
        for (int w = 1; w < WPI; ++w) {
            const uint4 x = s_hi[w][c], y = s_lo[w][c];
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hi[e] = max_bf16x2_nan(hi[e], xs[e]);
                lo[e] = min_bf16x2(lo[e], ys[e]);
            }
        }
    }
    float fh[2 * PAIRS], fl[2 * PAIRS], a = 0.f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < PAIRS; ++e) {
        uint32_t x = hi[e], y = lo[e];
#pragma unroll
        for (int g = 1; g < SHARES; ++g)
            if (share == g) x = hi[g * PAIRS + e], y = lo[g * PAIRS + e];
        fh[2 * e] = bf16_lo(x), fh[2 * e + 1] = bf16_hi(x);
        fl[2 * e] = bf16_lo(y), fl[2 * e + 1] = bf16_hi(y);
    }
#pragma unroll
    for (int e = 0; e < 2 * PAIRS; ++e) {
        bad |= !isfinite(fh[e]) || !isfinite(fl[e]);  // a NaN shows in the maximum, infinities in either
        a = fmaxf(a, fmaxf(fabsf(fh[e]), fabsf(fl[e])));
    }
    a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));  // (not negative: their bits are in order)
    bad = __any_sync(0xffffffffu, bad);
    const float s = bad ? __uint_as_float(0x7fffffffu) : __fdiv_rn(a, 127.f);
    const size_t at = (size_t)block * p.Hkv + h;
    if (lane == 0) p.scales[at] = s;
    uint32_t up[(PAIRS + 1) / 2] = {}, down[(PAIRS + 1) / 2] = {};
    if (!bad && s > 0.f) {
#pragma unroll
        for (int e = 0; e < 2 * PAIRS; ++e) {
            const int x = max(-127, min(127, __float2int_ru(__fdiv_rn(fh[e], s))));
            const int y = max(-127, min(127, __float2int_rd(__fdiv_rn(fl[e], s))));
            up[e >> 2] |= (uint32_t)(x & 0xff) << (8 * (e & 3));
            down[e >> 2] |= (uint32_t)(y & 0xff) << (8 * (e & 3));
        }
    }
    int8_t* dst = p.codes + at * 2 * D + 8 * c + 2 * PAIRS * share;
    if constexpr (PAIRS == 1) {
        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)up[0];
        *reinterpret_cast<uint16_t*>(dst + D) = (uint16_t)down[0];
    } else if constexpr (PAIRS == 2) {
        *reinterpret_cast<uint32_t*>(dst) = up[0];
        *reinterpret_cast<uint32_t*>(dst + D) = down[0];
    } else {
        *reinterpret_cast<uint2*>(dst) = make_uint2(up[0], up[1]);
        *reinterpret_cast<uint2*>(dst + D) = make_uint2(down[0], down[1]);
    }
}

cudaError_t launch_block_bounds(const BoundsParams& p, cudaStream_t stream) {
    const int per_seq = (int)(((long long)p.max_new + (1 << p.block_shift) - 1) >> p.block_shift);  // blocks max_new tokens can fill
    cudaLaunchConfig_t cfg = {};
    const long long items = (long long)p.B * per_seq * p.Hkv;
    const bool small = (p.D << p.block_shift) <= 4096;
    cfg.gridDim = dim3((unsigned)(small ? (items + 3) / 4 : items), 1, 1);
    cfg.blockDim = dim3(kBoundsThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto launch = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, p, (unsigned)per_seq, (unsigned)items); };
    switch (p.D) {
        case 64: return launch(small ? block_bounds_kernel<64, 1> : block_bounds_kernel<64, 4>);
        case 128: return launch(small ? block_bounds_kernel<128, 1> : block_bounds_kernel<128, 4>);
        case 256: return launch(small ? block_bounds_kernel<256, 1> : block_bounds_kernel<256, 4>);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvd
