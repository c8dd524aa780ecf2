// fp4 KV cache: the bulk conversion of a bf16 cache into blocks, and the read of
// blocks back to bf16 rows. D / 16 threads to a row, 16 columns (one scale) each. Both read
// and write every byte once and are bound by memory.
#include <algorithm>

#include "../../include/kvdecode.h"
#include "fp4.cuh"
#include "params.h"
#include "rope.cuh"

namespace kvd {

constexpr int kFp4Threads = 256;

template <int D>
__global__ void __launch_bounds__(kFp4Threads) quantize_fp4_kernel(const uint4* __restrict__ src,
                                                                   uint8_t* __restrict__ blocks,
                                                                   const int32_t* __restrict__ seq_lens, int B,
                                                                   int S_max, int S_blocks, int len_cap, int Hkv) {
    using Blk = Fp4Block<D>;
    constexpr int UN = D / 16;
    const int u = threadIdx.x % UN;
    const long long nblk = S_blocks >> 4, cap16 = (long long)(len_cap + 15) >> 4;
    // Rows in the blocks' order, (b, h, t): a warp writes neighbouring tokens of one block.
    const long long rows = (long long)B * Hkv * cap16 * 16;
    const long long groups = (long long)gridDim.x * (kFp4Threads / UN);
    const int g0 = threadIdx.x / UN;
    for (long long g = (long long)blockIdx.x * (kFp4Threads / UN) + g0; g - g0 < rows; g += groups) {
        const bool in = g < rows;
        const long long bh = in ? g / (cap16 * 16) : 0;
        const int t = in ? (int)(g - bh * cap16 * 16) : 0;
        const int b = (int)(bh / Hkv), h = (int)(bh - (long long)b * Hkv);
        int L = in ? __ldg(seq_lens + b) : 0;
        L = L < 0 ? 0 : (L > len_cap ? len_cap : L);
        const bool live = in && t < L;
        float a[8] = {}, c[8] = {};
        if (live) {
            const uint4* row = src + (((long long)b * S_max + t) * Hkv + h) * (D / 8) + 2 * u;
            unpack8(__ldg(row), a);
            unpack8(__ldg(row + 1), c);
        }
        float mb = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) mb = fmaxf(mb, fmaxf(fabsf(a[k]), fabsf(c[k])));
        float m = mb;
#pragma unroll
        for (int off = UN / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const uint32_t eb = fp4_row_exp(m);
        const float up = eb ? fp4_row_inv(eb) : 0.f;
        float inv, z[8];
        const uint32_t s = fp4_block_scale(mb * up, inv);
#pragma unroll
        for (int k = 0; k < 8; ++k) z[k] = __fmul_rn(__fmul_rn(a[k], up), inv);
        const uint32_t wa = e2m1x8(z);
#pragma unroll
        for (int k = 0; k < 8; ++k) z[k] = __fmul_rn(__fmul_rn(c[k], up), inv);
        const uint32_t wc = e2m1x8(z);
        if (live) {
            uint8_t* blk = blocks + (size_t)(bh * nblk + (t >> 4)) * Blk::BYTES;
            const int r = t & 15;
            *reinterpret_cast<uint2*>(blk + Blk::code(r, 16 * u)) = make_uint2(wa, wc);
            blk[Blk::scale(r, 16 * u)] = (uint8_t)s;
            if (u == 0) blk[Blk::exp(r)] = (uint8_t)eb;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kFp4Threads) read_fp4_kernel(const uint8_t* __restrict__ blocks, const PagedCache pg,
                                                               int S_blocks, uint4* __restrict__ out, int S_out,
                                                               const int32_t* __restrict__ seq_lens, int B,
                                                               int len_cap, int Hkv, int32_t* status) {
    using Blk = Fp4Block<D>;
    constexpr int UN = D / 16;
    const int u = threadIdx.x % UN;
    const long long cap16 = (long long)(len_cap + 15) >> 4;
    const long long rows = (long long)B * Hkv * cap16 * 16;
    const long long groups = (long long)gridDim.x * (kFp4Threads / UN);
    for (long long g = (long long)blockIdx.x * (kFp4Threads / UN) + threadIdx.x / UN; g < rows; g += groups) {
        const long long bh = g / (cap16 * 16);
        const int t = (int)(g - bh * cap16 * 16);
        const int b = (int)(bh / Hkv), h = (int)(bh - (long long)b * Hkv);
        int L = __ldg(seq_lens + b);
        L = L < 0 ? 0 : (L > len_cap ? len_cap : L);
        if (t >= L) continue;
        long long blk_i = bh * (S_blocks >> 4) + (t >> 4);
        bool ok = true;
        if (pg.block_table) {
            const int page = __ldg(pg.block_table + (size_t)b * pg.max_blocks + (t >> pg.page_shift));
            ok = page >= 0 && page < pg.num_pages;
            if (!ok && status && h == 0 && u == 0) atomicOr(status, KVD_STATUS_BAD_PAGE);
            const int in_page = t & ((1 << pg.page_shift) - 1);
            blk_i = (((long long)page * Hkv + h) << (pg.page_shift - 4)) + (in_page >> 4);
        }
        float f[8] = {}, f2[8] = {};
        if (ok) {
            const uint8_t* blk = blocks + (size_t)blk_i * Blk::BYTES;
            const int r = t & 15;
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(blk + Blk::code(r, 16 * u)));
            const uint32_t s = e4m3x2_to_f16x2(__ldg(blk + Blk::scale(r, 16 * u)) * 0x101u);
            const float up = fp4_row_scale(__ldg(blk + Blk::exp(r)));
            uint32_t v[4];
            e2m1x8_to_f16(w.x, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t x = hmul2(v[k], s);  // exact: 2 by 4 significant bits
                f[2 * k] = f16_lo(x) * up;
                f[2 * k + 1] = f16_hi(x) * up;
            }
            e2m1x8_to_f16(w.y, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t x = hmul2(v[k], s);
                f2[2 * k] = f16_lo(x) * up;
                f2[2 * k + 1] = f16_hi(x) * up;
            }
        }
        uint4* o = out + (((long long)b * S_out + t) * Hkv + h) * (D / 8) + 2 * u;
        o[0] = pack8(f);
        o[1] = pack8(f2);
    }
}

cudaError_t launch_quantize_fp4(const void* src, void* blocks, const int32_t* seq_lens, int B, int S_max, int S_blocks,
                                int len_cap, int Hkv, int D, int num_sms, cudaStream_t stream) {
    const long long rows = (long long)B * Hkv * ((len_cap + 15) / 16) * 16;
    const int per = kFp4Threads / (D / 16);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max(1LL, std::min((rows + per - 1) / per, 16LL * num_sms)), 1, 1);
    cfg.blockDim = dim3(kFp4Threads, 1, 1);
    cfg.stream = stream;
    auto* s = static_cast<const uint4*>(src);
    auto* d = static_cast<uint8_t*>(blocks);
#define KVD_Q4(DD) cudaLaunchKernelEx(&cfg, quantize_fp4_kernel<DD>, s, d, seq_lens, B, S_max, S_blocks, len_cap, Hkv)
    return D == 64 ? KVD_Q4(64) : D == 128 ? KVD_Q4(128) : D == 256 ? KVD_Q4(256) : cudaErrorInvalidValue;
#undef KVD_Q4
}

cudaError_t launch_read_fp4(const void* blocks, const PagedCache& pg, int S_blocks, void* out, int S_out,
                            const int32_t* seq_lens, int B, int len_cap, int Hkv, int D, int32_t* status, int num_sms,
                            cudaStream_t stream) {
    const long long rows = (long long)B * Hkv * ((len_cap + 15) / 16) * 16;
    const int per = kFp4Threads / (D / 16);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max(1LL, std::min((rows + per - 1) / per, 16LL * num_sms)), 1, 1);
    cfg.blockDim = dim3(kFp4Threads, 1, 1);
    cfg.stream = stream;
    auto* s = static_cast<const uint8_t*>(blocks);
    auto* d = static_cast<uint4*>(out);
#define KVD_R4(DD) cudaLaunchKernelEx(&cfg, read_fp4_kernel<DD>, s, pg, S_blocks, d, S_out, seq_lens, B, len_cap, Hkv, status)
    return D == 64 ? KVD_R4(64) : D == 128 ? KVD_R4(128) : D == 256 ? KVD_R4(256) : cudaErrorInvalidValue;
#undef KVD_R4
}

}  // namespace kvd
