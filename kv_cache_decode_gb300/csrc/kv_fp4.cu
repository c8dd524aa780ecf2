// fp4 KV cache: the bulk conversion of a bf16 cache into blocks, and the read of
// blocks back to bf16 rows. Both read and write every byte once and are bound by memory.
// A CTA takes 16 tokens of one sequence, the rows of a block, for all KV heads: the bf16
// side is then one contiguous stretch of 16 * n_heads_kv rows, and the divisions of the indexing are done once. A
// row is dealt to D / 16 threads (16 columns, one scale, each), and two passes' loads are in flight at a time.
// Measured: 32 sequences of up to 8,192 tokens, 8 heads of 128, 517 MB each way: to blocks 79 us (6.5 TB/s), back 90 (5.8).
#include "../../include/kvdecode.h"
#include "fp4.cuh"
#include "rope.cuh"

namespace kvd {

constexpr int kFp4Threads = 256;

// Rows of a pass of the CTA: 16 tokens of HP heads, thread = (token, head, unit). What a CTA takes: all heads of one block;
// where two passes hold more heads than there are, as many of 1 << sh consecutive blocks (64 sequences of up to 30,000
// tokens, one head of 64, to blocks and back: 101 us, 355 with a block to a CTA); or, where there are few blocks, a share
// of the heads of one (6 sequences of up to 432 tokens, 19 heads of 256: 16 us, 26 with all heads).
enum class Fp4Deal { kBlock, kBlocks, kHeads };
template <int D>
struct Fp4Pass {
    static constexpr int UN = D / 16, HP = kFp4Threads / (16 * UN);  // D 256: 1, 128: 2, 64: 4
};

template <int D, Fp4Deal DEAL>
__global__ void __launch_bounds__(kFp4Threads) quantize_fp4_kernel(const uint4* __restrict__ src,
                                                                   uint8_t* __restrict__ blocks,
                                                                   const int32_t* __restrict__ seq_lens, int n_grp, int sh,
                                                                   int S_max, int S_blocks, int len_cap, int Hkv) {
    using Blk = Fp4Block<D>;
    constexpr int UN = Fp4Pass<D>::UN, HP = Fp4Pass<D>::HP;
    if (DEAL != Fp4Deal::kBlocks) sh = 0;
    const int b = blockIdx.x / n_grp, blk0 = (blockIdx.x - b * n_grp) << sh;
    const int u = threadIdx.x % UN, hp = threadIdx.x / UN % HP, r = threadIdx.x / (UN * HP);
    int L = __ldg(seq_lens + b);
    L = L < 0 ? 0 : (L > len_cap ? len_cap : L);
    if (16 * blk0 >= L) return;
    constexpr int NP = DEAL == Fp4Deal::kBlocks ? 2 : 1;  // of a thread's two places, each its block, or both the one block
    bool live[NP];
    const uint4* row[NP];
    uint8_t* out[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int blk_i = blk0 + ((hp + k * HP) & ((1 << sh) - 1)), t = 16 * blk_i + r;
        live[k] = t < L;
        row[k] = src + ((size_t)b * S_max + t) * Hkv * (D / 8) + 2 * u;
        out[k] = blocks + ((size_t)b * Hkv * (S_blocks >> 4) + blk_i) * Blk::BYTES;
    }
    const size_t head_bytes = (size_t)(S_blocks >> 4) * Blk::BYTES;
    constexpr bool PARTS = DEAL == Fp4Deal::kHeads;
    for (int h0 = PARTS ? blockIdx.y * 2 * HP : 0; h0 < Hkv; h0 += PARTS ? gridDim.y * 2 * HP : 2 * HP >> sh) {
        uint4 v[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int h = h0 + ((hp + k * HP) >> sh);
            v[k][0] = v[k][1] = make_uint4(0u, 0u, 0u, 0u);
            if (live[k % NP] && h < Hkv) {
                v[k][0] = __ldcs(row[k % NP] + (size_t)h * (D / 8));
                v[k][1] = __ldcs(row[k % NP] + (size_t)h * (D / 8) + 1);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int h = h0 + ((hp + k * HP) >> sh);
            const uint32_t w[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w, v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
            // The largest magnitude, two bf16 values at a time (exact).
            __nv_bfloat162 m2 = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
            for (int i = 1; i < 8; ++i) m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
            const float mb = fmaxf(__low2float(m2), __high2float(m2));
            float m = mb;
#pragma unroll
            for (int off = UN / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            const uint32_t eb = fp4_row_exp(m);
            const float up = eb ? fp4_row_inv(eb) : 0.f;
            float inv, z[8];
            const uint32_t s = fp4_block_scale(mb * up, inv);
            // A power of two may be taken into the factor: the products round the same, unless it overflows
            // (rows below 2^-115), where the steps are taken one by one.
            const float c = up * inv;
            const bool fits = c < 1.7e38f;
            const float c1 = fits ? c : up, c2 = fits ? 1.f : inv;
            uint32_t code[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[2 * i] = __fmul_rn(bf16_lo(w[4 * q + i]), c1);
                    z[2 * i + 1] = __fmul_rn(bf16_hi(w[4 * q + i]), c1);
                }
                if (!fits) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[i] = __fmul_rn(z[i], c2);
                }
                code[q] = e2m1x8(z);
            }
            if (live[k % NP] && h < Hkv) {
                uint8_t* blk = out[k % NP] + h * head_bytes;
                *reinterpret_cast<uint2*>(blk + Blk::code(r, 16 * u)) = make_uint2(code[0], code[1]);
                blk[Blk::scale(r, 16 * u)] = (uint8_t)s;
                if (u == 0) blk[Blk::exp(r)] = (uint8_t)eb;
            }
        }
    }
}

template <int D, Fp4Deal DEAL>
__global__ void __launch_bounds__(kFp4Threads) read_fp4_kernel(const uint8_t* __restrict__ blocks, const PagedCache pg,
                                                               int S_blocks, uint4* __restrict__ out, int S_out,
                                                               const int32_t* __restrict__ seq_lens, int n_grp, int sh,
                                                               int len_cap, int Hkv, int32_t* status) {
    using Blk = Fp4Block<D>;
    constexpr int UN = Fp4Pass<D>::UN, HP = Fp4Pass<D>::HP;
    if (DEAL != Fp4Deal::kBlocks) sh = 0;
    const int b = blockIdx.x / n_grp, blk0 = (blockIdx.x - b * n_grp) << sh;
    const int u = threadIdx.x % UN, hp = threadIdx.x / UN % HP, r = threadIdx.x / (UN * HP);
    int L = __ldg(seq_lens + b);
    L = L < 0 ? 0 : (L > len_cap ? len_cap : L);
    if (16 * blk0 + r >= L) return;
    const size_t step = pg.block_table ? (size_t)1 << (pg.page_shift - 4) : (size_t)(S_blocks >> 4);
    constexpr int NP = DEAL == Fp4Deal::kBlocks ? 2 : 1;
    bool live[NP], ok[NP];
    size_t first[NP];  // block of head 0; the next head's is `step` further
    uint4* o[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int blk_i = blk0 + ((hp + k * HP) & ((1 << sh) - 1)), t = 16 * blk_i + r;
        live[k] = NP == 1 || t < L;
        ok[k] = live[k];
        first[k] = (size_t)b * Hkv * step + blk_i;
        if (pg.block_table && live[k]) {
            const int page = __ldg(pg.block_table + (size_t)b * pg.max_blocks + (t >> pg.page_shift));
            ok[k] = page >= 0 && page < pg.num_pages;
            if (!ok[k] && status && u == 0 && r == 0) atomicOr(status, KVD_STATUS_BAD_PAGE);
            first[k] = (size_t)(ok[k] ? page : 0) * Hkv * step + (blk_i & (step - 1));
        }
        o[k] = out + ((size_t)b * S_out + t) * Hkv * (D / 8) + 2 * u;
    }
    constexpr bool PARTS = DEAL == Fp4Deal::kHeads;
    for (int h0 = PARTS ? blockIdx.y * 2 * HP : 0; h0 < Hkv; h0 += PARTS ? gridDim.y * 2 * HP : 2 * HP >> sh) {
        uint2 w[2];
        uint32_t sb[2], eb[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int h = h0 + ((hp + k * HP) >> sh);
            w[k] = make_uint2(0u, 0u);
            sb[k] = eb[k] = 0u;
            if (ok[k % NP] && h < Hkv) {
                const uint8_t* blk = blocks + (first[k % NP] + h * step) * Blk::BYTES;
                w[k] = __ldcs(reinterpret_cast<const uint2*>(blk + Blk::code(r, 16 * u)));
                sb[k] = __ldg(blk + Blk::scale(r, 16 * u));
                eb[k] = __ldg(blk + Blk::exp(r));
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int h = h0 + ((hp + k * HP) >> sh);
            if (!live[k % NP] || h >= Hkv) continue;
            const uint32_t s = e4m3x2_to_f16x2(sb[k] * 0x101u);
            const float up = fp4_row_scale(eb[k]);
            uint4 q[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t v[4], f[4];
                e2m1x8_to_f16(x ? w[k].y : w[k].x, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t y = hmul2(v[i], s);  // exact: 2 by 4 significant bits
                    f[i] = pack_bf16x2(f16_lo(y) * up, f16_hi(y) * up);
                }
                q[x] = make_uint4(f[0], f[1], f[2], f[3]);
            }
            o[k % NP][(size_t)h * (D / 8)] = q[0];
            o[k % NP][(size_t)h * (D / 8) + 1] = q[1];
        }
    }
}

// log2 of the blocks a CTA takes: two passes' places over the heads, as far as about 8 CTAs per SM are left.
static int blocks_log2(int B, int n_blk, int Hkv, int D, int num_sms) {
    int sh = 0;
    while ((Hkv << (sh + 1)) <= 2 * kFp4Threads / D && ((long long)B * n_blk >> (sh + 1)) >= 8LL * num_sms) ++sh;
    return sh;
}

// CTAs that share a block's heads where there are few blocks: up to about 4 CTAs per SM, two passes each at least.
static unsigned head_parts(long long ctas, int Hkv, int D, int sh, int num_sms) {
    const int heads = 2 * kFp4Threads / D >> sh;
    const long long most = (Hkv + heads - 1) / heads, want = (4LL * num_sms + ctas - 1) / ctas;
    return (unsigned)(want < most ? want : most);
}

cudaError_t launch_quantize_fp4(const void* src, void* blocks, const int32_t* seq_lens, int B, int S_max, int S_blocks,
                                int len_cap, int Hkv, int D, int num_sms, cudaStream_t stream) {
    const int n_blk = (len_cap + 15) / 16, sh = blocks_log2(B, n_blk, Hkv, D, num_sms), n_grp = (n_blk + (1 << sh) - 1) >> sh;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)B * n_grp), head_parts((long long)B * n_grp, Hkv, D, sh, num_sms), 1);
    cfg.blockDim = dim3(kFp4Threads, 1, 1);
    cfg.stream = stream;
    auto* s = static_cast<const uint4*>(src);
    auto* d = static_cast<uint8_t*>(blocks);
#define KVD_Q4(DD)                                                                                       \
    cudaLaunchKernelEx(&cfg, sh ? quantize_fp4_kernel<DD, Fp4Deal::kBlocks> \
                             : cfg.gridDim.y > 1 ? quantize_fp4_kernel<DD, Fp4Deal::kHeads> \
                             : quantize_fp4_kernel<DD, Fp4Deal::kBlock>, s, d, seq_lens, n_grp, sh, S_max, S_blocks, len_cap, Hkv)
    return D == 64 ? KVD_Q4(64) : D == 128 ? KVD_Q4(128) : D == 256 ? KVD_Q4(256) : cudaErrorInvalidValue;
#undef KVD_Q4
}

cudaError_t launch_read_fp4(const void* blocks, const PagedCache& pg, int S_blocks, void* out, int S_out,
                            const int32_t* seq_lens, int B, int len_cap, int Hkv, int D, int32_t* status,
                            int num_sms, cudaStream_t stream) {
    const int n_blk = (len_cap + 15) / 16, sh = blocks_log2(B, n_blk, Hkv, D, num_sms), n_grp = (n_blk + (1 << sh) - 1) >> sh;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)B * n_grp), head_parts((long long)B * n_grp, Hkv, D, sh, num_sms), 1);
    cfg.blockDim = dim3(kFp4Threads, 1, 1);
    cfg.stream = stream;
    auto* s = static_cast<const uint8_t*>(blocks);
    auto* d = static_cast<uint4*>(out);
#define KVD_R4(DD)                                                                                       \
    cudaLaunchKernelEx(&cfg, sh ? read_fp4_kernel<DD, Fp4Deal::kBlocks> \
                             : cfg.gridDim.y > 1 ? read_fp4_kernel<DD, Fp4Deal::kHeads> \
                             : read_fp4_kernel<DD, Fp4Deal::kBlock>, s, pg, S_blocks, d, S_out, seq_lens, n_grp, sh, len_cap, Hkv, status)
    return D == 64 ? KVD_R4(64) : D == 128 ? KVD_R4(128) : D == 256 ? KVD_R4(256) : cudaErrorInvalidValue;
#undef KVD_R4
}

}  // namespace kvd
