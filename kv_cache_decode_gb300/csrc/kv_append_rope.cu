// The append with the rotation of the positions on the way: each new token's
// key heads are turned by the token's position and stored in the cache (bf16,
// int8, fp8 or fp4; contiguous or paged), its value heads stored as they are,
// and its query heads turned into q_out. One read of q, k, v and one write of
// each; a separate rotation would read and write q and k once more. Bound by
// memory for prompts and by latency for single tokens.
//
// A block takes a few tokens (fewer blocks per token for many tokens, several
// blocks per token for few): each token's sequence, position and place in the
// cache, then the rotary_dim / 2 cosines and sines, are worked out once in
// shared memory for all its heads. A head is dealt to D / 16 threads as in
// rope.cuh; where the cache is quantized these threads find the row's (and,
// fp4, the 16 columns') largest magnitude by shuffles, so a row goes from its
// load to its codes in registers.
#include <algorithm>

#include "../../include/kvdecode.h"
#include "fp4.cuh"
#include "rope.cuh"

namespace kvd {

constexpr int kAppThreads = 256;
constexpr int kAppRows = 4;  // tokens of a block, at most

// DD: head dimension of a quantized cache (64, 128, 256), 0 for bf16 (any multiple of 8).
template <CacheForm FORM, int DD>
__global__ void __launch_bounds__(kAppThreads) append_rope_kernel(const AppendTarget to, const RopeTable rope,
                                                                  const NewRows in, int rows_per_block,
                                                                  int32_t* status) {
    extern __shared__ float2 s_cs[];        // [tokens of the block][R / 2]
    __shared__ long long s_pos[kAppRows];   // position, or LLONG_MIN: the row belongs to no sequence
    __shared__ long long s_dst[kAppRows];   // cache row (fp4: block of head 0), or -1: not appended
    __shared__ int s_slot[kAppRows];        // fp4: token's place in its block
    pdl_launch_dependents();  // the attention that may follow waits for this grid before it reads anything
    const int tid = threadIdx.x, lane = tid & 31;
    const int D = DD ? DD : in.D;
    const int R = rope.turns ? rope.rotary_dim : 0, half = R >> 1, units = (D + 15) >> 4;
    const long long row0 = (long long)blockIdx.x * rows_per_block;
    const int n = (int)min((long long)rows_per_block, in.rows - row0);

    // ---- each token's sequence, position and place ----
    if (tid < 32 * n) {
        const int r = tid >> 5;
        const long long row = row0 + r;
        int b;
        long long i;
        bool live = true;
        if (in.offsets) {
            int cnt = 0;  // offsets <= row, counted over all of them at once rather than by dependent steps
            for (int j = lane; j <= in.B; j += 32) cnt += __ldg(in.offsets + j) <= row ? 1 : 0;
            b = __reduce_add_sync(0xffffffffu, cnt) - 1;
            live = b >= 0 && b < in.B;
            i = live ? row - __ldg(in.offsets + b) : 0;
            if (i < 0) live = false;
        } else {
            b = (int)(row / in.T);
            i = row - (long long)b * in.T;
        }
        if (lane == 0) {
            long long t = live ? (long long)__ldg(in.pos + b) + i : LLONG_MIN;
            long long dst = -1;
            int slot = 0;
            if (live && (t < 0 || t >= to.S_max)) {
                if (status && blockIdx.y == 0) atomicOr(status, KVD_STATUS_POS_OUT_OF_RANGE);
            } else if (live) {
                long long seq = b, cap = to.S_max, at = t;  // sequence (page), its capacity, place in it
                bool ok = true;
                if (to.pg.block_table) {
                    seq = __ldg(to.pg.block_table + (size_t)b * to.pg.max_blocks + (t >> to.pg.page_shift));
                    cap = 1LL << to.pg.page_shift;
                    at = t & (cap - 1);
                    ok = seq >= 0 && seq < to.pg.num_pages;
                    if (!ok && status && blockIdx.y == 0) atomicOr(status, KVD_STATUS_BAD_PAGE);
                }
                if (ok) {
                    dst = FORM == CacheForm::kFp4 ? seq * in.Hkv * (cap >> 4) + (at >> 4) : seq * cap + at;
                    slot = (int)(at & 15);
                }
            }
            s_pos[r] = t;
            s_dst[r] = dst;
            s_slot[r] = slot;
        }
    }
    __syncthreads();
    for (int i = tid; i < n * half; i += kAppThreads) {
        const int r = i / half;
        s_cs[i] = rope_cos_sin(s_pos[r], __ldg(rope.turns + (i - r * half)), rope.factor);
    }
    __syncthreads();

    const int start = blockIdx.y * kAppThreads + tid, step = gridDim.y * kAppThreads;
    // ---- queries ----
    if (in.q) {
        const int per_row = in.Hq * units;
        for (int i = start; i < n * per_row; i += step) {
            const int r = i / per_row, j = i - r * per_row, h = j / units, u = j - h * units;
            if (s_pos[r] == LLONG_MIN) continue;
            const RopeUnit ru = rope_unit(u, D, R, rope.interleaved);
            const size_t qe = (size_t)(row0 + r) * in.qs + (size_t)h * D, oe = (size_t)(row0 + r) * in.qos + (size_t)h * D;
            float a[8], b[8];
            load8<false>(in.q, qe + ru.ca, a);
            if (ru.cb >= 0) load8<false>(in.q, qe + ru.cb, b);
            if (ru.turn) rope_turn(a, b, s_cs + r * half + 8 * u, rope.interleaved);
            store8<false>(in.q_out, oe + ru.ca, a);
            if (ru.cb >= 0) store8<false>(in.q_out, oe + ru.cb, b);
        }
    }
    // ---- keys, then values; whole warps stay in the loop for the shuffles ----
    const int per_row = 2 * in.Hkv * units, total = n * per_row;
    for (int i = start; i - lane < total; i += step) {
        const bool live0 = i < total;
        const int ii = live0 ? i : 0;
        const int r = ii / per_row, j = ii - r * per_row, hh = j / units, u = j - hh * units;
        const bool value = hh >= in.Hkv;
        const int h = value ? hh - in.Hkv : hh;
        const long long dst = s_dst[r];
        const bool live = live0 && dst >= 0;
        const int Rh = value ? 0 : R;
        const RopeUnit ru = rope_unit(u, D, Rh, rope.interleaved);
        const void* src = value ? in.v : in.k;
        const size_t e = (size_t)(row0 + r) * (value ? in.vs : in.ks) + (size_t)h * D;
        float a[8] = {}, b[8] = {};
        if (live) {
            load8<false>(src, e + ru.ca, a);
            if (ru.cb >= 0) load8<false>(src, e + ru.cb, b);
            if (ru.turn) rope_turn(a, b, s_cs + r * half + 8 * u, rope.interleaved);
        }
        if constexpr (FORM == CacheForm::kBf16) {
            if (live) {
                void* cache = value ? to.v : to.k;
                const size_t o = ((size_t)dst * in.Hkv + h) * D;
                store8<false>(cache, o + ru.ca, a);
                if (ru.cb >= 0) store8<false>(cache, o + ru.cb, b);
            }
        } else {
            constexpr int UN = DD / 16;  // threads of a row
            unpack8(pack8(a), a);        // the rotated row as bf16, as the plain append would be given it
            unpack8(pack8(b), b);
            float ma = 0.f, mb = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                ma = fmaxf(ma, fabsf(a[k]));
                mb = fmaxf(mb, fabsf(b[k]));
            }
            float m = fmaxf(ma, mb);
#pragma unroll
            for (int off = UN / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            if constexpr (FORM == CacheForm::kFp4) {
                using Blk = Fp4Block<DD>;
                // The other 8 of each vector's 16 columns may lie with another thread (halves).
                const int R16 = (ru.turn && !rope.interleaved) ? Rh >> 4 : 0;  // this vector's unit map, see rope_unit
                auto partner = [&](int c) -> float {
                    const int v = (c >> 3) ^ 1;  // the neighbour vector of the row
                    const int pu = R16 ? (v < R16 ? v : v - R16) : v >> 1;
                    const bool second = R16 ? v >= R16 : (v & 1);
                    const int from = (lane & ~(UN - 1)) + pu;
                    const float xa = __shfl_sync(0xffffffffu, ma, from), xb = __shfl_sync(0xffffffffu, mb, from);
                    return second ? xb : xa;
                };
                const float na = fmaxf(ma, partner(ru.ca)), nb = fmaxf(mb, partner(ru.cb));
                const uint32_t eb = fp4_row_exp(m);
                const float up = eb ? fp4_row_inv(eb) : 0.f;
                float ia, ib, z[8];
                const uint32_t sa = fp4_block_scale(na * up, ia), sb = fp4_block_scale(nb * up, ib);
#pragma unroll
                for (int k = 0; k < 8; ++k) z[k] = __fmul_rn(__fmul_rn(a[k], up), ia);
                const uint32_t wa = e2m1x8(z);
#pragma unroll
                for (int k = 0; k < 8; ++k) z[k] = __fmul_rn(__fmul_rn(b[k], up), ib);
                const uint32_t wb = e2m1x8(z);
                if (live) {
                    const long long nblk = to.pg.block_table ? (1LL << to.pg.page_shift) >> 4 : to.S_max >> 4;
                    uint8_t* blk = static_cast<uint8_t*>(value ? to.v : to.k) + (size_t)(dst + h * nblk) * Blk::BYTES;
                    const int t = s_slot[r];
                    *reinterpret_cast<uint32_t*>(blk + Blk::code(t, ru.ca)) = wa;
                    *reinterpret_cast<uint32_t*>(blk + Blk::code(t, ru.cb)) = wb;
                    if (!(ru.ca & 8)) blk[Blk::scale(t, ru.ca)] = (uint8_t)sa;
                    if (!(ru.cb & 8)) blk[Blk::scale(t, ru.cb)] = (uint8_t)sb;
                    if (u == 0) blk[Blk::exp(t)] = (uint8_t)eb;
                }
            } else {
                constexpr bool FP8 = FORM == CacheForm::kFp8;
                const float sc = __fdiv_rn(m, FP8 ? 448.f : 127.f);
                auto codes = [&](const float(&f)[8]) {
                    uint32_t w[2] = {0u, 0u};
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        int c = 0;
                        if (m > 0.f) {
                            if constexpr (FP8) {
                                c = __nv_cvt_float_to_fp8(__fdiv_rn(f[k], sc), __NV_SATFINITE, __NV_E4M3);
                                if ((c & 0x7f) == 0) c = 0;
                            } else {
                                c = max(-127, min(127, __float2int_rn(__fdiv_rn(f[k], sc))));
                            }
                        }
                        w[k >> 2] |= (uint32_t)(c & 0xff) << (8 * (k & 3));
                    }
                    return make_uint2(w[0], w[1]);
                };
                const uint2 wa = codes(a), wb = codes(b);
                if (live) {
                    const size_t o = (size_t)dst * in.Hkv + h;
                    uint8_t* c = static_cast<uint8_t*>(value ? to.v : to.k) + o * DD;
                    *reinterpret_cast<uint2*>(c + ru.ca) = wa;
                    *reinterpret_cast<uint2*>(c + ru.cb) = wb;
                    if (u == 0) (value ? to.v_scale : to.k_scale)[o] = sc;
                }
            }
        }
    }
}

cudaError_t launch_append_rope(const AppendTarget& to, const RopeTable& rope, const NewRows& in, int32_t* status,
                               int num_sms, cudaStream_t stream) {
    const int rpb = (int)std::max(1LL, std::min((long long)kAppRows, in.rows / (4LL * num_sms)));
    const long long bx = (in.rows + rpb - 1) / rpb;
    const int units = (in.D + 15) / 16;
    const long long items = (long long)rpb * std::max(in.q ? in.Hq : 0, 2 * in.Hkv) * units;
    const int by = (int)std::max(1LL, std::min((items + kAppThreads - 1) / kAppThreads, 2LL * num_sms / bx));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)bx, (unsigned)by, 1);
    cfg.blockDim = dim3(kAppThreads, 1, 1);
    cfg.dynamicSmemBytes = rope.turns ? (size_t)rpb * (rope.rotary_dim / 2) * sizeof(float2) : 0;
    cfg.stream = stream;
#define KVD_APP(F, DD) cudaLaunchKernelEx(&cfg, append_rope_kernel<CacheForm::F, DD>, to, rope, in, rpb, status)
#define KVD_APP_D(F) (in.D == 64 ? KVD_APP(F, 64) : in.D == 128 ? KVD_APP(F, 128) : in.D == 256 ? KVD_APP(F, 256) : cudaErrorInvalidValue)
    switch (to.form) {
        case CacheForm::kBf16: return KVD_APP(kBf16, 0);
        case CacheForm::kInt8: return KVD_APP_D(kInt8);
        case CacheForm::kFp8: return KVD_APP_D(kFp8);
        case CacheForm::kFp4: return KVD_APP_D(kFp4);
    }
#undef KVD_APP_D
#undef KVD_APP
    return cudaErrorInvalidValue;
}

}  // namespace kvd
