// The append with the rotation of the positions on the way: each new token's
// key heads are turned by the token's position and stored in the cache (bf16,
// int8, fp8 or fp4; contiguous or paged), its value heads stored as they are,
// and its query heads turned into q_out. One read of q, k, v and one write of
// each; a separate rotation would read and write q and k once more. Bound by
// memory for prompts and by latency for single tokens.
//
// A warp takes a token (a share of its heads where there are few tokens): its
// sequence, position and place in the cache and its cosines and sines, then the heads, two steps'
// loads at a time; warps wait for nothing but their own loads. A head is dealt to D / 16
// threads as in rope.cuh; where the cache is quantized these threads find the row's (and,
// fp4, the 16 columns') largest magnitude by shuffles, so a row goes from its
// load to its codes in registers. Measured: 24 prompts of up to 4,096 tokens, 32 query and 8 KV heads of 128, into
// bf16 pages: 188 us (1.21 GB, 6.4 of 6.8 TB/s copied); a persistent loop over the tokens took 280. One token of each of
// 64 sequences: 3.6 us, where the rotation of as many query rows alone takes 2.45. Into contiguous caches, 24 prompts of 2,048 tokens
// of the same heads: bf16 178 us, int8 212, fp8 209, fp4 179; the token of 64 sequences 3.1, 4.2, 4.1 and 3.8.
#include <algorithm>

#include "../../include/kvdecode.h"
#include "fp4.cuh"
#include "rope.cuh"

namespace kvd {

// Blocks of 4 warps, 7 to an SM (72 registers a thread), although all fp4 forms and most of the kernel for few heads then spill 24 to 72 bytes: with the
// registers that the compiler takes by itself 8 prompts of up to 2,048 tokens, 40 and 40 heads of 80, bf16, take 75 us instead of
// 61, and the 24 of 2,048 above 178, 230, 225 and 197 (bf16, int8, fp8, fp4); with 6 blocks to an SM 75, and 176, 212, 208 and 182.
constexpr int kAppWarps = 4;

// Where sequence sq's token t goes: its cache row (fp4: the block of head 0, and the token's slot in it), or -1: nowhere.
// status: where to say so, or null.
template <CacheForm FORM>
__device__ __forceinline__ long long place_of(const AppendTarget& to, const NewRows& in, int sq, long long t, int32_t* status,
                                              int& slot) {
    long long dst = -1;
    slot = 0;
    if (t < 0 || t >= to.S_max) {
        if (status) atomicOr(status, KVD_STATUS_POS_OUT_OF_RANGE);
    } else {
        long long seq = sq, cap = to.S_max, at = t;  // sequence (page), its capacity, place in it
        bool ok = true;
        if (to.pg.block_table) {
            seq = __ldg(to.pg.block_table + (size_t)sq * to.pg.max_blocks + (t >> to.pg.page_shift));
            cap = 1LL << to.pg.page_shift;
            at = t & (cap - 1);
            ok = seq >= 0 && seq < to.pg.num_pages;
            if (!ok && status) atomicOr(status, KVD_STATUS_BAD_PAGE);
        }
        if (ok) {
            dst = FORM == CacheForm::kFp4 ? seq * in.Hkv * (cap >> 4) + (at >> 4) : seq * cap + at;
            slot = (int)(at & 15);
        }
    }
    return dst;
}

// One unit (two vectors of 8 columns) of a key or value row, turned, into the cache: unit u of head h at cache row (fp4:
// block of head 0) dst. R: the row's rotary columns (0 for values); turn: the rotation of its pairs. Whole warps call this,
// a row's threads side by side; live: this thread has a unit.
template <CacheForm FORM, int DD, class F>
__device__ __forceinline__ void put_unit(const AppendTarget& to, const NewRows& in, bool interleaved, const RopeRaw<false>& raw,
                                         const RopeUnit& ru, int R, bool value, int h, int u, int D, long long dst, int slot,
                                         bool live, F&& turn) {
    const int lane = threadIdx.x & 31;
    if constexpr (FORM == CacheForm::kBf16) {
        void* cache = value ? to.v : to.k;
        const size_t o = ((size_t)dst * in.Hkv + h) * D;
        if (live && !ru.turn) raw.copy(cache, o, ru);
        if (live && ru.turn) {
            float a[8], b[8];
            raw.get(a, b);
            turn(a, b);
            store8<false>(cache, o + ru.ca, a);
            store8<false>(cache, o + ru.cb, b);
        }
    } else {
        float a[8] = {}, b[8] = {};
        if (live) {
            raw.get(a, b);
            if (ru.turn) turn(a, b);
        }
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
            const int R16 = (ru.turn && !interleaved) ? R >> 4 : 0;  // this vector's unit map, see rope_unit
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
                const int t = slot;
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

// DD: head dimension 64, 128 or 256, or 0 for any other (bf16 cache only).
template <CacheForm FORM, int DD>
__global__ void __launch_bounds__(kAppWarps * 32, 7) append_rope_kernel(const AppendTarget to, const RopeTable rope,
                                                                     const NewRows in, int parts, int32_t* status) {
    extern __shared__ __align__(16) float2 s_cs[];  // [warps][R / 2]
    pdl_launch_dependents();  // the attention that may follow waits for this grid before it reads anything
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * kAppWarps + (threadIdx.x >> 5);
    const long long row = w / parts;
    const int part = (int)(w - row * parts);
    if (row >= in.rows) return;

    // ---- the token's sequence, position and place ----
    int sq;  // its sequence
    long long i;
    if (in.offsets) {
        if (row >= __ldg(in.offsets + in.B)) return;  // a buffer may be much longer than its sequences
        int cnt = 0;  // offsets <= row, counted over all of them at once rather than by dependent steps
        for (int j = lane; j <= in.B; j += 32) cnt += __ldg(in.offsets + j) <= row ? 1 : 0;
        sq = __reduce_add_sync(0xffffffffu, cnt) - 1;
        if (sq < 0 || sq >= in.B) return;
        i = row - __ldg(in.offsets + sq);
        if (i < 0) return;
    } else {
        sq = (int)(row / in.T);
        i = row - (long long)sq * in.T;
    }
    const long long t = (long long)__ldg(in.pos + sq) + i;
    int slot;
    const long long dst = place_of<FORM>(to, in, sq, t, part == 0 && lane == 0 ? status : nullptr, slot);
    RopeWarp<DD> rw;
    rw.init(rope, t, in.D, s_cs + (threadIdx.x >> 5) * (rope.rotary_dim >> 1));
    const int D = rw.D, units = rw.units;

    if (in.q) rw.template heads<false, false>(in.q, (size_t)row * in.qs, in.q_out, (size_t)row * in.qos, in.Hq, part, parts);
    if (dst < 0) return;
    // ---- keys, then values, likewise; whole warps stay in the loop for the shuffles ----
    const int total = 2 * in.Hkv * units;
    for (int base = 32 * part; base < total; base += 64 * parts) {
        RopeRaw<false> raw[2];
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            const int j = base + k2 * 32 * parts + lane, hh = j / units;
            const bool value = hh >= in.Hkv;
            if (j < total)
                raw[k2].load(value ? in.v : in.k, (size_t)row * (value ? in.vs : in.ks) + (size_t)(value ? hh - in.Hkv : hh) * D,
                             rope_unit(j - hh * units, D, value ? 0 : rw.R, rope.interleaved));
        }
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            const int j0 = base + k2 * 32 * parts;
            if (j0 >= total) break;
            const bool live = j0 + lane < total;
            const int j = live ? j0 + lane : 0, hh = j / units, u = j - hh * units;
            const bool value = hh >= in.Hkv;
            const int h = value ? hh - in.Hkv : hh;
            const int Rh = value ? 0 : rw.R;
            const RopeUnit ru = rope_unit(u, D, Rh, rope.interleaved);
            put_unit<FORM, DD>(to, in, rope.interleaved, raw[k2], ru, Rh, value, h, u, D, dst, slot, live,
                               [&](float(&a)[8], float(&b)[8]) { rw.turn(a, b, u); });
        }
    }
}

// Tokens of few heads: several to a warp, a lane each for their sequences, positions and places. 32 prompts of up to 4,096
// tokens, 8 query heads and one KV head of 64: 35 us, 70 by a warp each.
template <CacheForm FORM, int DD>
__global__ void __launch_bounds__(kAppWarps * 32, 7) append_rope_rows_kernel(const AppendTarget to, const RopeTable rope,
                                                                          const NewRows in, int per_warp, int32_t* status) {
    extern __shared__ __align__(16) float2 s_cs[];  // [warps][per_warp][R / 2]
    pdl_launch_dependents();  // as above
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row0 = ((long long)blockIdx.x * kAppWarps + warp) * per_warp;
    if (row0 >= in.rows) return;
    const int n = (int)min((long long)per_warp, in.rows - row0);
    const long long row = row0 + lane;
    bool ok = lane < n;
    int sq = 0;
    long long i = 0;
    if (in.offsets) {
        if (row0 >= __ldg(in.offsets + in.B)) return;
        int cnt = 0;  // the first row's sequence as above; the others' from there on
        for (int j = lane; j <= in.B; j += 32) cnt += __ldg(in.offsets + j) <= row0 ? 1 : 0;
        sq = min(max(__reduce_add_sync(0xffffffffu, cnt) - 1, 0), in.B - 1);
        while (sq + 1 < in.B && __ldg(in.offsets + sq + 1) <= row) ++sq;
        i = row - __ldg(in.offsets + sq);
        ok = ok && i >= 0 && row < __ldg(in.offsets + sq + 1);
    } else if (ok) {
        sq = (int)(row / in.T);
        i = row - (long long)sq * in.T;
    }
    const long long t = ok ? (long long)__ldg(in.pos + sq) + i : 0;
    int slot = 0;
    const long long dst = ok ? place_of<FORM>(to, in, sq, t, status, slot) : -1;

    const int R = rope.turns ? rope.rotary_dim : 0, D = DD ? DD : in.D, units = DD ? DD / 16 : (D + 15) >> 4;
    const RopeTokens rt{D, units, R, n, rope.interleaved != 0, __ballot_sync(0xffffffffu, ok),
                        s_cs + (size_t)warp * per_warp * (R >> 1)};
    if (in.q)
        rt.heads<false, false, false>(in.q, (size_t)row0 * in.qs, (size_t)in.qs, in.q_out, (size_t)row0 * in.qos, (size_t)in.qos, in.Hq, rope, t,
                               [&]() { rt.table(rope, t); });
    const int total = n * 2 * in.Hkv * units;
    for (int base = 0; base < total; base += 64) {
        RopeRaw<false> raw[2];
        RopeUnit ru[2];
        int hh[2], u[2], tok[2], at[2];
        long long to_row[2];
        bool live[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = base + 32 * k + lane;
            rt.item(j, 2 * in.Hkv, tok[k], hh[k], u[k]);
            to_row[k] = __shfl_sync(0xffffffffu, dst, tok[k] & 31);
            at[k] = __shfl_sync(0xffffffffu, slot, tok[k] & 31);
            live[k] = j < total && to_row[k] >= 0;
            const bool value = hh[k] >= in.Hkv;
            ru[k] = rope_unit(u[k], D, value ? 0 : R, rope.interleaved);
            if (live[k])
                raw[k].load(value ? in.v : in.k, (size_t)(row0 + tok[k]) * (value ? in.vs : in.ks) +
                                                     (size_t)(value ? hh[k] - in.Hkv : hh[k]) * D, ru[k]);
        }
        if (base == 0 && !in.q) rt.table(rope, t);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (base + 32 * k >= total) break;
            const bool value = hh[k] >= in.Hkv;
            put_unit<FORM, DD>(to, in, rope.interleaved, raw[k], ru[k], value ? 0 : R, value, value ? hh[k] - in.Hkv : hh[k], u[k],
                               D, to_row[k], at[k], live[k],
                               [&](float(&a)[8], float(&b)[8]) { rt.turn(a, b, tok[k], u[k]); });
        }
    }
}

cudaError_t launch_append_rope(const AppendTarget& to, const RopeTable& rope, const NewRows& in, int32_t* status,
                               int num_sms, cudaStream_t stream) {
    const long long units = (in.D + 15) / 16, hq = in.q ? in.Hq : 0;
    const int per_warp = rope_tokens(in.rows, (hq + 2LL * in.Hkv) * units, 256, num_sms);
    const long long steps = (std::max(hq, 2LL * in.Hkv) * units + 31) / 32;
    const int parts = per_warp > 1 ? 1 : rope_parts(in.rows, steps, num_sms);  // warps of a token
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(per_warp > 1 ? (in.rows + per_warp * kAppWarps - 1) / (per_warp * kAppWarps)
                                               : (in.rows * parts + kAppWarps - 1) / kAppWarps), 1, 1);
    cfg.blockDim = dim3(kAppWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = rope.turns ? (size_t)kAppWarps * per_warp * (rope.rotary_dim / 2) * sizeof(float2) : 0;
    cfg.stream = stream;
#define KVD_APP(F, DD)                                                                                                  \
    (per_warp > 1 ? cudaLaunchKernelEx(&cfg, append_rope_rows_kernel<CacheForm::F, DD>, to, rope, in, per_warp, status) \
                  : cudaLaunchKernelEx(&cfg, append_rope_kernel<CacheForm::F, DD>, to, rope, in, parts, status))
#define KVD_APP_D(F) (in.D == 64 ? KVD_APP(F, 64) : in.D == 128 ? KVD_APP(F, 128) : in.D == 256 ? KVD_APP(F, 256) : cudaErrorInvalidValue)
    switch (to.form) {
        case CacheForm::kBf16:
            return in.D == 64 ? KVD_APP(kBf16, 64) : in.D == 128 ? KVD_APP(kBf16, 128) : in.D == 256 ? KVD_APP(kBf16, 256) : KVD_APP(kBf16, 0);
        case CacheForm::kInt8: return KVD_APP_D(kInt8);
        case CacheForm::kFp8: return KVD_APP_D(kFp8);
        case CacheForm::kFp4: return KVD_APP_D(kFp4);
    }
#undef KVD_APP_D
#undef KVD_APP
    return cudaErrorInvalidValue;
}

}  // namespace kvd
