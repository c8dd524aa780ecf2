// A unit of a new key or value row on its way into the cache, turned and, where the cache is quantized, encoded
// in registers.
#pragma once

#include "../../include/kvdecode.h"
#include "fp4.cuh"
#include "rope.cuh"

namespace kvd {

// One unit (two vectors of 8 columns) of a key or value row, turned, into the cache: unit u of head h at cache
// row (fp4: block of head 0) dst. R: the row's rotary columns (0 for values); turn: the rotation of its pairs.
// Whole warps call this, a row's threads side by side; live: this thread has a unit.
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

}  // namespace kvd
