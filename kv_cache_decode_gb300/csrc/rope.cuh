// Rotary positions, device side: phases in 64-bit fixed point, their cosines and
// sines, and the rotation of 8 pairs held by one thread.
//
// A pair's frequency is given in turns per position as a fraction of 2^64, so
// position * turns modulo 2^64 (an integer product that wraps) is the exact
// fraction of a turn: no argument reduction is left to floating point, at any
// position. Its nearest quarter turn is taken off too, as an integer; only what is left, at most pi / 4, becomes a
// float32, which moves the angle by at most pi * 2^-27 = 2.4e-8 (of a half turn rounded whole it was up to 9.4e-8, the
// larger part of the error of a cosine or sine).
#pragma once

#include <algorithm>

#include "common.cuh"
#include "rope_fp4.h"

namespace kvd {

// factor * (cos, sin) of the pair's angle at position t. Within half a quarter turn of zero two short
// polynomials in u = x^2 do: interpolations of sin(pi x) / x and (cos(pi x) - 1) / u at the four Chebyshev nodes of
// [0, 1/16], pi as a float and what that lacks. Both stay within 1 unit in the last place (2 million x compared with
// 64 bits). The error of a cosine or sine is 1.7e-8 RMS. 500,000 bf16 rows of one head of 128 take 57 us; sincospif of the angle
// rounded whole took 66, with an error of 3.3e-8; sincospif behind the quarter turn 74. The step of 64 rows of 32 heads takes
// 2.45 us and took 2.35.
__device__ __forceinline__ float2 rope_cos_sin(long long t, uint64_t turns, float factor) {
    const uint64_t phase = (uint64_t)t * turns;
    const uint32_t near = (uint32_t)(phase >> 32) + 0x20000000u;  // the nearest quarter turn in the top two bits
    const float x = (float)(int32_t)(uint32_t)(phase >> 30) * 1.1641532182693481e-10f;  // 2^-33: half turns, [-1/4, 1/4]
    const float u = __fmul_rn(x, x);
    float s = __fmaf_rn(u, -0.5890751f, 2.549767f);
    s = __fmaf_rn(__fmaf_rn(s, u, -5.167708f), u, -9.71061e-8f);
    s = __fmaf_rn(x, 3.1415927f, __fmul_rn(x, s));
    float c = __fmaf_rn(u, 0.23212542f, -1.3351378f);
    c = __fmaf_rn(__fmaf_rn(c, u, 4.0587106f), u, -4.934802f);
    c = __fmaf_rn(c, u, 1.f);
    const bool odd = near & 0x40000000u;
    const uint32_t a = __float_as_uint(odd ? s : c), b = __float_as_uint(odd ? c : s);
    return make_float2(__fmul_rn(factor, __uint_as_float(a ^ ((near + 0x40000000u) & 0x80000000u))),
                       __fmul_rn(factor, __uint_as_float(b ^ (near & 0x80000000u))));
}

// A head's columns are dealt out to threads in units of two vectors of 8
// columns. Of the rotary columns [0, R) unit u holds pairs 8u .. 8u + 7: columns
// 8u and R/2 + 8u (halves), or the 16 columns from 16u (interleaved: the same
// columns a plain copy would give it). Units past R/16 hold 16 columns each; in a head of
// 8 mod 16 columns the last one has no second vector (cb = -1).
struct RopeUnit {
    int ca, cb;  // first column of each vector
    bool turn;   // rotary columns
};
__device__ __forceinline__ RopeUnit rope_unit(int u, int D, int R, bool interleaved) {
    RopeUnit r;
    r.turn = u < (R >> 4);
    r.ca = (r.turn && !interleaved) ? 8 * u : 16 * u;
    r.cb = (r.turn && !interleaved) ? (R >> 1) + 8 * u : 16 * u + 8;
    if (r.cb >= D) r.cb = -1;
    return r;
}

// (a, b) turned; the roundings are spelled out so that every kernel gives the same bits.
__device__ __forceinline__ void rope_pair(float& a, float& b, const float2& cs) {
    const float x = a;
    a = __fmaf_rn(x, cs.x, -__fmul_rn(b, cs.y));
    b = __fmaf_rn(b, cs.x, __fmul_rn(x, cs.y));
}

// The rotation of a unit's 8 pairs; cs: their factor * (cos, sin).
__device__ __forceinline__ void rope_turn(float (&a)[8], float (&b)[8], const float2* cs, bool interleaved) {
    if (interleaved) {  // pairs are neighbours: a holds pairs 0..3, b pairs 4..7
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rope_pair(a[2 * i], a[2 * i + 1], cs[i]);
            rope_pair(b[2 * i], b[2 * i + 1], cs[i + 4]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) rope_pair(a[i], b[i], cs[i]);
    }
}

// A table of cosines and sines in shared memory, 16-byte chunks of two entries: chunk c lies at c ^ (c / 8 % 4), so that
// threads with neighbouring units (8 entries each) read from different banks (30,000 rows of 40 heads of 80: 65 us, 75 without).
__device__ __forceinline__ void rope_table_put(float2* table, int e, const float2& cs) {
    const int c = e >> 1;
    table[2 * (c ^ ((c >> 3) & 3)) + (e & 1)] = cs;
}
__device__ __forceinline__ void rope_table_get(const float2* table, int e, float2 (&cs)[8]) {  // e: a multiple of 8
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = (e >> 1) + k;
        const float4 v = reinterpret_cast<const float4*>(table)[c ^ ((c >> 3) & 3)];
        cs[2 * k] = make_float2(v.x, v.y);
        cs[2 * k + 1] = make_float2(v.z, v.w);
    }
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, size_t e, const float (&f)[8]) {
    if constexpr (F32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + e);
        d[0] = make_float4(f[0], f[1], f[2], f[3]);
        d[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + e) = pack8(f);
    }
}

// A unit's two vectors as they lie in memory (plain loads, not the read-only path: rows may be turned in place), so that several units can be loaded before one is turned.
template <bool F32>
struct RopeRaw {
    uint4 a[F32 ? 2 : 1], b[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, size_t e, const RopeUnit& u) {
        if constexpr (F32) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + e + u.ca);
            a[0] = p[0], a[1] = p[1];
            if (u.cb >= 0) {
                const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + e + u.cb);
                b[0] = q[0], b[1] = q[1];
            }
        } else {
            a[0] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + e + u.ca);
            if (u.cb >= 0) b[0] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + e + u.cb);
        }
    }
    __device__ __forceinline__ void copy(void* base, size_t e, const RopeUnit& u) const {  // bit by bit, to the same type
        if constexpr (F32) {
            uint4* p = reinterpret_cast<uint4*>(static_cast<float*>(base) + e + u.ca);
            p[0] = a[0], p[1] = a[1];
            if (u.cb >= 0) {
                uint4* q = reinterpret_cast<uint4*>(static_cast<float*>(base) + e + u.cb);
                q[0] = b[0], q[1] = b[1];
            }
        } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + e + u.ca) = a[0];
            if (u.cb >= 0) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + e + u.cb) = b[0];
        }
    }
    __device__ __forceinline__ void get(float (&x)[8], float (&y)[8]) const {
        if constexpr (F32) {
            const uint32_t v[8] = {a[0].x, a[0].y, a[0].z, a[0].w, a[1].x, a[1].y, a[1].z, a[1].w};
            const uint32_t w[8] = {b[0].x, b[0].y, b[0].z, b[0].w, b[1].x, b[1].y, b[1].z, b[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[i]), y[i] = __uint_as_float(w[i]);
        } else {
            unpack8(a[0], x);
            unpack8(b[0], y);
        }
    }
};

// A warp's share of one token's work: its cosines and sines, and the turning of heads. DD: head dimension 64,
// 128 or 256, whose units divide the warp, so that a thread keeps one unit of every
// head and its 8 pairs' cosines and sines in registers; 0 for any other, with those in shared memory.
template <int DD>
struct RopeWarp {
    static constexpr int UN = DD / 16;
    float2 cs[DD ? 8 : 1];
    const float2* s_cs;
    int D, units, R;
    bool interleaved;

    // t: the token's position. buf: R / 2 entries of this warp's shared memory. Whole warps call this.
    __device__ __forceinline__ void init(const RopeTable& rope, long long t, int D_, float2* buf) {
        init(rope, D_, buf, [t](int) { return t; });
    }
    // The same, pair i turned by position at(i).
    template <class F>
    __device__ __forceinline__ void init(const RopeTable& rope, int D_, float2* buf, F&& at) {
        const int lane = threadIdx.x & 31;
        D = DD ? DD : D_;
        units = DD ? UN : (D + 15) >> 4;
        R = rope.turns ? rope.rotary_dim : 0;
        interleaved = rope.interleaved;
        s_cs = buf;
#pragma unroll 1  // (4 at most: unrolled it is 0.1 us slower for a few tokens)
        for (int i = lane; i < R >> 1; i += 32) rope_table_put(buf, i, rope_cos_sin(at(i), __ldg(rope.turns + i), rope.factor));
        __syncwarp();
        if constexpr (DD > 0) {
            if (lane % UN < R >> 4) rope_table_get(buf, 8 * (lane % UN), cs);
        }
    }
    __device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], int u) const {
        if constexpr (DD > 0) {
            rope_turn(a, b, cs, interleaved);
        } else {
            float2 w[8];
            rope_table_get(s_cs, 8 * u, w);
            rope_turn(a, b, w, interleaved);
        }
    }
    // Turns the heads of one row, src to dst, this warp's steps of them: part, part + parts, ... Two steps'
    // loads come before either is turned: one unit in flight per thread keeps too few bytes on the way.
    template <bool IN32, bool OUT32>
    __device__ __forceinline__ void heads(const void* src, size_t se, void* dst, size_t de, int H, int part, int parts) const {
        const int lane = threadIdx.x & 31, total = H * units;
        for (int base = 32 * part; base < total; base += 64 * parts) {
            RopeRaw<IN32> raw[2];
            RopeUnit ru[2];
            int h[2], u[2];
            bool live[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = base + k * 32 * parts + lane;
                live[k] = j < total;
                h[k] = j / units;
                u[k] = j - h[k] * units;
                ru[k] = rope_unit(u[k], D, R, interleaved);
                if (live[k]) raw[k].load(src, se + (size_t)h[k] * D, ru[k]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (!live[k]) continue;
                const size_t e = de + (size_t)h[k] * D;
                if (IN32 == OUT32 && !ru[k].turn) {
                    raw[k].copy(dst, e, ru[k]);
                    continue;
                }
                float a[8], b[8];
                raw[k].get(a, b);
                if (ru[k].turn) turn(a, b, u[k]);
                store8<OUT32>(dst, e + ru[k].ca, a);
                if (ru[k].cb >= 0) store8<OUT32>(dst, e + ru[k].cb, b);
            }
        }
    }
};

// A warp's work on several tokens at once, whose rows are too short to keep it busy one by one: the units of all of them
// are dealt to the lanes, and the cosines and sines of all lie in shared memory, [token][R / 2].
struct RopeTokens {
    int D, units, R, n;  // n: tokens
    bool interleaved;
    uint32_t ok;         // bit i: token i takes part
    float2* s_cs;

    // t: lane i's is token i's position. Whole warps call this.
    __device__ __forceinline__ void table(const RopeTable& rope, long long t) const {
        const int lane = threadIdx.x & 31, half = R >> 1;
        int tok = 0, i = lane;
        for (int e = 0; e < n * half; e += 32) {
            while (i >= half) i -= half, ++tok;
            const long long at = __shfl_sync(0xffffffffu, t, tok & 31);
            if (tok < n) rope_table_put(s_cs, tok * half + i, rope_cos_sin(at, __ldg(rope.turns + i), rope.factor));
            i += 32;
        }
        __syncwarp();
    }
    // Unit j of rows of H heads: its token, head and unit of the head.
    __device__ __forceinline__ void item(int j, int H, int& tok, int& h, int& u) const {
        tok = j / (H * units);
        const int m = j - tok * H * units;
        h = m / units;
        u = m - h * units;
    }
    __device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], int tok, int u) const {
        float2 cs[8];
        rope_table_get(s_cs, tok * (R >> 1) + 8 * u, cs);
        rope_turn(a, b, cs, interleaved);
    }
    // The tokens' rows (ss, ds elements apart), src to dst; ready() forms the table behind the first loads. ONE: rows of one
    // head, where no thread shares a pair's cosine and sine with another and each forms its own (t as for the table): 57 us instead of 86
    // for 500,000 rows of 128.
    template <bool IN32, bool OUT32, bool ONE, class F>
    __device__ __forceinline__ void heads(const void* src, size_t se, size_t ss, void* dst, size_t de, size_t ds, int H,
                                          const RopeTable& rope, long long t, F&& ready) const {
        const int lane = threadIdx.x & 31, total = n * H * units;
        for (int base = 0; base < total; base += 64) {
            RopeRaw<IN32> raw[2];
            RopeUnit ru[2];
            int tok[2], h[2], u[2];
            bool live[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = base + 32 * k + lane;
                item(j, H, tok[k], h[k], u[k]);
                live[k] = j < total && ((ok >> tok[k]) & 1u);
                ru[k] = rope_unit(u[k], D, R, interleaved);
                if (live[k]) raw[k].load(src, se + tok[k] * ss + (size_t)h[k] * D, ru[k]);
            }
            if (!ONE && base == 0) ready();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const long long at = ONE ? __shfl_sync(0xffffffffu, t, tok[k] & 31) : 0;
                if (!live[k]) continue;
                const size_t e = de + tok[k] * ds + (size_t)h[k] * D;
                if (IN32 == OUT32 && !ru[k].turn) {
                    raw[k].copy(dst, e, ru[k]);
                    continue;
                }
                float a[8], b[8];
                raw[k].get(a, b);
                if (ONE && ru[k].turn) {
                    float2 cs[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) cs[i] = rope_cos_sin(at, __ldg(rope.turns + 8 * u[k] + i), rope.factor);
                    rope_turn(a, b, cs, interleaved);
                } else if (ru[k].turn) {
                    turn(a, b, tok[k], u[k]);
                }
                store8<OUT32>(dst, e + ru[k].ca, a);
                if (ru[k].cb >= 0) store8<OUT32>(dst, e + ru[k].cb, b);
            }
        }
    }
};

// How many tokens a warp takes: as many as give it `want` units, as far as about 64 warps per SM are left.
inline int rope_tokens(long long rows, long long row_units, int want, int num_sms) {
    const long long n = std::min({want / row_units, rows / (64LL * num_sms), 32LL});
    return (int)(n < 1 ? 1 : n);
}

// How many warps share a row of `steps` steps: about 64 warps per SM, as many as it holds, where there are few rows.
inline int rope_parts(long long rows, long long steps, int num_sms) {
    const long long want = rows > 0 ? (64LL * num_sms + rows - 1) / rows : 1;
    return (int)(want < 1 ? 1 : want > steps ? (steps < 1 ? 1 : steps) : want);
}

}  // namespace kvd
