// Rotary positions, device side: phases in 64-bit fixed point, their cosines and
// sines, and the rotation of 8 pairs held by one thread.
//
// A pair's frequency is given in turns per position as a fraction of 2^64, so
// position * turns modulo 2^64 (an integer product that wraps) is the exact
// fraction of a turn: no argument reduction is left to floating point, at any
// position. The top 32 bits, signed, are then the angle in units of pi / 2^31;
// rounding them to float32's 24 bits moves it by at most pi * 2^-25 = 9.4e-8.
#pragma once

#include "common.cuh"
#include "params.h"

namespace kvd {

// factor * (cos, sin) of the pair's angle at position t.
__device__ __forceinline__ float2 rope_cos_sin(long long t, uint64_t turns, float factor) {
    const uint64_t phase = (uint64_t)t * turns;
    const float half_turns = (float)(int32_t)(phase >> 32) * 4.656612873077393e-10f;  // 2^-31: [-1, 1]
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(__fmul_rn(factor, c), __fmul_rn(factor, s));
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

// 8 consecutive elements of a bf16 or fp32 row. Plain loads, not the read-only path: the rows may be turned in place.
template <bool F32>
__device__ __forceinline__ void load8(const void* base, size_t e, float (&f)[8]) {
    if constexpr (F32) {
        const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + e);
        const float4 y = *(reinterpret_cast<const float4*>(static_cast<const float*>(base) + e) + 1);
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + e), f);
    }
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

}  // namespace kvd
