// fp4 KV cache, device side: the block layout, E2M1 conversions and the
// quantization of a thread's two vectors of 8 columns.
#pragma once

#include "common.cuh"

namespace kvd {

// A block holds 16 consecutive tokens of one KV head: codes (128 columns at a
// time, [16 tokens][W / 2] bytes, W = min(D, 128)), E4M3 scales [16][D / 16],
// row exponents [16].
template <int D>
struct Fp4Block {
    static constexpr int W = D < 128 ? D : 128;
    static constexpr int ROW = W / 2;          // bytes of a token's codes in one column group
    static constexpr int SCALES = 8 * D, EXPS = 9 * D, BYTES = 9 * D + 16;
    static_assert(BYTES % 16 == 0, "blocks stay 16-byte aligned");
    // Byte offset of column c's code (c even) of token t.
    __device__ static __forceinline__ int code(int t, int c) { return (c / W) * 16 * ROW + t * ROW + (c % W) / 2; }
    __device__ static __forceinline__ int scale(int t, int c) { return SCALES + t * (D / 16) + c / 16; }
    __device__ static __forceinline__ int exp(int t) { return EXPS + t; }
};

// Eight values as E2M1 codes (value i in bits 4i .. 4i + 3), round to nearest
// even, saturating at 6; a zero result loses its sign.
__device__ __forceinline__ uint32_t e2m1x8(const float (&z)[8]) {
    uint32_t w;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(w)
        : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
    const uint32_t nonzero = (w | (w >> 1) | (w >> 2)) & 0x11111111u;
    return w & (0x77777777u | (nonzero << 3));
}
// Four bytes of codes (8 columns) as four f16x2, exactly.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Two E4M3 bytes (low half of w) as f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t h;
    asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}

// 2^(byte - 127) of a row exponent byte (byte 0, an all-zero row's: 0).
__device__ __forceinline__ float fp4_row_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// The row exponent byte of a row whose largest magnitude is a (finite): the
// smallest e >= -126 with a <= 2688 * 2^e, plus 127; 0 when a = 0. 2688 is
// 1.3125 * 2^11, so e is the exponent of a less 11, or less 10 when a's
// significand is past 1.3125 (0x3fa80000).
__device__ __forceinline__ uint32_t fp4_row_exp(float a) {
    if (!(a > 0.f)) return 0u;
    const uint32_t b = __float_as_uint(a);
    const int e = (int)(b >> 23) - 11 + ((b & 0x7fffffu) > 0x280000u ? 1 : 0);  // biased by 127
    return (uint32_t)max(e, 1);
}
// 2^-e of a nonzero exponent byte (e = byte - 127 in [-126, 117]).
__device__ __forceinline__ float fp4_row_inv(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// The E4M3 scale byte of 16 columns whose largest |y| is m, and the factor fl(1 / s) its codes are taken with.
__device__ __forceinline__ uint32_t fp4_block_scale(float m, float& inv) {
    const uint32_t s = __nv_cvt_float_to_fp8(m * (1.f / 6.f), __NV_SATFINITE, __NV_E4M3);
    const float sv = f16_lo(e4m3x2_to_f16x2(s));
    inv = sv > 0.f ? __frcp_rn(sv) : 0.f;
    return s;
}

}  // namespace kvd
