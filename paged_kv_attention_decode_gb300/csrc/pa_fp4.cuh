// The 4-bit cache format shared by the kernels that write, widen and attend.
//
// A value is e2m1(code) * e4m3(scale of its group) * (scale of the pool); a
// group is 16 consecutive dims of one (token, kv head) row.  A tile holds the
// 16 rows of one (block, kv head):
//   codes   16 rows of D / 2 bytes, dims 2j and 2j + 1 in the low and high
//           nibble of byte j
//   scales  K: [16 tokens][D / 16 groups]; V: [D / 16 groups][16 tokens], one
//           E4M3 byte each
// so a tile is 9 D bytes (1152 at head_dim 128) and one contiguous read.  The
// scale orders are those in which the lanes of the attention kernel need them:
// a lane holds two tokens' groups of K, and four tokens of one group of V.
#pragma once

#include "pa_device.cuh"

namespace pa {

template <int D>
struct Fp4Tile {
    static constexpr int kRow = D / 2;             // code bytes of one token row
    static constexpr int kGroups = D / 16;         // scales of one token row
    static constexpr int kCodes = 16 * kRow;
    static constexpr int kBytes = kCodes + 16 * kGroups;
    static __device__ __forceinline__ int scale_off(bool v, int tok, int grp) {
        return kCodes + (v ? grp * 16 + tok : tok * kGroups + grp);
    }
};

// Eight E2M1 codes (two per byte, low nibble first) -> four fp16 pairs (exact).
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t codes, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(codes));
}

// Eight fp32 values -> eight E2M1 codes, round to nearest even, saturating at +-6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float* y) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}

__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Maximum that keeps a NaN of either operand.
__device__ __forceinline__ float fmax_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// One group of 16 values y (already divided by the pool's scale) -> its codes
// and its E4M3 scale: s = e4m3(max|y| / 6), code = e2m1(y / s), both rounded
// to nearest even and saturating; a group whose scale rounds to 0 has zero
// codes, and a NaN in it makes the scale NaN (zero codes).
__device__ __forceinline__ void quantise_group(const float (&y)[16], uint32_t& lo, uint32_t& hi, uint8_t& scale) {
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) mx = fmax_nan(mx, fabsf(y[j]));
    const uint16_t code = f32x2_to_e4m3x2(__fdiv_rn(mx, 6.f), 0.f);
    scale = static_cast<uint8_t>(code & 0xffu);
    const float s = Elem<__half>::to_float2(e4m3x2_to_f16x2(code)).x;
    float q[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) q[j] = s > 0.f ? __fdiv_rn(y[j], s) : 0.f;
    lo = f32x8_to_e2m1x8(q);
    hi = f32x8_to_e2m1x8(q + 8);
}

// The 16 values of one group as fp16 pairs: code times group scale, exact
// (E2M1 has 2 significant bits, E4M3 has 4, and the products lie in
// [2^-10, 2688]).
__device__ __forceinline__ void group_values(uint32_t lo, uint32_t hi, uint8_t scale, uint32_t (&h)[8]) {
    const uint32_t s2 = e4m3x2_to_f16x2(static_cast<uint16_t>(scale * 0x0101u));
    uint32_t a[4], b[4];
    e2m1x8_to_f16x2(lo, a);
    e2m1x8_to_f16x2(hi, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = hmul2_bits(a[j], s2);
        h[4 + j] = hmul2_bits(b[j], s2);
    }
}

// The same for 8 values of a group (one half's codes).
__device__ __forceinline__ void half_group_values(uint32_t codes, uint8_t scale, uint32_t (&h)[4]) {
    const uint32_t s2 = e4m3x2_to_f16x2(static_cast<uint16_t>(scale * 0x0101u));
    e2m1x8_to_f16x2(codes, h);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = hmul2_bits(h[j], s2);
}

}  // namespace pa
