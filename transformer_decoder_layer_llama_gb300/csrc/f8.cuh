// e4m3 codes and their power-of-two block scales.
#pragma once

#include "common.cuh"

namespace ll {

// Four codes of a word, lowest byte first, as two FP16 pairs, exactly (NaN codes give NaN).
LL_DEVINL void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Four float32 as e4m3 codes: nearest even, beyond +-448 saturating, NaN kept.
LL_DEVINL uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        " mov.b32 %0, {lo, hi};\n}\n"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// The smallest power of two s, at least 2^-117, with amax <= 448 s; 0 for 0.  448 = 1.75 * 2^8, so
// with amax = m 2^x (1 <= m < 2) the exponent is x - 8, or x - 7 where m > 1.75.  From 2^-117 on every
// code times its scale is a normal float32.  amax is finite and not negative.
LL_DEVINL float e4m3_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    if (u == 0u) return 0.f;
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);   // biased
    return __uint_as_float((uint32_t)max(e, 127 - 117) << 23);
}

// log2 of a V scale, exact for powers of two.  A scale of 0 becomes 2^-160: times a code and a probability that is
// below float32's smallest number.
constexpr float kLog2ZeroScale = -160.f;
LL_DEVINL float f8_log2_scale(float s) {
    if (!(s > 0.f)) return kLog2ZeroScale;
    const bool tiny = s < 1.17549435e-38f;                 // subnormal
    const uint32_t u = __float_as_uint(tiny ? s * 16777216.f : s);
    return (float)((int)(u >> 23) - 127 - (tiny ? 24 : 0)) + log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
}

// Four codes requantised from scale f_old to f_new: ratio = f_old / f_new.
LL_DEVINL uint32_t e4m3x4_rescale(uint32_t w, float ratio) {
    uint32_t lo, hi;
    e4m3x4_to_f16x4(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return f32x4_to_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

}  // namespace ll
