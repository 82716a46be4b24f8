// 16 bytes of BF16 or float32 as float32 values.
#pragma once

#include "common.cuh"

namespace ll {

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static LL_DEVINL void unpack(const uint4& w, float (&v)[8]) {
        v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
        v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
    }
    static LL_DEVINL uint4 pack(const float (&v)[8]) {
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7]));
    }
    static LL_DEVINL float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static LL_DEVINL void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static LL_DEVINL void unpack(const uint4& w, float (&v)[4]) {
        v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y);
        v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
    }
    static LL_DEVINL uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    static LL_DEVINL float get(const float* p) { return *p; }
    static LL_DEVINL void put(float* p, float x) { *p = x; }
};

}  // namespace ll
