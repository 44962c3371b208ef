// rows.cuh -- runs of 4 or 8 values of a row in the three element types, as the norm,
// rotation and cache kernels read and write them, and the symmetric Q8 code of a value.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace w4 {

// 4 values as they lie in memory.
template <typename T>
struct Raw4 {
    uint32_t r[sizeof(T)];
};

template <typename T>
W4_DEV Raw4<T> load4(const T *p) {
    Raw4<T> v;
    if constexpr (sizeof(T) == 4) {
        const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p));
        v.r[0] = w.x; v.r[1] = w.y; v.r[2] = w.z; v.r[3] = w.w;
    } else {
        const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(p));
        v.r[0] = w.x; v.r[1] = w.y;
    }
    return v;
}

template <typename T>
W4_DEV void unpack4(const Raw4<T> &raw, float *v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(raw.r[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float2 f;
            if constexpr (std::is_same<T, __half>::value) f = __half22float2(*reinterpret_cast<const __half2 *>(&raw.r[i]));
            else f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&raw.r[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// Two values rounded to a 16-bit type, in one word.
template <typename T>
W4_DEV uint32_t pack_pair(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

template <typename T>
W4_DEV void store4(T *p, const float *v) {
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_pair<T>(v[0], v[1]), pack_pair<T>(v[2], v[3]));
}

// One value.
W4_DEV float load_f32(float v) { return v; }
W4_DEV float load_f32(__half v) { return __half2float(v); }
W4_DEV float load_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
W4_DEV T from_f32(float v) {
    if constexpr (std::is_same<T, float>::value) return v;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// clamp(rint(fl(v / sx)), -127, 127), the code of w4_quantize_row_q8, for sx > 0; r = fl(1 / sx),
// fast: r is finite.  t = fl(v r) is within 2^-16 + 2^-24 of x = v / sx when |x| < 256 (two correctly rounded
// operations), and fl(x) within ulp(x) / 2 <= 2^-17 of x, so t and fl(x) lie within 2^-15 of each other: rint(t)
// decides unless t is within 2^-13 of a half-integer (about 1 value in 4000), where the IEEE quotient is taken.
W4_DEV int q8_code(float v, float sx, float r, bool fast) {
    const float t = __fmul_rn(v, r), rt = rintf(t);
    const int c = (fast && fabsf(t) < 256.0f && 0.5f - fabsf(t - rt) > 0x1p-13f) ? __float2int_rn(rt)
                                                                                  : __float2int_rn(__fdiv_rn(v, sx));
    return min(max(c, -127), 127);
}

// The low bytes of four words.
W4_DEV uint32_t pack_codes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return prmt(prmt(a, b, 0x0040), prmt(c, d, 0x0040), 0x5410);
}

}  // namespace w4
