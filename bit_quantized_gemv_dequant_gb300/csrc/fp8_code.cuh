// The 8-bit floating point format of the serving operators: e4m3 codes with one
// f32 scale per 128 values of a row.
#pragma once

#include <cuda_fp8.h>

#include "serve_common.cuh"

namespace qg {

constexpr int kFp8Block = 128;   // values per scale

// The largest magnitude of three, NaN above infinity.
__device__ __forceinline__ float fp8_largest(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The scale of a block whose largest |x| has the bits `top`.
__device__ __forceinline__ float fp8_scale(unsigned top) {
    const float scale = __fdiv_rn(__uint_as_float(top), 448.f);
    return scale == 0.f ? 1.f : scale;
}

// A division per value would bound the kernel instead. With r = 1 / scale
// correctly rounded, q' = q + r (x - scale q) after one such step is within an
// ulp of the quotient and after another the correctly rounded one (Markstein's
// theorem); the remainders are exact as long as nothing underflows, which the
// limits on scale see to for every quotient that does not end as code 0.
// The codes of PER values, from -x (so that a zero keeps its sign through the
// steps).
template <int PER>
__device__ __forceinline__ void fp8_encode(const float (&minus_x)[PER], float scale, uint32_t (&code)[PER / 4]) {
    float2 q[PER / 2];
    const bool plain = scale > 0x1p-80f && scale < 0x1p80f && (__float_as_uint(scale) & 0x7FFFFFu) != 0x7FFFFFu;
    if (plain) {
        const float rcp = __frcp_rn(scale);
        const float2 mr = make_float2(-rcp, -rcp), s2 = make_float2(scale, scale);
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) {
            const float2 mx = make_float2(minus_x[2 * i], minus_x[2 * i + 1]);
            q[i] = __fmul2_rn(mx, mr);
            q[i] = __ffma2_rn(__ffma2_rn(s2, q[i], mx), mr, q[i]);
            q[i] = __ffma2_rn(__ffma2_rn(s2, q[i], mx), mr, q[i]);
        }
    } else {  // far from 1, infinite, NaN, or a significand of ones
#pragma unroll
        for (int i = 0; i < PER / 2; ++i)
            q[i] = make_float2(__fdiv_rn(minus_x[2 * i], -scale), __fdiv_rn(minus_x[2 * i + 1], -scale));
    }
#pragma unroll
    for (int i = 0; i < PER / 4; ++i)
        code[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(q[2 * i], __NV_SATFINITE, __NV_E4M3) |
                  (uint32_t)__nv_cvt_float2_to_fp8x2(q[2 * i + 1], __NV_SATFINITE, __NV_E4M3) << 16;
}

}  // namespace qg
