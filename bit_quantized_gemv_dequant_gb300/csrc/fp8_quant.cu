// quantize_fp8_b128: one e4m3 code per value and one f32 scale per 128 values
// of a row.
#include <cuda_fp8.h>

#include "serve_common.cuh"

namespace qg {
namespace {

constexpr int kBlock = 128;   // values per scale
constexpr int kThreads = 256;

// scale = max |x| / 448, code = e4m3_rn(x / scale), both divisions correctly
// rounded f32 ones. The maximum is taken over the bit patterns of |x|, whose
// order is that of the values with infinity above them and NaN above that, so
// a NaN reaches the scale. PER values per lane, which are 16 bytes where the
// rows allow it (PER = 8 for 16-bit types), 128 / PER lanes per block; bound by
// the bytes of x and the codes (and by latency for few rows).
//
// A division per value would bound the kernel instead. With r = 1 / scale
// correctly rounded, q' = q + r (x - scale q) after one such step is within an
// ulp of the quotient and after another the correctly rounded one (Markstein's
// theorem); the remainders are exact as long as nothing underflows, which the
// limits on scale see to for every quotient that does not end as code 0.
// The codes of PER values, from -x (so that a zero keeps its sign through the
// steps).
template <int PER>
__device__ __forceinline__ void encode(const float (&minus_x)[PER], float scale, uint32_t (&code)[PER / 4]) {
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

template <class T, int PER, bool VEC, int kDeep>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* __restrict__ x, long long stride, uint8_t* __restrict__ codes,
                    float* __restrict__ scales, int M, int K, int KB) {
    constexpr int kLanes = kBlock / PER, kUnits = kThreads / kLanes;
    constexpr int kWords = PER * sizeof(T) / 4;
    const int lane = threadIdx.x % kLanes;
    const long long units = (long long)M * KB;
    const long long unit0 = (long long)blockIdx.x * (kUnits * kDeep) + threadIdx.x / kLanes;
    uint32_t w[kDeep][kWords];
    int at_m[kDeep], at_k[kDeep];
    // All of a thread's loads first.
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
        const long long unit = unit0 + d * kUnits;
        // a division of 64 bits would take longer than everything else
        const int m = unit >= units ? M : units <= 0xFFFFFFFFll ? (int)((uint32_t)unit / (uint32_t)KB) : (int)(unit / KB);
        const int k = (int)(unit - (long long)m * KB) * kBlock + lane * PER;
        at_m[d] = m;
        at_k[d] = k;
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[d][i] = 0;
        if (m < M && k < K) {
            const T* p = x + m * stride + k;
            if constexpr (VEC && kWords == 4) {  // K % PER == 0: a lane's values are all there
                const uint4 u = *reinterpret_cast<const uint4*>(p);
                w[d][0] = u.x; w[d][1] = u.y; w[d][2] = u.z; w[d][3] = u.w;
            } else if constexpr (VEC) {
                const uint2 u = *reinterpret_cast<const uint2*>(p);
                w[d][0] = u.x; w[d][1] = u.y;
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    if (k + i >= K) break;
                    if constexpr (sizeof(T) == 4) w[d][i] = __float_as_uint(p[i]);
                    else w[d][i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + i) << (16 * (i % 2));
                }
            }
        }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
        float v[PER];  // -x
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = __uint_as_float(w[d][i] ^ 0x80000000u);
            } else {
                const float2 f = unpack2<T>(w[d][i] ^ 0x80008000u);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        if constexpr (kLanes == 32) {
            top = __reduce_max_sync(0xFFFFFFFFu, top);
        } else {
#pragma unroll
            for (int i = kLanes / 2; i; i >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
        }
        float scale = __fdiv_rn(__uint_as_float(top), 448.f);
        if (scale == 0.f) scale = 1.f;
        uint32_t code[PER / 4];
        encode<PER>(v, scale, code);
        if (at_m[d] >= M) continue;
        uint8_t* out = codes + (long long)at_m[d] * K + at_k[d];
        if (VEC) {
            if (at_k[d] < K) {
                if constexpr (PER == 8) *reinterpret_cast<uint2*>(out) = make_uint2(code[0], code[1]);
                else *reinterpret_cast<uint32_t*>(out) = code[0];
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (at_k[d] + i < K) out[i] = (uint8_t)(code[i / 4] >> (8 * (i % 4)));
        }
        if (lane == 0) scales[unit0 + d * kUnits] = scale;
    }
}

// DEEP: a thread's loads under way at once.
template <class T, int PER, bool VEC, int DEEP>
int launch_deep(const void* x, long long stride, uint8_t* codes, float* scales, long long M, long long K, cudaStream_t s) {
    constexpr int kUnits = kThreads / (kBlock / PER) * DEEP;
    const long long KB = (K + kBlock - 1) / kBlock, grid = (M * KB + kUnits - 1) / kUnits;
    if (grid > 0x7FFFFFFFLL) return QG_ERR_UNSUPPORTED;
    quantize_kernel<T, PER, VEC, DEEP><<<(unsigned)grid, kThreads, 0, s>>>(static_cast<const T*>(x), stride, codes, scales,
                                                                     (int)M, (int)K, (int)KB);
    return launched();
}

// Two loads per thread once that leaves every SM several CTAs (4096 x 4096 bf16:
// 14.1 us, and 14.7 with one; 1 x 4096: 1.9 us, and 1.5 with one).
template <class T, int PER, bool VEC>
int launch(const DevCtx& dc, const void* x, long long stride, uint8_t* codes, float* scales, long long M, long long K,
           cudaStream_t s) {
    constexpr int kUnits = kThreads / (kBlock / PER);
    const bool many = M * ((K + kBlock - 1) / kBlock) >= 16LL * dc.num_sms * kUnits;
    return many ? launch_deep<T, PER, VEC, 2>(x, stride, codes, scales, M, K, s)
                : launch_deep<T, PER, VEC, 1>(x, stride, codes, scales, M, K, s);
}

}  // namespace

int fp8_quantize_launch(const DevCtx& dc, const void* x, int dtype, long long stride, uint8_t* codes,
                        float* scales, long long M, long long K, cudaStream_t s) {
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        // Whether every lane's values start on a boundary of their size, and its codes too.
        auto fits = [&](int per) {
            return K % per == 0 && stride % per == 0 && reinterpret_cast<uintptr_t>(x) % (per * sizeof(T)) == 0 &&
                   reinterpret_cast<uintptr_t>(codes) % per == 0;
        };
        if constexpr (sizeof(T) == 2)
            if (fits(8)) return launch<T, 8, true>(dc, x, stride, codes, scales, M, K, s);
        return fits(4) ? launch<T, 4, true>(dc, x, stride, codes, scales, M, K, s)
                       : launch<T, 4, false>(dc, x, stride, codes, scales, M, K, s);
    });
}

}  // namespace qg
