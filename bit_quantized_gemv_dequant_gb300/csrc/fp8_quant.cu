// quantize_fp8_b128: one e4m3 code per value and one f32 scale per 128 values
// of a row.
#include <cuda_fp8.h>

#include "serve_common.cuh"

namespace qg {
namespace {

constexpr int kBlock = 128;   // values per scale
constexpr int kWarps = 8;     // warps per CTA, one (row, block) each

// scale = max |x| / 448, code = e4m3_rn(x / scale), both divisions correctly
// rounded f32 ones. The maximum is taken over the bit patterns of |x|, whose
// order is that of the values with infinity above them and NaN above that, so
// a NaN reaches the scale. Four consecutive values per lane; bound by the
// bytes of x (and by latency for few rows).
template <class T, bool VEC>
__global__ void __launch_bounds__(kWarps * 32)
    quantize_kernel(const T* __restrict__ x, long long stride, uint8_t* __restrict__ codes,
                    float* __restrict__ scales, int M, int K, int KB) {
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= (long long)M * KB) return;
    const int m = (int)(unit / KB), b = (int)(unit % KB);
    const int k = b * kBlock + lane * 4;
    const T* row = x + m * stride;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (VEC) {
        if (k < K) {  // K % 4 == 0: a lane's four values are all there
            if constexpr (sizeof(T) == 4) {
                const float4 f = *reinterpret_cast<const float4*>(row + k);
                v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(row + k);
                const float2 a = unpack2<T>(w.x), c = unpack2<T>(w.y);
                v[0] = a.x; v[1] = a.y; v[2] = c.x; v[3] = c.y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i < K) v[i] = to_f32(row[k + i]);
    }
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    float scale = __fdiv_rn(__uint_as_float(top), 448.f);
    if (scale == 0.f) scale = 1.f;
    uint32_t code = 0;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float2 q = make_float2(__fdiv_rn(v[i], scale), __fdiv_rn(v[i + 1], scale));
        code |= (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) << (8 * i);
    }
    uint8_t* out = codes + (long long)m * K + k;
    if (VEC) {
        if (k < K) *reinterpret_cast<uint32_t*>(out) = code;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i < K) out[i] = (uint8_t)(code >> (8 * i));
    }
    if (lane == 0) scales[unit] = scale;
}

}  // namespace

int fp8_quantize_launch(const DevCtx&, const void* x, int dtype, long long stride, uint8_t* codes,
                        float* scales, long long M, long long K, cudaStream_t s) {
    const long long KB = (K + kBlock - 1) / kBlock;
    const long long grid = (M * KB + kWarps - 1) / kWarps;
    if (grid > 0x7FFFFFFFLL) return QG_ERR_UNSUPPORTED;
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        const uintptr_t step = 4 * sizeof(T);
        const bool vec = K % 4 == 0 && stride % 4 == 0 &&
                         reinterpret_cast<uintptr_t>(x) % step == 0 &&
                         reinterpret_cast<uintptr_t>(codes) % 4 == 0;
        auto kern = vec ? quantize_kernel<T, true> : quantize_kernel<T, false>;
        kern<<<(unsigned)grid, kWarps * 32, 0, s>>>(static_cast<const T*>(x), stride, codes, scales,
                                                   (int)M, (int)K, (int)KB);
        return launched();
    });
}

}  // namespace qg
