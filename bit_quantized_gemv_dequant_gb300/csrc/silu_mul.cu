// silu_mul, silu_mul_fp8_b128: the gate of a feed-forward layer, as values or as
// e4m3 codes with a scale per 128.
#include <algorithm>

#include "fp8_code.cuh"
#include "fp8_tc.cuh"
#include "row8.cuh"

namespace qg {
namespace {

constexpr int kThreads = 256;

// g / (1 + e^-g). The approximate division gives 0 where the sum is past 2^126
// (results below 2^-119) and NaN for -infinity, as the quotient does.
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.f + expf(-g)); }

// y = silu(g) u. Eight values per thread, 16 threads per scale; bound by the bytes
// of g, u and y.
template <class T, bool FP8, bool VEC>
__global__ void __launch_bounds__(kThreads) gate_kernel(const GateArgs a, const int K, const int KB) {
    constexpr int kUnits = kThreads / 16;
    fp8::pdl_wait();
    fp8::pdl_trigger();
    const int lane = threadIdx.x % 16;
    const long long unit = (long long)blockIdx.x * kUnits + threadIdx.x / 16, units = (long long)a.M * KB;
    // a division of 64 bits would take longer than everything else
    const long long m = units <= 0xFFFFFFFFll ? (uint32_t)unit / (uint32_t)KB : unit / KB;
    const int k = (int)(unit - m * KB) * kFp8Block + lane * 8, left = m < a.M ? K - k : 0;
    const Raw8<T> gr = load8<T, VEC>(static_cast<const T*>(a.gate) + m * a.gate_stride + k, left);
    const Raw8<T> ur = load8<T, VEC>(static_cast<const T*>(a.up) + m * a.up_stride + k, left);
    float g[8], y[8];
    to_f32(gr, g);
    to_f32(ur, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= silu(g[i]);
    if constexpr (FP8) {
        unsigned top = 0;
        float minus[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            minus[i] = -y[i];
            top = max(top, __float_as_uint(minus[i]) & 0x7FFFFFFFu);
        }
#pragma unroll
        for (int i = 8; i; i >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
        const float scale = fp8_scale(top);
        uint32_t code[2];
        fp8_encode<8>(minus, scale, code);
        store_codes8<VEC>(static_cast<uint8_t*>(a.y) + m * K + k, code, left);
        if (lane == 0 && left > 0) a.scales[unit] = scale;
    } else {
        store8<VEC>(a.y, m * K + k, a.y_dtype, y, left);
    }
}

}  // namespace

int gate_launch(const GateArgs& a, cudaStream_t s) {
    const long long KB = (a.K + kFp8Block - 1) / kFp8Block, grid = (a.M * KB + kThreads / 16 - 1) / (kThreads / 16);
    if (grid > 0x7FFFFFFFLL) return QG_ERR_UNSUPPORTED;
    return by_type(a.x_dtype, [&](auto t) {
        using T = decltype(t);
        const bool fp8 = a.scales != nullptr;
        const bool vec = in_eights(a.gate, a.gate_stride, a.K, sizeof(T)) && in_eights(a.up, a.up_stride, a.K, sizeof(T)) &&
                         (fp8 ? reinterpret_cast<uintptr_t>(a.y) % 8 == 0
                              : in_eights(a.y, a.K, a.K, type_bytes(a.y_dtype)));
        auto kern = fp8 ? (vec ? gate_kernel<T, true, true> : gate_kernel<T, true, false>)
                        : (vec ? gate_kernel<T, false, true> : gate_kernel<T, false, false>);
        return launch_after(kern, dim3((unsigned)grid), dim3(kThreads), 0, s, a, (int)a.K, (int)KB);
    });
}

}  // namespace qg
