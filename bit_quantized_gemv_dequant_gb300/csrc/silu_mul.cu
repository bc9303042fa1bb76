// silu_mul, silu_mul_fp8_b128: the gate of a feed-forward layer, as values or as
// e4m3 codes with a scale per 128.
#include <algorithm>

#include "fp8_code.cuh"
#include "fp8_tc.cuh"
#include "row8.cuh"

namespace qg {
namespace {

constexpr int kThreads = 128;
constexpr int kPer = 16;                      // values per thread
constexpr int kLanes = kFp8Block / kPer;      // threads per scale
constexpr int kUnits = kThreads / kLanes;     // scales per block

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// y = u g / (1 + e^-g) for two values at a time (SIGN = -1: -y). e^-g = 2^t (1 + s
// ln2), where t + s = -g log2 e: t is rounded, and its remainder s, which grows with
// g, is not lost. From g = -88 on the result is 0; of -infinity it is NaN, as the
// quotient is. An infinite g has no remainder: the minimum drops the NaN.
template <int SIGN>
__device__ __forceinline__ float2 gated(float2 g, float2 u) {
    constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f;  // log2 e = their sum
    constexpr float kLn2 = SIGN * 0x1.62e43p-1f, kOne = SIGN;
    const float2 minus = make_float2(-kLog2e, -kLog2e), one = make_float2(kOne, kOne), t = __fmul2_rn(g, minus);
    float2 s = __ffma2_rn(g, minus, make_float2(-t.x, -t.y));
    s = __ffma2_rn(g, make_float2(-kRest, -kRest), s);
    float2 f = __ffma2_rn(s, make_float2(kLn2, kLn2), one);
    f.x = SIGN > 0 ? fminf(f.x, 2.f) : fmaxf(f.x, -2.f);
    f.y = SIGN > 0 ? fminf(f.y, 2.f) : fmaxf(f.y, -2.f);
    const float2 d = __ffma2_rn(make_float2(exp2_approx(t.x), exp2_approx(t.y)), f, one);
    return __fmul2_rn(__fmul2_rn(g, make_float2(reciprocal_approx(d.x), reciprocal_approx(d.y))), u);
}

// Sixteen values per thread, eight threads per scale. Bound by the bytes of g, u and
// y next to instruction issue (72 % of all slots): 4096 x 12288 bf16 to codes 42.5 us,
// 6.0 TB/s; with a library's exponential and division and eight values per thread 58.7.
template <class T, bool FP8, bool VEC>
__global__ void __launch_bounds__(kThreads) gate_kernel(const GateArgs a, const int K, const int KB) {
    constexpr int kSign = FP8 ? -1 : 1;
    const int lane = threadIdx.x % kLanes;
    const long long units = (long long)a.M * KB, unit = (long long)blockIdx.x * kUnits + threadIdx.x / kLanes;
    // a division of 64 bits would take longer than everything else
    const long long m = units <= 0xFFFF0000ll ? (uint32_t)unit / (uint32_t)KB : unit / KB;
    // A thread has two runs of eight values: beside each other, or of f32 (whose runs are
    // two loads each) one in each half of the block: 4096 x 8192 f32 57.9 us, and 71 beside
    // each other; bf16 29.7 beside each other, 30.7 apart. Values of rows that do not lie
    // in eights are eight apart, so that threads read places beside each other.
    constexpr int kStep = VEC ? 1 : kLanes, kRun = VEC && sizeof(T) == 2 ? 8 : kFp8Block / 2;
    const int k = (int)(unit - m * KB) * kFp8Block + lane * (!VEC ? 1 : kRun == 8 ? 16 : 8), left = unit < units ? K - k : 0;
    const T* gate = static_cast<const T*>(a.gate) + m * a.gate_stride + k;
    const T* up = static_cast<const T*>(a.up) + m * a.up_stride + k;
    const long long at = m * K + k;
    fp8::pdl_wait();
    fp8::pdl_trigger();
    Raw8<T> gr[2], ur[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        gr[h] = load8<T, VEC, kStep>(gate + kRun * h, left - kRun * h);
        ur[h] = load8<T, VEC, kStep>(up + kRun * h, left - kRun * h);
    }
    float y[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float g[8];
        to_f32(gr[h], g);
        to_f32(ur[h], y[h]);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 v = gated<kSign>(make_float2(g[i], g[i + 1]), make_float2(y[h][i], y[h][i + 1]));
            y[h][i] = v.x;
            y[h][i + 1] = v.y;
        }
    }
    if constexpr (FP8) {
        float most = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 8; i += 2) most = fp8_largest(most, y[h][i], y[h][i + 1]);
        unsigned top = __float_as_uint(most) & 0x7FFFFFFFu;
#pragma unroll
        for (int i = kLanes / 2; i; i >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
        const float scale = fp8_scale(top);
        uint32_t code[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            fp8_encode<8>(y[h], scale, code[h]);
            store_codes8<VEC, kStep>(static_cast<uint8_t*>(a.y) + at + kRun * h, code[h], left - kRun * h);
        }
        if (lane == 0 && left > 0) a.scales[unit] = scale;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            with_type(a.y_dtype, [&](auto t) {
                using TY = decltype(t);
                store8<TY, VEC, kStep>(static_cast<TY*>(a.y) + at + kRun * h, y[h], left - kRun * h);
            });
    }
}

}  // namespace

int gate_launch(const GateArgs& a, cudaStream_t s) {
    const long long KB = (a.K + kFp8Block - 1) / kFp8Block, grid = (a.M * KB + kUnits - 1) / kUnits;
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
