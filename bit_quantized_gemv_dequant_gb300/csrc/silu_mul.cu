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

__device__ __forceinline__ float least_of(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f;  // log2 e = their sum

// y = u g / (1 + e^-g) for two values at a time (SIGN = -1: -y). e^-g = 2^t (1 + s
// ln2), where t + s = -g log2 e: t is rounded, and its remainder s, which grows with
// g, is not lost. From g = -87.3 on the quotient is below the normal numbers and becomes
// 0 (see gated_far); of -infinity it is NaN. An infinite g has no remainder: the minimum
// drops the NaN.
template <int SIGN>
__device__ __forceinline__ float2 gated(float2 g, float2 u) {
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

// y for kFarthest < g < kFar, where 1 + e^-g is e^-g: u g e^g, half of whose exponent
// comes before u and half after it, since u may be as large as e^g is small. e^g = 2^-4k
// 2^-r (1 - s ln2), where 4k + r + s = -g log2 e. Below kFarthest nothing is left of the
// largest u.
constexpr float kFar = -87.f, kFarthest = -340.f;
template <int SIGN>
__device__ __forceinline__ float gated_far(float g, float u) {
    const float t = g * -kLog2e, k = rintf(t * 0.25f);
    const float s = fmaf(g, -kRest, fmaf(g, -kLog2e, -t));
    float e = exp2_approx(fmaf(k, 4.f, -t));
    e = fmaf(e, s * -0x1.62e43p-1f, e);
    const float q = __int_as_float((127 - (int)k) << 23);
    return g * (SIGN * e) * q * q * u * q * q;
}

// The values of a thread of gate_kernel whose gates are that small, read again one by one:
// what the rare path needs it works out anew, and takes few registers from the other one
// (4096 x 12288 bf16 to codes with one such gate in 10^4: 48 us; with nothing else: 238).
template <class T, int SIGN, int RUN, int STEP>
__device__ __noinline__ void again(float* y, const GateArgs& a, long long unit, int lane, int apart) {
    const long long KB = (a.K + kFp8Block - 1) / kFp8Block, m = unit / KB;
    const int k = (int)(unit - m * KB) * kFp8Block + lane * apart, left = m < a.M ? (int)a.K - k : 0;
    const T* gate = static_cast<const T*>(a.gate) + m * a.gate_stride + k;
    const T* up = static_cast<const T*>(a.up) + m * a.up_stride + k;
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
        const int at = i / 8 * RUN + i % 8 * STEP;
        if (at >= left) continue;
        const float g = to_f32(gate[at]);
        if (g < kFar && g > kFarthest) y[i] = gated_far<SIGN>(g, to_f32(up[at]));
    }
}

// Sixteen values per thread, eight threads per scale. Bound by the bytes of g, u and
// y next to instruction issue (72 % of all slots): 4096 x 12288 bf16 to codes 44.3 us,
// 5.7 TB/s, 1.3 of which are the look for gates below kFar (46.2 without a limit on
// registers, whose blocks are fewer); with a library's exponential and division and eight
// values per thread 58.7.
template <class T, bool FP8, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC ? 16 : 8)
    gate_kernel(const __grid_constant__ GateArgs a, const int K, const int KB) {
    constexpr int kSign = FP8 ? -1 : 1;
    const int lane = threadIdx.x % kLanes;
    const long long units = (long long)a.M * KB, unit = (long long)blockIdx.x * kUnits + threadIdx.x / kLanes;
    // a division of 64 bits would take longer than everything else
    const long long m = units <= 0xFFFF0000ll ? (uint32_t)unit / (uint32_t)KB : unit / KB;
    // A thread has two runs of eight values: beside each other, or of f32 (whose runs are
    // two loads each) one in each half of the block: 4096 x 8192 f32 57.9 us, and 71 beside
    // each other; bf16 30.8 beside each other, 1.0 more apart. Values of rows that do not
    // lie in eights are eight apart, so that threads read places beside each other.
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
    float y[2][8], least = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float g[8];
        to_f32(gr[h], g);
        to_f32(ur[h], y[h]);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            least = least_of(least, g[i], g[i + 1]);
            const float2 v = gated<kSign>(make_float2(g[i], g[i + 1]), make_float2(y[h][i], y[h][i + 1]));
            y[h][i] = v.x;
            y[h][i + 1] = v.y;
        }
    }
    if (least < kFar) {
        float z[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) z[i] = y[i / 8][i % 8];
        again<T, kSign, kRun, kStep>(z, a, unit, lane, !VEC ? 1 : kRun == 8 ? 16 : 8);
#pragma unroll
        for (int i = 0; i < kPer; ++i) y[i / 8][i % 8] = z[i];
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
