// rms_norm, rms_norm_fp8_b128: the residual's addition, the root-mean-square norm
// of each row and its output as values or as e4m3 codes with a scale per 128.
#include <algorithm>

#include "fp8_code.cuh"
#include "fp8_tc.cuh"
#include "row8.cuh"

namespace qg {
namespace {

// h = x + r, s = 1 / sqrt(mean h^2 + eps), y = h s (offset + w). Bound by the bytes
// of x, r, the new r and y: a row is read once, its first 16 values per thread
// stay in registers as h until the row's sum is known. Rows of more than 16
// values for each of 1024 threads read the rest a second time (from L2, mostly).
//
// 8192 x 4096 bf16 with an f32 residual, to codes: 60.3 us, 6.1 TB/s; one row 2.6 us.
// With eight values per thread (and twice the threads) the former takes 100 us.
//
// A block of up to 1024 threads takes a row, or each warp of a small block does
// (rows of up to 512 values). 16 lanes hold the 128 values of a scale.
constexpr int kHeld = 2;            // units of eight values that a thread keeps
constexpr int kWarpRows = 4;        // warps, and rows, of a block of short rows

template <class TX, class TR, bool FP8, bool VEC>
__global__ void __launch_bounds__(1024)
    norm_kernel(const NormArgs a, const int K, const int threads) {
    __shared__ float sums[32];
    const int tid = threadIdx.x % threads;
    const long long m = (long long)blockIdx.x * (blockDim.x / threads) + threadIdx.x / threads;
    const TX* x = static_cast<const TX*>(a.x) + m * a.x_stride;
    const TR* r = static_cast<const TR*>(a.res) + m * a.res_stride;
    TR* r_out = static_cast<TR*>(a.res_out) + m * a.res_out_stride;
    const bool has_res = a.res != nullptr, live = m < a.M;
    fp8::pdl_wait();
    fp8::pdl_trigger();

    // Rows that do not lie in eights go through a warp's kilobyte of shared memory.
    extern __shared__ __align__(16) uint32_t tiles[];
    uint32_t* tile = tiles + (threadIdx.x / 32) * 256;
    const int lane8 = (threadIdx.x & 31) * 8;
    auto load = [&](auto* p, int k, int left, float (&v)[8]) {  // p[k .. k + 8), a warp's threads together
        using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
        if constexpr (VEC) to_f32(load8<T, true>(p + k, left), v);
        else load8_warp(p + k - lane8, left + lane8, tile, v);
    };
    auto store = [&](auto* p, int k, int left, const float (&v)[8]) {
        using T = std::remove_pointer_t<decltype(p)>;
        if constexpr (VEC) store8<T, true>(p + k, v, left);
        else store8_warp(p + k - lane8, v, left + lane8, tile);
    };
    auto load_h = [&](int k, float (&h)[8]) {
        const int left = live ? K - k : -lane8;
        load(x, k, left, h);
        if (has_res) {
            float f[8];
            load(r, k, left, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] += f[i];
        }
    };
    const int step = threads * 8;
    float h[kHeld][8], sum = 0.f;
#pragma unroll
    for (int c = 0; c < kHeld; ++c) load_h(tid * 8 + c * step, h[c]);
#pragma unroll
    for (int c = 0; c < kHeld; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);
    for (int k0 = kHeld * step; k0 < K; k0 += step) {
        float f[8];
        load_h(k0 + tid * 8, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
    }
#pragma unroll
    for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
    if (threads > 32) {
        if (tid % 32 == 0) sums[tid / 32] = sum;
        __syncthreads();
        sum = tid % 32 < threads / 32 ? sums[tid % 32] : 0.f;
#pragma unroll
        for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
    }
    // correctly rounded division and root: rows of few values are as exact as long ones
    const float root = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, (float)K) + a.eps));
    const float s = FP8 ? -root : root;  // codes are made from -y

    auto finish = [&](int k, const float (&f)[8]) {
        const int left = live ? K - k : -lane8;
        if (has_res) store(r_out, k, left, f);
        float y[8];
        const float s0 = VEC && left <= 0 ? 0.f : s;  // (behind the row's end f is 0 and s may be infinite)
        if (a.w) {
            float w[8];
            with_type(a.w_dtype, [&](auto t) { load(static_cast<const decltype(t)*>(a.w), k, K - k, w); });
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = f[i] * s0 * (w[i] + a.offset);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = f[i] * s0;
        }
        if constexpr (FP8) {
            if constexpr (!VEC) {  // what lies behind the row's end is 0 whatever s is
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= left) y[i] = 0.f;
            }
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) most = fp8_largest(most, y[i], y[i + 1]);
            unsigned top = __float_as_uint(most) & 0x7FFFFFFFu;
#pragma unroll
            for (int i = 8; i; i >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
            const float scale = fp8_scale(top);
            uint32_t code[2];
            fp8_encode<8>(y, scale, code);
            uint8_t* to = static_cast<uint8_t*>(a.y) + m * K + k;
            if constexpr (VEC) store_codes8<true>(to, code, left);
            else store_codes8_warp(to - lane8, code, left + lane8, tile);
            if (tid % 16 == 0 && left > 0) a.scales[m * ((K + 127) / 128) + k / 128] = scale;
        } else {
            with_type(a.y_dtype, [&](auto t) { store(static_cast<decltype(t)*>(a.y) + m * K, k, left, y); });
        }
    };
#pragma unroll
    for (int c = 0; c < kHeld; ++c) finish(tid * 8 + c * step, h[c]);
    // all threads of a warp together: 16 of them share a scale
    for (int k0 = kHeld * step; k0 < K; k0 += step) {
        float f[8];
        load_h(k0 + tid * 8, f);
        finish(k0 + tid * 8, f);
    }
}

template <class TX, class TR, bool FP8>
int launch(const NormArgs& a, cudaStream_t s) {
    const bool vec = in_eights(a.x, a.x_stride, a.K, sizeof(TX)) &&
                     (!a.res || (in_eights(a.res, a.res_stride, a.K, sizeof(TR)) &&
                                 in_eights(a.res_out, a.res_out_stride, a.K, sizeof(TR)))) &&
                     (!a.w || in_eights(a.w, 8, a.K, type_bytes(a.w_dtype))) &&
                     (FP8 ? reinterpret_cast<uintptr_t>(a.y) % 8 == 0 : in_eights(a.y, a.K, a.K, type_bytes(a.y_dtype)));
    const long long warps = std::min<long long>((a.K + 256 * kHeld - 1) / (256 * kHeld), 32);
    const int threads = (int)warps * 32, block = threads == 32 ? 32 * kWarpRows : threads;
    const long long grid = (a.M + block / threads - 1) / (block / threads);
    if (grid > 0x7FFFFFFFLL) return QG_ERR_UNSUPPORTED;
    return launch_after(vec ? norm_kernel<TX, TR, FP8, true> : norm_kernel<TX, TR, FP8, false>, dim3((unsigned)grid),
                        dim3(block), vec ? 0 : block * 32, s, a, (int)a.K, threads);
}

template <class TX, class TR>
int launch_out(const NormArgs& a, cudaStream_t s) {
    return a.scales ? launch<TX, TR, true>(a, s) : launch<TX, TR, false>(a, s);
}

}  // namespace

int norm_launch(const NormArgs& a, cudaStream_t s) {
    return by_type(a.x_dtype, [&](auto t) {
        using T = decltype(t);
        if (a.res && a.res_dtype != a.x_dtype) return launch_out<T, float>(a, s);
        return launch_out<T, T>(a, s);
    });
}

}  // namespace qg
