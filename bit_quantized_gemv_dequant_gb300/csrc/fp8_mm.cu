// qmm_fp8_b128: the product of e4m3 codes with one f32 scale per row and 128
// values of K on the left and per 128 x 128 values on the right.
#include <cuda_fp8.h>

#include "fp8_tc.cuh"

namespace qg {
namespace {

constexpr int kGTile = 64;    // rows of a and of w per CTA
constexpr int kGChunk = 32;   // k per step
constexpr int kGThreads = 256;

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// Any K and any alignment, on the CUDA cores: 64 x 64 outputs per CTA, 4 x 4
// per thread; each block of 128 k is summed on its own and enters the total
// times its two scales.
template <class TY>
__global__ void __launch_bounds__(kGThreads)
    general_kernel(const uint8_t* __restrict__ a, const float* __restrict__ sa,
                   const uint8_t* __restrict__ w, const float* __restrict__ sw,
                   TY* __restrict__ y, int M, int N, int K, int KB) {
    __shared__ float as[kGChunk][kGTile + 4];
    __shared__ float ws[kGChunk][kGTile + 4];
    const long long m0 = (long long)blockIdx.y * kGTile, n0 = (long long)blockIdx.x * kGTile;
    const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
    float total[4][4] = {}, part[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kGChunk) {
        for (int i = threadIdx.x; i < kGTile * kGChunk; i += kGThreads) {
            const int r = i / kGChunk, c = i % kGChunk;
            const bool in = k0 + c < K;
            as[c][r] = in && m0 + r < M ? e4m3_f32(a[(m0 + r) * K + k0 + c]) : 0.f;
            ws[c][r] = in && n0 + r < N ? e4m3_f32(w[(n0 + r) * K + k0 + c]) : 0.f;
        }
        __syncthreads();
#pragma unroll 8
        for (int c = 0; c < kGChunk; ++c) {
            const float4 av = *reinterpret_cast<const float4*>(&as[c][tm * 4]);
            const float4 wv = *reinterpret_cast<const float4*>(&ws[c][tn * 4]);
            const float ar[4] = {av.x, av.y, av.z, av.w}, wr[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) part[i][j] = fmaf(ar[i], wr[j], part[i][j]);
        }
        __syncthreads();
        if ((k0 + kGChunk) % 128 == 0 || k0 + kGChunk >= K) {
            const int b = k0 / 128;
            const float swb = sw[(n0 / 128) * KB + b];  // a tile of 64 lies in one block of 128 rows
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long m = m0 + tm * 4 + i;
                const float s = (m < M ? sa[m * KB + b] : 0.f) * swb;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    total[i][j] = fmaf(part[i][j], s, total[i][j]);
                    part[i][j] = 0.f;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long m = m0 + tm * 4 + i, n = n0 + tn * 4 + j;
            if (m < M && n < N) y[m * N + n] = from_f32<TY>(total[i][j]);
        }
}

template <class TY>
int general_launch(const Fp8Args& a, cudaStream_t s) {
    const long long gx = (a.N + kGTile - 1) / kGTile, gy = (a.M + kGTile - 1) / kGTile;
    if (gx > 0x7FFFFFFFLL || gy > 65535) return QG_ERR_UNSUPPORTED;
    general_kernel<TY><<<dim3((unsigned)gx, (unsigned)gy), kGThreads, 0, s>>>(
        a.a, a.sa, a.w, a.sw, static_cast<TY*>(a.y), (int)a.M, (int)a.N, (int)a.K,
        (int)((a.K + 127) / 128));
    return launched();
}

}  // namespace

int fp8_mm_launch(const DevCtx& dc, const Fp8Args& a, cudaStream_t s) {
    const bool tma = a.K % 16 == 0 && reinterpret_cast<uintptr_t>(a.a) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.w) % 16 == 0;
    if (tma) return fp8::swap_is_shorter(dc, a) ? fp8::launch_swap(dc, a, s) : fp8::launch_tile(dc, a, s);
    return a.y_dtype == QG_F32 ? general_launch<float>(a, s) : general_launch<__nv_bfloat16>(a, s);
}

}  // namespace qg
