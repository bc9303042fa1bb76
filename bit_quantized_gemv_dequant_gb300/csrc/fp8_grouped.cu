// qmm_fp8_b128_grouped: products of rows grouped by expert with that expert's
// weight, e4m3 codes and scales as in qmm_fp8_b128.
#include <cuda_fp8.h>

#include "fp8_groups.cuh"

namespace qg {
namespace {

constexpr int kGTile = 64;    // rows of a and of w per tile
constexpr int kGChunk = 32;   // k per step
constexpr int kGThreads = 256;
using GGroups = fp8::Groups<kGTile, 1>;

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// Any K and any alignment, on the CUDA cores: 64 x 64 outputs per CTA, 4 x 4 per
// thread; each block of 128 k is summed on its own and enters the total times its
// two scales.
template <class TY>
__global__ void __launch_bounds__(kGThreads)
    general_kernel(const GroupedArgs a, const int KB, unsigned* err) {
    extern __shared__ long long list[];
    __shared__ float as[kGChunk][kGTile + 4];
    __shared__ float ws[kGChunk][kGTile + 4];
    const int M = (int)a.M, N = (int)a.N, K = (int)a.K, nt = (N - 1) / kGTile + 1;
    GGroups groups(list, (int)a.E);
    if (threadIdx.x < 32) groups.build(a.offsets, M, nt, err);
    __syncthreads();
    TY* y = static_cast<TY*>(a.y);
    GGroups::Tile g{};
    const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
    for (long long t = blockIdx.x; t < groups.first[a.E]; t += gridDim.x) {
        groups.find(t, nt, g);
        const long long m0 = g.m0, n0 = (long long)g.n_tile * kGTile, end = g.m0 + g.rows;
        const uint8_t* w = a.w + (long long)g.e * N * K;
        const float* sw = a.sw + ((long long)g.e * ((N - 1) / 128 + 1) + n0 / 128) * KB;
        float total[4][4] = {}, part[4][4] = {};
        for (int k0 = 0; k0 < K; k0 += kGChunk) {
            for (int i = threadIdx.x; i < kGTile * kGChunk; i += kGThreads) {
                const int r = i / kGChunk, c = i % kGChunk;
                const bool in = k0 + c < K;
                as[c][r] = in && m0 + r < end ? e4m3_f32(a.a[(m0 + r) * K + k0 + c]) : 0.f;
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
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const long long m = m0 + tm * 4 + i;
                    const float s = (m < end ? a.sa[m * KB + b] : 0.f) * sw[b];
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
                if (m < end && n < N) y[m * N + n] = from_f32<TY>(total[i][j]);
            }
    }
}

template <class TY>
int general_launch(const DevCtx& dc, const GroupedArgs& a, cudaStream_t s) {
    general_kernel<TY><<<(unsigned)dc.num_sms * 4, kGThreads, GGroups::bytes(a.E), s>>>(a, (int)((a.K + 127) / 128), dc.err);
    return launched();
}

// On the tensor cores: by the kernel of few rows per expert, or that of many.
int tensor_launch(const DevCtx& dc, const GroupedArgs& a, cudaStream_t s) {
    if (!fp8::may_be_few(a.M, a.E)) return fp8::launch_grouped_tile(dc, a, s);
    fp8::FewPlan plan;
    const int rc = fp8::plan_grouped_few(dc, a, &plan);
    if (rc) return rc;
    return fp8::takes_few(plan, dc.num_sms, a.M, a.E, a.N, a.K) ? fp8::launch_grouped_few(dc, a, plan, s)
                                                                : fp8::launch_grouped_tile(dc, a, s);
}

}  // namespace

int fp8_grouped_launch(const DevCtx& dc, const GroupedArgs& args, void* ws, size_t ws_bytes, cudaStream_t s) {
    GroupedArgs a = args;
    const long long pitch = (a.K + 15) / 16 * 16;
    auto fits = [&](const uint8_t* p) { return a.K == pitch && reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    bool tma = fits(a.a) && fits(a.w);
    const size_t need = (size_t)((fits(a.a) ? 0 : a.M) + (fits(a.w) ? 0 : a.E * a.N)) * (size_t)pitch;
    if (!tma && pitch <= 0x7FFFFFFF && ws_bytes >= need) {
        // Zeros after the end of a row add nothing, and the blocks of 128 are the same. Of w
        // only the experts that have rows are copied.
        uint8_t* p = static_cast<uint8_t*>(ws);
        int rc = QG_OK;
        if (!fits(a.w)) {
            rc = fp8::pad_rows(dc, a.w, p, a.E * a.N, a.K, pitch, s, a.offsets, a.N);
            a.w = p;
            p += a.E * a.N * pitch;
        }
        if (rc == QG_OK && !fits(args.a)) {
            rc = fp8::pad_rows(dc, a.a, p, a.M, a.K, pitch, s);
            a.a = p;
        }
        if (rc) return rc;
        a.K = pitch;
        tma = true;
    }
    if (tma) return tensor_launch(dc, a, s);
    return a.y_dtype == QG_F32 ? general_launch<float>(dc, a, s) : general_launch<__nv_bfloat16>(dc, a, s);
}

}  // namespace qg
