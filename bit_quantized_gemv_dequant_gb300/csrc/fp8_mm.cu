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
    const unsigned nt = (N - 1) / kGTile + 1;
    const long long m0 = (long long)(blockIdx.x / nt) * kGTile, n0 = (long long)(blockIdx.x % nt) * kGTile;
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

// dst[r][c] = src[r][c] for c < K, 0 up to the pitch (a multiple of 16); src's
// rows start at any byte. 16 bytes per thread, from the five aligned words that
// hold them; where those are not all inside src, byte by byte.
constexpr int kPadThreads = 256;
__global__ void __launch_bounds__(kPadThreads)
    pad_kernel(const uint8_t* __restrict__ src, uint8_t* __restrict__ dst, long long rows, int K, int pitch) {
    const int per = pitch / 16;
    const uintptr_t begin = reinterpret_cast<uintptr_t>(src), end = begin + rows * K;
    for (long long i = (long long)blockIdx.x * kPadThreads + threadIdx.x; i < rows * per;
         i += (long long)gridDim.x * kPadThreads) {
        const long long r = i < 0x7FFFFFFF ? (int)i / per : i / per;
        const int c = (int)(i - r * per) * 16, n = min(16, K - c);
        const uintptr_t at = begin + r * K + c, word = at & ~(uintptr_t)3;
        const int shift = (int)(at - word) * 8;
        uint32_t v[5];
        if (word >= begin && word + 20 <= end) {
#pragma unroll
            for (int j = 0; j < 5; ++j) v[j] = __ldg(reinterpret_cast<const uint32_t*>(word) + j);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __funnelshift_r(v[j], v[j + 1], shift);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (4 * j + b < n) v[j] |= (uint32_t)reinterpret_cast<const uint8_t*>(at)[4 * j + b] << (8 * b);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int left = n - 4 * j;  // bytes of this word that belong to the row
            if (left < 4) v[j] &= left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        }
        *reinterpret_cast<uint4*>(dst + r * pitch + c) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

int pad_launch(const DevCtx& dc, const uint8_t* src, uint8_t* dst, long long rows, long long K, long long pitch,
               cudaStream_t s) {
    const long long ctas = (rows * (pitch / 16) + kPadThreads - 1) / kPadThreads;
    pad_kernel<<<(unsigned)(ctas < dc.num_sms * 16LL ? ctas : dc.num_sms * 16LL), kPadThreads, 0, s>>>(
        src, dst, rows, (int)K, (int)pitch);
    return launched();
}

template <class TY>
int general_launch(const Fp8Args& a, cudaStream_t s) {
    const long long tiles = ((a.N + kGTile - 1) / kGTile) * ((a.M + kGTile - 1) / kGTile);
    if (tiles > 0x7FFFFFFFLL) return QG_ERR_UNSUPPORTED;  // y alone would be 2^43 values
    general_kernel<TY><<<(unsigned)tiles, kGThreads, 0, s>>>(
        a.a, a.sa, a.w, a.sw, static_cast<TY*>(a.y), (int)a.M, (int)a.N, (int)a.K,
        (int)((a.K + 127) / 128));
    return launched();
}

}  // namespace

int fp8_mm_launch(const DevCtx& dc, const Fp8Args& args, void* ws, size_t ws_bytes, cudaStream_t s) {
    Fp8Args a = args;
    const long long pitch = (a.K + 15) / 16 * 16;
    auto fits = [&](const uint8_t* p) { return a.K == pitch && reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    bool tma = fits(a.a) && fits(a.w);
    if (!tma && pitch <= 0x7FFFFFFF && ws_bytes >= (size_t)((a.M + a.N) * pitch)) {
        // Zeros after the end of a row add nothing, and the blocks of 128 are the
        // same. (M = 37, N = 2200, K = 5201: 13 us, and 553 on the CUDA cores.)
        uint8_t* p = static_cast<uint8_t*>(ws);
        int rc = QG_OK;
        if (!fits(a.w)) {
            rc = pad_launch(dc, a.w, p, a.N, a.K, pitch, s);
            a.w = p;
            p += a.N * pitch;
        }
        if (rc == QG_OK && !fits(args.a)) {
            rc = pad_launch(dc, a.a, p, a.M, a.K, pitch, s);
            a.a = p;
        }
        if (rc) return rc;
        a.K = pitch;
        tma = true;
    }
    if (tma) return fp8::swap_is_shorter(dc, a) ? fp8::launch_swap(dc, a, s) : fp8::launch_tile(dc, a, s);
    return a.y_dtype == QG_F32 ? general_launch<float>(a, s) : general_launch<__nv_bfloat16>(a, s);
}

}  // namespace qg
