// qmm_fp8_b128 for many rows of a: persistent CTAs over tiles of 128 rows of a
// times 256 rows of w.
#include <algorithm>

#include "fp8_tc.cuh"

namespace qg {
namespace fp8 {
namespace {

// Bound by the tensor cores: 128 x 256 x 128 products of a k block take them
// 512 cycles, while the two epilogue warpgroups bring its accumulator, which
// has two places in tensor memory, into registers: thread = row of a and 128
// columns, which lie in one block of w's scales, so a k block enters the sum
// as fma(d, a_scale * w_scale, acc) with one factor per thread.
//
//   warps 0-7  epilogue (ten warps leave 200 registers: 128 sums fit)
//   warp 8     TMA producer (48 KB per k block, four stages)
//   warp 9     MMA issuer
constexpr int kThreads = 320;
constexpr int kBM = 128, kBN = 256;
constexpr int kStages = 4;
constexpr int kStage = (kBM + kBN) * 128;
constexpr int kBarOff = kStages * kStage;
constexpr int kSmem = 1024 + kBarOff + 256;
constexpr uint32_t kDesc = f8_idesc(kBM, kBN);

template <class TY>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                const Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const uint32_t bars = base + kBarOff;
    auto full = [&](int i) { return bars + 8u * i; };
    auto empty = [&](int i) { return bars + 8u * (kStages + i); };
    auto t_full = [&](int i) { return bars + 8u * (2 * kStages + i); };
    auto t_empty = [&](int i) { return bars + 8u * (2 * kStages + 2 + i); };
    const uint32_t done = bars + 8u * (2 * kStages + 4);
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kBarOff + 8 * (2 * kStages + 5));
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int mt = (p.M + kBM - 1) / kBM, nt = (p.N + kBN - 1) / kBN;
    const long long tiles = (long long)mt * nt;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(t_full(i), 1);
            mbar_init(t_empty(i), 8);
        }
        mbar_init(done, 1);
        fence_mbar_init();
        prefetch_tmap(&map_a);
        prefetch_tmap(&map_w);
    }
    if (warp == 9) tmem_alloc(smem_addr(slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    pdl_trigger();
    pdl_wait();

    if (warp >= 8) {
        if (warp == 8 && lane == 0) {
            int i = 0;
            bool ok = true;
            for (long long t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int m0 = (int)(t % mt) * kBM, n0 = (int)(t / mt) * kBN;
                for (int b = 0; b < p.KB; ++b, ++i) {
                    const int st = i % kStages;
                    if (i >= kStages && !bar_wait(empty(st), ((i / kStages) & 1) ^ 1)) {
                        report_error(p.err, DEVERR_TC_WAIT);
                        ok = false;
                        break;
                    }
                    const uint32_t sb = base + st * kStage;
                    mbar_arrive_expect_tx(full(st), kStage);
                    tma_load_2d(sb, &map_a, b * 128, m0, full(st));
                    tma_load_2d(sb + kBM * 128, &map_w, b * 128, n0, full(st));
                }
            }
            for (int j = max(0, i - kStages); j < i; ++j)
                if (!bar_wait(full(j % kStages), (j / kStages) & 1)) report_error(p.err, DEVERR_WAIT_DRAIN);
        } else if (warp == 9) {
            const uint64_t da = sw128_desc(base), dw = sw128_desc(base + kBM * 128);
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            int st = 0, tb = 0;
            uint32_t ph = 0, tph = 0;
            bool ok = true;
            for (long long t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                for (int b = 0; b < p.KB; ++b) {
                    if (!warp_bar_wait(full(st), ph) || !warp_bar_wait(t_empty(tb), tph ^ 1)) {
                        if (lane == 0) report_error(p.err, DEVERR_TC_WAIT);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a = da + (uint64_t)(st * (kStage >> 4)), w = dw + (uint64_t)(st * (kStage >> 4));
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_f8(tm + tb * kBN, a + 2 * k, w + 2 * k, kDesc, k > 0);
                        tc_commit(empty(st));
                        tc_commit(t_full(tb));
                    }
                    __syncwarp();
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1;
                    }
                    tb ^= 1;
                    tph ^= tb == 0;
                }
            }
            if (elect_one()) tc_commit(done);
            __syncwarp();
            if (!warp_bar_wait(done, 0) && lane == 0) report_error(p.err, DEVERR_WAIT_DRAIN);
        }
    } else {
        const int half = warp / 4;
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 128;
        int i = 0;
        bool ok = true;
        for (long long t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const int m = (int)(t % mt) * kBM + (warp & 3) * 32 + lane;
            const long long n0 = (t / mt) * kBN + half * 128;
            const bool live = m < p.M && n0 < p.N;
            const float* sa = p.sa + (long long)min(m, p.M - 1) * p.KB;
            const float* sw = p.sw + min(n0, (long long)p.N - 1) / 128 * p.KB;
            float2 acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
            // The scales of the next k block, loaded one k block ahead.
            float sa_next = __ldg(sa), sw_next = __ldg(sw);
            for (int b = 0; b < p.KB; ++b, ++i) {
                const int tb = i & 1;
                const float sc = sa_next * sw_next;
                const float2 s = make_float2(sc, sc);
                if (b + 1 < p.KB) {
                    sa_next = __ldg(sa + b + 1);
                    sw_next = __ldg(sw + b + 1);
                }
                if (!warp_bar_wait(t_full(tb), (i / 2) & 1)) {
                    if (lane == 0) report_error(p.err, DEVERR_TC_WAIT);
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t r[2][16];
                tmem_ld16_async(at + tb * kBN, r[0]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    tmem_wait16(r[c & 1]);
                    if (c < 7) {
                        tmem_ld16_async(at + tb * kBN + (c + 1) * 16, r[(c + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(t_empty(tb));
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        acc[c * 8 + j] = fma2(make_float2(__uint_as_float(r[c & 1][2 * j]),
                                                          __uint_as_float(r[c & 1][2 * j + 1])),
                                              s, acc[c * 8 + j]);
                }
            }
            if (!ok || !live) continue;
            TY* y = static_cast<TY*>(p.y) + (long long)m * p.N + n0;
            if (p.vec && n0 + 128 <= p.N) {
                constexpr int kPer = 32 / sizeof(TY);  // outputs per 32-byte store
#pragma unroll
                for (int c = 0; c < 128; c += kPer) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if constexpr (sizeof(TY) == 4)
                            w[j] = __float_as_uint(j & 1 ? acc[(c + j) / 2].y : acc[(c + j) / 2].x);
                        else
                            w[j] = pack2<TY>(acc[c / 2 + j].x, acc[c / 2 + j].y);
                    }
                    st_global_256(y + c, w);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if (n0 + c < p.N) y[c] = from_f32<TY>(c & 1 ? acc[c / 2].y : acc[c / 2].x);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <class TY>
int launch(const DevCtx& dc, const Fp8Args& a, cudaStream_t s) {
    static int configured[64] = {0};
    auto kern = tile_kernel<TY>;
    if (!configured[dc.device]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return cuda_fail(e);
        configured[dc.device] = 1;
    }
    CUtensorMap ma, mw;
    int rc = code_map(&ma, a.a, a.M, a.K, kBM);
    if (rc == QG_OK) rc = code_map(&mw, a.w, a.N, a.K, kBN);
    if (rc) return rc;
    const bool vec = reinterpret_cast<uintptr_t>(a.y) % 32 == 0 && a.N * sizeof(TY) % 32 == 0;
    const Params p{a.sa, a.sw, a.y, (int)a.M, (int)a.N, (int)((a.K + 127) / 128), vec, dc.err};
    const long long tiles = ((a.M + kBM - 1) / kBM) * ((a.N + kBN - 1) / kBN);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::min<long long>(tiles, dc.num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, ma, mw, p);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

}  // namespace

int launch_tile(const DevCtx& dc, const Fp8Args& a, cudaStream_t s) {
    return a.y_dtype == QG_F32 ? launch<float>(dc, a, s) : launch<__nv_bfloat16>(dc, a, s);
}

}  // namespace fp8
}  // namespace qg
