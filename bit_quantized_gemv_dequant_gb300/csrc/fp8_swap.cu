// qmm_fp8_b128 for few rows of a: 128 rows of w on the tensor cores' M side, the
// rows of a on the N side, K split over a thread-block cluster.
#include <algorithm>

#include "fp8_tc.cuh"

namespace qg {
namespace fp8 {
namespace {

// One CTA: 128 rows of w (one block of scales) times BN rows of a, over its
// share of the 128-wide k blocks. Bound by the bytes of w, so the shape is
// chosen for loads in flight: the ring holds up to 200 KB, and N / 128 tiles
// times the split give about one CTA per SM.
//
//   warp 0    TMA producer: w tile and a tile of each k block.
//   warp 1    issues the four MMAs of a k block into an accumulator of its own
//             (kBufs of them in tensor memory).
//   warps 4-7 (and 8-11 from BN = 64 on, for the second half of the rows of a)
//             take the accumulators into registers, times
//             a_scale[m, b] * w_scale[n / 128, b] (f32): thread = row of w.
//
// The ring takes all of an SM, so the split is chosen by how many clusters of its
// size the GPU can place at once (plan() below). Measured, product alone:
//   N = K = 4096, M = 1         6.3 us  2.7 TB/s of w (launch, first loads, joining)
//   N = 2200, K = 5200, M = 33  6.8 us  1.7 TB/s
//   N = K = 12288, M = 1        28.0 us 5.4 TB/s (96 of 152 SMs load: a split is the
//                               same for all tiles, and two each would not fit)
//
// The split's partial sums meet in shared memory over the cluster, each CTA
// adding up its share of the rows of a in the order of the split: the result
// does not depend on timing. Threads of a warp hold consecutive n, so stores
// of y are coalesced.
constexpr int kScaleBlocks = 16;  // k blocks whose scales are staged at a time

template <int BN>
struct Geo {
    static constexpr int kStage = 16384 + BN * 128;
    static constexpr int kStages = BN == 128 ? 6 : BN == 64 ? 8 : 10;
    static constexpr int kBufs = BN == 16 ? 8 : 256 / BN;  // accumulators of BN columns
    static constexpr int kGroups = BN >= 64 ? 2 : 1;       // epilogue warpgroups
    static constexpr int kThreads = 128 + 128 * kGroups;
    static constexpr int kEpi = 128 * kGroups;             // epilogue threads
    static constexpr int kOwn = BN / kGroups;              // rows of a per epilogue thread
    static constexpr int kCols = kBufs * BN < 32 ? 32 : kBufs * BN;
    static constexpr int kScaleOff = kStages * kStage;
    static constexpr int kBarOff = kScaleOff + kScaleBlocks * BN * 4;
    static constexpr int kSmem = 1024 + kBarOff + 512;
    static_assert(BN * 128 * 4 <= kStages * kStage, "partial sums reuse the ring");
    static_assert(8 * (2 * kStages + 2 * kBufs + 1) + 8 <= 512, "barriers");
};

template <int BN, class TY>
__global__ void __launch_bounds__(Geo<BN>::kThreads, 1)
    swap_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                const Params p) {
    using G = Geo<BN>;
    constexpr uint32_t kDesc = f8_idesc(128, BN);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    float* scales = reinterpret_cast<float*>(smem + G::kScaleOff);
    const uint32_t bars = base + G::kBarOff;
    auto full = [&](int i) { return bars + 8u * i; };
    auto empty = [&](int i) { return bars + 8u * (G::kStages + i); };
    auto t_full = [&](int i) { return bars + 8u * (2 * G::kStages + i); };
    auto t_empty = [&](int i) { return bars + 8u * (2 * G::kStages + G::kBufs + i); };
    const uint32_t done = bars + 8u * (2 * G::kStages + 2 * G::kBufs);
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + G::kBarOff + 8 * (2 * G::kStages + 2 * G::kBufs + 1));

    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int split = (int)gridDim.x, rank = (int)blockIdx.x;
    const int n0 = (int)blockIdx.y * 128, m0 = (int)blockIdx.z * BN;
    const int b0 = (int)((long long)p.KB * rank / split), b1 = (int)((long long)p.KB * (rank + 1) / split);
    const int nb = b1 - b0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < G::kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < G::kBufs; ++i) {
            mbar_init(t_full(i), 1);
            mbar_init(t_empty(i), 4 * G::kGroups);
        }
        mbar_init(done, 1);
        fence_mbar_init();
        prefetch_tmap(&map_w);
        prefetch_tmap(&map_a);
    }
    if (warp == 1) tmem_alloc(smem_addr(slot), G::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    pdl_wait();
    pdl_trigger();

    float2 acc[G::kOwn / 2];
#pragma unroll
    for (int i = 0; i < G::kOwn / 2; ++i) acc[i] = make_float2(0.f, 0.f);
    const int row = (warp & 3) * 32 + lane;
    const int own0 = (warp >> 2) > 1 ? ((warp >> 2) - 1) * G::kOwn : 0;  // first row of a of this thread

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int i = 0; i < nb; ++i) {
                const int st = i % G::kStages;
                if (i >= G::kStages && !bar_wait(empty(st), ((i / G::kStages) & 1) ^ 1)) {
                    report_error(p.err, DEVERR_TC_WAIT);
                    break;
                }
                const uint32_t sb = base + st * G::kStage;
                mbar_arrive_expect_tx(full(st), G::kStage);
                tma_load_2d(sb, &map_w, (b0 + i) * 128, n0, full(st));
                tma_load_2d(sb + 16384, &map_a, (b0 + i) * 128, m0, full(st));
                issued = i + 1;
            }
            for (int i = max(0, issued - G::kStages); i < issued; ++i)
                if (!bar_wait(full(i % G::kStages), (i / G::kStages) & 1))
                    report_error(p.err, DEVERR_WAIT_DRAIN);
        }
    } else if (warp == 1) {
        const uint64_t dw = sw128_desc(base), da = sw128_desc(base + 16384);
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
        int st = 0, tb = 0;
        uint32_t ph = 0, tph = 0;
        for (int i = 0; i < nb; ++i) {
            if (!warp_bar_wait(full(st), ph) || !warp_bar_wait(t_empty(tb), tph ^ 1)) {
                if (lane == 0) report_error(p.err, DEVERR_TC_WAIT);
                break;
            }
            tc_fence_after();
            const uint64_t w = dw + (uint64_t)(st * (G::kStage >> 4)), a = da + (uint64_t)(st * (G::kStage >> 4));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_f8(tm + tb * BN, w + 2 * k, a + 2 * k, kDesc, k > 0);
                tc_commit(empty(st));
                tc_commit(t_full(tb));
            }
            __syncwarp();
            if (++st == G::kStages) {
                st = 0;
                ph ^= 1;
            }
            if (++tb == G::kBufs) {
                tb = 0;
                tph ^= 1;
            }
        }
        if (elect_one()) tc_commit(done);
        __syncwarp();
        if (!warp_bar_wait(done, 0) && lane == 0) report_error(p.err, DEVERR_WAIT_DRAIN);
    } else if (warp >= 4) {
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float* sw = p.sw + (long long)blockIdx.y * p.KB + b0;
        bool ok = true;
        for (int i0 = 0; i0 < nb; i0 += kScaleBlocks) {
            // The scales of the next blocks: [block][row of a], both factors in one.
            const int nk = min(kScaleBlocks, nb - i0);
            if (i0) named_bar_sync(1, G::kEpi);
            for (int j = threadIdx.x - 128; j < nk * BN; j += G::kEpi) {
                const int m = j / nk, b = j % nk;  // consecutive threads, consecutive blocks of a row
                scales[b * BN + m] = m0 + m < p.M
                    ? __ldg(p.sa + (long long)(m0 + m) * p.KB + b0 + i0 + b) * __ldg(sw + i0 + b) : 0.f;
            }
            named_bar_sync(1, G::kEpi);
            for (int b = 0; b < nk; ++b) {
                const int i = i0 + b, tb = i % G::kBufs;
                if (ok && !warp_bar_wait(t_full(tb), (i / G::kBufs) & 1)) {
                    if (lane == 0) report_error(p.err, DEVERR_TC_WAIT);
                    ok = false;  // the sums are lost; the barriers are still met
                }
                tc_fence_after();
                const float4* sc = reinterpret_cast<const float4*>(scales + b * BN + own0);
                const uint32_t from = tmem + lanes + tb * BN + own0;
                constexpr int kChunk = 16, kChunks = G::kOwn / kChunk;
                uint32_t r2[2][kChunk];
                tmem_ld16_async(from, r2[0]);
#pragma unroll
                for (int c = 0; c < G::kOwn; c += kChunk) {
                    uint32_t(&r)[kChunk] = r2[(c / kChunk) & 1];
                    tmem_wait16(r);
                    if (c / kChunk + 1 < kChunks) {
                        tmem_ld16_async(from + c + kChunk, r2[(c / kChunk + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(t_empty(tb));
                    }
#pragma unroll
                    for (int j = 0; j < kChunk; j += 4) {
                        const float4 s = sc[(c + j) / 4];
                        float2& a0 = acc[(c + j) / 2];
                        float2& a1 = acc[(c + j) / 2 + 1];
                        a0 = fma2(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                  make_float2(s.x, s.y), a0);
                        a1 = fma2(make_float2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])),
                                  make_float2(s.z, s.w), a1);
                    }
                }
            }
        }
    }
    __syncthreads();

    TY* y = static_cast<TY*>(p.y);
    const long long n = n0 + row;
    if (split == 1) {
        if (warp >= 4 && n < p.N) {
#pragma unroll
            for (int c = 0; c < G::kOwn; ++c)
                if (m0 + own0 + c < p.M)
                    y[(m0 + own0 + c) * (long long)p.N + n] = from_f32<TY>(c & 1 ? acc[c / 2].y : acc[c / 2].x);
        }
    } else {
        float* part = reinterpret_cast<float*>(smem);  // [row of a][row of w]; the ring is idle
        const int rows = min(BN, p.M - m0);
        if (warp >= 4) {
#pragma unroll
            for (int c = 0; c < G::kOwn; ++c)
                if (own0 + c < rows) part[(own0 + c) * 128 + row] = c & 1 ? acc[c / 2].y : acc[c / 2].x;
        }
        cluster_sync();
        for (int e = rank * G::kThreads + threadIdx.x; e < rows * 32; e += split * G::kThreads) {
            float4 v[8];  // all parts under way at once
#pragma unroll
            for (int r = 0; r < 8; ++r)
                v[r] = r < split ? ld_cluster(base + e * 16, r) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 1; r < 8; ++r) {
                v[0].x += v[r].x; v[0].y += v[r].y; v[0].z += v[r].z; v[0].w += v[r].w;
            }
            const float o[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
            const long long m = m0 + e / 32, col = n0 + e % 32 * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < p.N) y[m * p.N + col + i] = from_f32<TY>(o[i]);
        }
        cluster_sync();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, G::kCols);
    }
}

// The tiles, and the largest split of K whose clusters all run at once with two
// k blocks per CTA at least; no split if the tiles fill more than half of the GPU.
// A second round costs more than a longer first one: N = K = 12288, M = 1, 96
// tiles: 28.0 us without a split, 36 to 50 with any (76 clusters of 2 run at
// once, 46 of 3, 36 of 4, 23 of 6, 15 of 8); N = K = 8192, 64 tiles: 14.4 us split
// in 2, 17.0 without and 17.8 in 4; N = 2200, K = 5200, 18 tiles: 5.65 us split in
// 6, 5.9 in 4, 9.6 in 8.
struct Plan {
    long long nt, mt, kb;
    int split;
    long long rounds;
};
template <int BN, class TY>
int plan(const DevCtx& dc, const Fp8Args& a, Plan* p) {
    const int* room = nullptr;
    const int rc = cluster_room<swap_kernel<BN, TY>>(dc, Geo<BN>::kThreads, Geo<BN>::kSmem, &room);
    if (rc) return rc;
    *p = Plan{(a.N + 127) / 128, (a.M + BN - 1) / BN, (a.K + 127) / 128, 1, 1};
    for (int i = 2; i < 9 && p->kb >= 2 * i; ++i)
        if (p->nt * p->mt <= room[i]) p->split = i;
    if (room[p->split] < 1) return QG_ERR_UNSUPPORTED;
    p->rounds = (p->nt * p->mt + room[p->split] - 1) / room[p->split];
    return QG_OK;
}

template <int BN, class TY>
int launch(const DevCtx& dc, const Fp8Args& a, cudaStream_t s) {
    using G = Geo<BN>;
    Plan pl;
    int rc = plan<BN, TY>(dc, a, &pl);
    CUtensorMap mw, ma;
    if (rc == QG_OK) rc = code_map(&mw, a.w, a.N, a.K, 128);
    if (rc == QG_OK) rc = code_map(&ma, a.a, a.M, a.K, BN);
    if (rc) return rc;
    if (pl.nt > 65535 || pl.mt > 65535) return QG_ERR_UNSUPPORTED;
    const Params p{a.sa, a.sw, a.y, (int)a.M, (int)a.N, (int)pl.kb, false, dc.err};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)pl.split, (unsigned)pl.nt, (unsigned)pl.mt);
    cfg.blockDim = dim3(G::kThreads);
    cfg.dynamicSmemBytes = G::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)pl.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = may_overlap() ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, swap_kernel<BN, TY>, mw, ma, p);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

template <class TY>
int launch_type(const DevCtx& dc, const Fp8Args& a, cudaStream_t s) {
    if (a.M <= 16) return launch<16, TY>(dc, a, s);
    if (a.M <= 32) return launch<32, TY>(dc, a, s);
    if (a.M <= 64) return launch<64, TY>(dc, a, s);
    return launch<128, TY>(dc, a, s);
}

}  // namespace

int launch_swap(const DevCtx& dc, const Fp8Args& a, cudaStream_t s) {
    return a.y_dtype == QG_F32 ? launch_type<float>(dc, a, s) : launch_type<__nv_bfloat16>(dc, a, s);
}

// Both kernels take about 0.5 us per k block and CTA, so the one with fewer k
// blocks one after the other is taken. M = 256, N = K = 4096: 11.7 us with the
// split, 18.1 in 256-wide tiles; M = 256, N = 12288, K = 4096: 32.9 and 18.1.
bool swap_is_shorter(const DevCtx& dc, const Fp8Args& a) {
    if (a.N > 65535 * 128LL || a.M > 65535 * 128LL) return false;  // more tiles than a grid's y or z has room for
    if (a.M <= 64) return true;
    Plan p;
    if (plan<128, float>(dc, a, &p) != QG_OK) return false;
    const long long tiles = 2 * ((a.M + 255) / 256) * ((a.N + 255) / 256);  // per SM
    return p.rounds * ((p.kb + p.split - 1) / p.split) <= (tiles + dc.num_sms - 1) / dc.num_sms * p.kb;
}

int code_map(CUtensorMap* m, const uint8_t* ptr, long long rows, long long cols, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    int rc = encoder(&encode);
    if (rc) return rc;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(ptr), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QG_OK
               : QG_ERR_UNSUPPORTED;
}

}  // namespace fp8
}  // namespace qg
