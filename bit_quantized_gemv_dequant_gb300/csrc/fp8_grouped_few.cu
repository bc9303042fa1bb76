// qmm_fp8_b128_grouped for experts of few rows: 128 rows of a weight on the tensor
// cores' M side, up to 64 rows of a on the N side, K split over a thread-block
// cluster where there are too few tiles for the GPU.
#include <algorithm>

#include "fp8_groups.cuh"

namespace qg {
namespace fp8 {
namespace {

// A persistent cluster of CTAs per tile: 128 rows of w (one block of scales) times
// up to 64 rows of one expert, in steps of 16 (the instruction's N, and what is
// loaded of a, follow the rows that there are). Bound by the bytes of w: its loads
// go on across tiles, 112 KB under way per SM.
//
//   warp 0      builds the list of tiles, then TMA producer
//   warp 1      issues the four MMAs of a k block into an accumulator of its own
//               (eight of them in tensor memory)
//   warps 2-3   scales
//   warps 4-11  take the accumulators into registers, times both scales (f32):
//               thread = row of w, and 32 of the 64 rows of a
//
// 256 rows on 64 experts, N = K = 4096, bf16: 156 us, 6.6 TB/s. 8 rows on 8 of them, N =
// 4096, K = 2048: 17.8 us, 3.8 TB/s: 256 tiles on 152 SMs, the second round as slow as
// the first; 3 us until the first k block is there.
//
// Tiles that do not fill a round of all CTAs are shared, by K, over a cluster (9
// experts of 34 rows, N = 2200, K = 5200: 27.5 us, 35 without). Its parts meet in
// shared memory over the cluster, each CTA adding up its share of the rows of a in the
// order of the split: the result does not depend on timing.
constexpr int kBN = 64;
constexpr int kThreads = 384, kEpi = 256;
constexpr int kStages = 7, kStage = 16384 + kBN * 128;
constexpr int kBufs = 8;
constexpr int kOwn = kBN / 2;  // rows of a per epilogue thread
constexpr int kPartOff = kStages * kStage;
constexpr int kPitch = scale_pitch(kBN);
constexpr int kScaleOff = kPartOff + kBN * 128 * 4;
constexpr int kBarOff = kScaleOff + kSets * kSetBlocks * kPitch * 4;
constexpr int kBars = 2 * kStages + 2 * kBufs + 2 * kSets + 3;
constexpr int kGroupOff = kBarOff + 8 * kBars + 8;
using FewGroups = Groups<kBN, 16>;
constexpr int smem_bytes(long long E) { return 1024 + kGroupOff + FewGroups::bytes(E); }
static_assert(smem_bytes(kMaxExperts) <= 227 * 1024, "shared memory");
static_assert(kGroupOff % 8 == 0, "tile numbers are 8 bytes");

__device__ __forceinline__ void arrive_in_cta(uint32_t bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_cta(bar, rank)) : "memory");
}
// Bounded wait for what other CTAs of the cluster did before they arrived.
__device__ __forceinline__ bool cluster_bar_wait(uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            uint32_t ok;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
            if (ok) return true;
        }
        if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
    }
}

template <class TY>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
               const GroupedParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    float* scales = reinterpret_cast<float*>(smem + kScaleOff);
    FewGroups groups(smem + kGroupOff, p.E);
    const uint32_t bars = base + kBarOff;
    auto full = [&](int i) { return bars + 8u * i; };
    auto empty = [&](int i) { return bars + 8u * (kStages + i); };
    auto t_full = [&](int i) { return bars + 8u * (2 * kStages + i); };
    auto t_empty = [&](int i) { return bars + 8u * (2 * kStages + kBufs + i); };
    auto s_full = [&](int i) { return bars + 8u * (2 * kStages + 2 * kBufs + i); };
    auto s_empty = [&](int i) { return bars + 8u * (2 * kStages + 2 * kBufs + kSets + i); };
    const uint32_t done = bars + 8u * (kBars - 3), p_full = bars + 8u * (kBars - 2), p_empty = bars + 8u * (kBars - 1);
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kBarOff + 8 * kBars);

    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int split = (int)gridDim.x, rank = (int)blockIdx.x;

    if (threadIdx.x == 64) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(t_full(i), 1);
            mbar_init(t_empty(i), 8);
        }
        for (int i = 0; i < kSets; ++i) {
            mbar_init(s_full(i), 64);
            mbar_init(s_empty(i), 8);
        }
        mbar_init(done, 1);
        mbar_init(p_full, split);
        mbar_init(p_empty, split);
        fence_mbar_init();
        prefetch_tmap(&map_w);
        prefetch_tmap(&map_a);
    }
    if (warp == 1) tmem_alloc(smem_addr(slot), 512);
    pdl_wait();
    pdl_trigger();
    if (warp == 0) groups.build(p.offsets, p.M, (p.N + 127) / 128, p.err);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (split > 1) {  // the other CTAs' barriers are there
        cluster_sync();
    }
    const uint32_t tmem = *slot;
    const long long tiles = groups.first[p.E];
    FewGroups::Tile g{};
    // This CTA's jobs: tiles of its own, all of K, as long as there are enough for all
    // CTAs, then shares of the rest, one tile per cluster at a time.
    const long long ctas = (long long)split * gridDim.y, own = blockIdx.y * (long long)split + rank;
    const long long whole = quotient(split > 1 ? tiles : tiles + ctas - 1 - own, ctas);
    int b0 = 0, b1 = p.KB;
    auto job = [&](long long i) {
        long long t = i * ctas + own;
        if (i >= whole) {
            t = split > 1 ? whole * ctas + (i - whole) * gridDim.y + blockIdx.y : tiles;
            b0 = (int)((long long)p.KB * rank / split);
            b1 = (int)((long long)p.KB * (rank + 1) / split);
        }
        if (t >= tiles) return false;
        groups.find(t, (p.N + 127) / 128, g);
        return true;
    };

    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            bool ok = true;
            for (long long t = 0; ok && job(t); ++t) {
                const int parts = (g.rows + 15) / 16;
                for (int b = b0; b < b1; ++b, ++i) {
                    const int st = i % kStages;
                    if (i >= kStages && !bar_wait(empty(st), ((i / kStages) & 1) ^ 1)) {
                        report_error(p.err, DEVERR_TC_WAIT);
                        ok = false;
                        break;
                    }
                    const uint32_t sb = base + st * kStage;
                    mbar_arrive_expect_tx(full(st), 16384 + parts * 2048);
                    tma_load_3d(sb, &map_w, b * 128, g.n_tile * 128, g.e, full(st));
                    for (int j = 0; j < parts; ++j)
                        tma_load_2d(sb + 16384 + j * 2048, &map_a, b * 128, g.m0 + j * 16, full(st));
                }
            }
            for (int j = max(0, i - kStages); j < i; ++j)
                if (!bar_wait(full(j % kStages), (j / kStages) & 1)) report_error(p.err, DEVERR_WAIT_DRAIN);
        }
    } else if (warp == 1) {
        const uint64_t dw = sw128_desc(base), da = sw128_desc(base + 16384);
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
        int st = 0, tb = 0;
        uint32_t ph = 0, tph = 0;
        bool ok = true, any = false;
        for (long long t = 0; ok && job(t); ++t) {
            const uint32_t desc = f8_idesc(128, (g.rows + 15) / 16 * 16);
            for (int b = b0; b < b1; ++b) {
                any = true;
                if (!warp_bar_wait(full(st), ph) || !warp_bar_wait(t_empty(tb), tph ^ 1)) {
                    if (lane == 0) report_error(p.err, DEVERR_TC_WAIT);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t w = dw + (uint64_t)(st * (kStage >> 4)), a = da + (uint64_t)(st * (kStage >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f8(tm + tb * kBN, w + 2 * k, a + 2 * k, desc, k > 0);
                    tc_commit(empty(st));
                    tc_commit(t_full(tb));
                }
                __syncwarp();
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
                if (++tb == kBufs) {
                    tb = 0;
                    tph ^= 1;
                }
            }
        }
        if (any) {
            if (elect_one()) tc_commit(done);
            __syncwarp();
            if (!warp_bar_wait(done, 0) && lane == 0) report_error(p.err, DEVERR_WAIT_DRAIN);
        }
    } else if (warp < 4) {
        const int tid = threadIdx.x - 64;
        int set = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (long long t = 0; ok && job(t); ++t) {
            const float* sw = p.sw + ((long long)g.e * ((p.N + 127) / 128) + g.n_tile) * p.KB;
            for (int b = b0; b < b1; b += kSetBlocks) {
                if (!warp_bar_wait(s_empty(set), ph ^ 1)) {
                    if (lane == 0) report_error(p.err, DEVERR_TC_WAIT);
                    ok = false;
                    break;
                }
                load_scales<kBN, 8>(scales + set * (kSetBlocks * kPitch), p, sw, nullptr, g.m0, g.rows, b, min(kSetBlocks, b1 - b), tid);
                mbar_arrive(s_full(set));
                if (++set == kSets) {
                    set = 0;
                    ph ^= 1;
                }
            }
        }
    } else {
        const int row = (warp & 3) * 32 + lane, own0 = (warp / 4 - 1) * kOwn;
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + own0;
        TY* y = static_cast<TY*>(p.y);
        int set = 0, tb = 0;
        uint32_t sph = 0, tph = 0, pph = 0;
        bool ok = true;  // false: the sums are lost; the barriers are still met
        auto lost = [&](unsigned code) {
            if (ok && lane == 0) report_error(p.err, code);
            ok = false;
        };
        for (long long t = 0; job(t); ++t) {
            float2 acc[kOwn / 2];
#pragma unroll
            for (int i = 0; i < kOwn / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            for (int i0 = b0; i0 < b1; i0 += kSetBlocks) {
                if (ok && !warp_bar_wait(s_full(set), sph)) lost(DEVERR_TC_WAIT);
                const int nk = min(kSetBlocks, b1 - i0);
                for (int b = 0; b < nk; ++b) {
                    if (ok && !warp_bar_wait(t_full(tb), tph)) lost(DEVERR_TC_WAIT);
                    tc_fence_after();
                    const float4* sc = reinterpret_cast<const float4*>(scales + (set * kSetBlocks + b) * kPitch + own0);
                    uint32_t r[2][16];
                    const bool low = own0 < g.rows, high = own0 + 16 < g.rows;
                    if (low) tmem_ld16_async(at + tb * kBN, r[0]);
                    if (high) tmem_ld16_async(at + tb * kBN + 16, r[1]);
                    tmem_wait16(r[0]);
                    tmem_wait16(r[1]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(t_empty(tb));
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (c ? !high : !low) continue;
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 s = sc[c * 4 + j / 4];
                            float2& a0 = acc[c * 8 + j / 2];
                            float2& a1 = acc[c * 8 + j / 2 + 1];
                            a0 = fma2(make_float2(__uint_as_float(r[c][j]), __uint_as_float(r[c][j + 1])),
                                      make_float2(s.x, s.y), a0);
                            a1 = fma2(make_float2(__uint_as_float(r[c][j + 2]), __uint_as_float(r[c][j + 3])),
                                      make_float2(s.z, s.w), a1);
                        }
                    }
                    if (++tb == kBufs) {
                        tb = 0;
                        tph ^= 1;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty(set));
                if (++set == kSets) {
                    set = 0;
                    sph ^= 1;
                }
            }
            const long long n = g.n_tile * 128LL + row;
            if (t < whole) {
                if (n < p.N) {
#pragma unroll
                    for (int c = 0; c < kOwn; ++c)
                        if (own0 + c < g.rows)
                            y[(g.m0 + own0 + c) * (long long)p.N + n] = from_f32<TY>(c & 1 ? acc[c / 2].y : acc[c / 2].x);
                }
                continue;
            }
            float* part = reinterpret_cast<float*>(smem + kPartOff);  // [row of a][row of w]
            if (t > whole && ok && !cluster_bar_wait(p_empty, pph ^ 1)) lost(DEVERR_TC_WAIT);
#pragma unroll
            for (int c = 0; c < kOwn; ++c)
                if (own0 + c < g.rows) part[(own0 + c) * 128 + row] = c & 1 ? acc[c / 2].y : acc[c / 2].x;
            named_bar_sync(1, kEpi);
            const int tid = threadIdx.x - 128;
            if (tid < split) arrive_in_cta(p_full, tid);
            if (ok && !cluster_bar_wait(p_full, pph)) lost(DEVERR_TC_WAIT);
            for (int e = rank * kEpi + tid; e < g.rows * 32; e += split * kEpi) {
                float4 v[8];  // all parts under way at once
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    v[r] = r < split ? ld_cluster(base + kPartOff + e * 16, r) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int r = 1; r < 8; ++r) {
                    v[0].x += v[r].x; v[0].y += v[r].y; v[0].z += v[r].z; v[0].w += v[r].w;
                }
                const float o[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
                const long long m = g.m0 + e / 32, col = g.n_tile * 128LL + e % 32 * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (col + i < p.N) y[m * p.N + col + i] = from_f32<TY>(o[i]);
            }
            named_bar_sync(1, kEpi);
            if (tid < split) arrive_in_cta(p_empty, tid);
            pph ^= 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (split > 1) {  // nobody reads this CTA's parts any more
        cluster_sync();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <class TY>
int room_of(const DevCtx& dc, const int** room) {
    return cluster_room<few_kernel<TY>>(dc, kThreads, smem_bytes(kMaxExperts), room);
}

template <class TY>
int launch(const DevCtx& dc, const GroupedArgs& a, int split, cudaStream_t s) {
    const int* room;
    int rc = room_of<TY>(dc, &room);
    CUtensorMap mw, ma;
    if (rc == QG_OK) rc = weight_map(&mw, a);
    if (rc == QG_OK) rc = code_map(&ma, a.a, a.M, a.K, 16);
    if (rc) return rc;
    const long long kb = (a.K + 127) / 128, most = (a.N + 127) / 128 * (std::min(a.M, a.E) + a.M / kBN);
    const GroupedParams p{a.sa, a.sw, a.offsets, a.y, (int)a.M, (int)a.E, (int)a.N, (int)kb, dc.err};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)split, (unsigned)std::min<long long>(most, room[split]));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(a.E);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = may_overlap() ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, few_kernel<TY>, mw, ma, p);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

}  // namespace

int plan_grouped_few(const DevCtx& dc, const GroupedArgs& a, FewPlan* plan) {
    const int* room;
    const int rc = a.y_dtype == QG_F32 ? room_of<float>(dc, &room) : room_of<__nv_bfloat16>(dc, &room);
    if (rc == QG_OK) *plan = few_plan(room, a.M, a.E, a.N, a.K);
    return rc;
}

int launch_grouped_few(const DevCtx& dc, const GroupedArgs& a, const FewPlan& plan, cudaStream_t s) {
    return a.y_dtype == QG_F32 ? launch<float>(dc, a, plan.split, s) : launch<__nv_bfloat16>(dc, a, plan.split, s);
}

int weight_map(CUtensorMap* m, const GroupedArgs& a) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    int rc = encoder(&encode);
    if (rc) return rc;
    const cuuint64_t dims[3] = {(cuuint64_t)a.K, (cuuint64_t)a.N, (cuuint64_t)a.E};
    const cuuint64_t strides[2] = {(cuuint64_t)a.K, (cuuint64_t)(a.K * a.N)};
    const cuuint32_t box[3] = {128, 128, 1}, es[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(a.w), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QG_OK
               : QG_ERR_UNSUPPORTED;
}

}  // namespace fp8
}  // namespace qg
