// qmm_fp8_b128_grouped for experts of many rows: persistent pairs of CTAs over
// tiles of 256 rows of a weight times up to 256 rows of one expert.
#include <algorithm>

#include "fp8_groups.cuh"

namespace qg {
namespace fp8 {
namespace {

// As in fp8_tile.cu a pair of SMs issues its MMAs as one (cta_group::2), each with
// half of both operands in its shared memory, and two epilogue warpgroups bring
// the accumulator of the k block before into registers meanwhile. But w is on the M
// side here: the rows of a, of which an expert has any number, are the
// instruction's N, which comes in steps of 32. A chunk of 140 rows takes 160 / 256
// of a whole one's time; tiles of 256 rows of a would take all of it.
//
// A thread of the epilogue has one row of w, so its 128 columns have a scale each:
// they come from shared memory (all lanes of a warp read the same 16 bytes), with
// w's, the same for all 128 rows of w that a CTA has, multiplied in.
//
//   warps 0-7    epilogue; 216 registers each, which warps 8-11 give up
//   warp 8       TMA producer, whose copies complete on the first CTA's barrier
//   warp 9       of the first CTA: MMA issuer for both
//   warps 10-11  scales
constexpr int kThreads = 384;
constexpr int kRegisters = 256 * 216 + 128 * 72;  // what setmaxnreg hands out
constexpr int kBM = 128, kBN = 256;               // rows of w per CTA, rows of a per pair
constexpr int kStep = 32;
constexpr int kStages = 5;
constexpr int kStage = (kBM + kBN / 2) * 128;     // per CTA
constexpr int kScaleOff = kStages * kStage;
constexpr int kBarOff = kScaleOff + kSets * kSetBlocks * kBN * 4;
constexpr int kBars = 2 * kStages + 4 + 2 * kSets + 1;
constexpr int kGroupOff = kBarOff + 8 * kBars + 8;
using TileGroups = Groups<kBN, kStep>;
constexpr int smem_bytes(long long E) { return 1024 + kGroupOff + TileGroups::bytes(E); }
static_assert(smem_bytes(kMaxExperts) <= 227 * 1024, "shared memory");
static_assert(kGroupOff % 8 == 0, "tile numbers are 8 bytes");

// The address of shared memory `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Loads into this CTA's shared memory that complete on a barrier of the pair.
__device__ __forceinline__ void load_a_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void load_w_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"(acc)
        : "memory");
}
// Arrives on the barrier at this place in both CTAs when the MMAs so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// Arrives on a barrier of the pair. What the arrival orders is reads of tensor
// memory, complete and behind a tcgen05 fence: no release over the cluster is
// needed.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <class TY>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_tile_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                        const GroupedParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    float* scales = reinterpret_cast<float*>(smem + kScaleOff);
    TileGroups groups(smem + kGroupOff, p.E);
    const uint32_t bars = base + kBarOff;
    auto full = [&](int i) { return bars + 8u * i; };
    auto empty = [&](int i) { return bars + 8u * (kStages + i); };
    auto t_full = [&](int i) { return bars + 8u * (2 * kStages + i); };
    auto t_empty = [&](int i) { return bars + 8u * (2 * kStages + 2 + i); };
    auto s_full = [&](int i) { return bars + 8u * (2 * kStages + 4 + i); };
    auto s_empty = [&](int i) { return bars + 8u * (2 * kStages + 4 + kSets + i); };
    const uint32_t done = bars + 8u * (kBars - 1);
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kBarOff + 8 * kBars);
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x & 1), nt128 = (p.N + 127) / 128;
    const long long first = blockIdx.x >> 1, step = gridDim.x >> 1;  // this pair's tiles

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(t_full(i), 1);
            mbar_init(t_empty(i), 16);  // of the first CTA: both CTAs' epilogue warps
        }
        for (int i = 0; i < kSets; ++i) {
            mbar_init(s_full(i), 64);
            mbar_init(s_empty(i), 8);
        }
        mbar_init(done, 1);
        fence_mbar_init();
        prefetch_tmap(&map_w);
        prefetch_tmap(&map_a);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();
    if (warp == 8) groups.build(p.offsets, p.M, (p.N + 2 * kBM - 1) / (2 * kBM), p.err);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers and tensor memory are there
    tc_fence_after();
    const uint32_t tmem = *slot;
    const long long tiles = groups.first[p.E];

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8 && lane == 0) {
            int i = 0;
            bool ok = true;
            for (long long t = first; t < tiles && ok; t += step) {
                const TileGroups::Tile g = groups.find(t);
                const int half = (g.rows + kStep - 1) / kStep * (kStep / 2);  // of the columns: each CTA holds its own
                const int boxes = (half + 31) / 32, bytes = 2 * (kBM * 128 + boxes * 4096);  // both CTAs'
                const int n0 = (2 * g.n_tile + rank) * kBM, m0 = g.m0 + rank * half;
                for (int b = 0; b < p.KB; ++b, ++i) {
                    const int st = i % kStages;
                    if (i >= kStages && !bar_wait(empty(st), ((i / kStages) & 1) ^ 1)) {
                        report_error(p.err, DEVERR_TC_WAIT);
                        ok = false;
                        break;
                    }
                    const uint32_t sb = base + st * kStage, bar = in_cta(full(st), 0);
                    if (rank == 0) mbar_arrive_expect_tx(full(st), bytes);
                    load_w_pair(sb, &map_w, b * 128, n0, g.e, bar);
                    for (int j = 0; j < boxes; ++j) load_a_pair(sb + kBM * 128 + j * 4096, &map_a, b * 128, m0 + j * 32, bar);
                }
            }
            // Both CTAs' copies are done when the first one's barrier says so; the
            // other CTA waits for that at the end, behind the cluster's barrier.
            for (int j = max(0, i - kStages); rank == 0 && j < i; ++j)
                if (!bar_wait(full(j % kStages), (j / kStages) & 1)) report_error(p.err, DEVERR_WAIT_DRAIN);
        } else if (warp == 9 && rank == 0) {
            const uint64_t dw = sw128_desc(base), da = sw128_desc(base + kBM * 128);
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            int st = 0, tb = 0;
            uint32_t ph = 0, tph = 0;
            bool ok = true;
            for (long long t = first; t < tiles && ok; t += step) {
                const uint32_t desc = f8_idesc(2 * kBM, (groups.find(t).rows + kStep - 1) / kStep * kStep);
                for (int b = 0; b < p.KB; ++b) {
                    if (!warp_bar_wait(full(st), ph) || !warp_bar_wait(t_empty(tb), tph ^ 1)) {
                        if (lane == 0) report_error(p.err, DEVERR_TC_WAIT);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t w = dw + (uint64_t)(st * (kStage >> 4)), a = da + (uint64_t)(st * (kStage >> 4));
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_pair(tm + tb * kBN, w + 2 * k, a + 2 * k, desc, k > 0);
                        commit_pair(empty(st));
                        commit_pair(t_full(tb));
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
            if (first < tiles) {
                if (elect_one()) commit_pair(done);
                __syncwarp();
                if (!warp_bar_wait(done, 0) && lane == 0) report_error(p.err, DEVERR_WAIT_DRAIN);
            }
        } else if (warp >= 10) {
            const int tid = threadIdx.x - 320;
            int set = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (long long t = first; t < tiles && ok; t += step) {
                const TileGroups::Tile g = groups.find(t);
                // a second CTA without rows of w of its own: any scales that are there
                const float* sw = p.sw + ((long long)g.e * nt128 + min(2 * g.n_tile + rank, nt128 - 1)) * p.KB;
                for (int b = 0; b < p.KB; b += kSetBlocks) {
                    if (!warp_bar_wait(s_empty(set), ph ^ 1)) {
                        if (lane == 0) report_error(p.err, DEVERR_TC_WAIT);
                        ok = false;
                        break;
                    }
                    load_scales<kBN>(scales + set * (kSetBlocks * kBN), p, sw, g.m0, g.rows, b, min(kSetBlocks, p.KB - b), tid);
                    mbar_arrive(s_full(set));
                    if (++set == kSets) {
                        set = 0;
                        ph ^= 1;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t empty0 = in_cta(t_empty(0), 0);
        TY* y = static_cast<TY*>(p.y);
        int set = 0, tb = 0;
        uint32_t sph = 0, tph = 0;
        bool ok = true;  // false: the sums are lost; the barriers are still met
        auto lost = [&] {
            if (ok && lane == 0) report_error(p.err, DEVERR_TC_WAIT);
            ok = false;
        };
        for (long long t = first; t < tiles; t += step) {
            const TileGroups::Tile g = groups.find(t);
            const int half = (g.rows + kStep - 1) / kStep * (kStep / 2);  // columns of a warpgroup, a multiple of 16
            const int own0 = warp / 4 * half;
            float2 acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
            for (int b0 = 0; b0 < p.KB; b0 += kSetBlocks) {
                if (ok && !warp_bar_wait(s_full(set), sph)) lost();
                const int nk = min(kSetBlocks, p.KB - b0);
                const float* sp = scales + set * (kSetBlocks * kBN) + own0;
#pragma unroll 1
                for (int b = 0; b < nk; ++b, sp += kBN) {
                    if (!mbar_try_wait(t_full(tb), tph) && ok && !bar_wait(t_full(tb), tph)) lost();
                    __syncwarp();
                    tc_fence_after();
                    const uint32_t from = lanes + tb * kBN + own0;
                    uint32_t r[2][16];
                    tmem_ld16_async(from, r[0]);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if (c * 16 >= half) break;
                        tmem_wait16(r[c & 1]);
                        if (c < 7 && (c + 1) * 16 < half) tmem_ld16_async(from + (c + 1) * 16, r[(c + 1) & 1]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 s = *reinterpret_cast<const float4*>(sp + c * 16 + j * 4);
                            float2& a0 = acc[c * 8 + j * 2];
                            float2& a1 = acc[c * 8 + j * 2 + 1];
                            a0 = fma2(make_float2(__uint_as_float(r[c & 1][4 * j]), __uint_as_float(r[c & 1][4 * j + 1])),
                                      make_float2(s.x, s.y), a0);
                            a1 = fma2(make_float2(__uint_as_float(r[c & 1][4 * j + 2]), __uint_as_float(r[c & 1][4 * j + 3])),
                                      make_float2(s.z, s.w), a1);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_cluster(empty0 + 8u * tb);
                    tb ^= 1;
                    tph ^= tb == 0;
                }
                if (lane == 0) mbar_arrive(s_empty(set));
                if (++set == kSets) {
                    set = 0;
                    sph ^= 1;
                }
            }
            const long long n = (2LL * g.n_tile + rank) * kBM + row;
            const int mine = min(half, g.rows - own0);  // of the second warpgroup: maybe none
            if (n < p.N) {
                TY* out = y + (long long)(g.m0 + own0) * p.N + n;
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if (c < mine) out[(long long)c * p.N] = from_f32<TY>(c & 1 ? acc[c / 2].y : acc[c / 2].x);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA's memory is in use any more
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <class TY>
int launch(const DevCtx& dc, const GroupedArgs& a, cudaStream_t s) {
    static int configured[64] = {0};
    auto kern = grouped_tile_kernel<TY>;
    if (!configured[dc.device]) {
        // Were the kernel launched with fewer registers than it hands out, the
        // increase would wait for ever.
        cudaFuncAttributes at{};
        cudaError_t e = cudaFuncGetAttributes(&at, kern);
        if (e != cudaSuccess) return cuda_fail(e);
        if (at.numRegs * kThreads < kRegisters) return QG_ERR_UNSUPPORTED;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kMaxExperts));
        if (e != cudaSuccess) return cuda_fail(e);
        configured[dc.device] = 1;
    }
    CUtensorMap mw, ma;
    int rc = weight_map(&mw, a);
    if (rc == QG_OK) rc = code_map(&ma, a.a, a.M, a.K, 32);
    if (rc) return rc;
    const GroupedParams p{a.sa, a.sw, a.offsets, a.y, (int)a.M, (int)a.E, (int)a.N, (int)((a.K + 127) / 128), dc.err};
    const long long tiles = (a.N + 2 * kBM - 1) / (2 * kBM) * (std::min(a.M, a.E) + a.M / kBN);  // at most
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * (unsigned)std::min<long long>(tiles, dc.num_sms / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(a.E);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = may_overlap() ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mw, ma, p);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

}  // namespace

int launch_grouped_tile(const DevCtx& dc, const GroupedArgs& a, cudaStream_t s) {
    return a.y_dtype == QG_F32 ? launch<float>(dc, a, s) : launch<__nv_bfloat16>(dc, a, s);
}

}  // namespace fp8
}  // namespace qg
