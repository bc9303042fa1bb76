// qmm_fp8_b128 for many rows of a: persistent pairs of CTAs over tiles of 256
// rows of a times 256 rows of w.
#include <algorithm>

#include "fp8_tc.cuh"

namespace qg {
namespace fp8 {
namespace {

// A tile's two SMs issue their MMAs as one (cta_group::2): each holds 128 rows of
// a, the sums of those rows, and half of the rows of w, which the other one
// reads from it. A k block is then 32 KB of shared memory written and read per
// SM; one SM alone would need 48 KB for the same products, and the 96 KB that
// pass through its shared memory took 850 of 1040 cycles per k block.
//
// The tensor cores take 512 cycles for a k block's 128 x 256 x 128 products, in
// which the two epilogue warpgroups bring the accumulator of the one before,
// which has two places in tensor memory, into registers: thread = row of a and
// 128 columns, which lie in one block of w's scales, so a k block enters the
// sum as fma(d, a_scale * w_scale, acc) with one factor per thread.
//
// The scales of 32 k blocks at a time come into shared memory by 4-byte
// asynchronous copies, the next 32 while these are used (read from global
// memory as they are needed, a column of a row-major array, they cost 29 us of
// 210 at M = 4096, N = 12288, K = 4096). Outputs leave through shared memory and
// TMA stores, which go on while the next tile is summed (32-byte stores of 32
// rows by each warp cost 33 us there).
//
// M = 4096, N = 12288, K = 4096, bf16 out, with the quantizer: 168 to 175 us, 2.36
// to 2.45 PFLOP/s, by the GPU: at the power limit (SM clock 1970 MHz). Alone a k block takes about 820 cycles instead of
// 512: the promotion.
//
//   warps 0-7  epilogue; 216 registers each (128 sums and two loads of 32
//              columns under way), which warps 8-11 give up
//   warp 8     TMA producer (32 KB per k block, five stages), whose copies
//              complete on the first CTA's barrier
//   warp 9     of the first CTA: MMA issuer for both
constexpr int kThreads = 384;
constexpr int kRegisters = 256 * 216 + 128 * 72;                 // what setmaxnreg hands out
constexpr int kBM = 128, kBN = 256;
constexpr int kStages = 5;
constexpr int kStage = (kBM + kBN / 2) * 128;                   // per CTA
constexpr int kScaleBlocks = 32;
constexpr int kScaleRow = kBM + 4;                              // floats per k block: a's 128 rows, w's 2 blocks
constexpr int kScaleSet = kScaleBlocks * kScaleRow * 4;
constexpr int kOutOff = kStages * kStage;                       // 4 KB per epilogue warp: 32 rows x 128 bytes
constexpr int kScaleOff = kOutOff + 8 * 4096;                   // two sets
constexpr int kBarOff = kScaleOff + 2 * kScaleSet;
constexpr int kSmem = 1024 + kBarOff + 256;
constexpr uint32_t kDesc = f8_idesc(2 * kBM, kBN);

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// The address of shared memory `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// A load into this CTA's shared memory that completes on a barrier of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(kDesc), "r"(acc)
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
// needed (one costs 1000 cycles here).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int c0, int c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
}

template <class TY>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ CUtensorMap map_y, const Params p) {
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
    const int mt = (p.M + 2 * kBM - 1) / (2 * kBM), nt = (p.N + kBN - 1) / kBN;
    const long long tiles = (long long)mt * nt;
    const int rank = (int)(blockIdx.x & 1);
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
        mbar_init(done, 1);
        fence_mbar_init();
        prefetch_tmap(&map_a);
        prefetch_tmap(&map_w);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers and tensor memory are there
    tc_fence_after();
    const uint32_t tmem = *slot;
    pdl_wait();
    pdl_trigger();

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8 && lane == 0) {
            int i = 0;
            bool ok = true;
            for (long long t = first; t < tiles && ok; t += step) {
                const int m0 = ((int)(t % mt) * 2 + rank) * kBM, n0 = (int)(t / mt) * kBN + rank * (kBN / 2);
                for (int b = 0; b < p.KB; ++b, ++i) {
                    const int st = i % kStages;
                    if (i >= kStages && !bar_wait(empty(st), ((i / kStages) & 1) ^ 1)) {
                        report_error(p.err, DEVERR_TC_WAIT);
                        ok = false;
                        break;
                    }
                    const uint32_t sb = base + st * kStage, bar = in_cta(full(st), 0);
                    if (rank == 0) mbar_arrive_expect_tx(full(st), 2 * kStage);  // both CTAs' bytes
                    tma_load_pair(sb, &map_a, b * 128, m0, bar);
                    tma_load_pair(sb + kBM * 128, &map_w, b * 128, n0, bar);
                }
            }
            // Both CTAs' copies are done when the first one's barrier says so; the
            // other CTA waits for that at the end, behind the cluster's barrier.
            for (int j = max(0, i - kStages); rank == 0 && j < i; ++j)
                if (!bar_wait(full(j % kStages), (j / kStages) & 1)) report_error(p.err, DEVERR_WAIT_DRAIN);
        } else if (warp == 9 && rank == 0) {
            const uint64_t da = sw128_desc(base), dw = sw128_desc(base + kBM * 128);
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            int st = 0, tb = 0;
            uint32_t ph = 0, tph = 0;
            bool ok = true;
            for (long long t = first; t < tiles && ok; t += step) {
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
                        for (int k = 0; k < 4; ++k) mma_pair(tm + tb * kBN, a + 2 * k, w + 2 * k, k > 0);
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
            if (elect_one()) commit_pair(done);
            __syncwarp();
            if (!warp_bar_wait(done, 0) && lane == 0) report_error(p.err, DEVERR_WAIT_DRAIN);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int half = warp / 4;
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 128;
        const uint32_t out = base + kOutOff + warp * 4096;
        const float* scales = reinterpret_cast<const float*>(smem + kScaleOff);
        // Starts the copies of a tile's scales of the k blocks from b0 into a
        // set: warp = 16 rows of a, lane = k block (a row's are consecutive).
        auto fetch = [&](long long t, int b0, int set) {
            if (t < tiles) {
                const int m0 = ((int)(t % mt) * 2 + rank) * kBM, n0 = (int)(t / mt) * kBN;
                const uint32_t dst = base + kScaleOff + set * kScaleSet + lane * (kScaleRow * 4);
                if (b0 + lane < p.KB) {
#pragma unroll
                    for (int i = 0; i < kBM / 8; ++i) {
                        const int row = warp * (kBM / 8) + i;
                        cp_async4(dst + row * 4, p.sa + (long long)min(m0 + row, p.M - 1) * p.KB + b0 + lane);
                    }
                    if (warp < 2)
                        cp_async4(dst + (kBM + warp) * 4,
                                  p.sw + (long long)min(n0 / 128 + warp, (p.N - 1) / 128) * p.KB + b0 + lane);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int set = 0, tb = 0;
        uint32_t tph = 0;
        bool ok = true;
        const uint32_t empty0 = in_cta(t_empty(0), 0);
        fetch(first, 0, 0);
        for (long long t = first; t < tiles; t += step) {
            const int row = (warp & 3) * 32 + lane;
            const int m0 = ((int)(t % mt) * 2 + rank) * kBM + (warp & 3) * 32, m = m0 + lane;
            const long long n0 = (t / mt) * kBN + half * 128;
            float2 acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
            for (int b0 = 0; b0 < p.KB; b0 += kScaleBlocks) {
                // The other set's last readers are past this barrier, this set's copies done.
                asm volatile("cp.async.wait_all;" ::: "memory");
                named_bar_sync(1, 256);
                const int nb = min(kScaleBlocks, p.KB - b0);
                const bool more = b0 + nb < p.KB;
                fetch(more ? t : t + step, more ? b0 + nb : 0, set ^ 1);
                const float* sp = scales + set * (kScaleSet / 4);
                set ^= 1;
                float sc = sp[row] * sp[kBM + half];
#pragma unroll 1
                for (int b = 0; b < nb; ++b) {
                    const float2 s = make_float2(sc, sc);
                    sp += b + 1 < nb ? kScaleRow : 0;
                    if (!mbar_try_wait(t_full(tb), tph) && ok && !bar_wait(t_full(tb), tph)) {
                        report_error(p.err, DEVERR_TC_WAIT);
                        ok = false;  // the sums are lost; the barriers are still met
                    }
                    __syncwarp();
                    tc_fence_after();
                    const uint32_t from = at + tb * kBN;
                    uint32_t r[2][32];
                    tmem_ld32_async(from, r[0]);
                    sc = sp[row] * sp[kBM + half];  // of the next block
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tmem_wait32(r[c & 1]);
                        if (c < 3) {
                            tmem_ld32_async(from + (c + 1) * 32, r[(c + 1) & 1]);
                        } else {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive_cluster(empty0 + 8u * tb);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            acc[c * 16 + j] = fma2(make_float2(__uint_as_float(r[c & 1][2 * j]),
                                                              __uint_as_float(r[c & 1][2 * j + 1])),
                                                  s, acc[c * 16 + j]);
                    }
                    tb ^= 1;
                    tph ^= tb == 0;
                }
            }
            if (p.vec) {
                constexpr int kPer = 128 / sizeof(TY);  // columns of a 128-byte row
#pragma unroll
                for (int c = 0; c < 128; c += kPer) {
                    // the buffer's last store has been read
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {  // 16-byte chunk q of the row, at q ^ (row % 8)
                        uint4 v;
                        if constexpr (sizeof(TY) == 4) {
                            const float2 a0 = acc[(c + q * 4) / 2], a1 = acc[(c + q * 4) / 2 + 1];
                            v = make_uint4(__float_as_uint(a0.x), __float_as_uint(a0.y), __float_as_uint(a1.x),
                                           __float_as_uint(a1.y));
                        } else {
                            const float2* a = acc + (c + q * 8) / 2;
                            v = make_uint4(pack2<TY>(a[0].x, a[0].y), pack2<TY>(a[1].x, a[1].y),
                                           pack2<TY>(a[2].x, a[2].y), pack2<TY>(a[3].x, a[3].y));
                        }
                        *reinterpret_cast<uint4*>(smem + (out - base) + lane * 128 + ((q ^ (lane & 7)) << 4)) = v;
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        if (m0 < p.M && n0 + c < p.N) tma_store_2d(&map_y, (int)n0 + c, m0, out);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                }
            } else if (m < p.M) {
                TY* y = static_cast<TY*>(p.y) + (long long)m * p.N + n0;
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if (n0 + c < p.N) y[c] = from_f32<TY>(c & 1 ? acc[c / 2].y : acc[c / 2].x);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA's memory is in use any more
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// y in boxes of 32 rows x 128 bytes.
template <class TY>
int out_map(CUtensorMap* m, const Fp8Args& a) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    int rc = encoder(&encode);
    if (rc) return rc;
    const cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.M};
    const cuuint64_t strides[1] = {(cuuint64_t)a.N * sizeof(TY)};
    const cuuint32_t box[2] = {128 / sizeof(TY), 32}, es[2] = {1, 1};
    return encode(m, sizeof(TY) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.y, dims,
                  strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QG_OK
               : QG_ERR_UNSUPPORTED;
}

template <class TY>
int launch(const DevCtx& dc, const Fp8Args& a, cudaStream_t s) {
    static int configured[64] = {0};
    auto kern = tile_kernel<TY>;
    if (!configured[dc.device]) {
        // Were the kernel launched with fewer registers than it hands out, the
        // increase would wait for ever.
        cudaFuncAttributes at{};
        cudaError_t e = cudaFuncGetAttributes(&at, kern);
        if (e != cudaSuccess) return cuda_fail(e);
        if (at.numRegs * kThreads < kRegisters) return QG_ERR_UNSUPPORTED;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return cuda_fail(e);
        configured[dc.device] = 1;
    }
    CUtensorMap ma, mw, my = {};
    int rc = code_map(&ma, a.a, a.M, a.K, kBM);
    if (rc == QG_OK) rc = code_map(&mw, a.w, a.N, a.K, kBN / 2);
    // TMA stores want rows of y on 16-byte boundaries
    const bool vec = reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && a.N * sizeof(TY) % 16 == 0;
    if (rc == QG_OK && vec) rc = out_map<TY>(&my, a);
    if (rc) return rc;
    const Params p{a.sa, a.sw, a.y, (int)a.M, (int)a.N, (int)((a.K + 127) / 128), vec, dc.err};
    const long long tiles = ((a.M + 2 * kBM - 1) / (2 * kBM)) * ((a.N + kBN - 1) / kBN);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * (unsigned)std::min<long long>(tiles, dc.num_sms / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = may_overlap() ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, ma, mw, my, p);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

}  // namespace

int launch_tile(const DevCtx& dc, const Fp8Args& a, cudaStream_t s) {
    return a.y_dtype == QG_F32 ? launch<float>(dc, a, s) : launch<__nv_bfloat16>(dc, a, s);
}

}  // namespace fp8
}  // namespace qg
