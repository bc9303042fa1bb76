// attn_paged for few rows per key head (single tokens, short drafts): bound by
// the bytes of the cache.
#include <algorithm>

#include "attn_join.cuh"

namespace qg {
namespace attn {
namespace {

// One CTA per SM streams its steps' keys and values, 64 keys at a time, with
// TMA through a ring that runs ahead across segments, so that the loads never
// pause; four warps keep up with warp-level 16 x 8 x 16 products (at most 64
// rows meet each key: the tensor cores' large tiles would be empty, and the
// products take a fraction of the time that the bytes need).
//
// RB: blocks of 16 rows, 1, 2 or 4. Warp w has row block w % RB and the
// 64 / (4 / RB) keys w / RB of each step; warps with the same rows and other
// keys keep their own softmax and meet at the end of the segment.
//
// Probabilities enter the product with V in 16 bits. HALF, for at most 8 rows:
// a product's rows 8-15 then hold what the rounding took off rows 0-7, and the two
// sums are added at the end, so outputs are as exact as with f32 probabilities
// at no cost (half the exponentials, in fact: 327.5 us for 128 single tokens
// without, 340 with a cap and 315). With more rows the remainders would be products
// of their own, 16 % of the time for 32 rows (428 and 498 us): outputs are off by 1.2
// to 1.4 times what their own rounding alone is instead.
//
// With the joining kernel: 128 single tokens over 65 to 8192 keys, 32/8 heads of
// 128: 325 us, 6.68 TB/s; one token over 700 keys: 7.5 us, most of it the
// latency of finding the step, its page and its keys, and of a second launch.
constexpr int kKT = 64;
constexpr int kWarps = 4;
constexpr int kThreads = (kWarps + 1) * 32;

template <int D>
struct Geo {
    static constexpr int kHalf = kKT * 128;                    // 64 columns of 64 keys
    static constexpr int kTile = kHalf * (D / 64);             // k or v of a step
    static constexpr int kStage = 2 * kTile;
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kMergeOff = kStages * kStage;         // [4][16][D] f32
    static constexpr int kMlOff = kMergeOff + 64 * D * 4;      // [4][16] float2
    static constexpr int kBarOff = kMlOff + 64 * 8;
    static constexpr int kScratchOff = kBarOff + 16 * kStages;
    static constexpr int kSmem = 1024 + kScratchOff + 128;
};

__device__ __forceinline__ void ldsm(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void ldsm_t(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
template <class T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same_v<T, __half>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of a 16-byte chunk of key `row` in a tile of 128-byte-swizzled
// halves of 64 columns.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    return (uint32_t)((chunk >> 3) * Geo<D>::kHalf + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

template <class T, int D, int RB, bool HALF, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const Work w) {
    using G = Geo<D>;
    constexpr int RT = 16 * RB, KS = kWarps / RB, KW = kKT / KS;  // keys of a step per warp
    constexpr int NT = D / 8;                                     // 8-column tiles of the output
    constexpr int RH = HALF ? 1 : 2;                              // rows g, g + 8 of a lane
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const uint32_t bars = base + G::kBarOff;
    auto full = [&](int i) { return bars + 8u * i; };
    auto empty = [&](int i) { return bars + 8u * (G::kStages + i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < G::kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), kWarps);
        }
        fence_mbar_init();
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    Cuts cuts;
    Place place;
    Seq seq;
    if (threadIdx.x == 0) w.notes[blockIdx.x].from = -1, w.notes[blockIdx.x].bad = 0;
    if (!locate<RT, kKT, kThreads>(w, blockIdx.x, &cuts, &place, &seq, reinterpret_cast<long long*>(smem + G::kScratchOff)))
        return;
    const long long n = cuts(blockIdx.x + 1) - cuts(blockIdx.x);
    if (threadIdx.x == 0) note_start(w, place, n);
    Walk<RT, kKT> walk(w, place, seq, n);

    if (warp == kWarps) {
        // ------------------------------------------------------------ producer
        const int rows = min(w.a.page_size, kKT);  // keys per copy
        int i = 0;
        bool ok = true;
        while (ok && walk.next()) {
            for (int t = walk.lo; t < walk.hi; ++t, ++i) {
                const int st = i % G::kStages;
                if (i >= G::kStages && !warp_bar_wait(empty(st), ((i / G::kStages) & 1) ^ 1)) {
                    if (lane == 0) report_error(w.err, DEVERR_TC_WAIT);
                    ok = false;
                    break;
                }
                const int keys = max(0, min(kKT, walk.span.end - t * kKT));
                const int copies = (keys + rows - 1) / rows;
                if (lane == 0) mbar_arrive_expect_tx(full(st), (uint32_t)(copies * rows * D * 2 * 2));
                __syncwarp();
                if (lane < copies) {
                    const int j = t * kKT + lane * rows;
                    const int page = page_from(w, walk.p.b, j, rows, walk.span.begin);
                    const int y = walk.p.head * w.a.page_size + j % w.a.page_size;
                    const uint32_t dst = base + st * G::kStage + lane * rows * 128;
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        tma_load_3d(dst + h * G::kHalf, &map_k, h * 64, y, page, full(st));
                        tma_load_3d(dst + G::kTile + h * G::kHalf, &map_v, h * 64, y, page, full(st));
                    }
                }
            }
        }
        for (int j = max(0, i - G::kStages); j < i; ++j)
            if (!warp_bar_wait(full(j % G::kStages), (j / G::kStages) & 1) && lane == 0)
                report_error(w.err, DEVERR_WAIT_DRAIN);
        return;
    }

    // ---------------------------------------------------------------- compute
    const int rb = warp % RB, wk = warp / RB;
    const int g = lane >> 2, c2 = (lane & 3) * 2;
    float* merge = reinterpret_cast<float*>(smem + G::kMergeOff);
    float2* mls = reinterpret_cast<float2*>(smem + G::kMlOff);
    int i = 0;
    bool ok = true;
    while (walk.next()) {
        const int r0 = walk.p.tile * RT;
        const Seq s = walk.s;
        // Q as the products' left operand: rows g and g + 8 of this warp's block.
        uint32_t q[D / 16][4];
        int pos[RH];
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            const int r = r0 + rb * 16 + g + 8 * h;
            const int tok = min(r, s.rows - 1) / w.group;
            pos[h] = s.ctx - s.n + tok;
            const uint32_t* qp = reinterpret_cast<const uint32_t*>(
                static_cast<const T*>(w.a.q) + (long long)(s.first + tok) * w.a.q_stride +
                (long long)(walk.p.head * w.group + min(r, s.rows - 1) % w.group) * D + c2);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                q[k][h] = __ldg(qp + k * 8);
                q[k][2 + h] = __ldg(qp + k * 8 + 4);
                if (HALF) q[k][1] = q[k][3] = 0;
            }
        }
        const int pos_lo = s.ctx - s.n + r0 / w.group;  // of the tile's rows
        const int pos_hi = walk.span.end - 1;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][e] = 0.f;

        for (int t = walk.lo; t < walk.hi; ++t, ++i) {
            const int st = i % G::kStages;
            // After a wait that gave up the error word is set and the results
            // are lost, but every barrier below is still met.
            if (ok && !warp_bar_wait(full(st), (i / G::kStages) & 1)) {
                if (lane == 0) report_error(w.err, DEVERR_TC_WAIT);
                ok = false;
            }
            const uint32_t kt = base + st * G::kStage, vt = kt + G::kTile;
            const int j0 = t * kKT + wk * KW;  // this warp's first key
            float x[KW / 8][4];
#pragma unroll
            for (int nb = 0; nb < KW / 16; ++nb) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[2 * nb][e] = x[2 * nb + 1][e] = 0.f;
                const int row = wk * KW + nb * 16 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t b[4];
                    ldsm(kt + chunk_at<D>(row, k * 2 + ((lane >> 3) & 1)), b);
                    mma<T>(x[2 * nb], q[k], b[0], b[1]);
                    mma<T>(x[2 * nb + 1], q[k], b[2], b[3]);
                }
            }
            constexpr int E = 2 * RH;  // a lane's scores of 8 keys
            scores<CAP, KW / 8 * E>(w, [&](int e) { return x[e / E][e % E]; }, [&](int e, float v) { x[e / E][e % E] = v; });
            const bool masked = j0 + KW - 1 > pos_lo || (w.a.window && j0 <= pos_hi - w.a.window);
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int nt = 0; nt < KW / 8; ++nt)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float v = x[nt][e];
                    if (masked) {
                        const int j = j0 + nt * 8 + c2 + (e & 1), p = pos[e >> 1];
                        if (j > p || (w.a.window && j <= p - w.a.window)) v = -INFINITY;
                    }
                    x[nt][e] = v;
                    top[e >> 1] = fmaxf(top[e >> 1], v);
                }
            float keep[2], ref[2];
#pragma unroll
            for (int h = 0; h < RH; ++h) {
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], 1));
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], 2));
                const float mn = fmaxf(m[h], top[h]);
                ref[h] = mn == -INFINITY ? 0.f : mn;  // a row that has seen nothing yet
                keep[h] = ex2(m[h] - ref[h]);
                m[h] = mn;
                l[h] *= keep[h];
            }
            if (HALF) keep[1] = keep[0];
            if (__any_sync(0xFFFFFFFFu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][e] *= keep[e >> 1];
            }
            const int from = walk.span.begin - j0, valid = walk.span.end - j0;  // keys of this warp that any row sees
#pragma unroll
            for (int nb = 0; nb < KW / 16; ++nb) {
                uint32_t pa[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float* v = x[2 * nb + h];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        v[e] = ex2(v[e] - ref[e >> 1]);
                        l[e >> 1] += v[e];
                    }
                    pa[2 * h] = pack2<T>(v[0], v[1]);
                    if constexpr (HALF) {  // the remainders
                        const float2 r = unpack2<T>(pa[2 * h]);
                        v[2] = v[0] - r.x;
                        v[3] = v[1] - r.y;
                    }
                    pa[2 * h + 1] = pack2<T>(v[2], v[3]);
                }
                // Places that no row sees may hold anything, NaN included.
                uint32_t mask[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                const bool edge = valid < nb * 16 + 16 || from > nb * 16;
                if (edge) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int k = nb * 16 + h * 8 + c2;
                        mask[h] = (k >= from && k < valid ? 0xFFFFu : 0u) |
                                  (k + 1 >= from && k + 1 < valid ? 0xFFFF0000u : 0u);
                    }
                }
                const int row = wk * KW + nb * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
                for (int nt = 0; nt < NT; nt += 2) {
                    uint32_t b[4];
                    ldsm_t(vt + chunk_at<D>(row, nt + (lane >> 4)), b);
                    if (edge) {
                        b[0] &= mask[0];
                        b[1] &= mask[1];
                        b[2] &= mask[0];
                        b[3] &= mask[1];
                    }
                    mma<T>(o[nt], pa, b[0], b[1]);
                    mma<T>(o[nt + 1], pa, b[2], b[3]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(st));
        }

        // --------------------------------------------------- end of a segment
        if constexpr (HALF) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // (an infinite value stays one: with a remainder of 0 or less it would be NaN)
#pragma unroll
                for (int e = 0; e < 2; ++e) o[nt][e] += isinf(o[nt][e]) ? 0.f : o[nt][2 + e];
            }
        }
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
            l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
        }
        if ((lane & 3) == 0) {
            mls[warp * 16 + g] = make_float2(m[0], l[0]);
            if (!HALF) mls[warp * 16 + g + 8] = make_float2(m[1], l[1]);
        }
        float* mine = merge + warp * 16 * D;
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            // 8-float groups rotate by the row, so that a warp's stores spread over the banks
            const int r = g + 8 * h;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                *reinterpret_cast<float2*>(mine + r * D + ((nt + r) % NT) * 8 + c2) =
                    make_float2(o[nt][2 * h], o[nt][2 * h + 1]);
        }
        named_bar_sync(1, kWarps * 32);
        constexpr int kVec = 8;  // columns per thread
        for (int e = threadIdx.x; e < RT * (D / kVec); e += kWarps * 32) {
            const int r = e / (D / kVec), nt = e % (D / kVec);
            if (r0 + r >= s.rows) continue;
            const int rw = r / 16, rr = r % 16;
            float mm = -INFINITY, ll = 0.f, v[kVec] = {};
#pragma unroll
            for (int k = 0; k < KS; ++k) mm = fmaxf(mm, mls[(k * RB + rw) * 16 + rr].x);
            const float rf = mm == -INFINITY ? 0.f : mm;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const float2 p = mls[(k * RB + rw) * 16 + rr];
                const float f = ex2(p.x - rf);
                ll += p.y * f;
                const float4* src = reinterpret_cast<const float4*>(
                    merge + ((k * RB + rw) * 16 + rr) * D + ((nt + rr) % NT) * 8);
                const float4 a = src[0], b = src[1];
                v[0] += a.x * f; v[1] += a.y * f; v[2] += a.z * f; v[3] += a.w * f;
                v[4] += b.x * f; v[5] += b.y * f; v[6] += b.z * f; v[7] += b.w * f;
            }
            if (walk.whole) {
                const float inv = ll == 0.f ? 0.f : 1.f / ll;  // NaN stays NaN
                const int tok = s.first + (r0 + r) / w.group, head = walk.p.head * w.group + (r0 + r) % w.group;
                const long long at = (long long)tok * w.a.hq + head;
                uint4 u;
                u.x = pack2<T>(v[0] * inv, v[1] * inv);
                u.y = pack2<T>(v[2] * inv, v[3] * inv);
                u.z = pack2<T>(v[4] * inv, v[5] * inv);
                u.w = pack2<T>(v[6] * inv, v[7] * inv);
                *reinterpret_cast<uint4*>(static_cast<T*>(w.a.out) + at * D + nt * 8) = u;
                if (ll == ll && !all_finite(v)) w.notes[blockIdx.x].bad = 1;
                if (w.a.lse && nt == 0)
                    w.a.lse[at] = ll == 0.f ? -INFINITY : fmaf(mm, w.to_ln, logf(ll));
            } else {
                const long long at = ((long long)blockIdx.x * 2 + walk.slot) * RT + r;
                float4* dst = reinterpret_cast<float4*>(w.part + at * D + nt * 8);
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                if (nt == 0) w.ml[at] = make_float2(mm, ll);
            }
        }
        if (threadIdx.x == 0) walk.note(cuts, RT, blockIdx.x);
        named_bar_sync(1, kWarps * 32);  // the buffers are free again
    }
}

template <class T, int D, int RB, bool HALF, bool CAP>
int launch_one(const DevCtx& dc, const Work& w, cudaStream_t s) {
    static std::atomic<int> configured[64];  // set by any thread, all to the same
    auto kern = few_kernel<T, D, RB, HALF, CAP>;
    if (!configured[dc.device]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kSmem);
        if (e != cudaSuccess) return cuda_fail(e);
        configured[dc.device] = 1;
    }
    CUtensorMap mk, mv;
    const int rows = std::min(w.a.page_size, kKT);
    int rc = cache_map(&mk, w.a, w.a.k, rows);
    if (rc == QG_OK) rc = cache_map(&mv, w.a, w.a.v, rows);
    if (rc == QG_OK) rc = launch(may_overlap(), kern, dim3(w.ctas), kThreads, Geo<D>::kSmem, s, mk, mv, w);
    if (rc) return rc;
    return launch_join<T, D, 16 * RB, kKT, 1, 12>(w, s);
}

template <class T, int D, int RB, bool HALF = false>
int launch_cap(const DevCtx& dc, const Work& w, cudaStream_t s) {
    return w.a.softcap > 0.f ? launch_one<T, D, RB, HALF, true>(dc, w, s) : launch_one<T, D, RB, HALF, false>(dc, w, s);
}

template <class T, int D>
int launch_rows(const DevCtx& dc, const Work& w, int rb, cudaStream_t s) {
    if ((long long)w.a.max_new * w.group <= 8) return launch_cap<T, D, 1, true>(dc, w, s);
    return rb == 1 ? launch_cap<T, D, 1>(dc, w, s) : rb == 2 ? launch_cap<T, D, 2>(dc, w, s)
                                                             : launch_cap<T, D, 4>(dc, w, s);
}

}  // namespace

int launch_few(const DevCtx& dc, const Work& w, int rb, cudaStream_t s) {
    if (w.a.dtype == QG_F16)
        return w.a.d == 64 ? launch_rows<__half, 64>(dc, w, rb, s) : launch_rows<__half, 128>(dc, w, rb, s);
    return w.a.d == 64 ? launch_rows<__nv_bfloat16, 64>(dc, w, rb, s) : launch_rows<__nv_bfloat16, 128>(dc, w, rb, s);
}

int cache_map(CUtensorMap* m, const AttnArgs& a, const void* p, int rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    int rc = prefill::encoder(&encode);
    if (rc) return rc;
    const cuuint64_t per = (cuuint64_t)a.hkv * a.page_size;
    const cuuint64_t dims[3] = {(cuuint64_t)a.d, per, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[2] = {(cuuint64_t)a.d * 2, per * a.d * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1}, es[3] = {1, 1, 1};
    const auto type = a.dtype == QG_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode(m, type, 3, const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QG_OK
               : QG_ERR_UNSUPPORTED;
}

}  // namespace attn
}  // namespace qg
