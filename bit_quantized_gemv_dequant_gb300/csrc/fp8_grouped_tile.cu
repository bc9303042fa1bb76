// qmm_fp8_b128_grouped for experts of many rows: persistent pairs of CTAs over
// tiles of 256 rows of a weight times up to 256 rows of one expert.
#include <algorithm>

#include "fp8_groups.cuh"

namespace qg {
namespace fp8 {
namespace {

// As in fp8_tile.cu a pair of SMs issues its MMAs as one (cta_group::2), each with
// half of both operands in its shared memory, and two epilogue warpgroups bring
// the accumulator of the k block before into registers meanwhile. An expert's rows
// are cut into chunks of 256 and one of what is left:
// - 256 rows of a, or nearly, are the M side: a thread of the epilogue has a row of a and 128
//   columns in one block of w's scales, so one factor per k block.
// - Fewer are the N side, which comes in steps of 32, and w is M: 140 rows take
//   160 / 256 of the products' time. Each column has a scale of its own then, so the
//   accumulators are read in 16 x 256-bit fragments: a thread has four rows and two
//   of every eight columns, and needs up to 24 scales per k block. (With a row and up to
//   96 columns it would need 96, and shared memory is busy with the operands. 16 lanes
//   at a time is half of what tensor memory delivers: uniform chunks of 256 rows
//   take 294 us like that and 243 as M, 16384 rows on 32 experts, N = K = 4096.)
//
// A k block of a whole chunk takes about 970 cycles (512 of products; the round trip
// of accumulators and their promotion), of one of 64 rows 640. 16384 rows unevenly on
// 32 experts: 290 to 309 us by the GPU, 1.78 to 1.90 PFLOP/s, SM clock 1950 to 2040 MHz
// at the power limit.
//
//   warps 0-7    epilogue; 216 registers each, which warps 8-11 give up
//   warp 8       TMA producer, whose copies complete on the first CTA's barrier
//   warp 9       of the first CTA: MMA issuer for both
//   warps 10-11  scales
constexpr int kThreads = 384;
constexpr int kRegisters = 256 * 216 + 128 * 72;  // what setmaxnreg hands out
constexpr int kBM = 128, kBN = 256;               // rows of w per CTA, rows of a per pair
constexpr int kStep = 32;                         // of the columns of a chunk that is not whole
constexpr int kWhole = 192;                       // the most rows of a chunk that is not whole
constexpr int kHalf = (kWhole + kStep - 1) / kStep * (kStep / 2);  // and the columns of one epilogue warpgroup then
constexpr int kStages = 5;
constexpr int kStage = (kBM + kBN / 2) * 128;     // per CTA
constexpr int kTileSets = 2;                       // of scales under way
constexpr int kPitch = scale_pitch(kBN);
constexpr int kOutOff = kStages * kStage;          // 4 KB per epilogue warp
constexpr int kScaleOff = kOutOff + 8 * 4096;
constexpr int kBarOff = kScaleOff + kTileSets * kSetBlocks * kPitch * 4;
constexpr int kBars = 2 * kStages + 4 + 2 * kTileSets + 1;
constexpr int kGroupOff = kBarOff + 8 * kBars + 8;
using TileGroups = Groups<kBN, kBN>;
constexpr int smem_bytes(long long E) { return 1024 + kGroupOff + TileGroups::bytes(E); }
static_assert(smem_bytes(kMaxExperts) <= 227 * 1024, "shared memory");
static_assert(kGroupOff % 8 == 0, "tile numbers are 8 bytes");

// Whether a chunk's rows are the M side: a whole one's, or nearly (215 rows take 1080
// cycles per k block as N, 970 as M). 16384 rows unevenly on 32 experts: 296 us with the
// border at 192, 297 at 160, 301 at 128, 300 with 256 rows alone.
__device__ __forceinline__ bool is_whole(int rows) { return rows > kWhole; }

// As tma_load_pair, from w [E, N, K].
__device__ __forceinline__ void load_w_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// 32 columns of 16 lanes in fragments: register 4 j + 2 i + c of a thread is lane
// thread / 4 + 8 i, column 8 j + 2 (thread % 4) + c.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// 32 columns of a warp's 32 lanes: two such fragments.
struct Frag {
    uint32_t lo[16], hi[16];
    __device__ __forceinline__ void load(uint32_t taddr) {
        tmem_ld_frag(taddr, lo);
        tmem_ld_frag(taddr + (16u << 16), hi);
    }
    __device__ __forceinline__ void wait() {
        tmem_wait16(lo);
        tmem_wait16(hi);
    }
};
struct Scales {
    float2 v[4];
    __device__ __forceinline__ void load(const float* sp) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float2*>(sp + 8 * j);
    }
};
// acc[4 j + i]: lane thread / 4 + 8 i, the two columns of 8 j.
__device__ __forceinline__ void add_scaled(float2* acc, const Frag& f, const Scales& s) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t* r = (i < 2 ? f.lo : f.hi) + 4 * j + 2 * (i & 1);
            acc[4 * j + i] = fma2(make_float2(__uint_as_float(r[0]), __uint_as_float(r[1])), s.v[j], acc[4 * j + i]);
        }
}
// Four 8 x 8 matrices of 16-bit values, transposed; lane l gives the address of row
// l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

template <class TY>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_tile_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                        const __grid_constant__ CUtensorMap map_y, const GroupedParams p, const bool vec) {
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
    auto s_empty = [&](int i) { return bars + 8u * (2 * kStages + 4 + kTileSets + i); };
    const uint32_t done = bars + 8u * (kBars - 1);
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kBarOff + 8 * kBars);
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x & 1), nt128 = (p.N + 127) / 128;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(t_full(i), 1);
            mbar_init(t_empty(i), 16);  // of the first CTA: both CTAs' epilogue warps
        }
        for (int i = 0; i < kTileSets; ++i) {
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
    const long long tiles = groups.first[p.E], first = blockIdx.x >> 1, step = gridDim.x >> 1;  // this pair's tiles
    TileGroups::Tile g{};

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8 && lane == 0) {
            int i = 0;
            bool ok = true;
            for (long long t = first; t < tiles && ok; t += step) {
                groups.find(t, (p.N + 2 * kBM - 1) / (2 * kBM), g);
                // of the rows of a: each CTA holds its own
                const int half = is_whole(g.rows) ? kBM : (g.rows + kStep - 1) / kStep * (kStep / 2);
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
                    for (int j = 0; j < boxes; ++j) tma_load_pair(sb + kBM * 128 + j * 4096, &map_a, b * 128, m0 + j * 32, bar);
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
                groups.find(t, (p.N + 2 * kBM - 1) / (2 * kBM), g);
                const bool whole = is_whole(g.rows);
                const uint32_t desc = f8_idesc(2 * kBM, whole ? kBN : (g.rows + kStep - 1) / kStep * kStep);
                const uint64_t dm = whole ? da : dw, dn = whole ? dw : da;
                for (int b = 0; b < p.KB; ++b) {
                    if (!warp_bar_wait(full(st), ph) || !warp_bar_wait(t_empty(tb), tph ^ 1)) {
                        if (lane == 0) report_error(p.err, DEVERR_TC_WAIT);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t m = dm + (uint64_t)(st * (kStage >> 4)), n = dn + (uint64_t)(st * (kStage >> 4));
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_pair(tm + tb * kBN, m + 2 * k, n + 2 * k, desc, k > 0);
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
                groups.find(t, (p.N + 2 * kBM - 1) / (2 * kBM), g);
                // rows of w that are not there: any scales that are
                const float* sw = p.sw + (long long)g.e * nt128 * p.KB;
                const float* own = sw + (long long)min(2 * g.n_tile + rank, nt128 - 1) * p.KB;
                const float* halves[2] = {sw + 2LL * g.n_tile * p.KB, sw + (long long)min(2 * g.n_tile + 1, nt128 - 1) * p.KB};
                for (int b = 0; b < p.KB; b += kSetBlocks) {
                    if (!warp_bar_wait(s_empty(set), ph ^ 1)) {
                        if (lane == 0) report_error(p.err, DEVERR_TC_WAIT);
                        ok = false;
                        break;
                    }
                    float* to = scales + set * (kSetBlocks * kPitch);
                    const int n = min(kSetBlocks, p.KB - b);
                    if (is_whole(g.rows)) {  // [half of the columns][this CTA's rows]
                        load_scales<kBN, 16, kBM>(to, p, halves[0], halves[1], g.m0 + rank * kBM,
                                                  min(kBM, g.rows - rank * kBM), b, n, tid);
                    } else {
                        load_scales<kBN, 16>(to, p, own, nullptr, g.m0, g.rows, b, n, tid);
                    }
                    mbar_arrive(s_full(set));
                    if (++set == kTileSets) {
                        set = 0;
                        ph ^= 1;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
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
        auto release = [&](int buf) {  // all of this warp's reads of the accumulator are done
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(empty0 + 8u * buf);
        };
        for (long long t = first; t < tiles; t += step) {
            groups.find(t, (p.N + 2 * kBM - 1) / (2 * kBM), g);
            if (is_whole(g.rows)) {
                const int half = warp / 4, row = (warp & 3) * 32 + lane;
                const uint32_t at = lanes + half * 128;
                float2 acc[64];
#pragma unroll
                for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
                for (int b0 = 0; b0 < p.KB; b0 += kSetBlocks) {
                    if (ok && !warp_bar_wait(s_full(set), sph)) lost();
                    const int nk = min(kSetBlocks, p.KB - b0);
                    const float* sp = scales + set * (kSetBlocks * kPitch) + half * kBM + row;
#pragma unroll 1
                    for (int b = 0; b < nk; ++b, sp += kPitch) {
                        const float2 s = make_float2(*sp, *sp);
                        if (!mbar_try_wait(t_full(tb), tph) && ok && !bar_wait(t_full(tb), tph)) lost();
                        __syncwarp();
                        tc_fence_after();
                        const uint32_t from = at + tb * kBN;
                        uint32_t r[2][32];
                        tmem_ld32_async(from, r[0]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            tmem_wait32(r[c & 1]);
                            if (c < 3) tmem_ld32_async(from + (c + 1) * 32, r[(c + 1) & 1]);
                            else release(tb);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                acc[c * 16 + j] = fma2(make_float2(__uint_as_float(r[c & 1][2 * j]),
                                                                  __uint_as_float(r[c & 1][2 * j + 1])),
                                                      s, acc[c * 16 + j]);
                        }
                        tb ^= 1;
                        tph ^= tb == 0;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty(set));
                    if (++set == kTileSets) {
                        set = 0;
                        sph ^= 1;
                    }
                }
                const int m = g.m0 + rank * kBM + (warp & 3) * 32, mine = g.m0 + g.rows - m;  // rows from m on
                const long long n0 = g.n_tile * (2LL * kBM) + half * 128;
                const uint32_t stage = base + kOutOff + warp * 4096;
                if (vec && mine >= 32) {
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
                            *reinterpret_cast<uint4*>(smem + (stage - base) + lane * 128 + ((q ^ (lane & 7)) << 4)) = v;
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            if (n0 + c < p.N) tma_store_2d(&map_y, (int)n0 + c, m, stage);
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        }
                    }
                } else if (lane < mine) {
                    TY* to = y + (long long)(m + lane) * p.N + n0;
                    constexpr int kPer = 16 / sizeof(TY);
#pragma unroll
                    for (int c = 0; c < 128; c += kPer) {
                        const float2* v = acc + c / 2;
                        if (vec) {
                            uint4 o;
                            if constexpr (sizeof(TY) == 4)
                                o = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                                               __float_as_uint(v[1].y));
                            else
                                o = make_uint4(pack2<TY>(v[0].x, v[0].y), pack2<TY>(v[1].x, v[1].y),
                                               pack2<TY>(v[2].x, v[2].y), pack2<TY>(v[3].x, v[3].y));
                            if (n0 + c < p.N) *reinterpret_cast<uint4*>(to + c) = o;
                        } else {
#pragma unroll
                            for (int i = 0; i < kPer; ++i)
                                if (n0 + c + i < p.N) to[c + i] = from_f32<TY>(i & 1 ? v[i / 2].y : v[i / 2].x);
                        }
                    }
                }
                continue;
            }
            const int half = (g.rows + kStep - 1) / kStep * (kStep / 2);  // columns of a warpgroup, a multiple of 16
            const int own0 = warp / 4 * half;
            static_assert(kHalf <= 96, "three units of 32 columns");
            float2 acc[48];
#pragma unroll
            for (int j = 0; j < 48; ++j) acc[j] = make_float2(0.f, 0.f);
            // 64 columns are under way at once: a load takes about 200 cycles, and a wait is for all of them.
            // (What is read past this group's columns is inside the accumulator and the set.)
            auto sum = [&](auto units) {
                constexpr int U = decltype(units)::value;  // 32 columns each
                for (int b0 = 0; b0 < p.KB; b0 += kSetBlocks) {
                    if (ok && !warp_bar_wait(s_full(set), sph)) lost();
                    const int nk = min(kSetBlocks, p.KB - b0);
                    const float* sp = scales + set * (kSetBlocks * kPitch) + own0 + 2 * (lane & 3);
#pragma unroll 1
                    for (int b = 0; b < nk; ++b, sp += kPitch) {
                        if (!mbar_try_wait(t_full(tb), tph) && ok && !bar_wait(t_full(tb), tph)) lost();
                        __syncwarp();
                        tc_fence_after();
                        const uint32_t from = lanes + tb * kBN + own0;
                        Frag f0, f1;
                        Scales s0, s1;
                        f0.load(from);
                        if constexpr (U > 1) f1.load(from + 32);
                        s0.load(sp);
                        if constexpr (U > 1) s1.load(sp + 32);
                        f0.wait();
                        if constexpr (U > 1) f1.wait();
                        if constexpr (U <= 2) release(tb);
                        add_scaled(acc, f0, s0);
                        if constexpr (U > 2) f0.load(from + 64);
                        if constexpr (U > 2) s0.load(sp + 64);
                        if constexpr (U > 1) add_scaled(acc + 16, f1, s1);
                        if constexpr (U > 2) {
                            f0.wait();
                            release(tb);
                            add_scaled(acc + 32, f0, s0);
                        }
                        tb ^= 1;
                        tph ^= tb == 0;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty(set));
                    if (++set == kTileSets) {
                        set = 0;
                        sph ^= 1;
                    }
                }
            };
            if (half > 64) sum(std::integral_constant<int, 3>{});
            else if (half > 32) sum(std::integral_constant<int, 2>{});
            else sum(std::integral_constant<int, 1>{});
            const long long n0 = (2LL * g.n_tile + rank) * kBM + (warp & 3) * 32;
            const int mine = min(half, g.rows - own0);  // of the second warpgroup: maybe none
            TY* out = y + (long long)(g.m0 + own0) * p.N;
            if constexpr (sizeof(TY) == 2) {
                // Through shared memory, 32 columns (rows of y) at a time: 64 bytes of each beside each other.
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // a whole chunk's last store
                __syncwarp();
                const uint32_t stage = base + kOutOff + warp * 4096;
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    if (c * 32 >= mine) break;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2* v = acc + c * 16 + j * 4;
                        const int m = 8 * j + (lane & 7);  // 16-byte chunk q of row m lies at q ^ (m / 2 % 4)
                        stmatrix_t(stage + m * 64 + (((lane >> 3) ^ (m >> 1 & 3)) << 4), pack2<TY>(v[0].x, v[0].y),
                                   pack2<TY>(v[1].x, v[1].y), pack2<TY>(v[2].x, v[2].y), pack2<TY>(v[3].x, v[3].y));
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int m = 8 * j + (lane >> 2), q = lane & 3;
                        const uint4 v = *reinterpret_cast<const uint4*>(smem + (stage - base) + m * 64 + ((q ^ (m >> 1 & 3)) << 4));
                        const long long n = n0 + q * 8;
                        if (c * 32 + m < mine) {
                            TY* to = out + (c * 32 + m) * (long long)p.N + n;
                            if (vec) {
                                if (n < p.N) *reinterpret_cast<uint4*>(to) = v;
                            } else {
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    if (n + i < p.N) {
                                        const uint16_t u = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
                                        to[i] = *reinterpret_cast<const TY*>(&u);
                                    }
                            }
                        }
                    }
                    __syncwarp();
                }
            } else {
#pragma unroll
                for (int j = 0; j < 12; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = 8 * j + 2 * (lane & 3);
                        const long long n = n0 + 8 * i + lane / 4;
                        if (n < p.N) {
                            if (m < mine) out[m * (long long)p.N + n] = acc[4 * j + i].x;
                            if (m + 1 < mine) out[(m + 1) * (long long)p.N + n] = acc[4 * j + i].y;
                        }
                    }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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
    static std::atomic<int> configured[64];  // set by any thread, all to the same
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
    CUtensorMap mw, ma, my = {};
    int rc = weight_map(&mw, a);
    if (rc == QG_OK) rc = code_map(&ma, a.a, a.M, a.K, 32);
    // 16-byte stores, TMA's too, want rows of y on 16-byte boundaries
    const bool vec = reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && a.N * sizeof(TY) % 16 == 0;
    if (rc == QG_OK && vec) rc = out_map(&my, a.y, a.y_dtype, a.M, a.N);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mw, ma, my, p, vec);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

}  // namespace

int launch_grouped_tile(const DevCtx& dc, const GroupedArgs& a, cudaStream_t s) {
    return a.y_dtype == QG_F32 ? launch<float>(dc, a, s) : launch<__nv_bfloat16>(dc, a, s);
}

}  // namespace fp8
}  // namespace qg
