// attn_paged for chunks of new tokens: bound by the tensor cores and by the
// exponentials.
#include <algorithm>

#include "attn_join.cuh"

namespace qg {
namespace attn {
namespace {

using namespace prefill;
using fp8::fma2;
using fp8::tmem_alloc;
using fp8::tmem_dealloc;
using fp8::tmem_ld32_async;
using fp8::tmem_wait32;

// A row tile is two blocks of 128 rows, a step 128 keys. Both blocks share the
// keys and values in shared memory, and while one block's scores are turned
// into probabilities by its warpgroup the tensor cores work on the other's:
//
//   S_t = Q_t K^T        t = 0, 1; 128 x 128 f32 in tensor memory
//   P_t = 2^(s S_t - m)  by warpgroup t, thread = row; over S_t's columns
//   O_t += P_t V         P_t from tensor memory
//
// in the order S0 S1 | O0 S0' O1 S1' | O0' S0'' ..., where the MMAs that one
// thread issues run in order, so that S_t' may overwrite P_t and "S_t' is
// there" implies "O_t is up to date".
//
// The maximum m follows the scores lazily: O and the sum are rescaled only when
// a row's new maximum is over 2^8 times the one in use (probabilities up to
// 2^8 cost nothing in f16 or bf16, and the quotient by the sum is the same).
// Probabilities enter the product with V rounded to its type, which the tensor
// cores ask of both operands; their remainders as a second product would be half as
// much tensor work again. Outputs are off by 1.2 to 1.4 times what their own rounding
// alone is (root mean square, over normal keys and values).
// Rows past the last one repeat it; their results are not stored.
//
//   warps 0-3, 4-7  softmax and output of block 0, 1; they also gather their
//                   block's rows of Q, those of the next segment as soon as the
//                   last scores of this one are there
//   warp 8          TMA producer: ring of K and V tiles, taken alternately
//   warp 9          MMA issuer
// Ten warps are three to some of the schedulers, which leaves 168 registers per
// thread: a row's 128 scores stay in them.
//
// With the joining kernel: 2 x 2048 new tokens over 16384 and 8200 keys, 32/8
// heads of 128, bf16: 556 to 583 us, 1.30 to 1.36 PFLOP/s, by the GPU: at the power
// limit (SM clock 1965 MHz); tensor pipes 52 % busy. 13 sequences of up to 130 new
// tokens, 20/4 heads of 64, capped, windowed: 43 us, 4 or 5 steps one after the
// other per CTA.
constexpr int kKT = 128;
constexpr int kRT = 256;
constexpr int kThreads = 320;
constexpr float kLazy = 8.f;

template <int D>
struct Geo {
    static constexpr int kHalf = 128 * 128;            // 64 columns of 128 rows
    static constexpr int kTile = kHalf * (D / 64);     // one K, V or Q block
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kRingOff = 2 * kTile;
    static constexpr int kBarOff = kRingOff + kStages * kTile;
    static constexpr int kScratchOff = kBarOff + 16 * kStages + 128;
    static constexpr int kStageOff = kScratchOff + 256;  // 4 KB per softmax warp, outputs on their way
    static constexpr int kSmem = 1024 + kStageOff + 8 * 4096;
    static constexpr uint32_t kO = 256;                // tensor memory: S0, S1, O0, O1
};

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Operand with its rows along the product's inner dimension (V: a row is a
// key): 128-byte-swizzled atoms of 64 columns x 8 rows, atoms of the next 8
// rows 1024 bytes on, of the next 64 columns `half` bytes on.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, uint32_t half) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(half >> 4) << 16) | (64ull << 32) | (1ull << 46) |
           (2ull << 61);
}

template <class T>
constexpr uint32_t idesc(int n, bool b_rows_are_k) {
    constexpr uint32_t type = std::is_same_v<T, __nv_bfloat16> ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | (b_rows_are_k ? 1u << 16 : 0u) |
           ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared16(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void fence_async_proxy() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// How scores come from dot products: times a positive scale, which is left to the
// exponential; capped; or times any scale, under which the largest product need
// not be the largest score. The latter two are formed before anything else.
enum Mode : int { kPositive, kCapped, kAnyScale };

template <class T, int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const Work w) {
    using G = Geo<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const uint32_t bars = base + G::kBarOff;
    auto full = [&](int i) { return bars + 8u * i; };
    auto empty = [&](int i) { return bars + 8u * (G::kStages + i); };
    const uint32_t more = bars + 16u * G::kStages;
    auto s_full = [&](int t) { return more + 8u * t; };
    auto p_full = [&](int t, int half) { return more + 16u + 16u * t + 8u * half; };  // 64 keys each
    auto o_full = [&](int t) { return more + 48u + 8u * t; };
    auto q_full = [&](int t) { return more + 64u + 8u * t; };
    const uint32_t tail = more + 80u, done = more + 88u;
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + G::kBarOff + 16 * G::kStages + 96);
    const int warp = warp_number(), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < G::kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t, 0), 4);
            mbar_init(p_full(t, 1), 4);
            mbar_init(o_full(t), 1);
            mbar_init(q_full(t), 4);
        }
        mbar_init(tail, 1);
        mbar_init(done, 1);
        fence_mbar_init();
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
    }
    if (warp == 9) tmem_alloc(smem_addr(slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    pdl_wait();
    pdl_trigger();
    Cuts cuts;
    Place place;
    Seq seq;
    if (threadIdx.x == 0) w.notes[blockIdx.x].from = -1, w.notes[blockIdx.x].bad = 0;
    if (locate<kRT, kKT, kThreads>(w, blockIdx.x, &cuts, &place, &seq, reinterpret_cast<long long*>(smem + G::kScratchOff))) {
        const long long n = cuts(blockIdx.x + 1) - cuts(blockIdx.x);
        if (threadIdx.x == 0) note_start(w, place, n);
        Walk<kRT, kKT> walk(w, place, seq, n);
        bool ok = true;
        if (warp == 8) {
            // -------------------------------------------------------- producer
            const int rows = min(w.a.page_size, kKT);
            int i = 0, tails = 0;
            while (ok && walk.next()) {
                for (int t = walk.lo; ok && t < walk.hi; ++t) {
                    const int keys = max(0, min(kKT, walk.span.end - t * kKT)), unseen = walk.span.begin - t * kKT;
                    const int copies = (keys + rows - 1) / rows;
                    int page = 0, y = 0;
                    if (lane < copies) {
                        const int j = t * kKT + lane * rows;
                        page = page_from(w, walk.p.b, j, rows, walk.span.begin);
                        y = walk.p.head * w.a.page_size + j % w.a.page_size;
                    }
                    for (int kv = 0; kv < 2; ++kv, ++i) {
                        const int st = i % G::kStages;
                        if (i >= G::kStages && !warp_bar_wait(empty(st), ((i / G::kStages) & 1) ^ 1)) {
                            if (lane == 0) report_error(w.err, DEVERR_TC_WAIT);
                            ok = false;
                            break;
                        }
                        const bool part = kv && (keys < kKT || unseen > 0);  // values that no row sees are cleared
                        const uint32_t bar = part ? tail : full(st);
                        const uint32_t dst = base + G::kRingOff + st * G::kTile;
                        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(copies * rows * D * 2));
                        __syncwarp();
                        if (lane < copies) {
#pragma unroll
                            for (int h = 0; h < D / 64; ++h)
                                tma_load_3d(dst + h * G::kHalf + lane * rows * 128, kv ? &map_v : &map_k, h * 64, y,
                                            page, bar);
                        }
                        if (part) {
                            if (!warp_bar_wait(tail, tails & 1)) {
                                if (lane == 0) report_error(w.err, DEVERR_WAIT_DRAIN);
                                ok = false;
                            }
                            ++tails;
                            uint4* v = reinterpret_cast<uint4*>(smem + G::kRingOff + st * G::kTile);
                            for (int h = 0; h < D / 64; ++h) {
                                for (int e = lane; e < unseen * 8; e += 32)
                                    v[h * (G::kHalf / 16) + e] = make_uint4(0u, 0u, 0u, 0u);
                                for (int e = keys * 8 + lane; e < kKT * 8; e += 32)
                                    v[h * (G::kHalf / 16) + e] = make_uint4(0u, 0u, 0u, 0u);
                            }
                            fence_async_proxy();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(full(st));
                        }
                    }
                }
            }
            for (int j = max(0, i - G::kStages); j < i; ++j)
                if (!warp_bar_wait(full(j % G::kStages), (j / G::kStages) & 1) && lane == 0)
                    report_error(w.err, DEVERR_WAIT_DRAIN);
        } else if (warp == 9) {
            // ------------------------------------------------------------- MMA
            constexpr uint32_t kQK = idesc<T>(128, false), kPV = idesc<T>(D, true);
            const uint64_t dq = sw128_desc(base), dk = sw128_desc(base + G::kRingOff);
            const uint64_t dv = mn_desc(base + G::kRingOff, G::kHalf);
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            int st = 0;                               // place of the next ring entry
            uint32_t ph = 0;                          // and its phase
            int steps[2] = {0, 0}, segs[2] = {0, 0};  // of each block
            auto wait = [&](uint32_t bar, uint32_t parity) {
                if (ok && !warp_bar_wait(bar, parity)) {
                    if (lane == 0) report_error(w.err, DEVERR_TC_WAIT);
                    ok = false;
                }
                return ok;
            };
            auto score_mma = [&](int t, int stage) {
                const uint64_t a = dq + (uint64_t)(t * (G::kTile >> 4)), b = dk + (uint64_t)(stage * (G::kTile >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            mma_ss(tm + t * 128, a + h * (G::kHalf >> 4) + 2 * c, b + h * (G::kHalf >> 4) + 2 * c, kQK,
                                   h + c > 0);
                    tc_commit(s_full(t));
                }
                __syncwarp();
            };
            auto out_mma = [&](int t, int stage, bool acc) {
                const uint64_t v = dv + (uint64_t)(stage * (G::kTile >> 4));
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!wait(p_full(t, half), steps[t] & 1)) return;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int c = half * 4; c < half * 4 + 4; ++c)  // 16 keys: 8 columns of P, 2048 bytes of V
                            tc_mma_ts(tm + G::kO + t * D, tm + t * 128 + c * 8, v + c * 128, kPV, acc || c > 0);
                    }
                    __syncwarp();
                }
                ++steps[t];
            };
            auto commit = [&](uint32_t bar) {
                if (elect_one()) tc_commit(bar);
                __syncwarp();
            };
            auto advance = [&] {
                if (++st == G::kStages) {
                    st = 0;
                    ph ^= 1;
                }
            };
            while (ok && walk.next()) {
                const bool two = walk.s.rows - walk.p.tile * kRT > 128;
                const int nt = walk.hi - walk.lo;
                if (!wait(full(st), ph)) break;
                for (int t = 0; t < 1 + two; ++t) {
                    if (!wait(q_full(t), segs[t]++ & 1)) break;
                    tc_fence_after();
                    score_mma(t, st);
                }
                commit(empty(st));
                advance();
                for (int j = 0; ok && j < nt; ++j) {
                    const int vs = st;
                    const bool last = j + 1 == nt;
                    if (!wait(full(vs), ph)) break;
                    advance();
                    out_mma(0, vs, j > 0);
                    if (last) {
                        commit(o_full(0));
                    } else {
                        if (!wait(full(st), ph)) break;
                        tc_fence_after();
                        score_mma(0, st);
                    }
                    if (two) {
                        out_mma(1, vs, j > 0);
                        if (last) commit(o_full(1));
                    }
                    commit(empty(vs));
                    if (!last) {
                        if (two) score_mma(1, st);
                        commit(empty(st));
                        advance();
                    }
                }
            }
            commit(done);
            if (!warp_bar_wait(done, 0) && lane == 0) report_error(w.err, DEVERR_WAIT_DRAIN);
        } else {
            // --------------------------------------------------------- softmax
            const int t = warp >> 2, row = (warp & 3) * 32 + lane;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + G::kO + t * D;
            int steps = 0, seg = 0;
            // This thread's row of Q in the next segment that has this block;
            // `ahead` is advanced to it.
            auto gather = [&](Walk<kRT, kKT>& ahead) {
                do {
                    if (!ahead.next()) return;
                } while (ahead.s.rows - ahead.p.tile * kRT <= t * 128);
                const int r = min(ahead.p.tile * kRT + t * 128 + row, ahead.s.rows - 1);
                const T* src = static_cast<const T*>(w.a.q) +
                               (long long)(ahead.s.first + r / w.group) * w.a.q_stride +
                               (long long)(ahead.p.head * w.group + r % w.group) * D;
                const uint32_t dst = base + t * G::kTile + row * 128;
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    cp_async16(dst + (c / 8) * G::kHalf + (((c & 7) ^ (row & 7)) << 4), src + c * 8);
            };
            auto gathered = [&] {
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full(t));
            };
            {
                Walk<kRT, kKT> ahead = walk;
                gather(ahead);
                gathered();
            }
            while (walk.next()) {
                const Seq s = walk.s;
                const int r0 = walk.p.tile * kRT, nt = walk.hi - walk.lo;
                if (s.rows - r0 <= t * 128) continue;  // no such block
                const int r = min(r0 + t * 128 + row, s.rows - 1);
                const int pos = s.ctx - s.n + r / w.group;
                const int pos_lo = __shfl_sync(0xFFFFFFFFu, pos, 0), pos_hi = __shfl_sync(0xFFFFFFFFu, pos, 31);
                float m = -INFINITY, l = 0.f;
                for (int j = 0; j < nt; ++j, ++steps) {
                    const int j0 = (walk.lo + j) * kKT;
                    if (ok && !warp_bar_wait(s_full(t), steps & 1)) {
                        if (lane == 0) report_error(w.err, DEVERR_TC_WAIT);
                        ok = false;  // the results are lost; the barriers are still met
                    }
                    tc_fence_after();
                    // All of this segment's scores of the block are there: its Q is free.
                    if (j + 1 == nt) {
                        Walk<kRT, kKT> ahead = walk;
                        gather(ahead);
                    }
                    uint32_t x[4][32];
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    const bool masked = j0 + kKT - 1 > pos_lo || (w.a.window && j0 <= pos_hi - w.a.window);
                    tmem_ld32_async(s_at, x[0]);
                    tmem_ld32_async(s_at + 32, x[1]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c % 2 == 0) {
                            tmem_wait32(x[c]);
                            tmem_wait32(x[c + 1]);
                            if (c == 0) {
                                tmem_ld32_async(s_at + 64, x[2]);
                                tmem_ld32_async(s_at + 96, x[3]);
                            }
                        }
                        if constexpr (MODE != kPositive)
                            scores<MODE == kCapped, 32>(w, [&](int e) { return __uint_as_float(x[c][e]); },
                                                        [&](int e, float v) { x[c][e] = __float_as_uint(v); });
                        if (masked) {
                            const int hi = pos - j0 - c * 32;                                // last key seen
                            const int lo = w.a.window ? pos - w.a.window - j0 - c * 32 : -1;  // first key seen - 1
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (e > hi || e <= lo) x[c][e] = 0xFF800000u;
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            tops[(e / 2) & 3] = fmaxf(fmaxf(tops[(e / 2) & 3], __uint_as_float(x[c][e])),
                                                      __uint_as_float(x[c][e + 1]));
                    }
                    float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    if (MODE == kPositive) top *= w.scale_log2;
                    if (__any_sync(0xFFFFFFFFu, top > m + kLazy)) {
                        const float mn = fmaxf(m, top);
                        const float f = ex2(m - (mn == -INFINITY ? 0.f : mn));
                        m = mn;
                        l *= f;
                        if (j) {
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(o_at + c, o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st16(o_at + c, o);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m;
                    const float2 sc = make_float2(MODE == kPositive ? w.scale_log2 : 1.f, MODE == kPositive ? w.scale_log2 : 1.f);
                    const float2 off = make_float2(-ref, -ref);
                    float2 sum[4] = {};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 v = fma2(make_float2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), sc, off);
                            v.x = ex2(v.x);
                            v.y = ex2(v.y);
                            sum[(e / 2) & 3] = __fadd2_rn(sum[(e / 2) & 3], v);
                            p[e / 2] = pack2<T>(v.x, v.y);
                        }
                        tmem_st16(s_at + c * 16, p);
                        if (c & 1) {
                            tmem_st_wait();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(p_full(t, c / 2));
                        }
                    }
                    const float2 s01 = __fadd2_rn(sum[0], sum[1]), s23 = __fadd2_rn(sum[2], sum[3]);
                    l += (s01.x + s23.x) + (s01.y + s23.y);
                }
                gathered();
                // ------------------------------------------- end of a segment
                if (ok && !warp_bar_wait(o_full(t), seg & 1)) {
                    if (lane == 0) report_error(w.err, DEVERR_TC_WAIT);
                    ok = false;
                }
                ++seg;
                tc_fence_after();
                const bool live = r0 + t * 128 + row < s.rows;
                const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
                const long long at = (long long)(s.first + r / w.group) * w.a.hq + walk.p.head * w.group + r % w.group;
                const long long pt = ((long long)blockIdx.x * 2 + walk.slot) * kRT + t * 128 + row;
                // 128 bytes of each row at a time through shared memory, so that eight
                // lanes store to one row (16 bytes of 32 rows by each store took
                // about 1000 cycles per 16 columns).
                const uint32_t stage = base + G::kStageOff + warp * 4096, mine = stage + lane * 128, swz = lane & 7;
                const int rows_left = s.rows - (r0 + t * 128 + (warp & 3) * 32);
                auto leave = [&](char* to, long long stride) {
                    __syncwarp();
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const int rr = i * 4 + (lane >> 3), ch = lane & 7;
                        const long long row_at = stride ? rr * stride : __shfl_sync(0xFFFFFFFFu, at, rr) * (D * 2);
                        if (rr < rows_left)
                            *reinterpret_cast<uint4*>(to + row_at + ch * 16) = ld_shared16(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
                    }
                    __syncwarp();
                };
                if (walk.whole) {
                    float finite = 0.f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 64) {
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            uint32_t o[16], h[8];
                            tmem_ld16(o_at + c + k * 16, o);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 v = make_float2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                                finite = fmaf(v.x, 0.f, fmaf(v.y, 0.f, finite));
                                h[e] = pack2<T>(v.x, v.y);
                            }
                            st_shared16(mine + ((2 * k ^ swz) << 4), make_uint4(h[0], h[1], h[2], h[3]));
                            st_shared16(mine + ((2 * k + 1 ^ swz) << 4), make_uint4(h[4], h[5], h[6], h[7]));
                        }
                        leave(static_cast<char*>(w.a.out) + c * 2, 0);
                    }
                    if (live && l == l && finite != finite) w.notes[blockIdx.x].bad = 1;
                } else {
                    const long long part0 = ((long long)blockIdx.x * 2 + walk.slot) * kRT + t * 128 + (warp & 3) * 32;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
#pragma unroll 1
                        for (int k = 0; k < 2; ++k) {
                            uint32_t o[16];
                            tmem_ld16(o_at + c + k * 16, o);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                st_shared16(mine + ((4 * k + e ^ swz) << 4),
                                            make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                        }
                        leave(reinterpret_cast<char*>(w.part + part0 * D + c), D * 4);
                    }
                }
                tc_fence_before();
                if (threadIdx.x == 0) walk.note(cuts, kRT, blockIdx.x);
                if (live) {
                    if (!walk.whole) w.ml[pt] = make_float2(m, l);
                    else if (w.a.lse) w.a.lse[at] = l == 0.f ? -INFINITY : fmaf(m, w.to_ln, logf(l));
                }
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

template <class T, int D, int MODE>
int launch_one(const DevCtx& dc, const Work& w, cudaStream_t s) {
    static std::atomic<int> configured[64];  // set by any thread, all to the same
    auto kern = chunk_kernel<T, D, MODE>;
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
    return launch_join<T, D, kRT, kKT, 4, 2>(w, s);
}

template <class T, int D>
int launch_mode(const DevCtx& dc, const Work& w, cudaStream_t s) {
    if (w.a.softcap > 0.f) return launch_one<T, D, kCapped>(dc, w, s);
    return w.scale_log2 > 0.f ? launch_one<T, D, kPositive>(dc, w, s) : launch_one<T, D, kAnyScale>(dc, w, s);
}

}  // namespace

int launch_chunk(const DevCtx& dc, const Work& w, cudaStream_t s) {
    if (w.a.dtype == QG_F16)
        return w.a.d == 64 ? launch_mode<__half, 64>(dc, w, s) : launch_mode<__half, 128>(dc, w, s);
    return w.a.d == 64 ? launch_mode<__nv_bfloat16, 64>(dc, w, s) : launch_mode<__nv_bfloat16, 128>(dc, w, s);
}

}  // namespace attn
}  // namespace qg
