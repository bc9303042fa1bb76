// token_logprobs: log probabilities of given tokens, entropy, rank and the
// largest alternatives of rows of logits.
#include <cooperative_groups.h>

#include <algorithm>

#include "fp8_tc.cuh"

namespace cg = cooperative_groups;

namespace qg {
namespace {

// A row is read once, by one CTA or, when there are few rows, by a cluster of
// them, each taking a share of it; bound by the bytes of the logits.
//
// Each thread keeps, in base 2 with d = x log2(e) - b, where c is a logit next to
// its running maximum and b = c log2(e) rounded to f32,
//     s = sum 2^d,  t = sum d 2^d,
// which a larger base b + g turns into 2^-g s and 2^-g (t - g s). The rounding of b
// is the same in every term and d is rounded once (a fused multiplication), so it
// moves s by 2^r, r = c log2(e) - b. At the end, with c, s, t of the whole row,
//     log p(x) = (x - c) - (ln s - r ln2),  entropy = ln s - ln2 t / s.
// Both are within a few 2^-24 of ln s and of themselves.
//
// A producer warp copies the row's aligned middle into a ring of 16 KB stages by
// bulk copies, and on into the CTA's next row, so that the loads go on while a row
// is being finished and cost the other warps no instructions (they issue almost
// all the time: some 8 instructions per logit).
//
// The k largest come almost for free: every thread also keeps its largest logit
// and the chunk that has it. If k of these (of equal ones the one in the earlier
// chunk first) are at least T, a logit below T has k before it; so only the threads
// with T and larger ones can hold any of the k largest, and their logits, a small
// part of the row, are read again. That and the joining of the
// statistics is the work of one more warp while the others read the next row
// (done by all warps between two rows it took 55 us of 159 for 2048 rows of
// 131072 bf16 logits with the 5 largest).
//
// 2048 x 131072 bf16, 5 largest: 121 us, 4.5 TB/s, two thirds of all issue slots
// taken. One row of 50021 f32, 20 largest: 11.0 us, the latency of the finish.
constexpr int kThreads = 256;               // that read logits; a producer and a finishing warp more
constexpr int kWarps = kThreads / 32;
constexpr int kTop = 32;                    // most alternatives
constexpr int kPer = 2;                     // chunks per thread and stage
constexpr int kStageChunks = kPer * kThreads;
constexpr int kStages = 6;
constexpr int kRing = kStages * kStageChunks * 32;
constexpr int kCtasPerSm = 2;
// The maximum is followed in steps of 2 bits: d up to 2 rounds no worse than the
// exponential does, and a row that is dominated by one logit has it as its base
// (otherwise another with a fourth of its probability). With steps of 29 bits log
// probabilities were off by 3e-6 and entropies by 1e-5.
constexpr float kLazy = 1.3862944f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

using Key = unsigned long long;

// The order of the logits as an order of whole numbers: larger value first,
// NaN above all, -0 equal to 0; then the lower id. 0 is below every logit.
__device__ __forceinline__ uint32_t value_key(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 + 0 = 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ Key key_of(float v, int id) {
    return (Key)value_key(v) << 32 | (0xFFFFFFFFu - (uint32_t)id);
}
__device__ __forceinline__ int id_of(Key k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }
__device__ __forceinline__ float value_of(Key k) {
    const uint32_t v = (uint32_t)(k >> 32);
    return __uint_as_float(v & 0x80000000u ? v & 0x7FFFFFFFu : ~v);
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 32 bytes of a row: 8 or 16 logits.
template <class T>
struct Chunk {
    static constexpr int kN = 32 / sizeof(T);
    uint32_t w[8];
    __device__ __forceinline__ void load(const T* p) {
        asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                       "=r"(w[7])
                     : "l"(p));
    }
    __device__ __forceinline__ void get(float (&v)[kN]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = unpack2<T>(w[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
};

// How many of the chunk's logits are greater than xt (or NaN); xt2: xt twice, in T.
template <class T>
__device__ __forceinline__ int count_above(const Chunk<T>& c, float xt, uint32_t xt2) {
    if constexpr (sizeof(T) == 4) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) n += !(__uint_as_float(c.w[i]) <= xt);
        return n;
    } else {
        using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
        const T2 x = *reinterpret_cast<const T2*>(&xt2);
        T2 n = __hgtu2(*reinterpret_cast<const T2*>(&c.w[0]), x);  // 1 or 0 each; sums to 8 are exact
#pragma unroll
        for (int i = 1; i < 8; ++i) n = __hadd2(n, __hgtu2(*reinterpret_cast<const T2*>(&c.w[i]), x));
        const float2 f = unpack2<T>(*reinterpret_cast<const uint32_t*>(&n));
        return (int)(f.x + f.y);
    }
}

// This CTA's share of a row, cut into 32-byte chunks from an aligned address
// at or before it: chunk i holds ids i * kN - off .. of which [lo, hi) are its.
template <class T>
struct Row {
    const T* x;     // the row
    const T* base;  // x - off
    int off, lo, hi;
    int c_lo, c_hi;  // its chunks

    __device__ __forceinline__ void set(const LogprobArgs& a, long long r, int part, int parts) {
        constexpr int N = Chunk<T>::kN;
        x = static_cast<const T*>(a.x) + r * a.stride;
        off = (int)(reinterpret_cast<uintptr_t>(x) % 32 / sizeof(T));
        base = x - off;
        const int chunks = (int)((a.V + off + N - 1) / N);
        c_lo = (int)((long long)chunks * part / parts);
        c_hi = (int)((long long)chunks * (part + 1) / parts);
        lo = max(0, c_lo * N - off);
        hi = (int)min((long long)a.V, (long long)c_hi * N - off);
    }
    __device__ __forceinline__ bool inside(int c) const {
        return c * Chunk<T>::kN - off >= lo && (c + 1) * Chunk<T>::kN - off <= hi;
    }
    // Chunk c; -infinity past the ends (nothing is read there).
    __device__ __forceinline__ void load(int c, Chunk<T>& ch) const {
        if (inside(c)) {
            ch.load(base + (long long)c * Chunk<T>::kN);
            return;
        }
        const int id = c * Chunk<T>::kN - off;
        auto at = [&](int i) { return id + i >= lo && id + i < hi ? to_f32(x[id + i]) : -INFINITY; };
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 4) ch.w[i] = __float_as_uint(at(i));
            else ch.w[i] = pack2<T>(at(2 * i), at(2 * i + 1));
        }
    }
};

struct Stats {
    float c, s, t;  // c = -infinity: nothing yet
};
// The base of c, and whether it is a number (it is not next to the type's largest,
// nor for nothing; differences come first then).
__device__ __forceinline__ float base_of(float c) { return __fmul_rn(c, kLog2e); }
__device__ __forceinline__ bool has_base(float c) { return fabsf(base_of(c)) <= 3.4028235e38f; }
// From base c to a's, which is not larger. (From nothing: cut to a finite number.)
__device__ __forceinline__ float gap(float a, float c) {
    const float g = has_base(c) ? base_of(a) - base_of(c) : (a - (c == -INFINITY ? 0.f : c)) * kLog2e;
    return fmaxf(g, -200.f);
}
// The same with c instead of a.c. (Without logits s = t = 0.)
__device__ __forceinline__ Stats rebased(const Stats& a, float c) {
    const float g = gap(a.c, c), f = ex2(g);
    return Stats{c, a.s * f, f * (a.t + g * a.s)};
}

struct Thread {
    Stats st;
    float minus_b;  // minus the base of st.c
    float best;     // the largest logit, NaN above all, and the first chunk with it
    int best_chunk;
    int above;

    template <class T>
    __device__ __forceinline__ void take(const float (&v)[Chunk<T>::kN], const Chunk<T>& raw, int chunk, float xt,
                                         uint32_t xt2) {
        constexpr int N = Chunk<T>::kN;
        float cm = max_nan(v[0], v[1]);
#pragma unroll
        for (int i = 2; i < N; i += 2) cm = max_nan(cm, v[i], v[i + 1]);
        if (!(cm <= xt)) above += count_above(raw, xt, xt2);
        if (!(cm <= best) && best == best) {
            best = cm;
            best_chunk = chunk;
        }
        if (cm > st.c + kLazy) {  // always at first: st.c is -infinity, s = t = 0
            // (where a base is not a number the old sums vanish beside the new logit)
            const float m = -base_of(cm), g = fmaxf(m - minus_b, -200.f), f = ex2(g);
            st.t = f * (st.t + g * st.s);
            st.s *= f;
            st.c = cm;
            minus_b = m;
        }
        const float2 l2 = make_float2(kLog2e, kLog2e);
        float2 ss = make_float2(0.f, 0.f), tt = make_float2(0.f, 0.f);
        {
            const float2 mc = make_float2(minus_b, minus_b);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float2 d = __ffma2_rn(make_float2(v[i], v[i + 1]), l2, mc);
                const float2 e = make_float2(ex2(d.x), ex2(d.y));
                ss = __fadd2_rn(ss, e);
                tt = __ffma2_rn(e, d, tt);
            }
        }
        // Not finite: a masked logit (0 times infinity), a value whose multiple by
        // log2(e) is out of range, or a NaN. Again, cut off, and difference first if
        // there is no base.
        if (!(fabsf(tt.x + tt.y) < 1e30f)) {
            const bool based = has_base(st.c);
            const float ref = based || st.c == -INFINITY ? 0.f : st.c, off = based ? minus_b : 0.f;
            const float2 mr = make_float2(-ref, -ref), mc = make_float2(off, off);
            ss = tt = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                float2 d = __ffma2_rn(__fadd2_rn(make_float2(v[i], v[i + 1]), mr), l2, mc);
                // 2^-200 is 0 in f32: a masked logit adds 0; NaN stays
                d.x = max_nan(d.x, -200.f);
                d.y = max_nan(d.y, -200.f);
                const float2 e = make_float2(ex2(d.x), ex2(d.y));
                ss = __fadd2_rn(ss, e);
                tt = __ffma2_rn(e, d, tt);
            }
        }
        st.s += ss.x + ss.y;
        st.t += tt.x + tt.y;
    }
};

// The larger 32 of the keys in two descending lists over the warp's lanes,
// descending: lane i's larger one of a[i] and b[31 - i] is a bitonic sequence.
__device__ __forceinline__ Key merge_top(Key a, Key b) {
    const int lane = threadIdx.x & 31;
    const Key r = __shfl_sync(0xFFFFFFFFu, b, 31 - lane);
    Key k = a > r ? a : r;
#pragma unroll
    for (int step = 16; step; step /= 2) {
        const Key o = __shfl_xor_sync(0xFFFFFFFFu, k, step);
        k = ((lane & step) == 0) == (k > o) ? k : o;
    }
    return k;
}

// The warp's keys, descending over its lanes.
__device__ __forceinline__ Key warp_sort(Key k) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int step = size / 2; step; step /= 2) {
            const Key o = __shfl_xor_sync(0xFFFFFFFFu, k, step);
            const bool low = (lane & step) == 0, down = (lane & size) == 0 || size == 32;
            k = (low == down) == (k > o) ? k : o;
        }
    return k;
}

// The lanes' statistics in one, the same on all lanes.
__device__ __forceinline__ void join_lanes(Stats& st, int& above) {
    float c = st.c;
#pragma unroll
    for (int i = 16; i; i >>= 1) c = fmaxf(c, __shfl_xor_sync(0xFFFFFFFFu, c, i));
    st = rebased(st, c);
#pragma unroll
    for (int i = 16; i; i >>= 1) {
        st.s += __shfl_xor_sync(0xFFFFFFFFu, st.s, i);
        st.t += __shfl_xor_sync(0xFFFFFFFFu, st.t, i);
        above += __shfl_xor_sync(0xFFFFFFFFu, above, i);
    }
}

// What a row's readers leave to the finishing warp.
struct Left {
    float c[kThreads], s[kThreads], t[kThreads], best[kThreads];
    int chunk[kThreads], above[kThreads];
};

// CTA x of a cluster (grid x) has share x of its rows: y, y + grid y, ...
template <class T>
__global__ void __launch_bounds__(kThreads + 64, kCtasPerSm) row_kernel(const LogprobArgs a, unsigned* err) {
    constexpr int N = Chunk<T>::kN;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t bars[2 * kStages];
    __shared__ __align__(8) uint64_t more[4];  // left[i] written, taken
    __shared__ Left left[2];
    __shared__ int owner[kThreads];            // the threads that can hold the share's largest
    __shared__ Key wait[64];                   // keys on their way into the list of those
    __shared__ __align__(16) uint8_t look[32 * 32];  // the chunks being looked through
    __shared__ Key found[kTop];
    __shared__ Stats all;                      // and its statistics
    __shared__ int all_above;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int parts = (int)gridDim.x, part = (int)blockIdx.x;
    const int V = (int)a.V;
    const bool top = a.k > 0;
    cg::cluster_group cl = cg::this_cluster();
    auto full = [&](int i) { return smem_addr(bars + i); };
    auto empty = [&](int i) { return smem_addr(bars + kStages + i); };
    auto left_full = [&](int i) { return smem_addr(more + i); };
    auto left_empty = [&](int i) { return smem_addr(more + 2 + i); };
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(left_full(i), kWarps);
            mbar_init(left_empty(i), 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), kWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    fp8::pdl_wait();
    fp8::pdl_trigger();
    int st = 0;          // place of the next stage in the ring
    uint32_t ph = 0;     // and its phase

    if (warp == kWarps) {
        // ------------------------------------------------------------ producer
        int i = 0;
        bool ok = true;
        for (long long r = blockIdx.y; r < a.M; r += gridDim.y) {
            Row<T> row;
            row.set(a, r, part, parts);
            const int in_lo = row.inside(row.c_lo) ? row.c_lo : row.c_lo + 1;
            const int in_hi = row.c_hi > row.c_lo && row.inside(row.c_hi - 1) ? row.c_hi : row.c_hi - 1;
            for (int c = row.c_lo; c < row.c_hi; c += kStageChunks, ++i) {
                if (i >= kStages && ok && !warp_bar_wait(empty(st), ph ^ 1)) {
                    if (lane == 0) report_error(err, DEVERR_WAIT_EMPTY);
                    ok = false;
                }
                if (lane == 0 && ok) {
                    const int lo = max(c, in_lo), hi = min(c + kStageChunks, in_hi);
                    const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) * 32u : 0u;
                    mbar_arrive_expect_tx(full(st), bytes);
                    if (bytes)
                        prefill::bulk_g2s_nohint(smem_addr(ring) + (st * kStageChunks + lo - c) * 32,
                                                 row.base + (long long)lo * N, bytes, full(st));
                }
                __syncwarp();
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (parts > 1) {  // the others' two meetings of this row
                cl.sync();
                cl.sync();
            }
        }
        // Every copy is waited for by the threads that read it, unless they gave up.
        for (int j = max(0, i - kStages); ok && j < i; ++j)
            if (!warp_bar_wait(full(j % kStages), (j / kStages) & 1) && lane == 0)
                report_error(err, DEVERR_WAIT_DRAIN);
        return;
    }

    if (warp < kWarps) {
        // ------------------------------------------------------------- readers
        int64_t target = blockIdx.y < a.M ? a.targets[blockIdx.y] : -1;
        float xt = target >= 0 && target < V ? to_f32(static_cast<const T*>(a.x)[blockIdx.y * a.stride + target])
                                             : INFINITY;  // without a target nothing is counted
        bool ok = true;
        int rows = 0;
        for (long long r = blockIdx.y; r < a.M; r += gridDim.y, ++rows) {
            Row<T> row;
            row.set(a, r, part, parts);
            const long long rn = r + gridDim.y;
            const int64_t target_n = rn < a.M ? a.targets[rn] : -1;
            uint32_t xt2 = 0;
            if constexpr (sizeof(T) == 2) xt2 = pack2<T>(xt, xt);  // exact: xt is a logit (or infinity)
            Thread th{{-INFINITY, 0.f, 0.f}, INFINITY, -INFINITY, row.c_lo + (int)threadIdx.x, 0};
#pragma unroll 1
            for (int c0 = row.c_lo; c0 < row.c_hi; c0 += kStageChunks) {
                if (ok && !warp_bar_wait(full(st), ph)) {
                    if (lane == 0) report_error(err, DEVERR_WAIT_FULL);
                    ok = false;  // the results are lost; the barriers are still met
                }
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const int c = c0 + u * kThreads + threadIdx.x;
                    if (c < row.c_hi) {
                        Chunk<T> ch;
                        if (row.inside(c)) {
                            const uint4* p = reinterpret_cast<const uint4*>(
                                ring + (st * kStageChunks + u * kThreads + threadIdx.x) * 32);
                            const uint4 lo = p[0], hi = p[1];
                            ch.w[0] = lo.x; ch.w[1] = lo.y; ch.w[2] = lo.z; ch.w[3] = lo.w;
                            ch.w[4] = hi.x; ch.w[5] = hi.y; ch.w[6] = hi.z; ch.w[7] = hi.w;
                        } else {
                            row.load(c, ch);
                        }
                        float v[N];
                        ch.get(v);
                        th.take<T>(v, ch, c, xt, xt2);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(st));
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            xt = target_n >= 0 && target_n < V ? to_f32(static_cast<const T*>(a.x)[rn * a.stride + target_n])
                                               : INFINITY;
            if (rows >= 2 && ok && !warp_bar_wait(left_empty(rows & 1), ((rows >> 1) & 1) ^ 1)) {
                if (lane == 0) report_error(err, DEVERR_WAIT_EMPTY);
                ok = false;
            }
            Left& l = left[rows & 1];
            l.c[threadIdx.x] = th.st.c;
            l.s[threadIdx.x] = th.st.s;
            l.t[threadIdx.x] = th.st.t;
            l.best[threadIdx.x] = th.best;
            l.chunk[threadIdx.x] = th.best_chunk;
            l.above[threadIdx.x] = th.above;
            __syncwarp();
            if (lane == 0) mbar_arrive(left_full(rows & 1));
            if (parts > 1) {
                cl.sync();
                cl.sync();
            }
        }
        return;
    }

    // ---------------------------------------------------------- finishing warp
    int rows = 0;
    bool ok = true;
    for (long long r = blockIdx.y; r < a.M; r += gridDim.y, ++rows) {
        Row<T> row;
        row.set(a, r, part, parts);
        const int64_t target = a.targets[r];
        const bool given = target >= 0 && target < V;
        if (target >= V && lane == 0 && part == 0) report_error(err, DEVERR_INDEX);
        const float xt = given ? to_f32(row.x[target]) : 0.f;
        if (ok && !warp_bar_wait(left_full(rows & 1), (rows >> 1) & 1)) {
            if (lane == 0) report_error(err, DEVERR_WAIT_FULL);
            ok = false;
        }
        const Left& l = left[rows & 1];
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) most = fmaxf(most, l.c[i * 32 + lane]);
        Stats st{most, 0.f, 0.f};
        int above = 0;
        Key own[kWarps];  // of threads lane, 32 + lane, ...: best logit, earlier chunk first
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const int t = i * 32 + lane;
            const Stats o = rebased(Stats{l.c[t], l.s[t], l.t[t]}, most);
            st.s += o.s;
            st.t += o.t;
            above += l.above[t];
            const int c = l.chunk[t];
            own[i] = c < row.c_hi ? (Key)value_key(l.best[t]) << 32 | (0xFFFFFFFFu - (uint32_t)c) : 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(left_empty(rows & 1));
        join_lanes(st, above);

        Key mine = 0;  // the share's largest, lane i the i-th
        if (top) {
            // T here is the k-th largest of the lanes' largest keys: as good a bound,
            // one sort away, which a few threads more than k reach (all, if there
            // are not k lanes with keys).
            Key m = own[0];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) m = own[i] > m ? own[i] : m;
            const Key t = __shfl_sync(0xFFFFFFFFu, warp_sort(m), a.k - 1);
            const float least = t ? value_of(t) : -INFINITY;
            int owners = 0;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const bool in = own[i] && own[i] >= t;
                const unsigned who = __ballot_sync(0xFFFFFFFFu, in);
                if (in) owner[owners + __popc(who & ((1u << lane) - 1))] = i * 32 + lane;
                owners += __popc(who);
            }
            __syncwarp();
            Key worst = 0;  // the k-th of `mine`
            int waiting = 0;
            // Takes the first 32 of the waiting keys into `mine`.
            auto flush = [&] {
                __syncwarp();
                mine = merge_top(mine, warp_sort(lane < waiting ? wait[lane] : 0));
                worst = __shfl_sync(0xFFFFFFFFu, mine, a.k - 1);
                const Key more = lane + 32 < waiting ? wait[lane + 32] : 0;
                __syncwarp();
                wait[lane] = more;
                waiting = max(0, waiting - 32);
                __syncwarp();
            };
            // The owners' chunks, all in a line, 32 at a time, the next ones on the way.
            const int per = (row.c_hi - row.c_lo + kThreads - 1) / kThreads, n = owners * per;
            Chunk<T> ch;
            int c = row.c_hi, cn;
#pragma unroll 1
            for (int q0 = -32; q0 < n; q0 += 32) {
                const int q = q0 + 32 + lane, o = q / per;
                cn = q < n ? row.c_lo + owner[o] + (q - o * per) * kThreads : row.c_hi;
                Chunk<T> next;
                if (cn < row.c_hi) row.load(cn, next);
                // Which of the chunk's logits may be among the largest, and those one
                // at a time (from shared memory: the code stays short, for the readers'
                // sake, who run from the same instruction cache).
                uint32_t may = 0;
                if (c < row.c_hi) {
                    float v[N];
                    ch.get(v);
#pragma unroll
                    for (int i = 0; i < N; ++i) may |= (uint32_t)!(v[i] < least) << i;
                    const int first = c * N - row.off;  // ids outside the share are padding
                    if (first < row.lo) may &= ~0u << (row.lo - first);
                    if (first + N > row.hi) may &= (1u << (row.hi - first)) - 1u;
                    uint4* to = reinterpret_cast<uint4*>(look + lane * 32);
                    to[0] = make_uint4(ch.w[0], ch.w[1], ch.w[2], ch.w[3]);
                    to[1] = make_uint4(ch.w[4], ch.w[5], ch.w[6], ch.w[7]);
                }
#pragma unroll 1
                while (__any_sync(0xFFFFFFFFu, may)) {
                    Key key = 0;
                    if (may) {
                        const int i = __ffs(may) - 1;
                        key = key_of(to_f32(reinterpret_cast<const T*>(look + lane * 32)[i]), c * N - row.off + i);
                        may &= may - 1;
                    }
                    const unsigned who = __ballot_sync(0xFFFFFFFFu, key > worst);
                    if (key > worst) wait[waiting + __popc(who & ((1u << lane) - 1))] = key;
                    waiting += __popc(who);
                    if (waiting >= 32) flush();
                }
                c = cn;
                ch = next;
            }
            while (waiting > 0) flush();
        }

        if (parts > 1) {  // the shares' results meet in the first CTA
            found[lane] = mine;
            if (lane == 0) {
                all = st;
                all_above = above;
            }
            cl.sync();
            if (part == 0) {
                const int p = lane % parts;
                st = *cl.map_shared_rank(&all, p);
                above = *cl.map_shared_rank(&all_above, p);
                if (lane >= parts) {
                    st = Stats{-INFINITY, 0.f, 0.f};
                    above = 0;
                }
                join_lanes(st, above);
                if (top) {
                    Key others[7];
#pragma unroll
                    for (int o = 0; o < 7; ++o) others[o] = o + 1 < parts ? *cl.map_shared_rank(&found[lane], o + 1) : 0;
#pragma unroll
                    for (int o = 0; o < 7; ++o)
                        if (o + 1 < parts) mine = merge_top(mine, others[o]);
                }
            }
        }
        if (part == 0) {
            const bool nan = st.s != st.s, none = st.c == -INFINITY && !nan;
            const float ln = logf(st.s), rest = has_base(st.c) ? fmaf(st.c, kLog2e, -base_of(st.c)) : 0.f;
            const float all_ln = fmaf(-kLn2, rest, ln);
            // (neither a probability over 1 nor an entropy below 0 by rounding)
            auto logp = [&](float x) { return nan ? NAN : x == -INFINITY ? -INFINITY : fminf((x - st.c) - all_ln, 0.f); };
            if (lane == 0) {
                a.logprobs[r] = given ? logp(xt) : 0.f;
                a.entropy[r] = nan ? NAN : none ? 0.f : fmaxf(fmaf(-kLn2, st.t / st.s, ln), 0.f);
                a.ranks[r] = !given ? -1 : xt != xt ? 0 : above;
            }
            if (lane < a.k) {
                a.top_ids[r * a.k + lane] = id_of(mine);
                a.top_values[r * a.k + lane] = logp(value_of(mine));
            }
        }
        if (parts > 1) cl.sync();  // the shares' results have been read
    }
}

}  // namespace

int logprobs_launch(const DevCtx& dc, const LogprobArgs& a, cudaStream_t s) {
    return by_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        // Few rows are shared by clusters of up to 8 CTAs, so that all SMs load,
        // while a share keeps at least two chunks per thread.
        int parts = 1;
        while (parts < 8 && a.M * parts * 2 <= 2 * dc.num_sms &&
               a.V >= (long long)parts * 2 * 2 * kThreads * Chunk<T>::kN)
            parts *= 2;
        static std::atomic<int> configured[64];  // set by any thread, all to the same
        if (!configured[dc.device]) {
            const cudaError_t e =
                cudaFuncSetAttribute(row_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
            if (e != cudaSuccess) return cuda_fail(e);
            configured[dc.device] = 1;
        }
        cudaLaunchConfig_t cfg{};
        const long long most = std::max(1, dc.num_sms * kCtasPerSm / parts);
        cfg.gridDim = dim3((unsigned)parts, (unsigned)std::min<long long>(a.M, most));
        cfg.dynamicSmemBytes = kRing;
        cfg.blockDim = dim3(kThreads + 64);
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)parts;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = may_overlap() ? 2 : 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, row_kernel<T>, a, dc.err);
        return e == cudaSuccess ? (int)QG_OK : cuda_fail(e);
    });
}

}  // namespace qg
