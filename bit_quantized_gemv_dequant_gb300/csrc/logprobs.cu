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
// Each thread keeps, in base 2 with d = x log2(e) - c (c: its running maximum
// times log2(e)),
//     s = sum 2^d,  t = sum d 2^d,
// which a larger maximum, c' = c + g, turns into 2^-g s and 2^-g (t - g s).
// At the end, with c, s, t of the whole row,
//     log p(x) = ln2 (x log2(e) - c - log2 s),  entropy = ln2 (log2 s - t / s).
//
// The k largest come almost for free: every thread also keeps its best logit
// as a key (value, then lower id). If T is the k-th largest of the threads'
// keys, a logit below T has k larger ones; so only the k threads with keys of T
// and more can hold any of the k largest, and their logits, a small part of
// the row, are read again.
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTop = 32;                    // most alternatives
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
__device__ __forceinline__ Stats join(const Stats& a, const Stats& b) {
    const float c = fmaxf(a.c, b.c);
    const float ref = c == -INFINITY ? 0.f : c;
    // A side without logits has s = t = 0; its distance is cut to a finite number.
    const float ga = fmaxf((a.c - ref) * kLog2e, -200.f), gb = fmaxf((b.c - ref) * kLog2e, -200.f);
    const float fa = ex2(ga), fb = ex2(gb);
    return Stats{c, a.s * fa + b.s * fb, fa * (a.t + ga * a.s) + fb * (b.t + gb * b.s)};
}

struct Thread {
    Stats st;       // NaN left out of the maximum
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
        if (cm > st.c) {
            const float g = fmaxf((st.c - cm) * kLog2e, -200.f);  // at first from -infinity, with s = t = 0
            const float f = ex2(g);
            st.t = f * (st.t + g * st.s);
            st.s *= f;
            st.c = cm;
        }
        const float ref = st.c == -INFINITY ? 0.f : st.c;
        const float2 l2 = make_float2(kLog2e, kLog2e), mc = make_float2(-ref, -ref);
        float2 ss = make_float2(0.f, 0.f), tt = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            float2 d = __fmul2_rn(__fadd2_rn(make_float2(v[i], v[i + 1]), mc), l2);
            // 2^-200 is 0 in f32: masked logits add 0, not 0 times infinity; NaN stays
            d.x = max_nan(d.x, -200.f);
            d.y = max_nan(d.y, -200.f);
            const float2 e = make_float2(ex2(d.x), ex2(d.y));
            ss = __fadd2_rn(ss, e);
            tt = __ffma2_rn(e, d, tt);
        }
        st.s += ss.x + ss.y;
        st.t += tt.x + tt.y;
    }
};

// The warp's 32 keys in descending order over its lanes.
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

// Puts key k (lists: n descending lists of kTop keys; this thread's is number
// `list`, place `lane`) to its place among all of them, if that is below `top`.
// Equal keys occur only as 0, the absent one, which has no place.
template <int NL>
__device__ __forceinline__ int rank_of(Key k, int list, int lane, const Key (*lists)[kTop]) {
    int rank = lane;
    auto get = [&](int o, int i) { return lists[o][i]; };
#pragma unroll
    for (int j = 1; j < NL; ++j) {  // the searches are independent of one another
        const int o = (list + j) % NL;
        int at = 0;  // keys of list o above k
#pragma unroll
        for (int step = 16; step; step /= 2)
            if (get(o, at + step - 1) > k) at += step;
        at += at == 31 && get(o, 31) > k;
        rank += at;
    }
    return rank;
}

// The statistics of the first W lanes in lane 0 (W a power of two; lanes hold
// theirs with period W). Both sides of an exchange join in the same order.
template <int W>
__device__ __forceinline__ void join_lanes(Stats& st, int& above) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = W / 2; i; i >>= 1) {
        const Stats o{__shfl_xor_sync(0xFFFFFFFFu, st.c, i), __shfl_xor_sync(0xFFFFFFFFu, st.s, i),
                      __shfl_xor_sync(0xFFFFFFFFu, st.t, i)};
        st = lane & i ? join(o, st) : join(st, o);
        above += __shfl_xor_sync(0xFFFFFFFFu, above, i);
    }
}

// The best key of a chunk.
template <class T>
__device__ __forceinline__ Key best_of(const Row<T>& row, int c) {
    constexpr int N = Chunk<T>::kN;
    Chunk<T> ch;
    row.load(c, ch);
    float v[N];
    ch.get(v);
    Key best = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int id = c * N - row.off + i;
        const Key k = id >= row.lo && id < row.hi ? key_of(v[i], id) : 0;
        best = k > best ? k : best;
    }
    return best;
}

template <class T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 4 : 3) row_kernel(const LogprobArgs a, unsigned* err) {
    constexpr int N = Chunk<T>::kN;
    __shared__ Key lists[kWarps][kTop];
    __shared__ Key found[kTop];      // the share's largest
    __shared__ int owner[kTop];      // the threads that can hold them
    __shared__ Stats stats[kWarps];
    __shared__ int aboves[kWarps];
    __shared__ Stats all;
    __shared__ int all_above;
    __shared__ Key threshold;
    fp8::pdl_trigger();
    fp8::pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int parts = (int)gridDim.x, part = (int)blockIdx.x;
    const long long r = blockIdx.y + (long long)gridDim.y * blockIdx.z;
    if (r >= a.M) return;  // the whole cluster: it has one row
    const int V = (int)a.V;
    Row<T> row;
    row.x = static_cast<const T*>(a.x) + r * a.stride;
    row.off = (int)(reinterpret_cast<uintptr_t>(row.x) % 32 / sizeof(T));
    row.base = row.x - row.off;
    const int chunks = (int)(((long long)V + row.off + N - 1) / N);
    row.c_lo = (int)((long long)chunks * part / parts);
    row.c_hi = (int)((long long)chunks * (part + 1) / parts);
    row.lo = max(0, row.c_lo * N - row.off);
    row.hi = (int)min((long long)V, (long long)row.c_hi * N - row.off);

    const int64_t target = a.targets[r];
    const bool given = target >= 0 && target < V;
    const float xt = given ? to_f32(row.x[target]) : INFINITY;  // without a target no count is needed
    if (target >= V && threadIdx.x == 0 && part == 0) report_error(err, DEVERR_INDEX);

    uint32_t xt2 = 0;
    if constexpr (sizeof(T) == 2) xt2 = pack2<T>(xt, xt);  // exact: xt is a logit (or infinity)
    Thread th{{-INFINITY, 0.f, 0.f}, -INFINITY, row.c_lo + (int)threadIdx.x, 0};
    const bool top = a.k > 0;
    // Chunk c_lo + threadIdx.x and every kThreads-th after it, four in flight.
    constexpr int U = 4;
    for (int c0 = row.c_lo + threadIdx.x; c0 < row.c_hi; c0 += U * kThreads) {
        Chunk<T> ch[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * kThreads;
            if (c < row.c_hi) row.load(c, ch[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * kThreads;
            if (c >= row.c_hi) break;
            float v[N];
            ch[u].get(v);
            th.take<T>(v, ch[u], c, xt, xt2);
        }
    }

    // ------------------------------------------------- the share's statistics
    Stats st = th.st;
    int above = th.above;
    join_lanes<32>(st, above);
    if (lane == 0) {
        stats[warp] = st;
        aboves[warp] = above;
    }
    if (top) {
        Key best = 0;
        if (th.best_chunk < row.c_hi) best = best_of(row, th.best_chunk);
        lists[warp][lane] = warp_sort(best);
        if (threadIdx.x < kTop) {
            owner[threadIdx.x] = -1;
            found[threadIdx.x] = 0;
        }
        if (threadIdx.x == 0) threshold = 0;
    }
    __syncthreads();
    if (warp == 0) {
        st = stats[lane % kWarps];
        above = aboves[lane % kWarps];
        join_lanes<kWarps>(st, above);
        if (lane == 0) {
            all = st;
            all_above = above;
        }
    }

    // --------------------------------------------------- the share's largest
    if (top) {
        const Key k = lists[warp][lane];
        const int rank = k ? rank_of<kWarps>(k, warp, lane, lists) : kTop;
        if (rank < a.k) {
            // the thread whose chunk holds that logit
            owner[rank] = ((id_of(k) + row.off) / N - row.c_lo) % kThreads;
            if (rank == a.k - 1) threshold = k;
        }
        __syncthreads();
        const Key least = threshold;
        __syncthreads();  // the lists are written again
        Key mine = 0, worst = 0;  // this warp's largest, lane i the i-th; the k-th of them
        for (int o = warp; o < a.k; o += kWarps) {
            const int t = owner[o];
            if (t < 0) break;
            const int n = (row.c_hi - row.c_lo - t + kThreads - 1) / kThreads;  // that thread's chunks
            for (int i0 = 0; i0 < n; i0 += 32) {
                const int c = row.c_lo + t + (i0 + lane) * kThreads;
                float v[N];
                const bool has = i0 + lane < n;
                if (has) {
                    Chunk<T> ch;
                    row.load(c, ch);
                    ch.get(v);
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int id = c * N - row.off + i;
                    const Key key = has && id >= row.lo && id < row.hi ? key_of(v[i], id) : 0;
                    unsigned who = __ballot_sync(0xFFFFFFFFu, key && key >= least && key > worst);
                    while (who) {
                        const int src = __ffs(who) - 1;
                        const Key in = __shfl_sync(0xFFFFFFFFu, key, src);
                        const int at = __popc(__ballot_sync(0xFFFFFFFFu, mine > in));
                        const Key up = __shfl_up_sync(0xFFFFFFFFu, mine, 1);
                        mine = lane == at ? in : lane > at ? up : mine;
                        worst = __shfl_sync(0xFFFFFFFFu, mine, a.k - 1);
                        who &= who - 1;
                        who &= __ballot_sync(0xFFFFFFFFu, key > worst);
                    }
                }
            }
        }
        lists[warp][lane] = mine;
        __syncthreads();
        const int place = mine ? rank_of<kWarps>(mine, warp, lane, lists) : kTop;
        if (place < a.k) found[place] = mine;
    }

    // --------------------------------------------------------- the whole row
    cg::cluster_group cl = cg::this_cluster();
    if (parts > 1) cl.sync();
    else __syncthreads();
    if (part == 0) {
        if (parts > 1) {  // the shares' results into this CTA's shared memory
            if (warp < parts) {
                if (top) lists[warp][lane] = *cl.map_shared_rank(&found[lane], warp);
                if (lane == 0) {
                    stats[warp] = *cl.map_shared_rank(&all, warp);
                    aboves[warp] = *cl.map_shared_rank(&all_above, warp);
                }
            } else {
                if (top) lists[warp][lane] = 0;
                if (lane == 0) {
                    stats[warp] = Stats{-INFINITY, 0.f, 0.f};
                    aboves[warp] = 0;
                }
            }
            __syncthreads();
        }
        Stats s = all;
        int n = all_above;
        if (parts > 1) {
            s = stats[lane % kWarps];
            n = aboves[lane % kWarps];
            join_lanes<kWarps>(s, n);
            s.c = __shfl_sync(0xFFFFFFFFu, s.c, 0);
            s.s = __shfl_sync(0xFFFFFFFFu, s.s, 0);
            s.t = __shfl_sync(0xFFFFFFFFu, s.t, 0);
        }
        const float ls = log2f(s.s);
        const bool nan = s.s != s.s, none = s.c == -INFINITY && !nan;
        auto logp = [&](float x) {
            return nan ? NAN : x == -INFINITY ? -INFINITY : (x - s.c) - kLn2 * ls;
        };
        if (threadIdx.x == 0) {
            a.logprobs[r] = given ? logp(xt) : 0.f;
            a.entropy[r] = nan ? NAN : none ? 0.f : kLn2 * (ls - s.t / s.s);
            a.ranks[r] = !given ? -1 : xt != xt ? 0 : n;
        }
        if (top && warp < parts) {
            const Key k = parts > 1 ? lists[warp][lane] : found[lane];
            const int rank = !k ? kTop : parts > 1 ? rank_of<kWarps>(k, warp, lane, lists) : lane;
            if (rank < a.k) {
                a.top_ids[r * a.k + rank] = id_of(k);
                a.top_values[r * a.k + rank] = logp(value_of(k));
            }
        }
    }
    if (parts > 1) cl.sync();  // shared memory is read until here
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
        cudaLaunchConfig_t cfg{};
        const long long y = std::min<long long>(a.M, 65535);
        cfg.gridDim = dim3((unsigned)parts, (unsigned)y, (unsigned)((a.M + y - 1) / y));
        cfg.blockDim = dim3(kThreads);
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)parts;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, row_kernel<T>, a, dc.err);
        return e == cudaSuccess ? (int)QG_OK : cuda_fail(e);
    });
}

}  // namespace qg
