// The second kernel of attn_paged, and launches.
#pragma once

#include "attn_work.cuh"

namespace qg {
namespace attn {
namespace {

constexpr int kJoinThreads = 128;

template <int N>
__device__ __forceinline__ bool all_finite(const float (&v)[N]) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) z = fmaf(v[i], 0.f, z);
    return z == z;
}

// One row of out by a warp, from the keys that it sees alone.
//
// In a product of tiles a key that a row does not see enters with the
// probability 0, and 0 times a value that is infinite or NaN is NaN. Values that
// no row of the tile sees are cleared before the product; where some rows see a
// key and some do not, an output that is not finite is found out here: either it
// stays so, or it came from values that the row does not see. Lane = key for
// the scores, columns for the output.
template <class T, int D>
__device__ __forceinline__ void redo_row(const Work& w, int b, int head, int r) {
    const Seq s = seq_at(w, b);
    const int lane = threadIdx.x & 31, tok = r / w.group, pos = s.ctx - s.n + tok;
    const int h = head * w.group + r % w.group, from = w.a.window && pos >= w.a.window ? pos - w.a.window + 1 : 0;
    const T* q = static_cast<const T*>(w.a.q) + (long long)(s.first + tok) * w.a.q_stride + (long long)h * D;
    constexpr int E = D / 32;
    float m = -INFINITY, l = 0.f, acc[E] = {};
    for (int j0 = from; j0 <= pos; j0 += 32) {
        const int j = j0 + lane;
        float x = -INFINITY;
        int page = w.a.num_pages;
        if (j <= pos) {
            page = page_of(w, b, j);
            float dot = 0.f;
            if (page < w.a.num_pages) {
                const T* k = static_cast<const T*>(w.a.k) +
                             (((long long)page * w.a.hkv + head) * w.a.page_size + j % w.a.page_size) * D;
                for (int c = 0; c < D; c += 2) {
                    const float2 a = unpack2<T>(*reinterpret_cast<const uint32_t*>(q + c));
                    const float2 e = unpack2<T>(*reinterpret_cast<const uint32_t*>(k + c));
                    dot = fmaf(a.x, e.x, fmaf(a.y, e.y, dot));
                }
            }
            const float2 z = make_float2(dot, 0.f);
            x = (w.a.softcap > 0.f ? score2<true>(w, z) : score2<false>(w, z)).x;
        }
        float top = x;
#pragma unroll
        for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
        const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn, keep = ex2(m - ref), p = ex2(x - ref);
        m = mn;
        l *= keep;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= keep;
        for (int i = 0; i < min(32, pos - j0 + 1); ++i) {
            const float pi = __shfl_sync(0xFFFFFFFFu, p, i);
            const int at = __shfl_sync(0xFFFFFFFFu, page, i);
            l += pi;
            if (at == w.a.num_pages) continue;
            const T* v = static_cast<const T*>(w.a.v) +
                         (((long long)at * w.a.hkv + head) * w.a.page_size + (j0 + i) % w.a.page_size) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 f = unpack2<T>(*reinterpret_cast<const uint32_t*>(v + e));
                acc[e] = fmaf(pi, f.x, acc[e]);
                acc[e + 1] = fmaf(pi, f.y, acc[e + 1]);
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long at = (long long)(s.first + tok) * w.a.hq + h;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(w.a.out) + at * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) out[e / 2] = pack2<T>(acc[e] * inv, acc[e + 1] * inv);
}

// Looks through rows r0 .. r1 - 1 of a sequence and key head, then through those
// that the main kernel's CTA of this number finished alone (if its note says
// that some are not finite), for rows to be done again; warp `warp` of `warps`.
template <class T, int D, int RT, int KT>
__device__ __noinline__ void redo_rows(const Work& w, int b, int head, int r0, int r1, int warp, int warps) {
    const Note& n = w.notes[blockIdx.x];
    Walk<RT, KT> walk(w, Place{n.first_b, n.first_head, n.first_tile, n.first_at},
                      n.bad ? seq_at(w, n.first_b) : Seq{}, n.bad ? n.steps : 0);
    const int lane = threadIdx.x & 31;
    int at = r0, step = 1;
    __syncwarp();  // the warp wrote r0 .. r1 - 1 itself
    for (;;) {
        for (; at < r1; at += step) {
            const Seq s = seq_at(w, b);
            const long long row = (long long)(s.first + at / w.group) * w.a.hq + head * w.group + at % w.group;
            float v[D / 32];
#pragma unroll
            for (int e = 0; e < D / 32; ++e) v[e] = to_f32(static_cast<const T*>(w.a.out)[row * D + e * 32 + lane]);
            if (!__all_sync(0xFFFFFFFFu, all_finite(v))) redo_row<T, D>(w, b, head, at);
        }
        do {
            if (!walk.next()) return;
        } while (!walk.whole);
        b = walk.p.b;
        head = walk.p.head;
        at = walk.p.tile * RT + warp;
        r1 = min(walk.s.rows, walk.p.tile * RT + RT);
        step = warps;
    }
}

// Joins the parts of row tiles that a cut fell into. CTA (x, y): the row tile
// that CTA x's note names and its rows R y .. R y + R - 1, ROWS of them at a
// time per warp. Parts come in the order of the keys: CTA `from`'s, then the
// first segments of the CTAs after it up to x. Bound by the latency of its
// loads, hence PARTS parts (many for short tiles that are cut finely, two for
// tall ones) and ROWS rows under way at once.
//
// REDO: rows of a tile may see different keys (sequences with several new
// tokens). Without it the kernel has none of that code, which cost 1.2 of 9.5 us
// with one token over 700 keys.
template <class T, int D, int RT, int KT, int R, int ROWS, int PARTS, bool REDO>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Work w) {
    static_assert(R == ROWS * (kJoinThreads / 32), "one round per warp");
    pdl_wait();
    pdl_trigger();
    const Note n = w.notes[blockIdx.x];
    const int lane = threadIdx.x & 31, x = blockIdx.x, r0 = blockIdx.y * R + (threadIdx.x >> 5) * ROWS;
    const bool mine = n.from >= 0 && n.r0 + r0 < n.rows;
    if (!mine && !(REDO && n.bad)) return;
    constexpr int E = D / 32;
    using V = std::conditional_t<E == 4, float4, float2>;
    float m[ROWS], l[ROWS], v[ROWS][E];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[i][e] = 0.f;
    }
    // The running maximum rescales what is there, as in the kernels.
    for (int k0 = mine ? n.from : x + 1; k0 <= x; k0 += PARTS) {
        float2 ml[ROWS][PARTS];
        V o[ROWS][PARTS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int j = 0; j < PARTS; ++j) {
                const int k = min(k0 + j, x);
                // rows past the last have parts too, of whatever is there
                const long long at = ((long long)k * 2 + (k == n.from ? n.slot : 0)) * RT + r0 + i;
                ml[i][j] = w.ml[at];
                o[i][j] = *reinterpret_cast<const V*>(w.part + at * D + lane * E);
            }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            float top = m[i];
#pragma unroll
            for (int j = 0; j < PARTS; ++j)
                if (k0 + j <= x) top = fmaxf(top, ml[i][j].x);
            const float ref = top == -INFINITY ? 0.f : top, keep = ex2(m[i] - ref);
            m[i] = top;
            l[i] *= keep;
#pragma unroll
            for (int e = 0; e < E; ++e) v[i][e] *= keep;
#pragma unroll
            for (int j = 0; j < PARTS; ++j) {
                if (k0 + j > x) continue;
                const float f = ex2(ml[i][j].x - ref);
                l[i] += ml[i][j].y * f;
                const float* p = reinterpret_cast<const float*>(&o[i][j]);
#pragma unroll
                for (int e = 0; e < E; ++e) v[i][e] += p[e] * f;
            }
        }
    }
    bool redo = n.bad;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = n.r0 + r0 + i;
        if (!mine || row >= n.rows) break;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const long long at = n.out_row + (long long)(row / w.group) * w.a.hq + n.head + row % w.group;
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(w.a.out) + at * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) out[e / 2] = pack2<T>(v[i][e] * inv, v[i][e + 1] * inv);
        if (w.a.lse && lane == 0) w.a.lse[at] = l[i] == 0.f ? -INFINITY : fmaf(m[i], w.to_ln, logf(l[i]));
        redo |= l[i] == l[i] && !all_finite(v[i]);
    }
    if constexpr (REDO) {
        if (__any_sync(0xFFFFFFFFu, redo))  // the note says nothing of rows if none are this warp's
            redo_rows<T, D, RT, KT>(w, mine ? n.b : 0, mine ? n.head / w.group : 0, mine ? n.r0 + r0 : 0,
                                    mine ? min(n.rows, n.r0 + r0 + ROWS) : 0,
                                    blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5),
                                    gridDim.y * (kJoinThreads / 32));
    }
}

template <class K, class... A>
int launch(bool overlap, K kern, dim3 grid, int threads, int smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

template <class T, int D, int RT, int KT, int ROWS, int PARTS>
int launch_join(const Work& w, cudaStream_t s) {
    constexpr int R = ROWS * (kJoinThreads / 32);
    return w.a.max_new > 1
               ? launch(true, join_kernel<T, D, RT, KT, R, ROWS, PARTS, true>, dim3(w.ctas, RT / R), kJoinThreads, 0, s, w)
               : launch(true, join_kernel<T, D, RT, KT, R, ROWS, PARTS, false>, dim3(w.ctas, RT / R), kJoinThreads, 0, s, w);
}

}  // namespace
}  // namespace attn
}  // namespace qg
