// The second kernel of attn_paged, and launches.
#pragma once

#include "attn_work.cuh"

namespace qg {
namespace attn {
namespace {

// Joins the parts of row tiles that a cut fell into. CTA (x, y): the row tile
// that CTA x's note names and its rows R y .. R y + R - 1, ROWS of them at a
// time per warp. Parts come in the order of the keys: CTA `from`'s, then the
// first segments of the CTAs after it up to x. Bound by the latency of its
// loads, hence PARTS parts (many for short tiles that are cut finely, two for
// tall ones) and ROWS rows under way at once.
constexpr int kJoinThreads = 128;

template <class T, int D, int RT, int R, int ROWS, int PARTS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Work w) {
    static_assert(R == ROWS * (kJoinThreads / 32), "one round per warp");
    pdl_trigger();
    pdl_wait();
    const Note n = w.notes[blockIdx.x];
    const int lane = threadIdx.x & 31, x = blockIdx.x, r0 = blockIdx.y * R + (threadIdx.x >> 5) * ROWS;
    if (n.from < 0 || n.r0 + r0 >= n.rows) return;
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
    for (int k0 = n.from; k0 <= x; k0 += PARTS) {
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
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = n.r0 + r0 + i;
        if (row >= n.rows) break;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const long long at = n.out_row + (long long)(row / w.group) * w.a.hq + n.head + row % w.group;
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(w.a.out) + at * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) out[e / 2] = pack2<T>(v[i][e] * inv, v[i][e + 1] * inv);
        if (w.a.lse && lane == 0) w.a.lse[at] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994531f;
    }
}

template <class K, class... A>
int launch(K kern, dim3 grid, int threads, int smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

template <class T, int D, int RT, int ROWS, int PARTS>
int launch_join(const Work& w, cudaStream_t s) {
    constexpr int R = ROWS * (kJoinThreads / 32);
    return launch(join_kernel<T, D, RT, R, ROWS, PARTS>, dim3(w.ctas, RT / R), kJoinThreads, 0, s, w);
}

}  // namespace
}  // namespace attn
}  // namespace qg
