// The second kernel of attn_paged, and launches.
#pragma once

#include "attn_work.cuh"

namespace qg {
namespace attn {
namespace {

// Joins the parts of row tiles that a cut fell into. CTA (x, y): the row tile
// that CTA x's note names and its rows R y .. R y + R - 1, one at a time per
// warp. Parts come in the order of the keys: CTA `from`'s, then the first
// segments of the CTAs after it up to x.
constexpr int kJoinThreads = 128;

template <class T, int D, int RT, int R>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Work w) {
    pdl_trigger();
    pdl_wait();
    const Note n = w.notes[blockIdx.x];
    if (n.from < 0) return;
    const int lane = threadIdx.x & 31, x = blockIdx.x;
    for (int r = blockIdx.y * R + (threadIdx.x >> 5); r < (blockIdx.y + 1) * R && n.r0 + r < n.rows;
         r += kJoinThreads / 32) {
        auto slot_of = [&](int k) { return ((long long)k * 2 + (k == n.from ? n.slot : 0)) * RT + r; };
        float m = -INFINITY;
        for (int k = n.from + lane; k <= x; k += 32) m = fmaxf(m, w.ml[slot_of(k)].x);
        for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, i));
        const float ref = m == -INFINITY ? 0.f : m;
        constexpr int E = D / 32;
        using V = std::conditional_t<E == 4, float4, float2>;
        float l = 0.f, v[E] = {};
        for (int k0 = n.from; k0 <= x; k0 += 8) {  // eight parts' loads at a time
            float2 ml[8];
            V o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const long long sl = slot_of(min(k0 + i, x));
                ml[i] = w.ml[sl];
                o[i] = *reinterpret_cast<const V*>(w.part + sl * D + lane * E);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = k0 + i <= x ? ex2(ml[i].x - ref) : 0.f;
                l += ml[i].y * f;
                const float* e = reinterpret_cast<const float*>(&o[i]);
#pragma unroll
                for (int j = 0; j < E; ++j) v[j] += e[j] * f;
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int row = n.r0 + r;
        const long long at = n.out_row + (long long)(row / w.group) * w.a.hq + n.head + row % w.group;
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(w.a.out) + at * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) out[e / 2] = pack2<T>(v[e] * inv, v[e + 1] * inv);
        if (w.a.lse && lane == 0) w.a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
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

template <class T, int D, int RT, int R>
int launch_join(const Work& w, cudaStream_t s) {
    return launch(join_kernel<T, D, RT, R>, dim3(w.ctas, RT / R), kJoinThreads, 0, s, w);
}

}  // namespace
}  // namespace attn
}  // namespace qg
