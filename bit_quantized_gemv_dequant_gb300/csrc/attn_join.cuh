// The second kernel of attn_paged, and launches.
#pragma once

#include "attn_work.cuh"

namespace qg {
namespace attn {
namespace {

// Joins the parts of row tiles that a cut fell into. CTA (x, y): cut x + 1 of
// the line, if it is the first inside its row tile, and rows R y .. R y + R - 1,
// one at a time per warp. Parts come in the order of the keys.
constexpr int kJoinThreads = 128;

template <class T, int D, int RT, int KT, int R>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Work w) {
    __shared__ long long scratch[kJoinThreads / 32 + 4];
    pdl_trigger();
    pdl_wait();
    long long total;
    locate<RT, KT, kJoinThreads>(w, -1, &total, scratch);
    const int c = blockIdx.x + 1;
    const long long at = cut(total, c, w.ctas);
    if (at >= total || at == cut(total, c - 1, w.ctas)) return;
    const Place p = locate<RT, KT, kJoinThreads>(w, at, &total, scratch);
    if (p.at == 0) return;  // the cut is between two row tiles
    const long long begin = at - p.at;
    // an earlier cut inside the same row tile has done it
    if (cut(total, c - 1, w.ctas) > begin) return;
    const Seq s = seq_at(w, p.b);
    const Span span = span_of<RT, KT>(w, s, p.tile);
    const long long end = begin + span.hi - span.lo;
    const int lane = threadIdx.x & 31;
    // Contributors: CTA c - 1 with its last segment, then CTAs c .. with their first.
    int last = c;
    while (cut(total, last + 1, w.ctas) < end) ++last;
    for (int r = blockIdx.y * R + (threadIdx.x >> 5); r < (blockIdx.y + 1) * R; r += kJoinThreads / 32) {
        const int row = p.tile * RT + r;
        if (row >= s.rows) return;
        auto slot_of = [&](int k) -> long long {
            return ((long long)k * 2 + (k == c - 1 && cut(total, k, w.ctas) < begin ? 1 : 0)) * RT + r;
        };
        auto idle = [&](int k) { return cut(total, k + 1, w.ctas) == cut(total, k, w.ctas); };
        float m = -INFINITY;
        for (int k = c - 1 + lane; k <= last; k += 32)
            if (!idle(k)) m = fmaxf(m, w.ml[slot_of(k)].x);
        for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, i));
        const float ref = m == -INFINITY ? 0.f : m;
        constexpr int E = D / 32;
        float l = 0.f, v[E] = {};
#pragma unroll 4
        for (int k = c - 1; k <= last; ++k) {
            if (idle(k)) continue;
            const long long sl = slot_of(k);
            const float2 p2 = w.ml[sl];
            const float f = ex2(p2.x - ref);
            l += p2.y * f;
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] += w.part[sl * D + lane * E + e] * f;
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const long long o = (long long)(s.first + row / w.group) * w.a.hq + p.head * w.group + row % w.group;
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(w.a.out) + o * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) out[e / 2] = pack2<T>(v[e] * inv, v[e + 1] * inv);
        if (w.a.lse && lane == 0) w.a.lse[o] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
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

template <class T, int D, int RT, int KT, int R>
int launch_join(const Work& w, cudaStream_t s) {
    if (w.ctas == 1) return QG_OK;
    return launch(join_kernel<T, D, RT, KT, R>, dim3(w.ctas - 1, RT / R), kJoinThreads, 0, s, w);
}

}  // namespace
}  // namespace attn
}  // namespace qg
