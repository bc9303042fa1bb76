// attn_paged: attention of new tokens over a paged cache.
#include "serve_common.cuh"

namespace qg {
namespace {

constexpr int kWarps = 4;

// One warp per (token, head), one key at a time: lane l holds D / 32 columns
// of q and of the output, and the running maximum m and sum l of the softmax
// rescale the output when m grows.
template <class T, int D>
__global__ void __launch_bounds__(kWarps * 32)
    row_kernel(const AttnArgs a, unsigned* err) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= (long long)a.tokens * a.hq) return;
    const int t = (int)(unit / a.hq), h = (int)(unit % a.hq), hk = h / (a.hq / a.hkv);
    int b = -1, first = 0, n = 0;
    for (int i = 0; i < a.batch; ++i) {
        const int lo = a.offsets[i], hi = a.offsets[i + 1];
        if (lo < 0 || hi < lo || hi > a.tokens) {
            report_error(err, DEVERR_INDEX);
            return;
        }
        if (t >= lo && t < hi) {
            b = i;
            first = lo;
            n = hi - lo;
            break;
        }
    }
    if (b < 0) return;
    if (t - first >= a.max_new) {
        if (lane == 0) report_error(err, DEVERR_INDEX);
        return;
    }
    int len = a.ctx[b];
    if (len < 0 || len > (long long)a.width * a.page_size) {
        if (lane == 0) report_error(err, DEVERR_INDEX);
        len = max(0, min(len, a.width * a.page_size));
    }
    const int pos = len - n + (t - first);
    const T* qp = static_cast<const T*>(a.q) + t * a.q_stride + (long long)h * D + lane * E;
    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = to_f32(qp[e]);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = a.window ? max(0, pos - a.window + 1) : 0; j <= pos; ++j) {
        const int page = a.table[(long long)b * a.width + j / a.page_size];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) report_error(err, DEVERR_INDEX);
            continue;
        }
        const long long at = (((long long)page * a.hkv + hk) * a.page_size + j % a.page_size) * D + lane * E;
        const T* kp = static_cast<const T*>(a.k) + at;
        const T* vp = static_cast<const T*>(a.v) + at;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x = fmaf(q[e], to_f32(kp[e]), x);
        for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, i);
        x *= a.scale;
        if (a.softcap > 0.f) x = tanhf(x / a.softcap) * a.softcap;
        const float top = fmaxf(m, x);
        const float keep = top == -INFINITY ? 0.f : expf(m - top), p = top == -INFINITY ? 0.f : expf(x - top);
        l = l * keep + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * keep + p * to_f32(vp[e]);
        m = top;
    }
    T* op = static_cast<T*>(a.out) + unit * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) op[e] = from_f32<T>(l > 0.f ? o[e] / l : 0.f);
    if (a.lse && lane == 0) a.lse[unit] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t attn_workspace_bytes(const DevCtx&, const AttnArgs&) { return 0; }

int attn_launch(const DevCtx& dc, const AttnArgs& a, void*, size_t, cudaStream_t s) {
    const unsigned grid = (unsigned)(((long long)a.tokens * a.hq + kWarps - 1) / kWarps);
    return by_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        if constexpr (sizeof(T) == 2) {
            if (a.d == 64) row_kernel<T, 64><<<grid, kWarps * 32, 0, s>>>(a, dc.err);
            else row_kernel<T, 128><<<grid, kWarps * 32, 0, s>>>(a, dc.err);
            return launched();
        } else {
            return (int)QG_ERR_INVALID_ARG;
        }
    });
}

}  // namespace qg
