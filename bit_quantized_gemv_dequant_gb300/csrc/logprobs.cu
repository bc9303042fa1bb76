// token_logprobs: log probabilities of given tokens, entropy, rank and the
// largest alternatives of rows of logits.
#include "serve_common.cuh"

namespace qg {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxTop = 32;

// The order of the logits as an order of whole numbers: larger value first,
// NaN above all, -0 equal to 0; then the lower id.
__device__ __forceinline__ uint32_t value_key(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 + 0 = 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(float v, int id) {
    return (unsigned long long)value_key(v) << 32 | (0xFFFFFFFFu - (uint32_t)id);
}

template <class T, class Op>
__device__ __forceinline__ T block_reduce(T v, Op op, T* scratch) {
    for (int i = 16; i; i >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, i));
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[threadIdx.x % (kThreads / 32)];
    for (int i = 16; i; i >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, i));
    __syncthreads();
    return v;
}

// One CTA per row, one pass per quantity.
template <class T>
__global__ void __launch_bounds__(kThreads) row_kernel(const LogprobArgs a, unsigned* err) {
    __shared__ unsigned long long s64[kThreads / 32];
    __shared__ float sf[kThreads / 32];
    __shared__ int si[kThreads / 32];
    const long long row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.stride;
    const int V = (int)a.V;
    const int64_t target = a.targets[row];
    const bool given = target >= 0 && target < V;
    if (target >= V && threadIdx.x == 0) report_error(err, DEVERR_INDEX);
    const float xt = given ? to_f32(x[target]) : 0.f;
    const uint32_t kt = value_key(xt);
    auto larger = [](unsigned long long p, unsigned long long q) { return p > q ? p : q; };
    auto add = [](float p, float q) { return p + q; };
    float m = -INFINITY;
    bool nan = false;
    int above = 0;
    for (int v = threadIdx.x; v < V; v += kThreads) {
        const float f = to_f32(x[v]);
        nan |= f != f;
        m = fmaxf(m, f);
        above += value_key(f) > kt;
    }
    m = block_reduce(m, [](float p, float q) { return fmaxf(p, q); }, sf);
    nan = __syncthreads_or(nan);
    above = block_reduce(above, [](int p, int q) { return p + q; }, si);
    above /= 32 / (kThreads / 32);  // the second stage counts each warp twice
    float s = 0.f, t = 0.f;
    for (int v = threadIdx.x; v < V; v += kThreads) {
        const float d = to_f32(x[v]) - m;
        const float e = expf(d);
        if (e > 0.f) {
            s += e;
            t += e * d;
        }
    }
    s = block_reduce(s, add, sf) / (32 / (kThreads / 32));
    t = block_reduce(t, add, sf) / (32 / (kThreads / 32));
    const float ln = logf(s);
    const bool none = m == -INFINITY && !nan;
    auto logp = [&](float f) { return nan ? NAN : f == -INFINITY ? -INFINITY : (f - m) - ln; };
    if (threadIdx.x == 0) {
        a.logprobs[row] = given ? logp(xt) : 0.f;
        a.entropy[row] = nan ? NAN : none ? 0.f : ln - t / s;
        a.ranks[row] = given ? above : -1;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < a.k; ++k) {
        unsigned long long best = 0;
        for (int v = threadIdx.x; v < V; v += kThreads) {
            const unsigned long long key = key_of(to_f32(x[v]), v);
            if (key < last && key > best) best = key;
        }
        last = block_reduce(best, larger, s64);
        if (threadIdx.x == 0) {
            const int id = (int)(0xFFFFFFFFu - (uint32_t)last);
            a.top_ids[row * a.k + k] = id;
            a.top_values[row * a.k + k] = logp(to_f32(x[id]));
        }
    }
}

}  // namespace

size_t logprobs_workspace_bytes(const DevCtx&, long long, long long, int) { return 0; }

int logprobs_launch(const DevCtx& dc, const LogprobArgs& a, void*, cudaStream_t s) {
    return by_type(a.dtype, [&](auto t) {
        row_kernel<decltype(t)><<<(unsigned)a.M, kThreads, 0, s>>>(a, dc.err);
        return launched();
    });
}

}  // namespace qg
