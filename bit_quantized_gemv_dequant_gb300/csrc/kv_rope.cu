// kv_append_rope: queries and keys rotated by their positions, keys and values
// into their pages.
#include <algorithm>

#include "fp8_tc.cuh"
#include "row8.cuh"

namespace qg {
namespace {

// The angle position * inv_freq, exactly, as a fraction of a turn. A float is
// m 2^e with whole m, so f / 2 pi is m times the bits of 1 / 2 pi, shifted. Of
// that only the 64 bits after the point matter, since positions are whole: times
// the position modulo 2^64 they are the angle's fraction to position * 2^-64 of a
// turn. (In f32 the angle of position 10^6 would be off by 0.03; f64 has few units.)
__device__ __forceinline__ uint64_t turn_fraction(float f) {
    // 1 / 2 pi = 0x.28BE60DB9391054A 7F09D5F47D4D3770...
    constexpr uint64_t kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;
    const uint32_t bits = __float_as_uint(f);
    const int e = (bits >> 23) & 0xFF;
    const uint64_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    // m (kHi 2^64 + kLo) in three words; the point lies 128 bits up, then e - 150.
    const uint64_t w0 = m * kLo, c = __umul64hi(m, kLo), t = m * kHi;
    const uint64_t w1 = t + c, w2 = __umul64hi(m, kHi) + (w1 < t);
    const int up = (e ? e : 1) - 150;  // the 64 bits below the point, of (w2 w1 w0) << up
    uint64_t r;
    if (up <= -128) r = 0;
    else if (up <= -64) r = w2 >> (-64 - up);
    else if (up < 0) r = (w2 << (64 + up)) | (w1 >> -up);
    else if (up == 0) r = w1;
    else if (up < 64) r = (w1 << up) | (w0 >> (64 - up));
    else r = up < 128 ? w0 << (up - 64) : 0;
    return bits >> 31 ? 0 - r : r;
}

// Cosine and sine of a fraction of a turn (2^-64 each), as the f32 nearest to its number of
// half turns between -1 and 1: 2^-24 of the angle, however small it is.
__device__ __forceinline__ float2 cos_sin(uint64_t fraction) {
    float s, c;
    sincospif(__ll2float_rn((int64_t)fraction) * 0x1p-63f, &s, &c);
    return make_float2(c, s);
}

constexpr int kThreads = 128;

// A block takes a token: its angles into shared memory (one for all heads), then the
// heads of q, k and v one after the other, a head by the threads of one threadIdx.y.
// Bound by the bytes of q, k and v, once each, next to instruction issue; a thread has
// the loads of kBatch heads under way, the first ones while the angles are worked out.
//
// PAIRED: 16 values of a head per thread, both members of eight pairs (or two runs
// of eight that are not turned), so a pair's angle is read and its place worked out
// once: 8192 tokens, 32 and 8 heads of 128, bf16: 34.5 us, 5.8 TB/s; 57 with eight values
// per thread, whose partners were loaded a second time. It needs D a multiple of 16 and
// pairs that lie apart by a multiple of eight; in other heads a run of eight has partners in
// two runs, so they are turned value by value, each loading its partner by itself (4096
// tokens, 36 of 128 values turned: 34 us for 17).
//
// Angle i lies at chunk (i % 8) / 2, place i / 8: threads beside each other, whose values
// are beside each other, read 16-byte words beside each other.
template <class TX, class TC, bool VEC, bool INTER, bool PAIRED>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const RopeArgs a, unsigned* err) {
    constexpr int kRuns = PAIRED ? 2 : 1;  // of eight values per thread and head
    constexpr int kBatch = sizeof(TX) == 4 ? 2 : 3;
    extern __shared__ __align__(16) float2 angles[];  // [4][places][2]
    const int n = a.rot / 2, places = (n + 7) / 8;
    const long long t = blockIdx.x;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    const int D = a.d, heads = a.hq + 2 * a.hkv, x = threadIdx.x;
    // Where this thread's runs begin: threads below n / 8 have the pairs that lie apart.
    const bool apart = PAIRED && !INTER && x < n / 8;
    const int d0 = !PAIRED || apart ? x * 8 : x * 16, d1 = apart ? d0 + n : d0 + 8;

    // Head h of those of q, k and v.
    auto source = [&](int h) {
        const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + a.hkv;
        const int skip = is_q ? 0 : is_k ? a.hq : a.hq + a.hkv;
        return static_cast<const TX*>(is_q ? a.q : is_k ? a.k : a.v) +
               t * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) + (h - skip) * D;
    };
    Raw8<TX> raw[kBatch][kRuns];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = h0 + i * blockDim.y;
            if (h >= heads) continue;
            const TX* src = source(h);
            raw[i][0] = load8<TX, VEC>(src + d0, 8);
            if constexpr (PAIRED) raw[i][1] = load8<TX, VEC>(src + d1, 8);
        }
    };
    // (cos, sin) of pairs p and p + 1, p even
    auto two_angles = [&](int p) { return reinterpret_cast<const float4*>(angles)[p % 8 / 2 * places + p / 8]; };

    fp8::pdl_wait();
    fp8::pdl_trigger();
    load(threadIdx.y);
    const int64_t slot = a.slots[t], page = slot >> (31 - __clz(a.page_size));
    const bool none = slot < 0 || page >= a.num_pages;
    const long long place = (page * a.hkv * a.page_size + (slot & (a.page_size - 1))) * D;  // of head 0
    for (int j = tid; j < n; j += threads)
        angles[(j % 8 / 2 * places + j / 8) * 2 + j % 2] = cos_sin(turn_fraction(a.inv_freq[j]) * (uint64_t)a.positions[t]);
    if (tid == 0 && page >= a.num_pages) report_error(err, DEVERR_INDEX);
    __syncthreads();

    for (int h0 = threadIdx.y; h0 < heads; h0 += kBatch * blockDim.y, load(h0)) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int h = h0 + b * blockDim.y;
            if (h >= heads) break;
            float y[kRuns][8];
#pragma unroll
            for (int r = 0; r < kRuns; ++r) to_f32(raw[b][r], y[r]);
            if (h >= a.hq + a.hkv) {
            } else if (INTER) {
#pragma unroll
                for (int r = 0; r < kRuns; ++r)
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const int p = (d0 + r * 8 + i) / 2;
                        if (p >= n) continue;
                        const float4 v = two_angles(p);
                        const float* f = &y[r][i];
                        const float o[4] = {fmaf(f[1], -v.y, f[0] * v.x), fmaf(f[0], v.y, f[1] * v.x),
                                            fmaf(f[3], -v.w, f[2] * v.z), fmaf(f[2], v.w, f[3] * v.z)};
                        y[r][i] = o[0];
                        y[r][i + 1] = o[1];
                        if (p + 1 < n) {
                            y[r][i + 2] = o[2];
                            y[r][i + 3] = o[3];
                        }
                    }
            } else if constexpr (PAIRED) {
                if (apart) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float4 v = two_angles(d0 + i);
                        const float2 c = make_float2(v.x, v.z), s = make_float2(v.y, v.w);
                        const float2 p = make_float2(y[0][i], y[0][i + 1]), q = make_float2(y[1][i], y[1][i + 1]);
                        const float2 u = __ffma2_rn(make_float2(-q.x, -q.y), s, __fmul2_rn(p, c));
                        const float2 w = __ffma2_rn(p, s, __fmul2_rn(q, c));
                        y[0][i] = u.x;
                        y[0][i + 1] = u.y;
                        y[1][i] = w.x;
                        y[1][i + 1] = w.y;
                    }
                }
            } else {
                const TX* src = source(h);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int d = d0 + i;
                    if (d < a.rot) {
                        const bool second = d >= n;
                        const int p = second ? d - n : d;
                        const float2 cs = angles[(p % 8 / 2 * places + p / 8) * 2 + p % 2];
                        const float o = to_f32(src[second ? p : d + n]);
                        y[0][i] = fmaf(o, second ? cs.y : -cs.y, y[0][i] * cs.x);
                    }
                }
            }
            TC* dst;
            if (h < a.hq) {
                dst = static_cast<TC*>(a.q_out) + (t * a.hq + h) * D;
            } else {
                if (none) continue;
                const bool is_k = h < a.hq + a.hkv;
                const long long at = h - a.hq - (is_k ? 0 : a.hkv);
                dst = static_cast<TC*>(is_k ? a.k_cache : a.v_cache) + place + at * a.page_size * D;
            }
            store8<TC, true>(dst + d0, y[0], 8);
            if constexpr (PAIRED) store8<TC, true>(dst + d1, y[1], 8);
        }
    }
}

}  // namespace

int kv_append_rope_launch(const DevCtx& dc, const RopeArgs& a, cudaStream_t s) {
    const int n = a.rot / 2;
    const bool paired = a.d % 16 == 0 && (a.interleaved || n % 8 == 0);
    const int cols = a.d / (paired ? 16 : 8), rows = std::max(1, kThreads / cols);
    const size_t smem = (size_t)((n + 7) / 8) * 64;
    return by_type(a.x_dtype, [&](auto tx) {
        using TX = decltype(tx);
        const int es = sizeof(TX);
        const bool vec = (!a.q || in_eights(a.q, a.q_stride, a.d, es)) && in_eights(a.k, a.k_stride, a.d, es) &&
                         in_eights(a.v, a.v_stride, a.d, es);
        return by_type(a.cache_dtype, [&](auto tc) {
            using TC = decltype(tc);
            if constexpr (sizeof(TC) == 2) {
                auto pick = [&](auto inter, auto pairs) {
                    constexpr bool I = decltype(inter)::value, P = decltype(pairs)::value;
                    return vec ? rope_kernel<TX, TC, true, I, P> : rope_kernel<TX, TC, false, I, P>;
                };
                using Yes = std::true_type;
                using No = std::false_type;
                auto kern = a.interleaved ? (paired ? pick(Yes{}, Yes{}) : pick(Yes{}, No{}))
                                          : (paired ? pick(No{}, Yes{}) : pick(No{}, No{}));
                return launch_after(kern, dim3((unsigned)a.tokens), dim3(cols, rows), smem, s, a, dc.err);
            } else {
                return (int)QG_ERR_INVALID_ARG;
            }
        });
    });
}

}  // namespace qg
