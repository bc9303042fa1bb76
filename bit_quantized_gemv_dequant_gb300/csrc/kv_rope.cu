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

// Cosine and sine of a fraction of a turn (2^-64 each). The nearest of +-1/2 turn
// as f32: 2^-24 of the angle, and 2^-33 of a turn where it is small.
__device__ __forceinline__ float2 cos_sin(uint64_t fraction) {
    float s, c;
    sincospif((float)(int32_t)(fraction >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c, s);
}

constexpr int kAngles = 256;  // angles of a block's tokens, if it has several
constexpr int kTokens = 8;    // tokens of a block at most

// A block of (D / 8) x rows threads takes `per` tokens: their angles into shared
// memory (one for all heads), then eight values of a head per thread, the heads of
// q, k and v one after the other. Bound by the bytes of q, k and v, once each.
// Angle i of a token lies at chunk (i % 8) / 2, place i / 8: threads beside each
// other, whose values are beside each other, read 16-byte words beside each other.
template <class TX, class TC, bool VEC, bool INTER>
__global__ void __launch_bounds__(1024) rope_kernel(const RopeArgs a, const int per, unsigned* err) {
    extern __shared__ float2 angles[];  // [per][4][places][2]
    const int n = a.rot / 2, places = (n + 7) / 8;
    const long long t0 = (long long)blockIdx.x * per;
    const int tokens = (int)min((long long)per, a.tokens - t0);
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    fp8::pdl_wait();
    fp8::pdl_trigger();
    for (int i = tid; i < tokens * n; i += threads) {
        const int t = i / n, j = i - t * n;
        angles[((t * 4 + j % 8 / 2) * places + j / 8) * 2 + j % 2] =
            cos_sin(turn_fraction(a.inv_freq[j]) * (uint64_t)a.positions[t0 + t]);
    }
    __syncthreads();

    const int d0 = threadIdx.x * 8, D = a.d;
    const int log_page = 31 - __clz(a.page_size);
    const int heads = a.hq + 2 * a.hkv;
    for (int t = 0; t < tokens; ++t) {
        const int64_t slot = a.slots[t0 + t];
        const int64_t page = slot >> log_page;
        const bool bad = page >= a.num_pages;
        if (bad && tid == 0) report_error(err, DEVERR_INDEX);
        for (int h = threadIdx.y; h < heads; h += blockDim.y) {
            const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + a.hkv;
            const int head = is_q ? h : is_k ? h - a.hq : h - a.hq - a.hkv;
            const TX* src = static_cast<const TX*>(is_q ? a.q : is_k ? a.k : a.v) +
                            (t0 + t) * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) + (long long)head * D;
            float x[8], y[8];
            to_f32(load8<TX, VEC>(src + d0, 8), x);
            if ((is_q || is_k) && d0 < a.rot) {
                if constexpr (INTER) {
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {  // pairs p and p + 1
                        const int p = d0 / 2 + i;
                        const float4 v = p < n ? reinterpret_cast<const float4*>(angles)[(t * 4 + p % 8 / 2) * places + p / 8]
                                               : make_float4(1.f, 0.f, 1.f, 0.f);
                        y[2 * i] = fmaf(x[2 * i + 1], -v.y, x[2 * i] * v.x);
                        y[2 * i + 1] = fmaf(x[2 * i], v.y, x[2 * i + 1] * v.x);
                        y[2 * i + 2] = fmaf(x[2 * i + 3], -v.w, x[2 * i + 2] * v.z);
                        y[2 * i + 3] = fmaf(x[2 * i + 2], v.w, x[2 * i + 3] * v.z);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (d0 + i >= a.rot) y[i] = x[i];
                } else if (n % 8 == 0) {  // all eight are first members of their pairs, or all second ones
                    const bool second = d0 >= n;
                    const int p0 = second ? d0 - n : d0;
                    float o[8];
                    to_f32(load8<TX, VEC>(src + (second ? p0 : d0 + n), 8), o);
                    const float4* cs = reinterpret_cast<const float4*>(angles) + t * 4 * places + p0 / 8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = cs[i * places];
                        const float s0 = second ? v.y : -v.y, s1 = second ? v.w : -v.w;
                        y[2 * i] = fmaf(o[2 * i], s0, x[2 * i] * v.x);
                        y[2 * i + 1] = fmaf(o[2 * i + 1], s1, x[2 * i + 1] * v.z);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int d = d0 + i;
                        y[i] = x[i];
                        if (d < a.rot) {
                            const bool second = d >= n;
                            const int p = second ? d - n : d;
                            const float2 cs = angles[((t * 4 + p % 8 / 2) * places + p / 8) * 2 + p % 2];
                            const float o = to_f32(src[second ? p : d + n]);
                            y[i] = fmaf(o, second ? cs.y : -cs.y, x[i] * cs.x);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = x[i];
            }
            TC* dst;
            if (is_q) {
                dst = static_cast<TC*>(a.q_out) + ((t0 + t) * a.hq + head) * D;
            } else {
                if (slot < 0 || bad) continue;
                dst = static_cast<TC*>(is_k ? a.k_cache : a.v_cache) +
                      ((page * a.hkv + head) * a.page_size + (slot & (a.page_size - 1))) * D;
            }
            store8<TC, true>(dst + d0, y, 8);
        }
    }
}

}  // namespace

int kv_append_rope_launch(const DevCtx& dc, const RopeArgs& a, cudaStream_t s) {
    const int cols = a.d / 8, rows = std::max(1, 256 / cols), n = a.rot / 2;
    // Enough tokens for an angle per thread, but first a block for every SM.
    const long long per = std::max<long long>(
        1, std::min<long long>(std::min(kAngles / n, kTokens), (a.tokens + dc.num_sms - 1) / dc.num_sms));
    const long long grid = (a.tokens + per - 1) / per;
    if (grid > 0x7FFFFFFFLL) return QG_ERR_UNSUPPORTED;
    const size_t smem = (size_t)per * ((n + 7) / 8) * 64;
    return by_type(a.x_dtype, [&](auto tx) {
        using TX = decltype(tx);
        const int es = sizeof(TX);
        const bool vec = (!a.q || in_eights(a.q, a.q_stride, a.d, es)) && in_eights(a.k, a.k_stride, a.d, es) &&
                         in_eights(a.v, a.v_stride, a.d, es);
        return by_type(a.cache_dtype, [&](auto tc) {
            using TC = decltype(tc);
            if constexpr (sizeof(TC) == 2) {
                auto kern = a.interleaved ? (vec ? rope_kernel<TX, TC, true, true> : rope_kernel<TX, TC, false, true>)
                                          : (vec ? rope_kernel<TX, TC, true, false> : rope_kernel<TX, TC, false, false>);
                return launch_after(kern, dim3((unsigned)grid), dim3(cols, rows), smem, s, a, (int)per, dc.err);
            } else {
                return (int)QG_ERR_INVALID_ARG;
            }
        });
    });
}

}  // namespace qg
