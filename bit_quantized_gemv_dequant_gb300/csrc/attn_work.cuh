// How attn_paged's work is cut up, and the pieces its kernels share.
//
// The rows of one sequence and key head are its new tokens times the query
// heads of the group, row r = token * group + head, in tiles of RT rows. A row
// tile meets the keys that any of its rows sees in tiles of KT keys. All
// (row tile, key tile) pairs of the batch, in the order sequence, key head,
// row tile, key tile, are one line of W steps; CTA c of G takes the steps
// W c / G .. W (c + 1) / G - 1 (G at most W), so every CTA has the same work to
// within one step whatever the lengths. Where a cut falls inside a row tile its
// parts leave (m, l, O) in the workspace and join_kernel joins them, in the
// order of the keys. A CTA has at most two such parts: its first segment (slot
// 0) and its last (slot 1). The CTA with a row tile's last part notes down
// which one that is and where the parts begin.
#pragma once

#include "fp8_tc.cuh"

namespace qg {
namespace attn {

using fp8::pdl_trigger;
using fp8::pdl_wait;
using prefill::prefetch_tmap;

struct Work {
    AttnArgs a;
    int group;
    float scale_log2;        // scale * log2(e): scores are in base 2
    float to_ln;             // what a score in base 2 is in base e, by the factor as rounded
    float small;             // products up to this in size are far from the cap
    float cap_in, cap_out;   // scale / softcap, softcap * log2(e)
    float* part;             // [G][2][RT][D] unnormalised outputs of cut row tiles
    float2* ml;              // [G][2][RT] their maximum (base 2) and sum
    struct Note* notes;      // [G]
    int ctas;
    unsigned* err;
};

// A row tile that ends in a CTA and was begun in another: CTA `from`, slot `slot`.
struct Note {
    int from, slot;  // from = -1: none
    int bad;         // a row that the CTA finished alone is not finite, though its sum is a number
    int b;           // the tile's sequence
    int out_row;     // row of q and out of the tile's first token's first head
    int rows, r0;    // rows of the sequence, first of the tile
    int head;
    int first_b, first_head, first_tile, first_at;  // the CTA's first step
    long long steps;
};

struct Seq {
    int first, n, rows, ctx;
};

__device__ __forceinline__ Seq seq_at(const Work& w, int b) {
    Seq s;
    const int lo = w.a.offsets[b], hi = w.a.offsets[b + 1];
    s.first = lo;
    s.n = hi - lo;
    s.ctx = w.a.ctx[b];
    bool bad = lo < 0 || hi < lo || hi > w.a.tokens;
    if (bad) s.n = 0;
    const long long most = (long long)w.a.width * w.a.page_size;
    if (s.ctx < 0 || s.ctx > most) {
        bad = true;
        s.ctx = s.ctx < 0 ? 0 : (int)most;
    }
    bad |= s.n > w.a.max_new;
    if (bad) report_error(w.err, DEVERR_INDEX);
    s.rows = min(s.n, w.a.max_new) * w.group;
    return s;
}

// The key tiles [lo, hi) that row tile i meets; its rows see the keys begin ..
// end - 1 and no others. A row tile that sees nothing has one (empty) step.
struct Span {
    int lo, hi, begin, end;
};
template <int RT, int KT>
__device__ __forceinline__ Span span_of(const Work& w, const Seq& s, int i) {
    const int r0 = i * RT, r1 = min(s.rows, r0 + RT) - 1;
    const int first = s.ctx - s.n + r0 / w.group, last = s.ctx - s.n + r1 / w.group;
    Span p;
    p.end = last + 1;
    if (p.end <= 0) return Span{0, 1, 0, 0};
    p.begin = w.a.window && first >= w.a.window ? first - w.a.window + 1 : 0;  // first may be far below 0
    p.lo = p.begin / KT;
    p.hi = (p.end + KT - 1) / KT;
    return p;
}

template <int RT, int KT>
__device__ __forceinline__ long long steps_of(const Work& w, const Seq& s) {
    long long t = 0;
    for (int i = 0; i * RT < s.rows; ++i) {
        const Span p = span_of<RT, KT>(w, s, i);
        t += p.hi - p.lo;
    }
    return t;
}

// Where a step lies: sequence, key head, row tile, and how many steps of the
// row tile come before it. b = batch: past the end.
struct Place {
    int b, head, tile;
    int at;
};

// The first step of CTA c: total c / n.
struct Cuts {
    long long each;  // total / n
    int rest, n;
    __device__ Cuts() {}
    __device__ Cuts(long long total, int ctas) {
        n = (int)min((long long)ctas, total);
        each = n == 0 ? 0 : total < 0x7FFFFFFF ? (int)total / n : total / n;
        rest = (int)(total - each * n);
    }
    __device__ __forceinline__ long long operator()(int c) const { return each * c + rest * c / n; }
    // The CTA whose steps hold step t.
    __device__ __forceinline__ int holder(long long t) const {
        int c = (int)min((long long)n - 1, t / each);  // at most a little too far
        while ((*this)(c) > t) --c;
        return c;
    }
};

// The scan of locate for up to 32 sequences, by each warp for itself: no
// barriers, and the sequence found comes from its lane.
template <int RT, int KT>
__device__ __forceinline__ bool locate_few(const Work& w, int cta, Cuts* cuts, Place* at, Seq* s, long long* per,
                                           long long* left) {
    const int lane = threadIdx.x & 31;
    Seq mine{};
    long long steps = 0;
    if (lane < w.a.batch) {
        mine = seq_at(w, lane);
        steps = steps_of<RT, KT>(w, mine);
    }
    const long long v = steps * w.a.hkv;
    long long x = v;
#pragma unroll
    for (int i = 1; i < 32; i *= 2) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, x, i);
        if (lane >= i) x += o;
    }
    *cuts = Cuts(__shfl_sync(0xFFFFFFFFu, x, 31), w.ctas);
    if (cta >= cuts->n) return false;
    const long long t = (*cuts)(cta);
    const int b = __ffs(__ballot_sync(0xFFFFFFFFu, t >= x - v && t < x)) - 1;
    at->b = b;
    *left = t - __shfl_sync(0xFFFFFFFFu, x - v, b);
    *per = __shfl_sync(0xFFFFFFFFu, steps, b);
    s->first = __shfl_sync(0xFFFFFFFFu, mine.first, b);
    s->n = __shfl_sync(0xFFFFFFFFu, mine.n, b);
    s->rows = __shfl_sync(0xFFFFFFFFu, mine.rows, b);
    s->ctx = __shfl_sync(0xFFFFFFFFu, mine.ctx, b);
    return true;
}

// The same for any number of sequences, by the whole block of NT threads; their
// counts stay in registers if there are no more than threads. scratch: NT / 32 + 2
// long longs of shared memory.
template <int RT, int KT, int NT>
__device__ __forceinline__ bool locate_many(const Work& w, int cta, Cuts* cuts, Place* at, Seq* s, long long* per,
                                            long long* rem, long long* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long* found = scratch + NT / 32;
    // Steps of sequence b0 + thread, those of the block's sequences before it,
    // and of all of them.
    auto scan = [&](int b0, long long* v, long long* begin) {
        const int b = b0 + threadIdx.x;
        *v = b < w.a.batch ? steps_of<RT, KT>(w, seq_at(w, b)) * w.a.hkv : 0;
        long long x = *v;
#pragma unroll
        for (int i = 1; i < 32; i *= 2) {
            const long long o = __shfl_up_sync(0xFFFFFFFFu, x, i);
            if (lane >= i) x += o;
        }
        __syncthreads();
        if (lane == 31) scratch[warp] = x;
        __syncthreads();
        long long base = 0, all = 0;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            if (i < warp) base += scratch[i];
            all += scratch[i];
        }
        *begin = base + x - *v;
        return all;
    };
    long long v = 0, begin = 0, total = 0;
    for (int b0 = 0; b0 < w.a.batch; b0 += NT) total += scan(b0, &v, &begin);
    *cuts = Cuts(total, w.ctas);
    if (cta >= cuts->n) return false;
    const long long t = (*cuts)(cta);
    long long before = 0;
    for (int b0 = 0; b0 < w.a.batch; b0 += NT) {
        const long long all = w.a.batch > NT ? scan(b0, &v, &begin) : total;
        if (t >= before + begin && t < before + begin + v) {
            found[0] = b0 + threadIdx.x;
            found[1] = t - before - begin;
        }
        before += all;
    }
    __syncthreads();
    at->b = (int)found[0];
    *rem = found[1];
    *s = seq_at(w, at->b);
    *per = steps_of<RT, KT>(w, *s);
    return true;
}

// The cuts, and the place of CTA `cta`'s first step: a scan over the sequences,
// then the head and the tile in the sequence s. False if the CTA has no steps.
// (A third of a short call's time was this scan; with one token over 700 keys
// the form for few sequences saves 0.65 us of 8.25.)
template <int RT, int KT, int NT>
__device__ __forceinline__ bool locate(const Work& w, int cta, Cuts* cuts, Place* at, Seq* seq, long long* scratch) {
    long long per = 0, left = 0;
    if (!(w.a.batch <= 32 ? locate_few<RT, KT>(w, cta, cuts, at, seq, &per, &left)
                          : locate_many<RT, KT, NT>(w, cta, cuts, at, seq, &per, &left, scratch)))
        return false;
    const Seq s = *seq;
    at->head = 0;
    while (left >= per) {  // few heads; a division of 64 bits takes longer
        left -= per;
        ++at->head;
    }
    for (at->tile = 0;; ++at->tile) {
        const Span p = span_of<RT, KT>(w, s, at->tile);
        if (left < p.hi - p.lo) break;
        left -= p.hi - p.lo;
    }
    at->at = (int)left;
    return true;
}

// Leaves where the CTA's steps begin, for whoever walks them again.
__device__ __forceinline__ void note_start(const Work& w, const Place& at, long long steps) {
    Note& n = w.notes[blockIdx.x];
    n.first_b = at.b;
    n.first_head = at.head;
    n.first_tile = at.tile;
    n.first_at = at.at;
    n.steps = steps;
}

// Walks the segments of a CTA's steps: for each, a row tile and the key tiles
// lo .. hi - 1 of it that are this CTA's.
template <int RT, int KT>
struct Walk {
    const Work& w;
    long long left;   // steps still to do
    Place p;
    Seq s;
    Span span;
    int lo, hi;
    bool whole;       // the segment is its row tile's only one
    int slot;         // where its part goes if not
    bool first;

    __device__ Walk(const Work& work, const Place& at, const Seq& seq, long long n)
        : w(work), left(n), p(at), s(seq), first(true) {
        if (left > 0) span = span_of<RT, KT>(w, s, p.tile);
    }
    // Leaves this segment's note, when it ends a row tile that another CTA began.
    __device__ void note(const Cuts& cuts, int rt, int cta) const {
        if (hi != span.hi || lo == span.lo) return;
        const long long start = cuts(cta) - (lo - span.lo);
        const int from = cuts.holder(start);
        Note& n = w.notes[cta];
        n.slot = cuts(from) < start ? 1 : 0;
        n.b = p.b;
        n.out_row = s.first * w.a.hq;
        n.rows = s.rows;
        n.r0 = p.tile * rt;
        n.head = p.head * w.group;
        n.from = from;
    }
    __device__ bool next() {
        if (left <= 0) return false;
        if (!first) {  // the row tile after the one just done
            p.at = 0;
            ++p.tile;
            if (p.tile * RT >= s.rows) {
                p.tile = 0;
                if (++p.head == w.a.hkv) {
                    p.head = 0;
                    do s = seq_at(w, ++p.b);
                    while (s.rows == 0);  // steps are left, so one with rows follows
                }
            }
            span = span_of<RT, KT>(w, s, p.tile);
        }
        lo = span.lo + p.at;
        const int n = (int)min((long long)(span.hi - lo), left);
        hi = lo + n;
        left -= n;
        whole = lo == span.lo && hi == span.hi;
        slot = first ? 0 : 1;
        first = false;
        return true;
    }
};

// Key `j` of sequence b: its page's number, or num_pages (whose rows TMA fills
// with zeros) where the table holds no page.
__device__ __forceinline__ int page_of(const Work& w, int b, int j) {
    const int page = w.a.table[(long long)b * w.a.width + j / w.a.page_size];
    if (page >= 0 && page < w.a.num_pages) return page;
    report_error(w.err, DEVERR_INDEX);
    return w.a.num_pages;
}

// The same for the `rows` keys from j on, of which those before `begin` are not seen.
__device__ __forceinline__ int page_from(const Work& w, int b, int j, int rows, int begin) {
    return j + rows <= begin ? w.a.num_pages : page_of(w, b, j);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float within(float x, float most) {  // NaN stays NaN
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(most));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(-most));
    return r;
}

// Scores of two dot products, in base 2. With a cap, softcap * tanh(z), z = scale x /
// softcap, as z P(z^2) / Q(z^2): P and Q of degree 4 with the least largest
// relative error for |z| up to 8.5 (1.2e-8, by least squares weighted anew until
// the errors are level), where tanh is 1 within 2^-23; in f32 within 9 units of 2^-24
// of the score itself (8.1 over 6 million z, with the reciprocal an ulp off). (1 - 2 / (1 + e^2z) is off by 2^-23 of the cap, which small
// scores feel.)
template <bool CAP>
__device__ __forceinline__ float2 score2(const Work& w, float2 x) {
    if (!CAP) return __fmul2_rn(x, make_float2(w.scale_log2, w.scale_log2));
    auto two = [](float v) { return make_float2(v, v); };
    x = __fmul2_rn(x, two(w.cap_in));
    const float2 z = make_float2(within(x.x, 8.5f), within(x.y, 8.5f)), s = __fmul2_rn(z, z);
    float2 p = two(1.4268720427e-8f), q = two(8.1449280742e-7f);
    p = __ffma2_rn(p, s, two(2.1250718418e-5f));
    q = __ffma2_rn(q, s, two(3.3488337938e-4f));
    p = __ffma2_rn(p, s, two(3.5340089817e-3f));
    q = __ffma2_rn(q, s, two(2.6022685692e-2f));
    p = __ffma2_rn(p, s, two(0.13413232565f));
    q = __ffma2_rn(q, s, two(0.46746554971f));
    p = __ffma2_rn(p, s, two(1.f));
    q = __ffma2_rn(q, s, two(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.x) : "f"(q.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.y) : "f"(q.y));
    return __fmul2_rn(__fmul2_rn(__fmul2_rn(z, two(w.cap_out)), p), q);
}

// N scores of each lane of a warp, get(i) and put(i, score). As long as no |z| is
// over a half, as is the rule (caps are there for the odd large score), tanh is
// z (1 + z^2 R(z^2)) with R of degree 3, fitted like P and Q to 1.5e-8.
// 13 sequences of up to 130 tokens: 43.0 us, and 48.6 with the quotient alone.
template <bool CAP, int N, class Get, class Put>
__device__ __forceinline__ void scores(const Work& w, const Get& get, const Put& put) {
    auto two = [](float v) { return make_float2(v, v); };
    if constexpr (CAP) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < N; i += 2) top = fmaxf(fmaxf(top, fabsf(get(i))), fabsf(get(i + 1)));
        if (!__any_sync(0xFFFFFFFFu, top > w.small)) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float2 x = make_float2(get(i), get(i + 1));
                const float2 z = __fmul2_rn(x, two(w.cap_in)), s = __fmul2_rn(z, z), y = __fmul2_rn(x, two(w.scale_log2));
                float2 r = __ffma2_rn(two(1.7241498455e-2f), s, two(-5.3045496345e-2f));
                r = __ffma2_rn(r, s, two(0.13325878978f));
                r = __ffma2_rn(r, s, two(-0.33333143592f));
                r = __ffma2_rn(__fmul2_rn(r, s), y, y);
                put(i, r.x);
                put(i + 1, r.y);
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 v = score2<CAP>(w, make_float2(get(i), get(i + 1)));
        put(i, v.x);
        put(i + 1, v.y);
    }
}

// Up to 16 * row_blocks rows per sequence and key head (row_blocks 1, 2, 4).
int launch_few(const DevCtx& dc, const Work& w, int row_blocks, cudaStream_t s);
// Any number of rows.
int launch_chunk(const DevCtx& dc, const Work& w, cudaStream_t s);

// A map of k or v: [num_pages][hkv * page_size][d], boxes of `rows` x 64 values.
int cache_map(CUtensorMap* m, const AttnArgs& a, const void* p, int rows);

}  // namespace attn
}  // namespace qg
