// Rows grouped by expert: how the products of all experts become one line of
// tiles, and what the two tensor-core kernels of qmm_fp8_b128_grouped share.
#pragma once

#include "fp8_group_rule.cuh"
#include "fp8_tc.cuh"

namespace qg {
namespace fp8 {

constexpr int kMaxExperts = 1024;

// The number of expert e's rows, and the first of them. A range that is none
// (outside of 0 .. M or backwards) is empty and recorded.
__device__ __forceinline__ int rows_of(const int32_t* offsets, int e, int M, int* first, unsigned* err) {
    const int lo = offsets[e], hi = offsets[e + 1];
    *first = lo;
    if (lo >= 0 && hi <= M && hi >= lo) return hi - lo;
    report_error(err, DEVERR_INDEX);
    return 0;
}

// a / b for a >= 0 and b > 0, in 32 bits where they do: several times shorter.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return (a | b) >> 32 ? a / b : (uint32_t)a / (uint32_t)b;
}

// The sum of v over this lane and those below it.
__device__ __forceinline__ long long warp_prefix(long long v) {
#pragma unroll
    for (int i = 1; i < 32; i *= 2) {
        const long long below = __shfl_up_sync(0xFFFFFFFFu, v, i);
        if ((threadIdx.x & 31) >= (unsigned)i) v += below;
    }
    return v;
}

// offsets[e] .. offsets[e + 1] - 1 are expert e's rows. Only the device knows
// them, so each block finds the tiles of all experts by itself: an expert with n
// rows has ceil(n / BN) chunks of rows, as even as whole STEPs allow, times nt
// tiles of its weight's rows. Tiles are numbered by expert, then chunks, then weight
// rows: tiles side by side share rows of a and take the same time, and an expert's
// weight is in the L2 for its next chunk. (With chunks last tiles side by side share
// weights: 16384 rows unevenly on 32 experts, N = K = 4096, take 290 us like this and 296
// like that; 24576 on 128 experts, N = 1024, K = 4096, 170 and 165.)
template <int BN, int STEP>
struct Groups {
    long long* first;  // the number of expert e's first tile; [E]: of tiles
    int* begin;
    int* rows;
    int E;

    static constexpr int bytes(long long E) { return (int)(E + 1) * 16; }

    __device__ Groups(void* smem, int experts)
        : first(static_cast<long long*>(smem)), begin(reinterpret_cast<int*>(first + experts + 1)),
          rows(begin + experts + 1), E(experts) {}

    struct Tile {
        int e, n_tile, m0, rows;  // rows m0 .. m0 + rows - 1 of a
    };

    // By one whole warp.
    __device__ void build(const int32_t* offsets, int M, int nt, unsigned* err) {
        const int lane = threadIdx.x & 31;
        long long base = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            int lo = 0, n = 0;
            if (e < E) {
                n = rows_of(offsets, e, M, &lo, err);
                begin[e] = lo;
                rows[e] = n;
            }
            const long long tiles = (long long)((n + BN - 1) / BN) * nt;
            const long long sum = warp_prefix(tiles);
            if (e < E) first[e] = base + sum - tiles;
            base += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (lane == 0) first[E] = base;
        __syncwarp();
    }

    // Tile t < first[E], from one before it (or Tile{}).
    __device__ void find(long long t, int nt, Tile& g) const {
        if (first[g.e + 1] <= t) {  // the last expert whose first tile is at most t: it has some
            ++g.e;
            for (int i = 1 << (31 - __clz(E)); i; i /= 2)
                if (g.e + i < E && first[g.e + i] <= t) g.e += i;
        }
        const int n = rows[g.e], chunks = (n + BN - 1) / BN;
        const long long at = t - first[g.e];
        const int c = (int)quotient(at, nt);
        g.n_tile = (int)(at - (long long)c * nt);
        const int each = ((n + chunks - 1) / chunks + STEP - 1) / STEP * STEP;
        g.m0 = begin[g.e] + c * each;
        g.rows = min(each, n - c * each);
    }
};

struct GroupedParams {
    const float* sa;         // [M, KB]
    const float* sw;         // [E, ceil(N / 128), KB]
    const int32_t* offsets;  // [E + 1]
    void* y;                 // [M, N]
    int M, E, N, KB;
    unsigned* err;
};

// Scales come through shared memory in sets of kSetBlocks k blocks, of which
// kSets are under way: [k block][row of a] with w's scale of the tile's 128 weight
// rows multiplied in. Two warps bring them, running ahead of the products. Eight
// lanes read the k blocks of a row, which lie beside each other; the pitch puts
// what a warp writes (8 blocks of 4 rows) into 32 banks.
constexpr int kSetBlocks = 8, kSets = 4;
constexpr int scale_pitch(int BN) { return BN + 4; }

// One set: k blocks b .. b + n - 1 of the rows m0 .. m0 + rows - 1, by 64 threads, with
// the factors of one block of w's rows, or of two (the second one's products from
// column kSecond on). 8 LOADS rows are under way at a time: loads are slow beside the
// operands' (many rows per expert: 305 us with 64 rows at a time and a reading of sa for
// each of two factors, 299 with 128 rows and one).
template <int BN, int LOADS, int kSecond = 0>
__device__ __forceinline__ void load_scales(float* set, const GroupedParams& p, const float* sw, const float* sw2, int m0,
                                            int rows, int b, int n, int tid) {
    const int i = tid % 8, m1 = tid / 8;
    if (i >= n) return;
    const float f = __ldg(sw + b + i), f2 = kSecond ? __ldg(sw2 + b + i) : 0.f;
    const float* sa = p.sa + (long long)m0 * p.KB + b + i;
    float* to = set + i * scale_pitch(BN);
#pragma unroll 1
    for (int j = m1; j < rows; j += 8 * LOADS) {
        float v[LOADS];
#pragma unroll
        for (int k = 0; k < LOADS; ++k) v[k] = j + k * 8 < rows ? __ldg(sa + (long long)(j + k * 8) * p.KB) : 0.f;
#pragma unroll
        for (int k = 0; k < LOADS; ++k)
            if (j + k * 8 < rows) {
                to[j + k * 8] = v[k] * f;
                if (kSecond) to[kSecond + j + k * 8] = v[k] * f2;
            }
    }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// w [E, N, K] in boxes of 128 rows of one expert x 128.
int weight_map(CUtensorMap* m, const GroupedArgs& a);

int plan_grouped_few(const DevCtx& dc, const GroupedArgs& a, FewPlan* plan);
int launch_grouped_few(const DevCtx& dc, const GroupedArgs& a, const FewPlan& plan, cudaStream_t s);
int launch_grouped_tile(const DevCtx& dc, const GroupedArgs& a, cudaStream_t s);

}  // namespace fp8
}  // namespace qg
