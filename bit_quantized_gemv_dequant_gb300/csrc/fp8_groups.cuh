// Rows grouped by expert: how the products of all experts become one line of
// tiles, and what the two tensor-core kernels of qmm_fp8_b128_grouped share.
#pragma once

#include "fp8_tc.cuh"

namespace qg {
namespace fp8 {

constexpr int kMaxExperts = 1024;

// offsets[e] .. offsets[e + 1] - 1 are expert e's rows. Only the device knows
// them, so each block finds the tiles of all experts by itself: an expert with n
// rows has ceil(n / BN) chunks of rows, as even as whole STEPs allow, times nt
// tiles of its weight's rows. Tiles are numbered by expert, then weight rows, then
// chunks, so tiles that run side by side share weights.
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

    // By one whole warp. Ranges that are none (outside of 0 .. M or backwards) count
    // as empty and are recorded.
    __device__ void build(const int32_t* offsets, int M, int nt, unsigned* err) {
        const int lane = threadIdx.x & 31;
        long long base = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            int lo = 0, n = 0;
            if (e < E) {
                lo = offsets[e];
                const int hi = offsets[e + 1];
                if (lo < 0 || hi > M || hi < lo) report_error(err, DEVERR_INDEX);
                else n = hi - lo;
                begin[e] = lo;
                rows[e] = n;
            }
            const long long tiles = (long long)((n + BN - 1) / BN) * nt;
            long long sum = tiles;
#pragma unroll
            for (int i = 1; i < 32; i *= 2) {
                const long long below = __shfl_up_sync(0xFFFFFFFFu, sum, i);
                if (lane >= i) sum += below;
            }
            if (e < E) first[e] = base + sum - tiles;
            base += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (lane == 0) first[E] = base;
        __syncwarp();
    }

    // Tile t < first[E].
    __device__ Tile find(long long t) const {
        int e = 0;  // the last expert whose first tile is at most t: it has some
        for (int i = kMaxExperts / 2; i; i /= 2)
            if (e + i < E && first[e + i] <= t) e += i;
        const int n = rows[e], chunks = (n + BN - 1) / BN;
        const long long at = t - first[e];
        const int n_tile = at <= 0x7FFFFFFF ? (int)at / chunks : (int)(at / chunks);
        const int c = (int)(at - (long long)n_tile * chunks);
        const int each = ((n + chunks - 1) / chunks + STEP - 1) / STEP * STEP;
        return Tile{e, n_tile, begin[e] + c * each, min(each, n - c * each)};
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
// rows multiplied in. Two warps of 32 bring them (rows of a by thread, whose
// blocks lie beside each other), running ahead of the products.
constexpr int kSetBlocks = 8, kSets = 4;

// One set: k blocks b .. b + n - 1 of the rows m0 .. m0 + rows - 1, by 64 threads.
template <int BN>
__device__ __forceinline__ void load_scales(float* set, const GroupedParams& p, const float* sw, int m0, int rows, int b,
                                            int n, int tid) {
    float f[kSetBlocks];
#pragma unroll
    for (int i = 0; i < kSetBlocks; ++i) f[i] = i < n ? __ldg(sw + b + i) : 0.f;
#pragma unroll
    for (int j = 0; j < BN; j += 64) {
        const int m = j + tid;
        if (m < rows) {
            const float* sa = p.sa + (long long)(m0 + m) * p.KB + b;
            float v[kSetBlocks];
#pragma unroll
            for (int i = 0; i < kSetBlocks; ++i) v[i] = i < n ? __ldg(sa + i) : 0.f;
#pragma unroll
            for (int i = 0; i < kSetBlocks; ++i) set[i * BN + m] = v[i] * f[i];
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

int launch_grouped_few(const DevCtx& dc, const GroupedArgs& a, cudaStream_t s);
int launch_grouped_tile(const DevCtx& dc, const GroupedArgs& a, cudaStream_t s);

}  // namespace fp8
}  // namespace qg
