// Rows grouped by expert: how the products of all experts become one line of
// tiles. offsets[e] .. offsets[e + 1] - 1 are expert e's rows; only the device
// knows them, so each block finds the tiles of all experts by itself.
#pragma once

#include "fp8_tc.cuh"

namespace qg {
namespace fp8 {

constexpr int kMaxExperts = 1024;

// In shared memory. An expert with n rows has ceil(n / BN) chunks of rows, as
// even as whole STEPs allow, times nt tiles of its weight's rows. Tiles are
// numbered by expert, then weight rows, then chunks, so tiles that run side by
// side share weights.
template <int BN, int STEP>
struct Groups {
    long long first[kMaxExperts + 1];  // the number of expert e's first tile; [E]: of tiles
    int begin[kMaxExperts + 1];
    int rows[kMaxExperts + 1];

    struct Tile {
        int e, n_tile, m0, rows;  // rows m0 .. m0 + rows - 1 of a
    };

    // By one whole warp. Ranges that are none (outside of 0 .. M or backwards) count
    // as empty and are recorded.
    __device__ void build(const int32_t* offsets, int E, int M, int nt, unsigned* err) {
        const int lane = threadIdx.x & 31;
        long long base = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            int lo = 0, n = 0;
            if (e < E) {
                lo = offsets[e];
                const int hi = offsets[e + 1];
                if (lo < 0 || hi > M || hi < lo) {
                    if (blockIdx.x == 0) report_error(err, DEVERR_INDEX);
                } else {
                    n = hi - lo;
                }
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
    __device__ Tile find(long long t, int E) const {
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

}  // namespace fp8
}  // namespace qg
