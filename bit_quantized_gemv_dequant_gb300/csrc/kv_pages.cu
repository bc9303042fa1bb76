// Upkeep of a paged cache: new tokens into their pages, copies, forks, freeing
// and compaction. The tables and counts are handled by one thread-block
// cluster (its barrier orders the steps, so a call is one such kernel and one
// that copies pages); the copies by the whole GPU.
#include <cooperative_groups.h>

#include <algorithm>

#include "fp8_tc.cuh"

namespace cg = cooperative_groups;

namespace qg {
namespace {

// ------------------------------------------------------------------- append
constexpr int kAppendThreads = 256;

// Eight elements of a row of k or v per thread, rounded to the cache's type.
// Bound by the bytes read and written; a token's rows land in one run of
// head_dim elements per head. 3001 tokens of 8 heads of 128, f32 to bf16: 7.5 us,
// 4.9 TB/s (two short waves).
template <class TX, class TC, bool VEC>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a, unsigned* err) {
    const int per_row = a.heads * a.d / 8;
    const long long unit = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
    const long long half = a.tokens * per_row;
    if (unit >= 2 * half) return;
    const bool is_v = unit >= half;
    const long long u = is_v ? unit - half : unit;
    // 32 bits where they do, and the source under way with the slot: 7.5 us, 9.0 without.
    const long long t = half <= 0xFFFFFFFFLL ? (uint32_t)u / (uint32_t)per_row : u / per_row;
    const int e = (int)(u - t * per_row) * 8, h = e / a.d, c = e % a.d;
    const int64_t slot = a.slots[t];
    // The source is loaded while the slot is on its way, also where that says: none.
    const TX* src = static_cast<const TX*>(is_v ? a.v : a.k) + t * (is_v ? a.v_stride : a.k_stride) + e;
    uint4 out;
    if constexpr (VEC && std::is_same_v<TX, TC>) {
        out = *reinterpret_cast<const uint4*>(src);
    } else {
        float f[8];
        if constexpr (VEC && sizeof(TX) == 4) {
            const float4 lo = reinterpret_cast<const float4*>(src)[0];
            const float4 hi = reinterpret_cast<const float4*>(src)[1];
            f[0] = lo.x; f[1] = lo.y; f[2] = lo.z; f[3] = lo.w;
            f[4] = hi.x; f[5] = hi.y; f[6] = hi.z; f[7] = hi.w;
        } else if constexpr (VEC) {
            const uint4 w = *reinterpret_cast<const uint4*>(src);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 p = unpack2<TX>(ws[i]);
                f[2 * i] = p.x;
                f[2 * i + 1] = p.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = to_f32(src[i]);
        }
        out = make_uint4(pack2<TC>(f[0], f[1]), pack2<TC>(f[2], f[3]), pack2<TC>(f[4], f[5]),
                         pack2<TC>(f[6], f[7]));
    }
    if (slot < 0) return;
    const int log_page = 31 - __clz(a.page_size);  // a power of two
    const int64_t page = slot >> log_page;
    if (page >= a.num_pages) {
        report_error(err, DEVERR_INDEX);
        return;
    }
    TC* dst = static_cast<TC*>(is_v ? a.v_cache : a.k_cache) +
              ((page * a.heads + h) * a.page_size + (slot & (a.page_size - 1))) * a.d + c;
    *reinterpret_cast<uint4*>(dst) = out;
}

// ------------------------------------------------------------------- copies
constexpr int kCopyThreads = 256;
constexpr int kPiece = 8 * kCopyThreads;  // 16-byte words

// The pairs to copy: src[i] -> dst[i], i < n; with `count` set, *count of
// them, their sources listed backwards (see compact_kernel).
struct CopyList {
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;
    long long n;
};

// Remaps a page table in the same launch (kv_compact); table null: nothing.
struct Remap {
    const int32_t* table;
    const int32_t* map;
    int32_t* out;
    long long n;
};

__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const PagePlanes p, const CopyList l, const Remap r, unsigned* err) {
    fp8::pdl_wait();
    fp8::pdl_trigger();
    for (long long i = (long long)blockIdx.x * kCopyThreads + threadIdx.x; r.table && i < r.n;
         i += (long long)gridDim.x * kCopyThreads) {
        const int32_t page = r.table[i];
        r.out[i] = page >= 0 && page < p.num_pages ? r.map[page] : -1;
        if (page >= p.num_pages) report_error(err, DEVERR_INDEX);
    }
    const long long n = l.count ? *l.count : l.n;
    // Pieces of 32 KB, all of whose loads are under way at once: whole pages leave the
    // last round of CTAs partly idle (48 pages of 64 KB in 32 planes: 31.7 us with the
    // tables, 33.1 by whole pages, 33.3 by 16 KB).
    const long long vecs = p.page_bytes / 16, pieces = (vecs + kPiece - 1) / kPiece;
    const long long all = n * p.planes * pieces;
    auto quotient = [&](long long x, long long by) {  // in 32 bits where they do: several times shorter
        return all <= 0xFFFFFFFFLL ? (uint32_t)x / (uint32_t)by : x / by;
    };
    for (long long u = blockIdx.x; u < all; u += gridDim.x) {
        const long long at = quotient(u, pieces), i = quotient(at, p.planes), plane = at - i * p.planes;
        const int32_t src = l.src[l.count ? n - 1 - i : i], dst = l.dst[i];
        if (src < 0 || dst < 0) continue;
        if (src >= p.num_pages || dst >= p.num_pages) {
            if (threadIdx.x == 0) report_error(err, DEVERR_INDEX);
            continue;
        }
        const uint4* from = reinterpret_cast<const uint4*>(p.cache + (plane * p.num_pages + src) * p.page_bytes);
        uint4* to = reinterpret_cast<uint4*>(p.cache + (plane * p.num_pages + dst) * p.page_bytes);
        const long long v0 = (u - at * pieces) * kPiece;
        const int left = (int)min((long long)kPiece, vecs - v0);
        from += v0 + threadIdx.x;
        to += v0 + threadIdx.x;
        constexpr int kEach = kPiece / kCopyThreads;
        uint4 d[kEach];
        if (left == kPiece) {
#pragma unroll
            for (int j = 0; j < kEach; ++j) d[j] = __ldcs(from + j * kCopyThreads);
#pragma unroll
            for (int j = 0; j < kEach; ++j) __stcs(to + j * kCopyThreads, d[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                if ((int)threadIdx.x + j * kCopyThreads < left) d[j] = __ldcs(from + j * kCopyThreads);
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                if ((int)threadIdx.x + j * kCopyThreads < left) __stcs(to + j * kCopyThreads, d[j]);
        }
    }
}

int copy_launch(const DevCtx& dc, const PagePlanes& p, const CopyList& l, const Remap& r,
                long long most, bool overlap, cudaStream_t s) {
    const long long pieces = (p.page_bytes / 16 + kPiece - 1) / kPiece;
    const long long work = std::max(most * p.planes * pieces, (r.n + kCopyThreads - 1) / kCopyThreads);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::max(1LL, std::min<long long>(work, (long long)dc.num_sms * 8)));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = s;
    // after the kernel with the tables it starts while that one ends, and waits for it
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, copy_kernel, p, l, r, dc.err);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

// --------------------------------------------------------- tables and counts
constexpr int kCluster = 8;
constexpr int kThreads = 1024;

// Exclusive prefix of `v` over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* total) {
    __shared__ int sums[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int i = 1; i < 32; i *= 2) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, x, i);
        if (lane >= i) x += o;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int t = sums[lane];
#pragma unroll
        for (int i = 1; i < 32; i *= 2) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, t, i);
            if (lane >= i) t += o;
        }
        sums[lane] = t;
    }
    __syncthreads();
    const int before = warp ? sums[warp - 1] : 0;
    *total = sums[kThreads / 32 - 1];
    __syncthreads();
    return before + x - v;
}

// Sum over the cluster's blocks of `mine`, and over the blocks before this one.
__device__ __forceinline__ void cluster_scan(int mine, int* before, int* total) {
    __shared__ int slot;
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x == 0) slot = mine;
    cl.sync();
    int b = 0, t = 0;
    for (unsigned i = 0; i < kCluster; ++i) {
        const int v = *cl.map_shared_rank(&slot, i);
        t += v;
        if (i < cl.block_rank()) b += v;
    }
    cl.sync();
    *before = b;
    *total = t;
}

// kv_fork's tables. Every block ranks its share of the free pages and, after
// the barrier, writes the rows of its share of the children.
__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkArgs a, unsigned* err) {
    fp8::pdl_trigger();
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), np = (int)a.p.num_pages;
    int32_t* ws_src = a.ws;
    int32_t* ws_dst = a.ws + a.children;
    int32_t* ws_free = a.ws + 2 * (long long)a.children;
    const int share = (np + kCluster - 1) / kCluster;
    const int lo = min(np, rank * share), hi = min(np, lo + share);
    int mine = 0;
    for (int p = lo + threadIdx.x; p < hi; p += kThreads) {
        const int ref = a.refs[p];
        a.new_refs[p] = ref;
        mine += ref <= 0;
    }
    int sum, before, nfree;
    block_scan(mine, &sum);
    cluster_scan(sum, &before, &nfree);
    for (int p0 = lo; p0 < hi && before < a.children; p0 += kThreads) {
        const int p = p0 + threadIdx.x;
        const bool is_free = p < hi && a.refs[p] <= 0;
        const int at = before + block_scan(is_free, &sum);
        if (is_free && at < a.children) ws_free[at] = p;
        before += sum;
    }
    cl.sync();  // new_refs and the free pages are written
    __shared__ int s_at[kThreads], s_len[kThreads], s_row[kThreads];
    int used = 0;
    for (int c0 = 0; c0 < a.children; c0 += kThreads) {
        const int c = c0 + threadIdx.x;
        int row = -1, len = 0;
        if (c < a.children) {
            row = a.parents[c];
            if (row < 0 || row >= a.rows) {
                report_error(err, DEVERR_INDEX);
                row = -1;
            } else {
                len = a.lens[row];
                if (len < 0 || len > (long long)a.width * a.page_size) {
                    report_error(err, DEVERR_INDEX);
                    len = 0;
                }
            }
        }
        const bool part = len % a.page_size != 0;
        const int at = used + block_scan(part, &sum);
        used += sum;
        s_at[threadIdx.x] = at;
        s_len[threadIdx.x] = len;
        s_row[threadIdx.x] = row;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        for (int i = (threadIdx.x >> 5) * kCluster + rank; i < kThreads && c0 + i < a.children;
             i += kThreads / 32 * kCluster) {
            const int n = s_len[i], whole = n / a.page_size;
            const bool want = n % a.page_size != 0;
            const int fresh = want && s_at[i] < nfree ? ws_free[s_at[i]] : -1;
            const int32_t* old = a.table + (long long)max(s_row[i], 0) * a.width;
            int32_t* out = a.child_table + (long long)(c0 + i) * a.width;
            for (int j = lane; j < a.width; j += 32) {
                int page = -1;
                if (j < whole) {
                    page = old[j];
                    if (page < 0 || page >= np) {
                        report_error(err, DEVERR_INDEX);
                        page = -1;
                    } else {
                        atomicAdd(a.new_refs + page, 1);
                    }
                } else if (j == whole) {
                    page = fresh;
                }
                out[j] = page;
            }
            if (lane == 0) {
                if (fresh >= 0) atomicAdd(a.new_refs + fresh, 1 - min(0, a.refs[fresh]));
                if (want && fresh < 0) report_error(err, DEVERR_NO_PAGE);
                a.child_lens[c0 + i] = want && fresh < 0 ? whole * a.page_size : n;
                const int last = fresh >= 0 ? old[whole] : -1;
                if (fresh >= 0 && last < 0) report_error(err, DEVERR_INDEX);  // the copies report those past the last page
                ws_src[c0 + i] = last;
                ws_dst[c0 + i] = fresh;
            }
        }
        __syncthreads();
    }
}

// kv_free: counts are copied, then lowered by the dropped rows' entries.
__global__ void __launch_bounds__(kThreads) free_kernel(const FreeArgs a, unsigned* err) {
    cg::cluster_group cl = cg::this_cluster();
    const int id = (int)cl.block_rank() * kThreads + threadIdx.x;
    for (int p = id; p < a.num_pages; p += kCluster * kThreads) a.new_refs[p] = a.refs[p];
    cl.sync();
    const long long n = (long long)a.rows * a.width;
    for (long long i = id; i < n; i += kCluster * kThreads) {
        int page = a.table[i];
        if (a.drop[i / a.width]) {
            if (page >= a.num_pages) {
                report_error(err, DEVERR_INDEX);
            } else if (page >= 0 && atomicSub(a.new_refs + page, 1) <= 0) {
                atomicAdd(a.new_refs + page, 1);
                report_error(err, DEVERR_COUNT);
            }
            page = -1;
        }
        a.new_table[i] = page;
    }
    for (int r = id; r < a.rows; r += kCluster * kThreads) a.new_lens[r] = a.drop[r] ? 0 : a.lens[r];
}

// kv_compact's numbering. With live(p) = the pages in use before page p and n
// = all of them, the free pages below n, in order, are the destinations (the
// one at p is number p - live(p)) and the pages in use at n or above the
// sources; source number i counted from the last one has n - 1 - live(p) = i,
// which needs no second count. There are as many of the one as of the other.
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
    fp8::pdl_trigger();
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), np = (int)a.p.num_pages;
    int32_t* ws_src = a.ws + 4;
    int32_t* ws_dst = ws_src + (np + 1) / 2;
    const int share = (np + kCluster - 1) / kCluster;
    const int lo = min(np, rank * share), hi = min(np, lo + share);
    int mine = 0, sum, before, n, moves;
    for (int p = lo + threadIdx.x; p < hi; p += kThreads) mine += a.refs[p] > 0;
    block_scan(mine, &sum);
    cluster_scan(sum, &before, &n);
    int low_free = 0;
    for (int p0 = lo; p0 < hi; p0 += kThreads) {
        const int p = p0 + threadIdx.x;
        const int ref = p < hi ? a.refs[p] : 0;
        const int live = before + block_scan(ref > 0, &sum);
        before += sum;
        if (p < hi) {
            a.map[p] = ref > 0 ? p : -1;
            if (p >= n) a.new_refs[p] = 0;
            else if (ref > 0) a.new_refs[p] = ref;
            if (ref > 0 && p >= n) ws_src[n - 1 - live] = p;
            if (ref <= 0 && p < n) {
                ws_dst[p - live] = p;
                ++low_free;
            }
        }
    }
    block_scan(low_free, &sum);
    cluster_scan(sum, &before, &moves);  // also orders the lists above before their use
    for (int i = rank * kThreads + threadIdx.x; i < moves; i += kCluster * kThreads) {
        const int src = ws_src[moves - 1 - i], dst = ws_dst[i];
        a.map[src] = dst;
        a.new_refs[dst] = a.refs[src];
    }
    if (rank == 0 && threadIdx.x == 0) {
        a.ws[0] = moves;
        a.live[0] = n;
    }
}

template <class... P, class... A>
int cluster_launch(void (*kern)(P...), cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

}  // namespace

int kv_append_launch(const DevCtx& dc, const AppendArgs& a, cudaStream_t s) {
    const long long units = 2 * a.tokens * (a.heads * (long long)a.d / 8);
    const long long grid = (units + kAppendThreads - 1) / kAppendThreads;
    if (grid > 0x7FFFFFFFLL) return QG_ERR_UNSUPPORTED;
    return by_type(a.x_dtype, [&](auto tx) {
        using TX = decltype(tx);
        const uintptr_t at = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                             (uintptr_t)(a.k_stride * sizeof(TX)) | (uintptr_t)(a.v_stride * sizeof(TX));
        const bool vec = at % 16 == 0;
        return by_type(a.cache_dtype, [&](auto tc) {
            using TC = decltype(tc);
            if constexpr (sizeof(TC) == 2) {
                auto kern = vec ? append_kernel<TX, TC, true> : append_kernel<TX, TC, false>;
                kern<<<(unsigned)grid, kAppendThreads, 0, s>>>(a, dc.err);
                return launched();
            } else {
                return (int)QG_ERR_INVALID_ARG;
            }
        });
    });
}

int kv_copy_launch(const DevCtx& dc, const PagePlanes& p, const int32_t* src, const int32_t* dst,
                   long long n, cudaStream_t s) {
    return copy_launch(dc, p, CopyList{src, dst, nullptr, n}, Remap{}, n, may_overlap(), s);
}

int kv_fork_launch(const DevCtx& dc, const ForkArgs& a, cudaStream_t s) {
    int rc = cluster_launch(fork_kernel, s, a, dc.err);
    if (rc || a.children == 0) return rc;
    return copy_launch(dc, a.p, CopyList{a.ws, a.ws + a.children, nullptr, a.children}, Remap{},
                       a.children, true, s);
}

int kv_free_launch(const DevCtx& dc, const FreeArgs& a, cudaStream_t s) {
    return cluster_launch(free_kernel, s, a, dc.err);
}

int kv_compact_launch(const DevCtx& dc, const CompactArgs& a, cudaStream_t s) {
    int rc = cluster_launch(compact_kernel, s, a);
    if (rc) return rc;
    const long long most = (a.p.num_pages + 1) / 2;
    const int32_t* src = a.ws + 4;
    return copy_launch(dc, a.p, CopyList{src, src + most, a.ws, 0},
                       Remap{a.table, a.map, a.new_table, (long long)a.rows * a.width}, most, true, s);
}

}  // namespace qg
