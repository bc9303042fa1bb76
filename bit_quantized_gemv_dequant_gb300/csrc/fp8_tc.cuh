// The tensor-core kernels of qmm_fp8_b128 and what they share: PTX wrappers on
// top of the prefill kernels' ones.
#pragma once

#include <mutex>

#include "prefill_common.cuh"
#include "serve_common.cuh"

namespace qg {
namespace fp8 {

using namespace prefill;

// D[tmem] (+)= A[smem] * B[smem], e4m3 operands, f32 accumulate, 32 k.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Instruction descriptor, kind::f8f6f4: f32 accumulator, e4m3 A and B, both
// K-major, M x N.
__host__ __device__ constexpr uint32_t f8_idesc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// 32 consecutive 32-bit columns of this thread's lane, without waiting;
// tmem_wait32 completes it (the registers pass through the wait, so no use of
// them moves before it).
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                   "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                   "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                   "+r"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t tmem, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

// The address of shared memory `addr` in CTA `rank` of the cluster, and what lies there.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(in_cta(addr, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Pairs of CTAs (cta_group::2). A load into this CTA's shared memory that completes on a
// barrier of the pair:
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"(acc)
        : "memory");
}
// Arrives on the barrier at this place in both CTAs when the MMAs so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// Arrives on a barrier of the pair. What the arrival orders is reads of tensor
// memory, complete and behind a tcgen05 fence: no release over the cluster is
// needed (one costs 1000 cycles in fp8_tile.cu).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int c0, int c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
}

// Programmatic dependent launch: wait for the kernels before this one on the
// stream; let the next one start its prologue.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

struct Params {
    const float* sa;   // [M, KB]
    const float* sw;   // [ceil(N / 128), KB]
    void* y;           // [M, N]
    int M, N, KB;
    bool vec;          // y's rows start on 16-byte boundaries (tile_kernel)
    unsigned* err;
};

int launch_swap(const DevCtx& dc, const Fp8Args& a, cudaStream_t s);
bool swap_is_shorter(const DevCtx& dc, const Fp8Args& a);
int launch_tile(const DevCtx& dc, const Fp8Args& a, cudaStream_t s);

// dst = src's rows of K bytes, which start at any byte, with zeros up to the pitch, a
// multiple of 16 (fp8_mm.cu). With offsets, which say what groups of rows are for, those
// of a group that has nothing (offsets[g] .. offsets[g + 1] - 1) are left out.
int pad_rows(const DevCtx& dc, const uint8_t* src, uint8_t* dst, long long rows, long long K, long long pitch, cudaStream_t s,
             const int32_t* offsets = nullptr, long long group = 0);

// How many clusters of i CTAs of a kernel the GPU holds at once, i = 1 .. 8, asked once per
// kernel and device; the kernel may have that much shared memory from then on.
template <auto KERN>
int cluster_room(const DevCtx& dc, int threads, int smem, const int** room) {
    static std::once_flag once[64];
    static cudaError_t error[64];
    static int held[64][9];
    std::call_once(once[dc.device], [&] {
        cudaError_t& e = error[dc.device];
        e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        for (int i = 1; i < 9 && e == cudaSuccess; ++i) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(i);
            cfg.blockDim = dim3(threads);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = i;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&held[dc.device][i], KERN, &cfg);
        }
    });
    *room = held[dc.device];
    return error[dc.device] == cudaSuccess ? QG_OK : cuda_fail(error[dc.device]);
}

// A 2-D map of rows x cols e4m3 codes, boxes of box_rows x 128, 128-byte swizzle.
int code_map(CUtensorMap* m, const uint8_t* p, long long rows, long long cols, int box_rows);

// y [rows, cols] of f32 or bf16 in boxes of 32 rows x 128 bytes, 128-byte swizzle (fp8_tile.cu).
int out_map(CUtensorMap* m, void* y, int dtype, long long rows, long long cols);

}  // namespace fp8
}  // namespace qg
