// Pieces shared by the serving operators' kernels: element types, conversions
// and 16-byte loads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "qg_internal.cuh"

namespace qg {

template <class T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (std::is_same_v<T, __half>) return __half2float(v);
    else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __bfloat162float(v);
    else return v;
}

template <class T>
__device__ __forceinline__ T from_f32(float v) {
    if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
    else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __float2bfloat16_rn(v);
    else return v;
}

// Two f32 values as one word of two 16-bit ones, the first in the low half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (std::is_same_v<T, __half>)
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// f(T{}) for the element type that `dtype` names.
template <class F>
int by_type(int dtype, F&& f) {
    switch (dtype) {
        case QG_F32: return f(float{});
        case QG_F16: return f(__half{});
        case QG_BF16: return f(__nv_bfloat16{});
        default: return QG_ERR_INVALID_ARG;
    }
}

// Bounded wait; the thread is suspended between polls, which would take issue
// slots from the warps that it waits for.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) { return mbar_wait_sleep(bar, parity); }
// The same for a whole warp.
__device__ __forceinline__ bool warp_bar_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity));
}

// True in one lane of a converged warp, the same one every time. The tensor-core
// instructions take their operands from uniform registers: a warp that stays
// together and issues them under this predicate has its addresses there, while
// a loop that one lane runs alone moves every operand over for every instruction
// (about 100 cycles each: more than the instruction itself takes).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// The warp's number in its block, known to be the same in all its lanes.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0); }

inline int launched() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

}  // namespace qg
