// Rows in units of eight values, for the kernels that pass over rows once: 16
// bytes of a 16-bit type, twice that of f32.
#pragma once

#include "serve_common.cuh"

namespace qg {

template <class T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};

// The values p[0 .. 8), of which `left` are inside the row (VEC: all or none, and
// p on a 16-byte boundary); those that are not are 0. Without VEC they may lie STEP
// apart, so that threads beside each other read places beside each other.
template <class T, bool VEC, int STEP = 1>
__device__ __forceinline__ Raw8<T> load8(const T* p, int left) {
    Raw8<T> r;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            r.w[i] = left > 0 ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0, 0, 0, 0);
    } else {
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u[i] = 0;
            if (i * STEP < left) {
                if constexpr (sizeof(T) == 4) u[i] = __float_as_uint(p[i * STEP]);
                else u[i] = *reinterpret_cast<const uint16_t*>(p + i * STEP);
            }
        }
        if constexpr (sizeof(T) == 4) {
            r.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
            r.w[1] = make_uint4(u[4], u[5], u[6], u[7]);
        } else {
            r.w[0] = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
        }
    }
    return r;
}

template <class T>
__device__ __forceinline__ void to_f32(const Raw8<T>& r, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(r.w[i].x);
            v[4 * i + 1] = __uint_as_float(r.w[i].y);
            v[4 * i + 2] = __uint_as_float(r.w[i].z);
            v[4 * i + 3] = __uint_as_float(r.w[i].w);
        }
    } else {
        const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<T>(u[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// p[0 .. min(8, left)) = v; VEC as above.
template <class T, bool VEC, int STEP = 1>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int left) {
    if constexpr (VEC) {
        if (left <= 0) return;
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(p) =
                make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * STEP < left) p[i * STEP] = from_f32<T>(v[i]);
    }
}

// Eight codes (VEC: on an 8-byte boundary).
template <bool VEC, int STEP = 1>
__device__ __forceinline__ void store_codes8(uint8_t* p, const uint32_t (&code)[2], int left) {
    if constexpr (VEC) {
        if (left > 0) *reinterpret_cast<uint2*>(p) = make_uint2(code[0], code[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * STEP < left) p[i * STEP] = (uint8_t)(code[i / 4] >> (8 * (i % 4)));
    }
}

// The same for a warp's 256 values that lie anywhere: 32 places beside each other at a
// time, by way of 1 KB of shared memory (`tile`, the warp's own). p is the place of
// its first value, `left` how many of the row there are from there on. Of 37 rows of
// 5201 f32 values value by value took rms_norm 7.1 us.
template <class T>
__device__ __forceinline__ void load8_warp(const T* p, int left, uint32_t* tile, float (&v)[8]) {
    const int lane = threadIdx.x & 31;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i * 32 + lane < left ? to_f32(p[i * 32 + lane]) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[i * 32 + lane] = __float_as_uint(f[i]);
    __syncwarp();
    Raw8<float> r;
    r.w[0] = reinterpret_cast<const uint4*>(tile)[2 * lane];
    r.w[1] = reinterpret_cast<const uint4*>(tile)[2 * lane + 1];
    to_f32(r, v);
    __syncwarp();
}
template <class T>
__device__ __forceinline__ void store8_warp(T* p, const float (&v)[8], int left, uint32_t* tile) {
    const int lane = threadIdx.x & 31;
    store8<float, true>(reinterpret_cast<float*>(tile) + 8 * lane, v, 8);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i * 32 + lane < left) p[i * 32 + lane] = from_f32<T>(__uint_as_float(tile[i * 32 + lane]));
    __syncwarp();
}
__device__ __forceinline__ void store_codes8_warp(uint8_t* p, const uint32_t (&code)[2], int left, uint32_t* tile) {
    const int lane = threadIdx.x & 31;
    reinterpret_cast<uint2*>(tile)[lane] = make_uint2(code[0], code[1]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i * 32 + lane < left) p[i * 32 + lane] = reinterpret_cast<const uint8_t*>(tile)[i * 32 + lane];
    __syncwarp();
}

// f(T{}) for an element type known at run time, in a kernel.
template <class F>
__device__ __forceinline__ void with_type(int dtype, F&& f) {
    if (dtype == QG_F32) f(float{});
    else if (dtype == QG_F16) f(__half{});
    else f(__nv_bfloat16{});
}

// Whether rows of `width` values that lie `stride` elements apart can be moved in
// units of eight.
inline bool in_eights(const void* p, long long stride, long long width, int elem_bytes) {
    return width % 8 == 0 && (stride * elem_bytes) % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

inline int type_bytes(int dtype) { return dtype == QG_F32 ? 4 : 2; }

// A launch that may start while the kernel before it ends (it waits for it with
// griddepcontrol.wait before it touches memory).
template <class... P, class... A>
int launch_after(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = may_overlap() ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e == cudaSuccess ? QG_OK : cuda_fail(e);
}

}  // namespace qg
