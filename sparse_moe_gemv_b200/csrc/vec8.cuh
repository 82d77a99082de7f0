// Chunks of eight consecutive row elements, the unit of the row-wise operators (norm.cu,
// balance.cu): one 16-byte load of bf16, two of fp32. Loading and converting are separate
// steps, so that all of a row's loads can be in flight before the first conversion waits.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace redmoe {
namespace {

// Row data is used once per call: streamed past L1, which keeps the weights that every row
// shares. Not a read-only (.nc) load: some outputs may be written over their own input.
__device__ __forceinline__ uint4 ld_row(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
template <int DT> struct Raw8;
template <> struct Raw8<DT_BF16> {
    uint4 a;
    __device__ __forceinline__ void load(const void* p, size_t chunk) {
        a = ld_row(static_cast<const uint4*>(p) + chunk);
    }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16lo(w[i]);
            v[2 * i + 1] = bf16hi(w[i]);
        }
    }
};
template <> struct Raw8<DT_F32> {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* p, size_t chunk) {
        a = ld_row(static_cast<const uint4*>(p) + 2 * chunk);
        b = ld_row(static_cast<const uint4*>(p) + 2 * chunk + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);  // round to nearest even, NaN stays NaN
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int DT>
__device__ __forceinline__ void store8(void* p, size_t chunk, const float (&v)[8]) {
    if (DT == DT_BF16) {
        static_cast<uint4*>(p)[chunk] =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
        float4* q = static_cast<float4*>(p) + 2 * chunk;
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// Vectors shared by all rows (weights, channel gates), type known at run time: cached loads.
__device__ __forceinline__ void load8_shared(const void* p, bool f32, size_t chunk, float (&v)[8]) {
    if (f32) {
        const float4 a = __ldg(static_cast<const float4*>(p) + 2 * chunk);
        const float4 b = __ldg(static_cast<const float4*>(p) + 2 * chunk + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = __ldg(static_cast<const uint4*>(p) + chunk);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16lo(w[i]);
            v[2 * i + 1] = bf16hi(w[i]);
        }
    }
}
__device__ __forceinline__ float load1(const void* p, bool f32, size_t i) {
    return f32 ? __ldg(static_cast<const float*>(p) + i) : bf16f(__ldg(static_cast<const uint16_t*>(p) + i));
}

}  // namespace
}  // namespace redmoe
