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

// Powers and logarithms to the base of two and reciprocals as one instruction each, off by one or
// two units; results below the smallest normal number are zero.
__device__ __forceinline__ float ex2(float a) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}
__device__ __forceinline__ float lg2(float a) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}
__device__ __forceinline__ float rcp(float a) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}
constexpr float LOG2E = 1.44269504088896341f, LN2 = 0.693147180559945309f;

// Eight fp32 values as pairs: one packed instruction works on two.
struct F8 {
    float2 v[4];
};
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ F8 mul(const F8& a, const F8& b) {
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = __fmul2_rn(a.v[i], b.v[i]);
    return r;
}
__device__ __forceinline__ F8 mul(const F8& a, float b) {
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = __fmul2_rn(a.v[i], both(b));
    return r;
}
__device__ __forceinline__ F8 fma(const F8& a, const F8& b, const F8& c) {
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = __ffma2_rn(a.v[i], b.v[i], c.v[i]);
    return r;
}
__device__ __forceinline__ F8 fma(const F8& a, float b, const F8& c) {
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = __ffma2_rn(a.v[i], both(b), c.v[i]);
    return r;
}
__device__ __forceinline__ F8 add(const F8& a, float b) {
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = __fadd2_rn(a.v[i], both(b));
    return r;
}
__device__ __forceinline__ void dot(const F8& a, const F8& b, float2& s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __ffma2_rn(a.v[i], b.v[i], s);
}
__device__ __forceinline__ F8 fill8(float a) {
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = both(a);
    return r;
}
__device__ __forceinline__ F8 bf16x8(const uint4& a) {
    F8 r;
    r.v[0] = make_float2(bf16lo(a.x), bf16hi(a.x));
    r.v[1] = make_float2(bf16lo(a.y), bf16hi(a.y));
    r.v[2] = make_float2(bf16lo(a.z), bf16hi(a.z));
    r.v[3] = make_float2(bf16lo(a.w), bf16hi(a.w));
    return r;
}
__device__ __forceinline__ F8 f32x8(const uint4& a, const uint4& b) {
    F8 r;
    r.v[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
    r.v[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
    r.v[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
    r.v[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
    return r;
}

// One chunk as it comes from memory.
template <int DT> struct Raw8;
template <> struct Raw8<DT_BF16> {
    uint4 a;
    __device__ __forceinline__ void load(const void* p, size_t chunk) { a = ld_row(static_cast<const uint4*>(p) + chunk); }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ F8 get() const { return bf16x8(a); }
};
template <> struct Raw8<DT_F32> {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* p, size_t chunk) {
        a = ld_row(static_cast<const uint4*>(p) + 2 * chunk);
        b = ld_row(static_cast<const uint4*>(p) + 2 * chunk + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ F8 get() const { return f32x8(a, b); }
};

// A chunk whose type is known at run time (weights and gates: cached loads).
struct RawAny {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* p, bool f32, size_t chunk) {
        const uint4* q = static_cast<const uint4*>(p) + (f32 ? 2 * chunk : chunk);
        a = *q;
        if (f32) b = q[1];
    }
    __device__ __forceinline__ F8 get(bool f32) const { return f32 ? f32x8(a, b) : bf16x8(a); }
};
__device__ __forceinline__ float load1(const void* p, bool f32, size_t i) {
    return f32 ? static_cast<const float*>(p)[i] : bf16f(static_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);  // round to nearest even, NaN stays NaN
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int DT>
__device__ __forceinline__ void store8(void* p, size_t chunk, const F8& f) {
    if (DT == DT_BF16) {
        static_cast<uint4*>(p)[chunk] = make_uint4(pack_bf16(f.v[0].x, f.v[0].y), pack_bf16(f.v[1].x, f.v[1].y),
                                                   pack_bf16(f.v[2].x, f.v[2].y), pack_bf16(f.v[3].x, f.v[3].y));
    } else {
        float4* q = static_cast<float4*>(p) + 2 * chunk;
        q[0] = make_float4(f.v[0].x, f.v[0].y, f.v[1].x, f.v[1].y);
        q[1] = make_float4(f.v[2].x, f.v[2].y, f.v[3].x, f.v[3].y);
    }
}

}  // namespace
}  // namespace redmoe
