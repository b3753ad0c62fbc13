// dq_types.cuh -- the element types of the row operators: four consecutive
// elements to and from fp32.
#pragma once

#include <cuda_bf16.h>

#include "dq_common.cuh"

namespace dq {

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __half* p)
{
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p)
{
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}

// Two fp32 as one register of the type's pairs, each rounded once to nearest.
__device__ __forceinline__ uint32_t pack2(float a, float b, const __half*)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __nv_bfloat16*)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v)
{
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v.x, v.y, p), pack2(v.z, v.w, p));
}

// Pairs of fp32 in one 64-bit register, for the two-wide fp32 instructions.
__device__ __forceinline__ uint64_t f2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 un2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t half2_f2(uint32_t h)
{
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return f2(v.x, v.y);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace dq

namespace dqhost {

inline bool valid_type(int t) { return t == DQ_TYPE_F32 || t == DQ_TYPE_F16 || t == DQ_TYPE_BF16; }
inline int type_bytes(int t) { return t == DQ_TYPE_F32 ? 4 : 2; }

// f(pointer of the type) for one of the three element types.
template <typename F>
cudaError_t with_type(int type, F f)
{
    if (type == DQ_TYPE_F32)
        return f(static_cast<float*>(nullptr));
    if (type == DQ_TYPE_F16)
        return f(static_cast<__half*>(nullptr));
    return f(static_cast<__nv_bfloat16*>(nullptr));
}

}  // namespace dqhost
