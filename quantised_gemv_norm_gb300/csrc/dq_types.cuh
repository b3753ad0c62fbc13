// dq_types.cuh -- the element types of the row operators: four consecutive
// elements to and from fp32.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

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

// Eight consecutive elements (16-byte aligned), one or two 16-byte accesses.
__device__ __forceinline__ void load8(const float* p, float (&x)[8])
{
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8])
{
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (std::is_same<T, __half>::value) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = v.x, x[2 * i + 1] = v.y;
        } else {
            x[2 * i] = bf16lo(w[i]), x[2 * i + 1] = bf16hi(w[i]);
        }
    }
}
// store8 is called by both lanes of a pair (2 i, 2 i + 1) for 16 consecutive elements: in
// fp32 they trade halves, so that each 16-byte access of the two fills a sector.
__device__ __forceinline__ void store8(float* p, const float (&x)[8])
{
    const bool odd = threadIdx.x & 1;
    const unsigned pair = 3u << (threadIdx.x & 30);
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = __shfl_xor_sync(pair, odd ? x[i] : x[4 + i], 1);
    float4* at = reinterpret_cast<float4*>(p) - (odd ? 1 : 0);
    at[0] = odd ? make_float4(y[0], y[1], y[2], y[3]) : make_float4(x[0], x[1], x[2], x[3]);
    at[2] = odd ? make_float4(x[4], x[5], x[6], x[7]) : make_float4(y[0], y[1], y[2], y[3]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8])
{
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2(x[0], x[1], p), pack2(x[2], x[3], p), pack2(x[4], x[5], p), pack2(x[6], x[7], p));
}

// n / d for 0 <= n < 2^31 and a divisor known to the host: two instructions.
struct FastDiv {
    uint32_t mul, shift, d;
};
__device__ __forceinline__ uint32_t fast_div(uint32_t n, const FastDiv& f) { return (__umulhi(n, f.mul) + n) >> f.shift; }

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

inline dq::FastDiv fast_divisor(uint32_t d)  // 1 <= d < 2^31
{
    uint32_t shift = 0;
    while ((1ull << shift) < d)
        ++shift;
    return {static_cast<uint32_t>((((1ull << shift) - d) << 32) / d + 1), shift, d};
}

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
