// dq_kv4.cu -- rows into a paged 4-bit cache and back (dq_kv4_append,
// dq_kv4_read).
//
// Half a warp takes one head's key and value row, eight dims a lane: 16 bytes of a
// 16-bit row, one 32-bit word of key codes, two halves of value words.  A group of 32
// dims with one scale is four lanes: its extremes are two shuffles.  A warp and a
// division for each code took 55 us for 8000 rows of 8 heads stored and read back;
// now the store takes 17 us (33 MB of fp16 in, 10 MB out; its 360 instructions for two
// rows are issued at 0.7 of the rate) and the read to fp32 14 us (76 MB, 5.4 TB/s).
// 16000 rows to bf16: 20.5 us, 86 MB, 4.2 TB/s.
#include "dq_kv4.cuh"

namespace dq {

constexpr int KV4_WARPS = 8;

struct Kv4AppendArgs {
    const void* k;
    const void* v;
    long long k_row, k_head, v_row, v_head;  // strides in elements
    const int* slots;
    unsigned char* pool;
    int rows;
    Kv4Shape s;
    FastDiv by_kv, by_page;
    int* err;
};

// The cache block of a slot (a page's rows are consecutive) and head; null, and the
// error bit, where the slot is past the pool.  Sets j, the row in the block.
__device__ __forceinline__ unsigned char* kv4_find(unsigned char* pool, const Kv4Shape& s, const FastDiv& by_page, int slot,
                                                   int g, int* err, int& j)
{
    const int page = static_cast<int>(fast_div(static_cast<uint32_t>(slot), by_page));
    const int off = slot - page * s.page_rows;
    j = off % KV4_ROWS;
    if (page >= s.n_pages) {
        if ((threadIdx.x & 15) == 0)
            set_error(err, DEVERR_BAD_ARG);
        return nullptr;
    }
    return pool + ((static_cast<size_t>(page) * s.n_kv + g) * (s.page_rows / KV4_ROWS) + off / KV4_ROWS) * KV4_BYTES;
}

__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// d, z and eight codes of a lane's dims, code i at bits SHIFT(i) of the word; the group
// is the lane and its three neighbours.  Extremes, d, z and x - z are the format's IEEE
// operations.  The quotient is a product with 1 / d, off by less than 1e-5 where it is
// below 16: only within that of a half can the rounding differ from the quotient's own,
// and there the division is done.
template <typename Shift>
__device__ __forceinline__ uint32_t kv4_quantise(const float (&x)[8], float& d, float& z, Shift shift)
{
    float lo = min_nan(min_nan(min_nan(x[0], x[1]), min_nan(x[2], x[3])), min_nan(min_nan(x[4], x[5]), min_nan(x[6], x[7])));
    float hi = max_nan(max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])), max_nan(max_nan(x[4], x[5]), max_nan(x[6], x[7])));
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    // (hi - lo) / 15 as IEEE division rounds it: the product with 1 / 15, corrected once by
    // its exact remainder (the method of P. Markstein, IBM Journal of Research and Development
    // 34(1), 1990); the tests go through every fp32 mantissa
    const float range = __fsub_rn(hi, lo), part = __fmul_rn(range, 1.f / 15.f);
    d = __half2float(__float2half_rn(__fmaf_rn(__fmaf_rn(-15.f, part, range), 1.f / 15.f, part)));
    z = __half2float(__float2half_rn(__fadd_rn(lo, 8.0f * d)));
    if (!(d <= 65504.f) || !(fabsf(z) <= 65504.f))  // also an infinity or NaN among them
        d = z = __int_as_float(0x7fc00000);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
    inv = d > 0.f ? inv : 0.f;
    constexpr float M = 12582912.f;  // 1.5 2^23: adding it rounds to an integer, halves to even
    const uint64_t z2 = f2(-z, -z), inv2 = f2(inv, inv), eight = f2(8.f, 8.f), m2 = f2(M, M), nm2 = f2(-M, -M);
    uint32_t word = 0, base = 0;
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = un2(fma2(add2(f2(x[2 * i], x[2 * i + 1]), z2), inv2, eight));
        const uint64_t c = f2(fminf(fmaxf(t.x, 0.f), 15.f), fminf(fmaxf(t.y, 0.f), 15.f));
        const uint64_t u = add2(c, m2);
        const float2 e = un2(fma2(add2(u, nm2), f2(-1.f, -1.f), c)), bits = un2(u);
        off = fmaxf(off, fmaxf(fabsf(e.x), fabsf(e.y)));
        // the integer in M's low mantissa bits, M's own bits taken off at the end
        word += __float_as_uint(bits.x) << shift(2 * i);
        word += __float_as_uint(bits.y) << shift(2 * i + 1);
        base += 0x4B400000u << shift(2 * i);
        base += 0x4B400000u << shift(2 * i + 1);
    }
    word -= base;
    if (off > 0.49998f) {
        word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = rintf(__fdiv_rn(__fsub_rn(x[i], z), d)) + 8.f;
            word |= static_cast<uint32_t>(fminf(fmaxf(t, 0.f), 15.f)) << shift(i);
        }
    }
    return word;
}

template <typename T>
__global__ void __launch_bounds__(32 * KV4_WARPS) kv4_append_kernel(const Kv4AppendArgs a)
{
    // a warp takes rows 2 i and 2 i + 1 of one head
    const uint32_t item = blockIdx.x * KV4_WARPS + (threadIdx.x >> 5);
    const uint32_t pair = fast_div(item, a.by_kv), g = item - pair * a.by_kv.d;
    const int row = static_cast<int>(2 * pair + ((threadIdx.x >> 4) & 1));
    const int slot = row < a.rows ? __ldg(a.slots + row) : -1;
    int j = 0;
    unsigned char* b = slot < 0 ? nullptr : kv4_find(a.pool, a.s, a.by_page, slot, g, a.err, j);
    if (!__any_sync(0xffffffffu, b != nullptr))
        return;
    const int dim = threadIdx.x & 15, grp = dim >> 2, t = dim & 3;
    float x[2][8] = {};
    if (b) {
        load8(static_cast<const T*>(a.k) + row * a.k_row + g * a.k_head + 8 * dim, x[0]);
        load8(static_cast<const T*>(a.v) + row * a.v_row + g * a.v_head + 8 * dim, x[1]);
    }
    float kd, kz, vd, vz;
    const uint32_t kw = kv4_quantise(x[0], kd, kz, [](int i) { return 4 * (i >> 1) + 16 * (i & 1); });
    const uint32_t vw = kv4_quantise(x[1], vd, vz, [](int i) { return 4 * i; });
    if (!b)
        return;
    *reinterpret_cast<uint32_t*>(b + kv4_key_word(j, t, grp)) = kw;
    unsigned short* p = reinterpret_cast<unsigned short*>(b + kv4_value_half(j, t, grp));
    p[0] = static_cast<unsigned short>(vw);
    p[32] = static_cast<unsigned short>(vw >> 16);
    // the four scales of a group, one a lane: d and z of the key, d and z of the value
    *reinterpret_cast<__half*>(b + kv4_scale(t & 2 ? KV4_VSCALES : KV4_KSCALES, j, grp) + 4 * (t & 1)) =
        __float2half_rn(t & 2 ? (t & 1 ? vz : vd) : (t & 1 ? kz : kd));
}

struct Kv4ReadArgs {
    unsigned char* pool;  // read
    const int* slots;
    int rows;
    Kv4Shape s;
    FastDiv by_kv, by_page;
    int* err;
};

template <typename T>
__global__ void __launch_bounds__(32 * KV4_WARPS) kv4_read_kernel(const Kv4ReadArgs a, T* __restrict__ k, T* __restrict__ v)
{
    const uint32_t item = 2 * (blockIdx.x * KV4_WARPS + (threadIdx.x >> 5)) + ((threadIdx.x >> 4) & 1);
    const uint32_t row = fast_div(item, a.by_kv), g = item - row * a.by_kv.d;
    const int slot = row < static_cast<uint32_t>(a.rows) ? __ldg(a.slots + row) : -1;
    int j = 0;
    const unsigned char* b = slot < 0 ? nullptr : kv4_find(a.pool, a.s, a.by_page, slot, g, a.err, j);
    if (!b)
        return;
    const int dim = threadIdx.x & 15, grp = dim >> 2, t = dim & 3;
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(b + kv4_key_word(j, t, grp));
    const unsigned short* vp = reinterpret_cast<const unsigned short*>(b + kv4_value_half(j, t, grp));
    const uint32_t vw = vp[0] | static_cast<uint32_t>(vp[32]) << 16;
    const __half* ks = reinterpret_cast<const __half*>(b + kv4_scale(KV4_KSCALES, j, grp));
    const __half* vs = reinterpret_cast<const __half*>(b + kv4_scale(KV4_VSCALES, j, grp));
    const float kd = __half2float(ks[0]), kz = __half2float(ks[2]), vd = __half2float(vs[0]), vz = __half2float(vs[2]);
    // a code at bits n .. n + 3 (n < 20) under 2^23 is 2^23 + 2^n c exactly, and d 2^-n exact
    uint32_t e23;  // 2^23's bits in a register: as a constant beside the mask they cost an instruction more
    asm volatile("mov.b32 %0, 0x4B000000;" : "=r"(e23));
    auto value = [&](uint32_t w, int n, float d, float z) {
        const float s = static_cast<float>(1 << n);
        uint32_t u;
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(w), "r"(15u << n), "r"(e23));
        return fmaf(d * (1.f / s), __uint_as_float(u) - (8388608.f + 8.f * s), z);
    };
    const size_t at = static_cast<size_t>(item) * ATT_HD + 8 * dim;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = value(i & 1 ? kw >> 16 : kw, 4 * (i >> 1), kd, kz);
    store8(k + at, x);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = value(i & 4 ? vw >> 16 : vw, 4 * (i & 3), vd, vz);
    store8(v + at, x);
}

}  // namespace dq

extern "C" {

DQ_API int dq_kv4_append(const void* k, const void* v, int type, long long k_row_stride, long long k_head_stride,
                         long long v_row_stride, long long v_head_stride, const int* slots, void* pool, int rows,
                         int n_kv, int head_dim, int n_pages, int page_size, void* stream)
{
    if (!k || !v || !slots || !pool)
        return DQ_ERR_NULL;
    if (rows < 1 || !dqhost::valid_type(type))
        return DQ_ERR_SHAPE;
    const int st = dqhost::kv4_check_shape(n_kv, head_dim, n_pages, page_size);
    if (st != DQ_OK)
        return st;
    if ((rows > 1 && (k_row_stride < dq::ATT_HD || v_row_stride < dq::ATT_HD)) ||
        (n_kv > 1 && (k_head_stride < dq::ATT_HD || v_head_stride < dq::ATT_HD)))
        return DQ_ERR_SHAPE;
    const int quad = 16 / dqhost::type_bytes(type);
    if (!dqhost::aligned16(k) || !dqhost::aligned16(v) || !dqhost::aligned16(pool) ||
        (rows > 1 && (k_row_stride % quad || v_row_stride % quad)) ||
        (n_kv > 1 && (k_head_stride % quad || v_head_stride % quad)))
        return DQ_ERR_ALIGN;
    dq::Kv4AppendArgs a{k, v, k_row_stride, k_head_stride, v_row_stride, v_head_stride, slots,
                        static_cast<unsigned char*>(pool), rows, {n_kv, n_pages, page_size}, dqhost::fast_divisor(n_kv),
                        dqhost::fast_divisor(page_size), dqhost::device_error_flag()};
    const long long items = (static_cast<long long>(rows) + 1) / 2 * n_kv, blocks = (items + dq::KV4_WARPS - 1) / dq::KV4_WARPS;
    if (items > 0x7fffff00ll)
        return DQ_ERR_UNSUPPORTED;
    cudaError_t e = dqhost::with_type(type, [&](auto* t) {
        dq::kv4_append_kernel<std::remove_pointer_t<decltype(t)>>
            <<<static_cast<unsigned>(blocks), 32 * dq::KV4_WARPS, 0, static_cast<cudaStream_t>(stream)>>>(a);
        return cudaGetLastError();
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

DQ_API int dq_kv4_read(const void* pool, const int* slots, int type, void* k_out, void* v_out, int rows, int n_kv,
                       int head_dim, int n_pages, int page_size, void* stream)
{
    if (!pool || !slots || !k_out || !v_out)
        return DQ_ERR_NULL;
    if (rows < 1 || !dqhost::valid_type(type))
        return DQ_ERR_SHAPE;
    const int st = dqhost::kv4_check_shape(n_kv, head_dim, n_pages, page_size);
    if (st != DQ_OK)
        return st;
    if (!dqhost::aligned16(pool) || !dqhost::aligned16(k_out) || !dqhost::aligned16(v_out))
        return DQ_ERR_ALIGN;
    dq::Kv4ReadArgs a{static_cast<unsigned char*>(const_cast<void*>(pool)), slots, rows, {n_kv, n_pages, page_size},
                      dqhost::fast_divisor(n_kv), dqhost::fast_divisor(page_size), dqhost::device_error_flag()};
    const long long items = static_cast<long long>(rows) * n_kv;
    const long long blocks = (items + 2 * dq::KV4_WARPS - 1) / (2 * dq::KV4_WARPS);
    if (items > 0x7fffff00ll)
        return DQ_ERR_UNSUPPORTED;
    cudaError_t e = dqhost::with_type(type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        dq::kv4_read_kernel<T>
            <<<static_cast<unsigned>(blocks), 32 * dq::KV4_WARPS, 0, static_cast<cudaStream_t>(stream)>>>(
                a, static_cast<T*>(k_out), static_cast<T*>(v_out));
        return cudaGetLastError();
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
