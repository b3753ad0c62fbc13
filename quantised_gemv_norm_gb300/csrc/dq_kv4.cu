// dq_kv4.cu -- rows into a paged 4-bit cache and back (dq_kv4_append,
// dq_kv4_read).
//
// One warp takes one head's key or value row, four dims a lane, so a group of 32
// dims with one scale is eight lanes: its extremes are three shuffles.
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
    int* err;
};

// d, z and the four codes (nibbles 0..3, unsigned) of a lane's dims; the group is
// the lane's eight neighbours.  Every step is one IEEE operation, as the format
// defines it.
__device__ __forceinline__ uint32_t kv4_quantise(float4 x, float& d, float& z)
{
    float lo = fminf(fminf(x.x, x.y), fminf(x.z, x.w)), hi = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
    // 0 * x is NaN for an infinity or NaN, which fminf and fmaxf would pass over
    bool bad = !(0.f * x.x + 0.f * x.y + 0.f * x.z + 0.f * x.w == 0.f);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const uint32_t group = 0xffu << (threadIdx.x & 24);
    bad = (__ballot_sync(0xffffffffu, bad) & group) != 0u;
    d = __half2float(__float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f)));
    z = __half2float(__float2half_rn(__fadd_rn(lo, 8.0f * d)));
    if (bad || !(fabsf(d) <= 65504.f) || !(fabsf(z) <= 65504.f)) {
        d = z = __int_as_float(0x7fc00000);
        return 0x8888u;
    }
    if (d == 0.f)
        return 0x8888u;
    const float v[4] = {x.x, x.y, x.z, x.w};
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float t = rintf(__fdiv_rn(__fsub_rn(v[i], z), d)) + 8.0f;
        c |= static_cast<uint32_t>(fminf(fmaxf(t, 0.f), 15.f)) << (4 * i);
    }
    return c;
}

template <typename T>
__global__ void __launch_bounds__(32 * KV4_WARPS) kv4_append_kernel(Kv4AppendArgs a)
{
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * KV4_WARPS + (threadIdx.x >> 5);
    const int per = 2 * a.s.n_kv;
    if (item >= static_cast<long long>(a.rows) * per)
        return;
    const int row = static_cast<int>(item / per), hh = static_cast<int>(item % per);
    const int g = hh >> 1, value = hh & 1;
    const int slot = __ldg(a.slots + row);
    if (slot < 0)
        return;
    const int page = slot / a.s.page_rows, off = slot % a.s.page_rows, j = off % KV4_ROWS;
    if (page >= a.s.n_pages) {
        if (lane == 0)
            set_error(a.err, DEVERR_BAD_ARG);
        return;
    }
    const T* src = value ? static_cast<const T*>(a.v) + row * a.v_row + g * a.v_head
                         : static_cast<const T*>(a.k) + row * a.k_row + g * a.k_head;
    float d, z;
    uint32_t c = kv4_quantise(load4(src + 4 * lane), d, z);
    unsigned char* b = a.pool + kv4_block(a.s, page, off, g);
    const int grp = lane >> 3, w = lane & 7;
    if (value) {
        *reinterpret_cast<unsigned short*>(b + kv4_value_half(j, w, grp)) = static_cast<unsigned short>(c);
    } else {
        // dims e = 0..3 (even lane) or 4..7: e = 2 i + s at bits 4 i + 16 s
        c = (c & 0xfu) | ((c >> 4) & 0xfu) << 16 | ((c >> 8) & 0xfu) << 4 | ((c >> 12) & 0xfu) << 20;
        c <<= 8 * (lane & 1);
        c |= __shfl_xor_sync(0xffffffffu, c, 1);
        if (!(lane & 1))
            *reinterpret_cast<uint32_t*>(b + kv4_key_word(j, w >> 1, grp)) = c;
    }
    if (w == 0) {
        __half* p = reinterpret_cast<__half*>(b + kv4_scale(value ? KV4_VSCALES : KV4_KSCALES, j, grp));
        p[0] = __float2half_rn(d);
        p[2] = __float2half_rn(z);
    }
}

struct Kv4ReadArgs {
    const unsigned char* pool;
    const int* slots;
    int rows;
    Kv4Shape s;
    int* err;
};

template <typename T>
__global__ void __launch_bounds__(32 * KV4_WARPS) kv4_read_kernel(Kv4ReadArgs a, T* __restrict__ k, T* __restrict__ v)
{
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * KV4_WARPS + (threadIdx.x >> 5);
    if (item >= static_cast<long long>(a.rows) * a.s.n_kv)
        return;
    const int row = static_cast<int>(item / a.s.n_kv), g = static_cast<int>(item % a.s.n_kv);
    const int slot = __ldg(a.slots + row);
    if (slot < 0)
        return;
    const int page = slot / a.s.page_rows, off = slot % a.s.page_rows, j = off % KV4_ROWS;
    if (page >= a.s.n_pages) {
        if (lane == 0)
            set_error(a.err, DEVERR_BAD_ARG);
        return;
    }
    const unsigned char* b = a.pool + kv4_block(a.s, page, off, g);
    const int grp = lane >> 3, w = lane & 7;
#pragma unroll
    for (int value = 0; value < 2; ++value) {
        uint32_t c;
        if (value) {
            c = *reinterpret_cast<const unsigned short*>(b + kv4_value_half(j, w, grp));
        } else {
            c = *reinterpret_cast<const uint32_t*>(b + kv4_key_word(j, w >> 1, grp)) >> (8 * (lane & 1));
            c = (c & 0xfu) | ((c >> 16) & 0xfu) << 4 | ((c >> 4) & 0xfu) << 8 | ((c >> 20) & 0xfu) << 12;
        }
        const __half* p = reinterpret_cast<const __half*>(b + kv4_scale(value ? KV4_VSCALES : KV4_KSCALES, j, grp));
        const float d = __half2float(p[0]), z = __half2float(p[2]);
        float4 x;
        x.x = fmaf(d, static_cast<float>(static_cast<int>(c & 15u) - 8), z);
        x.y = fmaf(d, static_cast<float>(static_cast<int>((c >> 4) & 15u) - 8), z);
        x.z = fmaf(d, static_cast<float>(static_cast<int>((c >> 8) & 15u) - 8), z);
        x.w = fmaf(d, static_cast<float>(static_cast<int>((c >> 12) & 15u) - 8), z);
        store4((value ? v : k) + (static_cast<size_t>(row) * a.s.n_kv + g) * ATT_HD + 4 * lane, x);
    }
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
                        static_cast<unsigned char*>(pool), rows, {n_kv, n_pages, page_size}, dqhost::device_error_flag()};
    const long long blocks = (2ll * rows * n_kv + dq::KV4_WARPS - 1) / dq::KV4_WARPS;
    if (blocks > 0x7fffffffll)
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
    dq::Kv4ReadArgs a{static_cast<const unsigned char*>(pool), slots, rows, {n_kv, n_pages, page_size},
                      dqhost::device_error_flag()};
    const long long blocks = (static_cast<long long>(rows) * n_kv + dq::KV4_WARPS - 1) / dq::KV4_WARPS;
    if (blocks > 0x7fffffffll)
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
