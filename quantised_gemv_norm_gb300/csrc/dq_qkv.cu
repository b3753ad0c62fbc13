// dq_qkv.cu -- head norm and rotary embedding of many rows of projections
// (dq_qkv_rope): the Qwen3 inputs of dq_attention_decode_rope for a prompt's or a
// batch's rows, with the values converted beside them.
//
// Half a warp takes one head, a warp eight heads of one row: lane i of 16 holds dims
// 4 i .. 4 i + 3 and 64 + 4 i .., so a rotation's two dims are in one lane, the sum of
// squares of two heads is four shuffles, and the row's angles are loaded once.  All
// eight heads' loads are issued first.  Memory bounds it: 8191 rows of 48 heads to
// fp16, 306 MB, 55.8 us, 5.5 TB/s (0.81 of the measured copy rate; one warp a head, with
// the partner dims 16 lanes away and divisions for the index, was bound by its 150
// instructions: 80 us).
#include "dq_attn.cuh"
#include "dq_types.cuh"

namespace dq {

struct QkvArgs {
    const float* qkv;
    long long ld;
    const int* pos;
    const float* q_norm;
    const float* k_norm;
    const float2* rope;
    float eps;
    int rows, n_q, n_kv, max_ctx;
    FastDiv by_chunks;  // warps a row
    int* err;
};

constexpr int QKV_WARPS = 8;
constexpr int QKV_PAIRS = 4;  // pairs of heads a warp

template <typename T>
__global__ void __launch_bounds__(32 * QKV_WARPS) qkv_rope_kernel(const QkvArgs a, T* __restrict__ q, T* __restrict__ k,
                                                                  T* __restrict__ v)
{
    const int lane = threadIdx.x & 31, half = lane >> 4, i = lane & 15;
    const uint32_t item = blockIdx.x * QKV_WARPS + (threadIdx.x >> 5);
    const uint32_t row = fast_div(item, a.by_chunks), chunk = item - row * a.by_chunks.d;
    if (row >= static_cast<uint32_t>(a.rows))
        return;
    const int pos = __ldg(a.pos + row);
    if (pos < 0 || pos >= a.max_ctx) {
        if (pos >= 0 && lane == 0)
            set_error(a.err, DEVERR_BAD_ARG);
        return;
    }
    const int heads = a.n_q + 2 * a.n_kv, turned = a.n_q + a.n_kv, h0 = 2 * QKV_PAIRS * chunk + half;
    const float* src = a.qkv + row * a.ld + 4 * i;
    float4 x[QKV_PAIRS], y[QKV_PAIRS];
#pragma unroll
    for (int p = 0; p < QKV_PAIRS; ++p) {
        const int h = h0 + 2 * p;
        if (h < heads) {
            x[p] = __ldcs(reinterpret_cast<const float4*>(src + h * ATT_HD));
            y[p] = __ldcs(reinterpret_cast<const float4*>(src + h * ATT_HD + 64));
        }
    }
    const float4* cs = reinterpret_cast<const float4*>(a.rope + static_cast<size_t>(pos) * (ATT_HD / 2) + 4 * i);
    const float4 c01 = __ldg(cs), c23 = __ldg(cs + 1);  // cos, sin, cos, sin
#pragma unroll
    for (int p = 0; p < QKV_PAIRS; ++p) {
        const int h = h0 + 2 * p;
        if (a.q_norm && h - half < turned) {  // not for a pair of value heads
            float s = 0.f;
            if (h < turned)
                s = (x[p].x * x[p].x + x[p].y * x[p].y + x[p].z * x[p].z + x[p].w * x[p].w) +
                    (y[p].x * y[p].x + y[p].y * y[p].y + y[p].z * y[p].z + y[p].w * y[p].w);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, o);
            if (h < turned) {
                const float r = rsqrtf(s * (1.0f / ATT_HD) + a.eps);
                const float4* w = reinterpret_cast<const float4*>(h < a.n_q ? a.q_norm : a.k_norm) + i;
                const float4 u = __ldg(w), t = __ldg(w + 16);
                x[p] = make_float4(x[p].x * r * u.x, x[p].y * r * u.y, x[p].z * r * u.z, x[p].w * r * u.w);
                y[p] = make_float4(y[p].x * r * t.x, y[p].y * r * t.y, y[p].z * r * t.z, y[p].w * r * t.w);
            }
        }
        if (h >= heads)
            continue;
        T* out = h < a.n_q   ? q + (static_cast<size_t>(row) * a.n_q + h) * ATT_HD
                 : h < turned ? k + (static_cast<size_t>(row) * a.n_kv + (h - a.n_q)) * ATT_HD
                              : v + (static_cast<size_t>(row) * a.n_kv + (h - turned)) * ATT_HD;
        if (h < turned) {
            const float4 b = x[p], c = y[p];
            x[p] = make_float4(fmaf(b.x, c01.x, -(c.x * c01.y)), fmaf(b.y, c01.z, -(c.y * c01.w)),
                               fmaf(b.z, c23.x, -(c.z * c23.y)), fmaf(b.w, c23.z, -(c.w * c23.w)));
            y[p] = make_float4(fmaf(c.x, c01.x, b.x * c01.y), fmaf(c.y, c01.z, b.y * c01.w),
                               fmaf(c.z, c23.x, b.z * c23.y), fmaf(c.w, c23.z, b.w * c23.w));
        }
        store4(out + 4 * i, x[p]);
        store4(out + 64 + 4 * i, y[p]);
    }
}

}  // namespace dq

extern "C" {

DQ_API int dq_qkv_rope(const float* qkv, long long row_stride, const int* positions, const float* q_norm,
                       const float* k_norm, const float* rope_table, float eps, int rows, int n_q, int n_kv,
                       int head_dim, int max_ctx, int type, void* q_out, void* k_out, void* v_out, void* stream)
{
    if (!qkv || !positions || !rope_table || !q_out || !k_out || !v_out || !q_norm != !k_norm)
        return DQ_ERR_NULL;
    if (rows < 1 || n_q < 1 || n_kv < 1 || max_ctx < 1 || !dqhost::valid_eps(eps) || !dqhost::valid_type(type))
        return DQ_ERR_SHAPE;
    if (head_dim != dq::ATT_HD || n_q > (1 << 16) || n_kv > (1 << 16))
        return DQ_ERR_UNSUPPORTED;
    const long long heads = n_q + 2ll * n_kv;
    if (row_stride < heads * dq::ATT_HD)
        return DQ_ERR_SHAPE;
    if (row_stride % 4 || !dqhost::aligned16(qkv) || !dqhost::aligned16(rope_table) || !dqhost::aligned16(q_out) ||
        !dqhost::aligned16(k_out) || !dqhost::aligned16(v_out) || !dqhost::aligned16(q_norm) ||
        !dqhost::aligned16(k_norm))
        return DQ_ERR_ALIGN;
    dq::QkvArgs a{qkv,  row_stride, positions, q_norm,  k_norm, reinterpret_cast<const float2*>(rope_table), eps,
                  rows, n_q,        n_kv,      max_ctx};
    const int chunks = static_cast<int>((heads + 2 * dq::QKV_PAIRS - 1) / (2 * dq::QKV_PAIRS));
    const long long items = static_cast<long long>(rows) * chunks, blocks = (items + dq::QKV_WARPS - 1) / dq::QKV_WARPS;
    if (items > 0x7fffff00ll)
        return DQ_ERR_UNSUPPORTED;
    a.by_chunks = dqhost::fast_divisor(chunks);
    a.err = dqhost::device_error_flag();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dqhost::with_type(type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        dq::qkv_rope_kernel<T><<<static_cast<unsigned>(blocks), 32 * dq::QKV_WARPS, 0, s>>>(
            a, static_cast<T*>(q_out), static_cast<T*>(k_out), static_cast<T*>(v_out));
        return cudaGetLastError();
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
