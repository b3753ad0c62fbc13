// dq_qkv.cu -- head norm and rotary embedding of many rows of projections
// (dq_qkv_rope): the Qwen3 inputs of dq_attention_decode_rope for a prompt's or a
// batch's rows, with the values converted beside them.
//
// One warp takes one head of one row, four dims a lane: the head's sum of squares
// is one warp reduction, a dim's rotation partner sits 16 lanes away.
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
    int* err;
};

constexpr int QKV_WARPS = 8;

template <typename T>
__global__ void __launch_bounds__(32 * QKV_WARPS) qkv_rope_kernel(QkvArgs a, T* __restrict__ q, T* __restrict__ k,
                                                                  T* __restrict__ v)
{
    const int lane = threadIdx.x & 31;
    const int heads = a.n_q + 2 * a.n_kv;
    const long long item = static_cast<long long>(blockIdx.x) * QKV_WARPS + (threadIdx.x >> 5);
    if (item >= static_cast<long long>(a.rows) * heads)
        return;
    const int row = static_cast<int>(item / heads), h = static_cast<int>(item % heads);
    const int pos = __ldg(a.pos + row);
    if (pos < 0 || pos >= a.max_ctx) {
        if (pos >= 0 && lane == 0)
            set_error(a.err, DEVERR_BAD_ARG);
        return;
    }
    float4 x = load4(a.qkv + row * a.ld + static_cast<long long>(h) * ATT_HD + 4 * lane);
    T* out = h < a.n_q ? q + (static_cast<size_t>(row) * a.n_q + h) * ATT_HD
             : h < a.n_q + a.n_kv ? k + (static_cast<size_t>(row) * a.n_kv + (h - a.n_q)) * ATT_HD
                                  : v + (static_cast<size_t>(row) * a.n_kv + (h - a.n_q - a.n_kv)) * ATT_HD;
    if (h < a.n_q + a.n_kv) {
        const float2* cs = a.rope + static_cast<size_t>(pos) * (ATT_HD / 2);
        const float* w = h < a.n_q ? a.q_norm : a.k_norm;
        x = w ? head_norm_rope(x, load_norm_rope(w, cs, lane), a.eps, lane) : head_rope(x, cs, lane);
    }
    store4(out + 4 * lane, x);
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
                  rows, n_q,        n_kv,      max_ctx, dqhost::device_error_flag()};
    const long long blocks = (rows * heads + dq::QKV_WARPS - 1) / dq::QKV_WARPS;
    if (blocks > 0x7fffffffll)
        return DQ_ERR_UNSUPPORTED;
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
