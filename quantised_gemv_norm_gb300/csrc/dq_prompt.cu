// dq_prompt.cu -- causal attention of packed prompts (dq_attention_prompt).
//
// One warp takes one query row of one head and walks the keys it sees with a
// running maximum and sum, four dims a lane.
#include "dq_attn.cuh"
#include "dq_types.cuh"

namespace dq {

struct PromptArgs {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    long long q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;
    const int* cu_q;
    const int* cu_k;
    int n_seq, total_q, total_k, n_q, group;
    int* err;
};

// Rows [a, b) of sequence s: false (and the error bit) where the offsets do not
// ascend within their total.
__device__ __forceinline__ bool prompt_range(const int* cu, int s, int total, int& a, int& b)
{
    a = cu[s];
    b = cu[s + 1];
    return a >= 0 && a <= b && b <= total;
}

constexpr int PROMPT_WARPS = 4;

template <typename T>
__global__ void __launch_bounds__(32 * PROMPT_WARPS) prompt_kernel(PromptArgs a)
{
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * PROMPT_WARPS + (threadIdx.x >> 5);
    if (item >= static_cast<long long>(a.total_q) * a.n_q)
        return;
    const int row = static_cast<int>(item / a.n_q), h = static_cast<int>(item % a.n_q), g = h / a.group;
    int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    bool found = false;
    for (int s = 0; s < a.n_seq && !found; ++s) {
        const bool ok = prompt_range(a.cu_q, s, a.total_q, q0, q1) && prompt_range(a.cu_k, s, a.total_k, k0, k1);
        if (!ok && lane == 0)
            set_error(a.err, DEVERR_BAD_ARG);
        found = ok && row >= q0 && row < q1;
    }
    if (!found)
        return;
    const int n = min(k1 - k0, row - q0 + (k1 - k0) - (q1 - q0) + 1);
    const float4 q = load4(static_cast<const T*>(a.q) + row * a.q_row + h * a.q_head + 4 * lane);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < n; ++j) {
        const float4 k = load4(static_cast<const T*>(a.k) + (k0 + j) * a.k_row + g * a.k_head + 4 * lane);
        const float4 v = load4(static_cast<const T*>(a.v) + (k0 + j) * a.v_row + g * a.v_head + 4 * lane);
        const float s = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w) * 0.08838834764831845f;
        const float mn = fmaxf(m, s);
        const float corr = expf(m - mn), e = expf(s - mn);
        m = mn;
        l = l * corr + e;
        o.x = o.x * corr + e * v.x;
        o.y = o.y * corr + e * v.y;
        o.z = o.z * corr + e * v.z;
        o.w = o.w * corr + e * v.w;
    }
    const float inv = n < 1 ? 0.f : 1.0f / l;
    store4(static_cast<T*>(a.out) + row * a.o_row + h * a.o_head + 4 * lane,
           make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

}  // namespace dq

extern "C" {

DQ_API size_t dq_attention_prompt_workspace_bytes(int n_seq, int total_q, int total_k, int n_q, int n_kv) { return 0; }

DQ_API int dq_attention_prompt(const dq_prompt* p, void* stream)
{
    if (!p || !p->q || !p->k || !p->v || !p->out || !p->cu_q)
        return DQ_ERR_NULL;
    if (p->n_seq < 1 || p->total_q < 1 || p->total_k < 1 || p->n_q < 1 || p->n_kv < 1 || p->n_q % p->n_kv ||
        (p->type != DQ_TYPE_F16 && p->type != DQ_TYPE_BF16))
        return DQ_ERR_SHAPE;
    const long long rows[4] = {p->q_row_stride, p->k_row_stride, p->v_row_stride, p->out_row_stride};
    const long long heads[4] = {p->q_head_stride, p->k_head_stride, p->v_head_stride, p->out_head_stride};
    for (int i = 0; i < 4; ++i) {
        const bool kv = i == 1 || i == 2;
        if (((kv ? p->total_k : p->total_q) > 1 && rows[i] < dq::ATT_HD) ||
            ((kv ? p->n_kv : p->n_q) > 1 && heads[i] < dq::ATT_HD))
            return DQ_ERR_SHAPE;
    }
    if (p->head_dim != dq::ATT_HD || p->n_q / p->n_kv > 128 || p->total_q > (1 << 30) || p->total_k > (1 << 30))
        return DQ_ERR_UNSUPPORTED;
    for (int i = 0; i < 4; ++i)
        if (rows[i] % 8 || heads[i] % 8)
            return DQ_ERR_ALIGN;
    if (!dqhost::aligned16(p->q) || !dqhost::aligned16(p->k) || !dqhost::aligned16(p->v) || !dqhost::aligned16(p->out))
        return DQ_ERR_ALIGN;
    dq::PromptArgs a{p->q, p->k, p->v, p->out, rows[0], heads[0], rows[1], heads[1], rows[2], heads[2], rows[3], heads[3],
                     p->cu_q, p->cu_k ? p->cu_k : p->cu_q, p->n_seq, p->total_q, p->total_k, p->n_q, p->n_q / p->n_kv,
                     dqhost::device_error_flag()};
    const long long blocks = (static_cast<long long>(p->total_q) * p->n_q + dq::PROMPT_WARPS - 1) / dq::PROMPT_WARPS;
    if (blocks > 0x7fffffffll)
        return DQ_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->type == DQ_TYPE_F16)
        dq::prompt_kernel<__half><<<static_cast<unsigned>(blocks), 32 * dq::PROMPT_WARPS, 0, s>>>(a);
    else
        dq::prompt_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), 32 * dq::PROMPT_WARPS, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
