// dq_kv4_attn.cu -- single-token attention of a batch of sequences over the paged
// 4-bit cache (dq_attention_decode_kv4).
//
// One warp takes one query head of one sequence and walks its keys with a running
// maximum and sum.
#include "dq_kv4.cuh"

namespace dq {

struct Kv4AttnArgs {
    const void* q;
    void* out;
    const unsigned char* pool;
    const int* pages;
    const int* n_keys;
    int n_seq, n_q, group;
    Kv4Shape s;
    int max_pages, max_keys;
    int* err;
};

template <typename T>
__global__ void __launch_bounds__(32) kv4_attn_kernel(Kv4AttnArgs a)
{
    const int lane = threadIdx.x;
    const int b = blockIdx.x / a.n_q, h = blockIdx.x % a.n_q, g = h / a.group;
    const size_t at = static_cast<size_t>(blockIdx.x) * ATT_HD + 4 * lane;
    const float4 q = load4(static_cast<const T*>(a.q) + at);
    int n = a.n_keys[b];
    if (n < 0 || n > a.max_keys) {
        if (lane == 0)
            set_error(a.err, DEVERR_BAD_ARG);
        n = 0;
    }
    const int grp = lane >> 3, w = lane & 7;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < n; ++j) {
        const int page = a.pages[static_cast<size_t>(b) * a.max_pages + j / a.s.page_rows];
        if (page < 0 || page >= a.s.n_pages) {
            if (lane == 0)
                set_error(a.err, DEVERR_BAD_ARG);
            continue;
        }
        const unsigned char* p = a.pool + kv4_block(a.s, page, j % a.s.page_rows, g);
        const int r = j % KV4_ROWS;
        const uint32_t kc = *reinterpret_cast<const uint32_t*>(p + kv4_key_word(r, w >> 1, grp)) >> (8 * (lane & 1));
        const uint32_t vc = *reinterpret_cast<const unsigned short*>(p + kv4_value_half(r, w, grp));
        const __half* ks = reinterpret_cast<const __half*>(p + kv4_scale(KV4_KSCALES, r, grp));
        const __half* vs = reinterpret_cast<const __half*>(p + kv4_scale(KV4_VSCALES, r, grp));
        const float kd = __half2float(ks[0]), kz = __half2float(ks[2]);
        const float vd = __half2float(vs[0]), vz = __half2float(vs[2]);
        auto val = [](uint32_t c, int bit, float d, float z) {
            return fmaf(d, static_cast<float>(static_cast<int>((c >> bit) & 15u) - 8), z);
        };
        float s = q.x * val(kc, 0, kd, kz) + q.y * val(kc, 16, kd, kz) + q.z * val(kc, 4, kd, kz) +
                  q.w * val(kc, 20, kd, kz);
        s = warp_sum(s) * 0.08838834764831845f;
        const float mn = fmaxf(m, s);
        const float corr = expf(m - mn), e = expf(s - mn);
        m = mn;
        l = l * corr + e;
        o.x = o.x * corr + e * val(vc, 0, vd, vz);
        o.y = o.y * corr + e * val(vc, 4, vd, vz);
        o.z = o.z * corr + e * val(vc, 8, vd, vz);
        o.w = o.w * corr + e * val(vc, 12, vd, vz);
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    store4(static_cast<T*>(a.out) + at, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

}  // namespace dq

extern "C" {

DQ_API size_t dq_attention_decode_kv4_workspace_bytes(int n_seq, int n_q, int n_kv, int max_keys)
{
    return 0;
}

DQ_API int dq_attention_decode_kv4(const void* q, int type, const void* pool, const int* pages, const int* n_keys,
                                   void* out, int n_seq, int n_q, int n_kv, int head_dim, int n_pages, int page_size,
                                   int max_pages, int max_keys, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!q || !pool || !pages || !n_keys || !out)
        return DQ_ERR_NULL;
    if (n_seq < 1 || n_q < 1 || n_kv < 1 || n_q % n_kv || max_pages < 1 || max_keys < 1 || !dqhost::valid_type(type))
        return DQ_ERR_SHAPE;
    const int st = dqhost::kv4_check_shape(n_kv, head_dim, n_pages, page_size);
    if (st != DQ_OK)
        return st;
    if (max_keys > static_cast<long long>(max_pages) * page_size)
        return DQ_ERR_SHAPE;
    if (n_q / n_kv > 8 || static_cast<long long>(n_seq) * n_q > 0x7fffffffll)
        return DQ_ERR_UNSUPPORTED;
    if (!dqhost::aligned16(q) || !dqhost::aligned16(pool) || !dqhost::aligned16(out))
        return DQ_ERR_ALIGN;
    dq::Kv4AttnArgs a{q,     out,      static_cast<const unsigned char*>(pool), pages,     n_keys,   n_seq,
                      n_q,   n_q / n_kv, {n_kv, n_pages, page_size},             max_pages, max_keys, dqhost::device_error_flag()};
    cudaError_t e = dqhost::with_type(type, [&](auto* t) {
        dq::kv4_attn_kernel<std::remove_pointer_t<decltype(t)>>
            <<<n_seq * n_q, 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
        return cudaGetLastError();
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
