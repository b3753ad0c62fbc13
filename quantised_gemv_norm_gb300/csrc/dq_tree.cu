// dq_tree.cu -- attention of a few new tokens of each sequence, a drafted tree, a chain
// or one, over a paged 16-bit cache (dq_attention_tree).
#include <algorithm>

#include "dq_kv16.cuh"

namespace dq {

constexpr float TR_C = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(128)
constexpr int TR_MAX_NEW = 64, TR_MAX_GROUP = 64;

struct TreeArgs {
    const void* q;
    void* out;
    long long q_row, q_head, o_row, o_head;
    const void* pool;
    const int* pages;
    const int* n_past;
    const int* cu_new;
    const unsigned long long* seen;
    int n_seq, total_new, max_new, n_q, group, max_pages;
    Kv16Shape s;
    int* err;
};

// A sequence's new rows, and the keys before them; no rows where cu_new is not in order.
struct TreeSeq {
    int row0, rows, past;
    bool bad;  // no keys: n_past does not fit
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int s)
{
    TreeSeq t;
    int r1;
    if (a.cu_new) {
        t.row0 = __ldg(a.cu_new + s);
        r1 = __ldg(a.cu_new + s + 1);
    } else {
        t.row0 = s * a.max_new;
        r1 = t.row0 + a.max_new;
    }
    t.past = __ldg(a.n_past + s);
    const bool in_order = t.row0 >= 0 && r1 >= t.row0 && r1 <= a.total_new && r1 - t.row0 <= a.max_new;
    t.rows = in_order ? r1 - t.row0 : 0;
    t.bad = t.past < 0 || static_cast<long long>(t.past) + t.rows > static_cast<long long>(a.max_pages) * a.s.page_rows;
    if (t.bad || !in_order)
        set_error(a.err, DEVERR_BAD_ARG);
    if (t.bad)
        t.past = 0;
    return t;
}

// One block a new token and query head; a warp takes every fourth key, four dims a lane.
template <typename T>
__global__ void __launch_bounds__(128) tree_simple_kernel(const TreeArgs a)
{
    __shared__ float ml[4][2];
    __shared__ float4 sums[4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.x / a.max_new, i = blockIdx.x % a.max_new, h = blockIdx.y, g = h / a.group;
    const TreeSeq t = tree_seq(a, s);
    if (i >= t.rows)
        return;
    const int row = t.row0 + i;
    const unsigned long long seen = a.seen ? a.seen[row] : (2ull << i) - 1;
    const float4 q = load4(static_cast<const T*>(a.q) + row * a.q_row + h * a.q_head + 4 * lane);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const int keys = t.bad ? 0 : t.past + t.rows;
    for (int j = warp; j < keys; j += 4) {
        if (j >= t.past && !(seen >> (j - t.past) & 1))
            continue;
        const int page = a.pages[static_cast<size_t>(s) * a.max_pages + j / a.s.page_rows];
        if (page < 0 || page >= a.s.n_pages) {
            set_error(a.err, DEVERR_BAD_ARG);
            continue;
        }
        const T* pool = static_cast<const T*>(a.pool);
        const float4 k = load4(pool + (kv16_row(a.s, page, 0, g) + j % a.s.page_rows) * ATT_HD + 4 * lane);
        const float4 v = load4(pool + (kv16_row(a.s, page, 1, g) + j % a.s.page_rows) * ATT_HD + 4 * lane);
        const float x = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w);
        const float mn = fmaxf(m, x), f = mn == m ? 1.f : ex2((m - mn) * TR_C), p = mn == -INFINITY ? 0.f : ex2((x - mn) * TR_C);
        m = mn;
        l = l * f + p;
        o = make_float4(o.x * f + p * v.x, o.y * f + p * v.y, o.z * f + p * v.z, o.w * f + p * v.w);
    }
    if (lane == 0) {
        ml[warp][0] = m;
        ml[warp][1] = l;
    }
    sums[warp][lane] = o;
    __syncthreads();
    if (warp)
        return;
    for (int w = 1; w < 4; ++w)
        m = fmaxf(m, ml[w][0]);
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < 4; ++w) {
        const float f = ml[w][0] == m ? 1.f : ex2((ml[w][0] - m) * TR_C);
        const float4 y = sums[w][lane];
        l += f * ml[w][1];
        o = make_float4(o.x + f * y.x, o.y + f * y.y, o.z + f * y.z, o.w + f * y.w);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    store4(static_cast<T*>(a.out) + row * a.o_row + h * a.o_head + 4 * lane,
           l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

}  // namespace dq

extern "C" {

DQ_API size_t dq_attention_tree_workspace_bytes(int n_seq, int max_new, int n_q, int n_kv)
{
    if (n_seq < 1 || max_new < 1 || max_new > dq::TR_MAX_NEW || n_q < 1 || n_kv < 1 || n_q % n_kv ||
        n_q / n_kv > dq::TR_MAX_GROUP)
        return 0;
    return 16;
}

DQ_API int dq_attention_tree(const dq_tree* t, void* stream)
{
    if (!t || !t->q || !t->out || !t->pool || !t->pages || !t->n_past || !t->workspace)
        return DQ_ERR_NULL;
    if (t->n_seq < 1 || t->total_new < 1 || t->max_new < 1 || t->n_q < 1 || t->n_kv < 1 || t->n_q % t->n_kv || t->max_pages < 1)
        return DQ_ERR_SHAPE;
    const int st = dqhost::kv16_check_shape(t->type, t->n_kv, t->head_dim, t->n_pages, t->page_size);
    if (st != DQ_OK)
        return st;
    const long long rows[2] = {t->q_row_stride, t->out_row_stride}, heads[2] = {t->q_head_stride, t->out_head_stride};
    for (int i = 0; i < 2; ++i)
        if ((t->total_new > 1 && rows[i] < dq::ATT_HD) || (t->n_q > 1 && heads[i] < dq::ATT_HD))
            return DQ_ERR_SHAPE;
    if (!t->cu_new && t->total_new != static_cast<long long>(t->n_seq) * t->max_new)
        return DQ_ERR_SHAPE;
    if (t->max_new > dq::TR_MAX_NEW || t->n_q / t->n_kv > dq::TR_MAX_GROUP || t->total_new > (1 << 30) ||
        static_cast<long long>(t->max_pages) * t->page_size > (1 << 30) ||
        static_cast<long long>(t->n_seq) * t->n_kv >= (1 << 24))
        return DQ_ERR_UNSUPPORTED;
    for (int i = 0; i < 2; ++i) {
        if (rows[i] % 8 || heads[i] % 8)
            return DQ_ERR_ALIGN;
        if (rows[i] >= (1ll << 38) || heads[i] >= (1ll << 38))
            return DQ_ERR_UNSUPPORTED;
    }
    if (!dqhost::aligned16(t->q) || !dqhost::aligned16(t->out) || !dqhost::aligned16(t->pool) ||
        !dqhost::aligned16(t->workspace) || (reinterpret_cast<uintptr_t>(t->pages) & 3) ||
        (reinterpret_cast<uintptr_t>(t->n_past) & 3) || (reinterpret_cast<uintptr_t>(t->cu_new) & 3) ||
        (reinterpret_cast<uintptr_t>(t->seen) & 7))
        return DQ_ERR_ALIGN;
    if (t->workspace_bytes < dq_attention_tree_workspace_bytes(t->n_seq, t->max_new, t->n_q, t->n_kv))
        return DQ_ERR_SHAPE;
    const dq::TreeArgs a{t->q, t->out, rows[0], heads[0], rows[1], heads[1], t->pool, t->pages, t->n_past, t->cu_new, t->seen,
                         t->n_seq, t->total_new, t->max_new, t->n_q, t->n_q / t->n_kv, t->max_pages,
                         {t->n_kv, t->n_pages, t->page_size}, dqhost::device_error_flag()};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dqhost::with_type16(t->type, [&](auto* p) {
        dq::tree_simple_kernel<std::remove_pointer_t<decltype(p)>>
            <<<dim3(static_cast<unsigned>(t->n_seq) * t->max_new, t->n_q), 128, 0, s>>>(a);
        return cudaGetLastError();
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
