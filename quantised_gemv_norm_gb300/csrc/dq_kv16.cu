// dq_kv16.cu -- projections into a paged 16-bit cache with head norm and rotary
// embedding on the way (dq_kv16_append), and accepted rows moved within it
// (dq_kv16_keep).
//
// The store: half a warp takes one head, a warp four heads of one row; lane i of 16 holds
// dims 4 i .. 4 i + 3 and 64 + 4 i .., so a rotation's two dims are in one lane, the sum of
// squares of two heads is four shuffles, the row's angles are loaded once and all four heads'
// loads are issued first.  Memory bounds it: 8191 rows of 48 heads from fp32, 306 MB, 48.3
// us, 6.3 TB/s (0.95 of the measured copy rate).  The stores are streaming ones: written
// back late, as plain stores are, the rows took 55.8 us.  Eight heads a warp 50.1 us (one row
// 3.1 us, with four heads 2.6), blocks of 16 warps 54.3.
#include <algorithm>

#include "dq_kv16.cuh"

namespace dq {

struct Kv16AppendArgs {
    const void* qkv;
    long long ld;
    const int* pos;
    const int* slots;
    const float* q_norm;
    const float* k_norm;
    const float2* rope;
    void* q;
    void* pool;
    float eps;
    int rows, n_q, max_ctx;
    Kv16Shape s;
    FastDiv by_chunks, by_page;  // warps a row
    int* err;
};

constexpr int KV16_WARPS = 4;
constexpr int KV16_PAIRS = 2;  // pairs of heads a warp

// Four consecutive elements, read once.
__device__ __forceinline__ float4 stream4(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
template <typename T>
__device__ __forceinline__ float4 stream4(const T* p)
{
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
    const float2 a = un2(std::is_same<T, __half>::value ? half2_f2(u.x) : f2(bf16lo(u.x), bf16hi(u.x)));
    const float2 b = un2(std::is_same<T, __half>::value ? half2_f2(u.y) : f2(bf16lo(u.y), bf16hi(u.y)));
    return make_float4(a.x, a.y, b.x, b.y);
}

// Four elements to where they are not read again soon.
template <typename T>
__device__ __forceinline__ void stream_store4(T* p, float4 v)
{
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack2(v.x, v.y, p), pack2(v.z, v.w, p)));
}

template <typename In, typename T>
__global__ void __launch_bounds__(32 * KV16_WARPS) kv16_append_kernel(const Kv16AppendArgs a)
{
    const int lane = threadIdx.x & 31, half = lane >> 4, i = lane & 15;
    const uint32_t item = blockIdx.x * KV16_WARPS + (threadIdx.x >> 5);
    const uint32_t row = fast_div(item, a.by_chunks), chunk = item - row * a.by_chunks.d;
    if (row >= static_cast<uint32_t>(a.rows))
        return;
    const int pos = __ldg(a.pos + row), slot = __ldg(a.slots + row);
    if (pos < 0 || pos >= a.max_ctx) {
        if (pos >= 0 && lane == 0)
            set_error(a.err, DEVERR_BAD_ARG);
        return;
    }
    const int heads = a.n_q + 2 * a.s.n_kv, turned = a.n_q + a.s.n_kv, h0 = 2 * KV16_PAIRS * chunk + half;
    const In* src = static_cast<const In*>(a.qkv) + row * a.ld + 4 * i;
    float4 x[KV16_PAIRS], y[KV16_PAIRS];
#pragma unroll
    for (int p = 0; p < KV16_PAIRS; ++p) {
        const int h = h0 + 2 * p;
        if (h < heads) {
            x[p] = stream4(src + h * ATT_HD);
            y[p] = stream4(src + h * ATT_HD + 64);
        }
    }
    // the slot's row of key head 0 in the pool; below 0 where the row is not stored
    long long first = -1;
    if (slot >= 0) {
        const int page = static_cast<int>(fast_div(static_cast<uint32_t>(slot), a.by_page));
        if (page < a.s.n_pages)
            first = kv16_row(a.s, page, 0, 0) + (slot - page * a.s.page_rows);
        else if (lane == 0)
            set_error(a.err, DEVERR_BAD_ARG);
    }
    const float4* cs = reinterpret_cast<const float4*>(a.rope + static_cast<size_t>(pos) * (ATT_HD / 2) + 4 * i);
    const float4 c01 = __ldg(cs), c23 = __ldg(cs + 1);  // cos, sin, cos, sin
#pragma unroll
    for (int p = 0; p < KV16_PAIRS; ++p) {
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
        if (h < turned) {
            const float4 b = x[p], c = y[p];
            x[p] = make_float4(fmaf(b.x, c01.x, -(c.x * c01.y)), fmaf(b.y, c01.z, -(c.y * c01.w)),
                               fmaf(b.z, c23.x, -(c.z * c23.y)), fmaf(b.w, c23.z, -(c.w * c23.w)));
            y[p] = make_float4(fmaf(c.x, c01.x, b.x * c01.y), fmaf(c.y, c01.z, b.y * c01.w),
                               fmaf(c.z, c23.x, b.z * c23.y), fmaf(c.w, c23.z, b.w * c23.w));
        }
        T* out = static_cast<T*>(a.q) + (static_cast<size_t>(row) * a.n_q + h) * ATT_HD;
        if (h >= a.n_q) {
            if (first < 0)
                continue;
            // heads n_q .. are the pool's planes [2][n_kv] in order
            out = static_cast<T*>(a.pool) + (first + static_cast<long long>(h - a.n_q) * a.s.page_rows) * ATT_HD;
        }
        stream_store4(out + 4 * i, x[p]);
        stream_store4(out + 64 + 4 * i, y[p]);
    }
}

struct Kv16KeepArgs {
    unsigned char* pool;
    long long layer;  // bytes
    const int* pages;
    const int* n_past;
    const int* path;
    const int* n_path;
    int max_new, max_pages, n_layers, each;  // layers a block
    Kv16Shape s;
    FastDiv by_page, by_groups;  // groups of layers
    int* err;
};

constexpr int KV16_KEEP_THREADS = 256;
constexpr int KV16_KEEP_EACH = 4;  // 16-byte pieces a thread has in registers
constexpr int KV16_MAX_NEW = 64;
static_assert(KV16_KEEP_THREADS * KV16_KEEP_EACH >= KV16_MAX_NEW * 16, "a plane's rows are moved at once");

// One block a sequence, group of layers and half (keys or values).  The moved rows' places
// are found once, a thread a row; then, layer by layer, as many heads at a time as the
// block's registers hold go through them, all their rows read before the first is written (a
// row may be another's place).  A block has as many layers as leave eight blocks an SM:
// finding the places is three waits for memory in a row.  64 sequences' rows in 36 layers, 113
// MB: 23.3 us (one layer a block 25.5, a block a head, each finding the rows for itself, 59);
// the rows' bytes take 17.
__global__ void __launch_bounds__(KV16_KEEP_THREADS) kv16_keep_kernel(const Kv16KeepArgs a)
{
    __shared__ long long from[KV16_MAX_NEW], to[KV16_MAX_NEW];  // in rows from the pool's start, of head 0
    __shared__ int moved;
    const int tid = threadIdx.x, lane = tid & 31, kv = blockIdx.x & 1;
    const uint32_t x = blockIdx.x >> 1;
    const uint32_t b = fast_div(x, a.by_groups), group = x - b * a.by_groups.d;
    if (tid < 32) {
        const int n = __ldg(a.n_path + b), past = __ldg(a.n_past + b);
        int nodes[KV16_MAX_NEW / 32];
#pragma unroll
        for (int e = 0; e < KV16_MAX_NEW / 32; ++e)
            nodes[e] = 32 * e + lane < a.max_new ? __ldg(a.path + static_cast<size_t>(b) * a.max_new + 32 * e + lane) : 0;
        const bool bad = n < 0 || n > a.max_new || past < 0;
        if (bad && lane == 0)
            set_error(a.err, DEVERR_BAD_ARG);
        const int* pages = a.pages + static_cast<size_t>(b) * a.max_pages;
        // a row's place, below 0 where it does not exist
        auto at = [&](uint32_t j) -> long long {
            if (j > 0x7fffffffu)
                return -1;
            const int k = static_cast<int>(fast_div(j, a.by_page));
            if (k >= a.max_pages)
                return -1;
            const int page = __ldg(pages + k);
            return page < 0 || page >= a.s.n_pages ? -1 : kv16_row(a.s, page, kv, 0) + (static_cast<int>(j) - k * a.s.page_rows);
        };
        int count = 0;
#pragma unroll
        for (int e = 0; e < KV16_MAX_NEW / 32; ++e) {
            const int i = 32 * e + lane;
            bool go = !bad && i < n;
            long long f = -1, t = -1;
            if (go) {
                const int node = nodes[e];
                go = node != i;
                if (go) {
                    if (node >= 0 && node < a.max_new)
                        f = at(static_cast<uint32_t>(past) + node);
                    t = at(static_cast<uint32_t>(past) + i);
                    if (f < 0 || t < 0) {
                        set_error(a.err, DEVERR_BAD_ARG);
                        go = false;
                    }
                }
            }
            const unsigned who = __ballot_sync(0xffffffffu, go);
            if (go) {
                const int place = count + __popc(who & ((1u << lane) - 1));
                from[place] = f;
                to[place] = t;
            }
            count += __popc(who);
        }
        if (lane == 0)
            moved = count;
    }
    __syncthreads();
    const int n = moved;
    if (n == 0)
        return;
    const int pieces = 16 * n, heads = KV16_KEEP_THREADS * KV16_KEEP_EACH / pieces;  // at a time
    const int last = min(a.n_layers, static_cast<int>(group + 1) * a.each);
    for (int layer = static_cast<int>(group) * a.each; layer < last; ++layer) {
        uint4* base = reinterpret_cast<uint4*>(a.pool + layer * a.layer);
        for (int h0 = 0; h0 < a.s.n_kv; h0 += heads) {
            uint4 v[KV16_KEEP_EACH];
            long long dst[KV16_KEEP_EACH];
#pragma unroll
            for (int e = 0; e < KV16_KEEP_EACH; ++e) {
                const int i = tid + e * KV16_KEEP_THREADS, h = i / pieces, row = (i - h * pieces) >> 4;
                dst[e] = -1;
                if (h < heads && h0 + h < a.s.n_kv) {
                    const long long head = static_cast<long long>(h0 + h) * a.s.page_rows;
                    v[e] = __ldcg(base + (from[row] + head) * 16 + (i & 15));
                    dst[e] = (to[row] + head) * 16 + (i & 15);
                }
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < KV16_KEEP_EACH; ++e)
                if (dst[e] >= 0)
                    base[dst[e]] = v[e];
        }
    }
}

}  // namespace dq

extern "C" {

DQ_API int dq_kv16_append(const void* qkv, int in_type, long long row_stride, const int* positions, const int* slots,
                          const float* q_norm, const float* k_norm, const float* rope_table, float eps, int rows,
                          int n_q, int n_kv, int head_dim, int max_ctx, int type, void* q_out, void* pool, int n_pages,
                          int page_size, void* stream)
{
    if (!qkv || !positions || !slots || !rope_table || !q_out || !pool || !q_norm != !k_norm)
        return DQ_ERR_NULL;
    if (rows < 1 || n_q < 1 || n_kv < 1 || max_ctx < 1 || !dqhost::valid_eps(eps) || !dqhost::valid_type(in_type))
        return DQ_ERR_SHAPE;
    const int st = dqhost::kv16_check_shape(type, n_kv, head_dim, n_pages, page_size);
    if (st != DQ_OK)
        return st;
    if (n_q > (1 << 16))
        return DQ_ERR_UNSUPPORTED;
    const long long heads = n_q + 2ll * n_kv;
    if (row_stride < heads * dq::ATT_HD)
        return DQ_ERR_SHAPE;
    const int chunks = static_cast<int>((heads + 2 * dq::KV16_PAIRS - 1) / (2 * dq::KV16_PAIRS));
    const long long items = static_cast<long long>(rows) * chunks, blocks = (items + dq::KV16_WARPS - 1) / dq::KV16_WARPS;
    if (items > 0x7fffff00ll)
        return DQ_ERR_UNSUPPORTED;
    if (row_stride % (in_type == DQ_TYPE_F32 ? 4 : 8) || !dqhost::aligned16(qkv) || !dqhost::aligned16(rope_table) ||
        !dqhost::aligned16(q_out) || !dqhost::aligned16(pool) || !dqhost::aligned16(q_norm) ||
        !dqhost::aligned16(k_norm) || (reinterpret_cast<uintptr_t>(positions) & 3) || (reinterpret_cast<uintptr_t>(slots) & 3))
        return DQ_ERR_ALIGN;
    const dq::Kv16AppendArgs a{qkv,  row_stride, positions, slots, q_norm, k_norm, reinterpret_cast<const float2*>(rope_table),
                               q_out, pool, eps, rows, n_q, max_ctx, {n_kv, n_pages, page_size}, dqhost::fast_divisor(chunks),
                               dqhost::fast_divisor(page_size), dqhost::device_error_flag()};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dqhost::with_type(in_type, [&](auto* in) {
        return dqhost::with_type16(type, [&](auto* t) {
            using In = std::remove_pointer_t<decltype(in)>;
            using T = std::remove_pointer_t<decltype(t)>;
            dq::kv16_append_kernel<In, T><<<static_cast<unsigned>(blocks), 32 * dq::KV16_WARPS, 0, s>>>(a);
            return cudaGetLastError();
        });
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

DQ_API int dq_kv16_keep(void* pool, int type, const int* pages, const int* n_past, const int* path, const int* n_path,
                        int n_layers, long long layer_stride, int n_seq, int max_new, int n_kv, int head_dim,
                        int n_pages, int page_size, int max_pages, void* stream)
{
    if (!pool || !pages || !n_past || !path || !n_path)
        return DQ_ERR_NULL;
    if (n_layers < 1 || n_seq < 1 || max_new < 1 || max_pages < 1)
        return DQ_ERR_SHAPE;
    const int st = dqhost::kv16_check_shape(type, n_kv, head_dim, n_pages, page_size);
    if (st != DQ_OK)
        return st;
    const long long bytes = static_cast<long long>(n_pages) * page_size * 2 * n_kv * dq::ATT_HD * 2;
    if (n_layers > 1 && layer_stride < bytes)
        return DQ_ERR_SHAPE;
    // the grid, two blocks a sequence and group of layers, stays below 2^31
    if (max_new > dq::KV16_MAX_NEW || n_layers > (1 << 16) || n_seq > (1 << 29) ||
        static_cast<long long>(n_seq) * n_layers > 0x7fffffffll / n_kv)
        return DQ_ERR_UNSUPPORTED;
    if (!dqhost::aligned16(pool) || (n_layers > 1 && layer_stride % 16) || (reinterpret_cast<uintptr_t>(pages) & 3) ||
        (reinterpret_cast<uintptr_t>(n_past) & 3) || (reinterpret_cast<uintptr_t>(path) & 3) ||
        (reinterpret_cast<uintptr_t>(n_path) & 3))
        return DQ_ERR_ALIGN;
    const long long each = std::min<long long>(n_layers, std::max(1ll, 2ll * n_seq * n_layers / (8ll * dqhost::sm_count())));
    const int groups = static_cast<int>((n_layers + each - 1) / each);
    const unsigned grid = static_cast<unsigned>(2ll * n_seq * groups);
    const dq::Kv16KeepArgs a{static_cast<unsigned char*>(pool), layer_stride, pages, n_past, path, n_path, max_new, max_pages,
                             n_layers, static_cast<int>(each), {n_kv, n_pages, page_size}, dqhost::fast_divisor(page_size),
                             dqhost::fast_divisor(groups), dqhost::device_error_flag()};
    dq::kv16_keep_kernel<<<grid, dq::KV16_KEEP_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
