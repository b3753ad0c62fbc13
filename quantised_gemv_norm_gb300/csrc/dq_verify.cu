// dq_verify.cu -- drafted tokens against the target's logits (dq_verify_draft).
//
// Two kernels.  The first reads every node's logits once, in pieces of 8192: a piece's
// largest logit with its lowest place, and the sum of exp((l - largest) / temperature).
// The second, a cluster of eight blocks a sequence, joins the pieces, walks the tree
// over numbers that are all in shared memory by then (a node's probability needs its
// parent's logits at one place and their sum), and looks for the next token: one pass
// over one node's logits, the random numbers and, for a rejected token of a chain, the
// draft's probabilities.
//
// The next token is the largest r(v) / noise(v) instead of the place where a cumulated
// sum passes one random number: of 10^5 such places some lie within the rounding of any
// 32-bit sum, where two ratios are seldom that close.  The pass runs in fp32; every
// thread whose best is within 1e-5 of the largest computes that one ratio again in
// 64 bits, and those decide.
#include <cooperative_groups.h>

#include "dq_types.cuh"

namespace dq {

constexpr int VF_PIECE = 8192;   // logits a block of the first kernel
constexpr int VF_THREADS = 256;
constexpr int VF_EACH = VF_PIECE / VF_THREADS;
constexpr int VF_CLUSTER = 8;    // blocks a sequence
constexpr int VF_MAX_NEW = 64;

struct VerifyArgs {
    const void* logits;
    long long ld;
    const float* draft;
    long long draft_ld;
    const float* noise;
    long long noise_ld;
    const int* tokens;
    const int* parents;
    const float* uniform;
    const float* temperature;
    const int* cu;
    int* path;
    int* n_path;
    int* next;
    int n_seq, total_new, max_new, vocab, pieces;
    float4* part;  // [total_new][pieces]: largest logit, its place, sum
    int* err;
};

// A sequence's first node and how many it has.
__device__ __forceinline__ int2 verify_nodes(const VerifyArgs& a, int s, bool& ok)
{
    if (!a.cu) {
        ok = true;
        return make_int2(s * a.max_new, a.max_new);
    }
    const int r0 = __ldg(a.cu + s), r1 = __ldg(a.cu + s + 1);
    ok = r0 >= 0 && r1 >= r0 && r1 <= a.total_new && r1 - r0 <= a.max_new;
    return make_int2(r0, ok ? r1 - r0 : 0);
}

__device__ __forceinline__ float verify_one(const float* p) { return *p; }
__device__ __forceinline__ float verify_one(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float verify_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// A logit as the definition takes it: NaN counts as -infinity.
__device__ __forceinline__ float verify_clean(float x) { return x == x ? x : -INFINITY; }

// log2(e) / temperature in two parts.
struct VerifyScale {
    float hi, lo;
};
__device__ __forceinline__ VerifyScale verify_scale(float temperature)
{
    constexpr float L = 1.4426950408889634f, REST = static_cast<float>(1.4426950408889634 - static_cast<double>(L));
    const float hi = __fdiv_rn(L, temperature);
    const float lo = __fdiv_rn(fmaf(-hi, temperature, L) + REST, temperature);
    return {hi, hi > 0.f && hi < INFINITY ? lo : 0.f};
}
// exp((x - m) / temperature) for x <= m, m > -infinity: 1 at m even where m is infinite, 0
// at -infinity.  The product's rounding error goes back in as a factor 1 + e ln 2.
__device__ __forceinline__ float verify_exp(float x, float m, VerifyScale c)
{
    const float d = x - m, t = d * c.hi, e = fmaf(d, c.lo, fmaf(d, c.hi, -t));
    const float w = ex2(t);
    return x == m ? 1.f : w == 0.f || x == -INFINITY ? 0.f : fmaf(w, e * 0.6931471805599453f, w);
}

struct Best {
    float v;
    int at;  // -1: none
};
__device__ __forceinline__ Best better(Best a, Best b)
{
    const bool take = b.at >= 0 && (a.at < 0 || b.v > a.v || (b.v == a.v && b.at < a.at));
    return take ? b : a;
}
__device__ __forceinline__ Best warp_best(Best x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x = better(x, Best{__shfl_xor_sync(0xffffffffu, x.v, o), __shfl_xor_sync(0xffffffffu, x.at, o)});
    return x;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(VF_THREADS) verify_stats_kernel(const VerifyArgs a)
{
    __shared__ Best tops[VF_THREADS / 32];
    __shared__ float sums[VF_THREADS / 32];
    __shared__ int seq_of;
    const int row = blockIdx.x / a.pieces, piece = blockIdx.x - row * a.pieces;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_trigger();
    const T* src = static_cast<const T*>(a.logits) + row * a.ld;
    constexpr int W = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;  // elements an access
    float x[VF_EACH];
    // element i = W k + e of a thread is at base + W VF_THREADS k + W tid + e: ascending in i
    const int base = piece * VF_PIECE + W * tid;
#pragma unroll
    for (int k = 0; k < VF_EACH / W; ++k) {
        const int at = base + W * VF_THREADS * k;
        if (VEC && at + W <= a.vocab) {
            const uint4 u = __ldcg(reinterpret_cast<const uint4*>(src + at));
            const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
            for (int i = 0; i < W; ++i)
                x[W * k + i] = verify_clean(verify_one(e + i));
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                x[W * k + i] = at + i < a.vocab ? verify_clean(verify_one(src + at + i)) : -INFINITY;
        }
    }
    if (tid == 0)
        seq_of = -1;
    __syncthreads();
    if (!a.cu) {
        if (tid == 0)
            seq_of = row / a.max_new;
    } else {
        for (int s = tid; s < a.n_seq; s += VF_THREADS) {
            bool ok;
            const int2 n = verify_nodes(a, s, ok);
            if (row >= n.x && row < n.x + n.y)
                seq_of = s;
        }
    }
    Best top{-INFINITY, -1};
#pragma unroll
    for (int i = 0; i < VF_EACH; ++i)
        if (x[i] > top.v)
            top = {x[i], base + W * VF_THREADS * (i / W) + i % W};
    top = warp_best(top);
    if (lane == 0)
        tops[warp] = top;
    __syncthreads();
    const int s = seq_of;
    if (s < 0)
        return;  // a row of no sequence
    top = tops[0];
#pragma unroll
    for (int w = 1; w < VF_THREADS / 32; ++w)
        top = better(top, tops[w]);
    const float temp = a.temperature ? __ldg(a.temperature + s) : 1.f;
    float sum = 0.f;
    if (temp > 0.f && top.at >= 0) {
        const VerifyScale c = verify_scale(temp);
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < VF_EACH; ++i)
            part[i & 3] += verify_exp(x[i], top.v, c);
        sum = warp_sum((part[0] + part[1]) + (part[2] + part[3]));
    }
    if (lane == 0)
        sums[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        float z = 0.f;
#pragma unroll
        for (int w = 0; w < VF_THREADS / 32; ++w)
            z += sums[w];
        a.part[static_cast<size_t>(row) * a.pieces + piece] = make_float4(top.v, __int_as_float(top.at), z, 0.f);
    }
}

struct VerifyShared {
    Best top[VF_MAX_NEW];      // a node's largest logit
    double sum[VF_MAX_NEW];    // of its weights
    double p[VF_MAX_NEW];      // of a node's token at its parent
    float u[VF_MAX_NEW], q[VF_MAX_NEW];
    int parent[VF_MAX_NEW], token[VF_MAX_NEW];
    int gone[VF_MAX_NEW], n_gone;  // rejected tokens at the last node
    int last, turned_down;         // the rejected node of a chain, or 0
    Best warp[VF_THREADS / 32];
    double exact_v[VF_THREADS / 32];
    int exact_at[VF_THREADS / 32];
    float best;          // the block's
    double best_exact;
    int best_at;
};

template <typename T>
__global__ void __cluster_dims__(VF_CLUSTER, 1, 1) __launch_bounds__(VF_THREADS) verify_pick_kernel(const VerifyArgs a)
{
    namespace cg = cooperative_groups;
    __shared__ VerifyShared sh;
    const int s = blockIdx.x / VF_CLUSTER, rank = blockIdx.x % VF_CLUSTER;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool ok;
    const int2 nodes = verify_nodes(a, s, ok);
    const int row0 = nodes.x, n = nodes.y;
    int* path = a.path + static_cast<size_t>(s) * a.max_new;
    if (n == 0) {  // the same in the whole cluster
        pdl_wait();
        if (rank == 0) {
            if (!ok && tid == 0)
                set_error(a.err, DEVERR_BAD_ARG);
            if (tid < a.max_new)
                path[tid] = -1;
            if (tid == 0) {
                a.n_path[s] = 0;
                a.next[s] = -1;
            }
        }
        return;
    }
    const T* logits = static_cast<const T*>(a.logits);
    const float temp = a.temperature ? __ldg(a.temperature + s) : 1.f;
    const bool greedy = !(temp > 0.f);
    const VerifyScale c = verify_scale(greedy ? 1.f : temp);

    float own = -INFINITY;  // a node's token's logit at its parent
    int parent = -1, token = -1;
    if (tid < n) {
        token = __ldg(a.tokens + row0 + tid);
        parent = tid == 0 ? -1 : a.parents ? __ldg(a.parents + row0 + tid) : tid - 1;
        if (tid > 0 && (parent < 0 || parent >= tid)) {
            parent = -1;
            if (rank == 0)
                set_error(a.err, DEVERR_BAD_ARG);
        }
        if (token < 0 || token >= a.vocab)
            token = -1;
        if (parent >= 0 && token >= 0) {
            own = verify_clean(verify_one(logits + (row0 + parent) * a.ld + token));
            sh.u[tid] = __ldg(a.uniform + row0 + tid);
            sh.q[tid] = a.draft ? __ldg(a.draft + (row0 + tid) * a.draft_ld + token) : 1.f;
        }
        sh.parent[tid] = parent;
        sh.token[tid] = token;
    }
    pdl_wait();
    // four threads a node join its pieces
    {
        const int node = tid >> 2, k0 = tid & 3;
        Best top{-INFINITY, -1};
        double sum = 0.0;
        if (node < n) {
            const float4* part = a.part + static_cast<size_t>(row0 + node) * a.pieces;
            for (int k = k0; k < a.pieces; k += 4) {
                const float4 x = __ldcg(part + k);
                const Best b{x.x, __float_as_int(x.y)};
                if (b.at < 0)
                    continue;
                const Best t = better(top, b);
                sum = (top.at < 0 ? 0.0 : sum * verify_exp(top.v, t.v, c)) +
                      static_cast<double>(x.z) * verify_exp(b.v, t.v, c);
                top = t;
            }
        }
#pragma unroll
        for (int o = 2; o > 0; o >>= 1) {
            const Best b{__shfl_xor_sync(0xffffffffu, top.v, o), __shfl_xor_sync(0xffffffffu, top.at, o)};
            const double z = __shfl_xor_sync(0xffffffffu, sum, o);
            const Best t = better(top, b);
            sum = (top.at < 0 ? 0.0 : sum * verify_exp(top.v, t.v, c)) + (b.at < 0 ? 0.0 : z * verify_exp(b.v, t.v, c));
            top = t;
        }
        if (node < n && k0 == 0) {
            sh.top[node] = top;
            sh.sum[node] = sum;
        }
    }
    __syncthreads();
    if (tid < n && parent >= 0) {
        const Best t = sh.top[parent];
        sh.p[tid] = token < 0 || t.at < 0 || greedy ? 0.0 : verify_exp(own, t.v, c) / sh.sum[parent];
    }
    __syncthreads();

    // ---- the walk: a node's children are above it, so one pass in ascending order
    if (tid == 0) {
        int cur = 0, len = 1, gone = 0, down = 0;
        double left = 1.0;
        if (rank == 0)
            path[0] = 0;
        for (int j = 1; j < n; ++j) {
            if (sh.parent[j] != cur)
                continue;
            const int x = sh.token[j];
            bool take;
            if (greedy) {
                take = x >= 0 && x == sh.top[cur].at;
            } else if (a.draft) {
                take = x >= 0 && static_cast<double>(sh.u[j]) * sh.q[j] < sh.p[j];
                down = take ? 0 : j;
            } else {
                bool again = x < 0;
                for (int k = 0; k < gone; ++k)
                    again |= sh.gone[k] == x;
                take = !again && sh.u[j] * left < sh.p[j];
                if (!again && !take) {
                    sh.gone[gone++] = x;
                    left -= sh.p[j];
                }
            }
            if (take) {
                if (rank == 0)
                    path[len] = j;
                cur = j;
                ++len;
                gone = 0;
                left = 1.0;
            }
        }
        sh.last = cur;
        sh.n_gone = gone;
        sh.turned_down = down;
        if (rank == 0) {
            a.n_path[s] = len;
            for (int k = len; k < a.max_new; ++k)
                path[k] = -1;
        }
    }
    __syncthreads();
    const int last = sh.last, n_gone = sh.n_gone, down = sh.turned_down;
    const Best top = sh.top[last];
    if (greedy || top.at < 0) {
        if (rank == 0 && tid == 0)
            a.next[s] = top.at;
        return;
    }

    // ---- the next token
    const T* row = logits + (row0 + last) * a.ld;
    const float* noise = a.noise + s * a.noise_ld;
    const float* draft = down ? a.draft + (row0 + down) * a.draft_ld : nullptr;
    const float z = static_cast<float>(sh.sum[last]);
    const int slice = (a.vocab + VF_CLUSTER - 1) / VF_CLUSTER, v0 = rank * slice, v1 = min(a.vocab, v0 + slice);
    Best best{0.f, -1};
    float size = 0.f;  // of the numbers that the best's r is a difference of, over its noise
    for (int v = v0 + tid; v < v1; v += VF_THREADS) {
        const float w = verify_exp(verify_clean(verify_one(row + v)), top.v, c), q = draft ? z * draft[v] : 0.f;
        const float e = noise[v], score = (w - q) / e;
        if (score > best.v) {
            bool out = false;
            for (int k = 0; k < n_gone; ++k)
                out |= sh.gone[k] == v;
            if (!out) {
                best = {score, v};
                size = (w + q) / e;
            }
        }
    }
    Best b = warp_best(best);
    if (lane == 0)
        sh.warp[warp] = b;
    __syncthreads();
    cg::cluster_group cluster = cg::this_cluster();
    if (tid == 0) {
        for (int w = 1; w < VF_THREADS / 32; ++w)
            b = better(b, sh.warp[w]);
        sh.best = b.at < 0 ? 0.f : b.v;
    }
    cluster.sync();
    float most = 0.f;
    for (int k = 0; k < VF_CLUSTER; ++k)
        most = fmaxf(most, *cluster.map_shared_rank(&sh.best, k));
    double v64 = 0.0;
    int at64 = -1;
    if (best.at >= 0 && best.v + 1e-5f * size >= most * (1.f - 1e-5f)) {
        const float x = verify_one(row + best.at);
        const double w = x == top.v ? 1.0 : exp((static_cast<double>(x) - top.v) / temp);
        v64 = (w - (draft ? sh.sum[last] * draft[best.at] : 0.0)) / noise[best.at];
        at64 = best.at;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const double v = __shfl_xor_sync(0xffffffffu, v64, o);
        const int at = __shfl_xor_sync(0xffffffffu, at64, o);
        if (at >= 0 && (at64 < 0 || v > v64 || (v == v64 && at < at64))) {
            v64 = v;
            at64 = at;
        }
    }
    if (lane == 0) {
        sh.exact_v[warp] = v64;
        sh.exact_at[warp] = at64;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < VF_THREADS / 32; ++w)
            if (sh.exact_at[w] >= 0 && (at64 < 0 || sh.exact_v[w] > v64 || (sh.exact_v[w] == v64 && sh.exact_at[w] < at64))) {
                v64 = sh.exact_v[w];
                at64 = sh.exact_at[w];
            }
        sh.best_exact = v64;
        sh.best_at = at64;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
        for (int k = 1; k < VF_CLUSTER; ++k) {
            const double v = *cluster.map_shared_rank(&sh.best_exact, k);
            const int at = *cluster.map_shared_rank(&sh.best_at, k);
            if (at >= 0 && (at64 < 0 || v > v64 || (v == v64 && at < at64))) {
                v64 = v;
                at64 = at;
            }
        }
        a.next[s] = at64 >= 0 ? at64 : top.at;
    }
    cluster.sync();  // a block's shared memory is read by the first until here
}

}  // namespace dq

namespace dqhost {

static int verify_pieces(int vocab) { return (vocab + dq::VF_PIECE - 1) / dq::VF_PIECE; }

}  // namespace dqhost

extern "C" {

DQ_API size_t dq_verify_draft_workspace_bytes(int total_new, int vocab)
{
    if (total_new < 1 || vocab < 1 || total_new > (1 << 24) || vocab > (1 << 24))
        return 0;
    return static_cast<size_t>(total_new) * dqhost::verify_pieces(vocab) * sizeof(float4);
}

DQ_API int dq_verify_draft(const dq_verify* v, void* stream)
{
    if (!v || !v->logits || !v->noise || !v->tokens || !v->uniform || !v->path || !v->n_path || !v->next || !v->workspace)
        return DQ_ERR_NULL;
    if (v->n_seq < 1 || v->total_new < 1 || v->max_new < 1 || v->vocab < 1 || !dqhost::valid_type(v->type))
        return DQ_ERR_SHAPE;
    if ((v->total_new > 1 && v->logits_stride < v->vocab) || (v->n_seq > 1 && v->noise_stride < v->vocab) ||
        (v->draft_probs && v->total_new > 1 && v->draft_stride < v->vocab) ||
        (!v->cu_new && v->total_new != static_cast<long long>(v->n_seq) * v->max_new))
        return DQ_ERR_SHAPE;
    const int pieces = dqhost::verify_pieces(v->vocab);
    if (v->max_new > dq::VF_MAX_NEW || (v->draft_probs && v->parents) || v->vocab > (1 << 24) || v->total_new > (1 << 24) ||
        v->n_seq > (1 << 24) || static_cast<long long>(v->total_new) * pieces > (1 << 30))
        return DQ_ERR_UNSUPPORTED;
    const void* words[11] = {v->draft_probs, v->noise, v->tokens, v->parents, v->uniform, v->temperature, v->cu_new,
                             v->path, v->n_path, v->next, nullptr};
    for (const void* w : words)
        if (reinterpret_cast<uintptr_t>(w) & 3)
            return DQ_ERR_ALIGN;
    const int size = dqhost::type_bytes(v->type);
    if ((reinterpret_cast<uintptr_t>(v->logits) & (size - 1)) || !dqhost::aligned16(v->workspace))
        return DQ_ERR_ALIGN;
    if (v->workspace_bytes < dq_verify_draft_workspace_bytes(v->total_new, v->vocab))
        return DQ_ERR_SHAPE;
    const dq::VerifyArgs a{v->logits, v->logits_stride, v->draft_probs, v->draft_stride, v->noise, v->noise_stride,
                           v->tokens, v->parents, v->uniform, v->temperature, v->cu_new, v->path, v->n_path, v->next,
                           v->n_seq, v->total_new, v->max_new, v->vocab, pieces, static_cast<float4*>(v->workspace),
                           dqhost::device_error_flag()};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = dqhost::aligned16(v->logits) && (v->total_new == 1 || v->logits_stride * size % 16 == 0);
    cudaError_t e = dqhost::with_type(v->type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const unsigned grid = static_cast<unsigned>(v->total_new) * pieces;
        if (vec)
            dq::verify_stats_kernel<T, true><<<grid, dq::VF_THREADS, 0, s>>>(a);
        else
            dq::verify_stats_kernel<T, false><<<grid, dq::VF_THREADS, 0, s>>>(a);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess)
            return err;
        // a dependent launch: it gathers the tree's numbers while the last pieces run
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(v->n_seq) * dq::VF_CLUSTER);
        cfg.blockDim = dim3(dq::VF_THREADS);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, dq::verify_pick_kernel<T>, a);
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
