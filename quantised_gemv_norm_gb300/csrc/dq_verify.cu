// dq_verify.cu -- drafted tokens against the target's logits (dq_verify_draft).
//
// Two kernels.  The first reads every node's logits once, in pieces of a row: a piece's
// largest logit with its lowest place, and the sum of exp((l - largest) / temperature).
// The second, a cluster of up to 16 blocks a sequence, joins the pieces, tests every node as
// if its turn came (a node's probability needs its parent's logits at one place and their
// sum; all its siblings before it were rejected then), walks from the root along the nodes
// that passed, and looks for the next token: one pass over one node's logits, the random
// numbers and, for a rejected token of a chain, the draft's probabilities.
//
// The next token is the largest r(v) / noise(v) instead of the place where a cumulated
// sum passes one random number: of 10^5 such places some lie within the rounding of any
// 32-bit sum, where two ratios are seldom that close.  The pass runs in fp32 and has for
// every place what its ratio is at least and at most, by bounds on all that fp32 may have
// rounded (slack, verify_exp_off; before a draft's part cancels).  The places whose most
// reaches the largest least can be the best: where that is one, it is; else they are compared in
// 64 bits, with the sum of weights that a draft is multiplied by taken again to 2^-38.  The
// acceptance of a token is open within the same bound of its border, and is then decided again
// like that when its turn comes (what rejected siblings leave of 1 may be small).  Either happens
// about once in 10^4 tokens, and costs 10 us for one sequence of 151936 logits.
//
// 64 sequences of up to 9 nodes, 151936 fp32 logits each, 193 MB and 78 MB of random numbers
// and draft probabilities: 52 us (floor 40): 32 us the first kernel (6.0 TB/s), the rest the
// pass (13 us, the same memory) and the second kernel's steps.  405 nodes of 100003 bf16
// logits in 16 trees: 36 us (13): the first kernel 24 us, 3.4 TB/s, two rounds of four blocks
// an SM: a block's start and the chain of each of its nine steps, 9.7 instructions a logit
// counted, issue 0.5 of its rate (10.8 before 16-bit logits were widened in pairs: 0.8 us more).
// One sequence of 6: 11.6 us: 2.5 the first kernel, then waits for memory in a row (lengths,
// tokens, their logits; sums; two rounds of the pass) and two meetings of the cluster.  64 nodes
// of one sequence, 5000 logits: a chain 9.4 us, breadth first with 4 children each 10.0, with 8
// 11.6, a root with 63 children 28.6: siblings are gone through one by one.
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "dq_types.cuh"

namespace dq {

constexpr int VF_THREADS = 256;
constexpr int VF_EACH = 16;      // logits a thread has of a step of the first kernel
constexpr int VF_STEP = VF_THREADS * VF_EACH;
constexpr int VF_CLUSTER = 16;   // blocks a sequence, at most (8 is the portable limit)
constexpr int VF_PICK = 512;     // threads each
constexpr int VF_BATCH = 12;     // places a thread has in flight there
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
    int n_seq, total_new, max_new, vocab, pieces, steps;  // pieces of a row, a block each; steps a piece
    float4* part;  // [total_new][pieces]: largest logit, its place, sum
    float slack;   // relative error of a node's sum, at most, and of a weight (VerifyCut)
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
__device__ __forceinline__ float verify_clean(float x) { return fmaxf(x, -INFINITY); }

// What exp((x - m) / temperature) needs: log2(e) / temperature in two parts, and the
// difference beyond which it is 0 (2^-200).  The temperature is kept within 2^-60 .. 2^60.
struct VerifyScale {
    float hi, lo, least;
};
__device__ __forceinline__ VerifyScale verify_scale(float temperature)
{
    constexpr float L = 1.4426950408889634f, REST = static_cast<float>(1.4426950408889634 - static_cast<double>(L));
    const float t = fminf(fmaxf(temperature, 8.673617e-19f), 1.1529215e18f);
    const float hi = __fdiv_rn(L, t);
    return {hi, __fdiv_rn(fmaf(-hi, t, L) + REST, t), __fdiv_rn(-200.f, hi)};
}
// exp((x - m) / temperature) of two x <= m, m finite: exactly 1 at m, 0 at -infinity and
// for a NaN.  Off by 2^-24 of the exponent, where a weight is large less than ex2's 2^-22.
__device__ __forceinline__ uint64_t verify_exp2(uint64_t x, uint64_t minus_m, const VerifyScale& c)
{
    const float2 d0 = un2(add2(x, minus_m));
    const uint64_t d = f2(fmaxf(d0.x, c.least), fmaxf(d0.y, c.least));
    const float2 t = un2(fma2(d, f2(c.lo, c.lo), mul2(d, f2(c.hi, c.hi))));
    return f2(ex2(t.x), ex2(t.y));
}
// The same of one, 1 at m even where m is infinite; the product's rounding error goes back
// in as a factor 1 + e ln 2, which leaves the difference's, 2^-24 of an exponent of at most 126,
// and ex2's (verify_exp_off).  Below 2^-126 it is 0.
__device__ __forceinline__ float verify_exp(float x, float m, const VerifyScale& c)
{
    const float d = fmaxf(x - m, c.least), t = d * c.hi, e = fmaf(d, c.lo, fmaf(d, c.hi, -t)), w = ex2(t);
    return x == m ? 1.f : isinf(m) ? 0.f : fmaf(w, e * 0.6931471805599453f, w);
}

// What that is off by, at most, relative to itself: the rounding of the difference, ex2's 2^-22, and
// 4.6e-7 for the product with it, a division by the noise (2^-22) and a rounding.
__device__ __forceinline__ float verify_exp_off(float x, float m, const VerifyScale& c)
{
    return fmaf(fmaxf((x - m) * c.hi, -130.f), -4.2e-8f, 7e-7f);
}
// In 64 bits, of one that is no NaN.
__device__ __forceinline__ double verify_exp64(float x, float m, double temperature)
{
    return x == m ? 1.0 : exp((static_cast<double>(x) - m) / temperature);
}
__device__ __forceinline__ double verify_temperature64(float t)
{
    return fmin(fmax(static_cast<double>(t), 8.673617379884035e-19), 1.152921504606847e18);
}

// The warp's largest, in one instruction.
__device__ __forceinline__ float verify_warp_max(float x)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
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

// The sequence that a row belongs to, by one warp; -1: none.  Its temperature comes with the
// sequences' ends, not after them.
__device__ __forceinline__ int verify_seq(const VerifyArgs& a, int row, int lane, float& temp)
{
    temp = 1.f;
    if (!a.cu) {
        const int s = row / a.max_new;
        if (a.temperature)
            temp = __ldg(a.temperature + s);
        return s;
    }
    for (int s0 = 0; s0 < a.n_seq; s0 += 128) {
        unsigned hit[4];
        float each[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int s = s0 + 32 * e + lane;
            each[e] = a.temperature && s < a.n_seq ? __ldg(a.temperature + s) : 1.f;
            bool ok = false;
            int2 n = make_int2(0, 0);
            if (s < a.n_seq)
                n = verify_nodes(a, s, ok);
            hit[e] = __ballot_sync(0xffffffffu, ok && row >= n.x && row < n.x + n.y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (hit[e]) {
                temp = __shfl_sync(0xffffffffu, each[e], __ffs(hit[e]) - 1);
                return s0 + 32 * e + __ffs(hit[e]) - 1;
            }
    }
    return -1;
}

// One step's logits of a thread, in 16-byte accesses wherever the row begins: element 0 of a
// row is element `skew` of its first one; element W k + e of a thread is at first + W
// VF_THREADS k + e.
template <typename T>
struct VerifyStep {
    static constexpr int W = 16 / static_cast<int>(sizeof(T)), N = VF_EACH / W;
    uint4 u[N];
    // `whole`: the block's step lies within the row
    __device__ __forceinline__ void load(const T* src, int first, int vocab, bool whole)
    {
        if (whole) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                u[k] = __ldcg(reinterpret_cast<const uint4*>(src + first + W * VF_THREADS * k));
            return;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int at = first + W * VF_THREADS * k;
            if (at >= 0 && at + W <= vocab) {
                u[k] = __ldcg(reinterpret_cast<const uint4*>(src + at));
            } else {
                T x[W];
#pragma unroll
                for (int i = 0; i < W; ++i)
                    x[i] = at + i >= 0 && at + i < vocab ? src[at + i] : static_cast<T>(-INFINITY);
                memcpy(&u[k], x, 16);
            }
        }
    }
    // the largest, NaN passed over; 16-bit logits in pairs
    __device__ __forceinline__ float top() const
    {
        float m = -INFINITY;
        if constexpr (sizeof(T) == 4) {
            float m4[4] = {m, m, m, m};
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    m4[i] = fmaxf(m4[i], reinterpret_cast<const float*>(&u[k])[i]);
            return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        } else {
            using P = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
            const P* p = reinterpret_cast<const P*>(u);
            P m2[2] = {p[0], p[1]};
#pragma unroll
            for (int i = 2; i < VF_EACH / 2; ++i)
                m2[i & 1] = __hmax2(m2[i & 1], p[i]);
            m2[0] = __hmax2(m2[0], m2[1]);
            return fmaxf(m, fmaxf(verify_one(&m2[0].x), verify_one(&m2[0].y)));
        }
    }
    __device__ __forceinline__ void get(float (&x)[VF_EACH]) const
    {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
#pragma unroll
            for (int i = 0; i < VF_EACH / 2; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else if constexpr (std::is_same_v<T, __half>) {
#pragma unroll
            for (int i = 0; i < VF_EACH / 2; ++i) {
                const float2 f = __half22float2(reinterpret_cast<const __half2*>(w)[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VF_EACH; ++i)
                x[i] = __uint_as_float(w[i]);
        }
    }
};

// The largest logit with its lowest place and the sum of weights of a piece: `steps` steps
// of one row, the next one's logits on their way while one is added up.  A warp has a
// running maximum of its own; the block's warps meet at the end.
template <typename T>
__global__ void __launch_bounds__(VF_THREADS) verify_stats_kernel(const VerifyArgs a)
{
    constexpr int WARPS = VF_THREADS / 32, W = VerifyStep<T>::W;
    __shared__ Best tops[WARPS];
    __shared__ float sums[WARPS], row_temp;
    __shared__ VerifyScale row_scale;
    __shared__ int row_seq;
    const int row = blockIdx.x / a.pieces, piece = blockIdx.x - row * a.pieces;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_trigger();
    const T* src = static_cast<const T*>(a.logits) + row * a.ld;
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    int base = piece * a.steps * VF_STEP - skew;  // the step's first element
    auto whole = [&](int b) { return b >= 0 && b + VF_STEP <= a.vocab; };
    const int steps = min(a.steps, (a.vocab + skew + VF_STEP - 1) / VF_STEP - piece * a.steps);
    // 64 bytes a thread on their way
    constexpr int DEPTH = 4 / static_cast<int>(sizeof(T));
    VerifyStep<T> next[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (d == 0 || d < steps)
            next[d].load(src, base + d * VF_STEP + W * tid, a.vocab, whole(base + d * VF_STEP));
    if (warp == 0) {
        float t;
        const int s = verify_seq(a, row, lane, t);
        if (lane == 0) {
            row_temp = t;
            row_seq = s;
            row_scale = verify_scale(row_temp > 0.f ? row_temp : 1.f);
        }
    }
    __syncthreads();
    if (row_seq < 0)
        return;  // a row of no sequence
    const float temp = row_temp;
    const VerifyScale c = row_scale;
    Best top{-INFINITY, -1};  // the warp's
    float sum = 0.f;          // the lane's
    for (int k = 0; k < steps; ++k, base += VF_STEP) {
        float x[VF_EACH];
        next[0].get(x);
        const float m = verify_warp_max(next[0].top());
#pragma unroll
        for (int d = 0; d + 1 < DEPTH; ++d)
            next[d] = next[d + 1];
        if (k + DEPTH < steps)
            next[DEPTH - 1].load(src, base + DEPTH * VF_STEP + W * tid, a.vocab, whole(base + DEPTH * VF_STEP));
        if (m > top.v) {  // the same in the whole warp
            int at = 0x7fffffff;
#pragma unroll
            for (int i = VF_EACH - 1; i >= 0; --i)
                if (x[i] == m)
                    at = base + W * tid + W * VF_THREADS * (i / W) + i % W;
            sum = top.at < 0 ? 0.f : sum * verify_exp(top.v, m, c);
            top = Best{m, static_cast<int>(__reduce_min_sync(0xffffffffu, at))};
        }
        if (temp > 0.f && top.at >= 0) {
            if (top.v < INFINITY) {
                uint64_t part[2] = {0ull, 0ull};
                const uint64_t minus = f2(-top.v, -top.v);
#pragma unroll
                for (int i = 0; i < VF_EACH / 2; ++i)
                    part[i & 1] = add2(part[i & 1], verify_exp2(f2(x[2 * i], x[2 * i + 1]), minus, c));
                const float2 p = un2(add2(part[0], part[1]));
                sum += p.x + p.y;
            } else {
#pragma unroll
                for (int i = 0; i < VF_EACH; ++i)
                    sum += x[i] == top.v ? 1.f : 0.f;
            }
        }
    }
    sum = warp_sum(sum);
    if (lane == 0) {
        tops[warp] = top;
        sums[warp] = sum;
    }
    __syncthreads();
    if (warp)
        return;
    const Best b = lane < WARPS ? tops[lane] : Best{-INFINITY, -1};
    top = warp_best(b);
    sum = warp_sum(b.at >= 0 ? sums[lane] * verify_exp(b.v, top.v, c) : 0.f);
    if (lane == 0)
        a.part[static_cast<size_t>(row) * a.pieces + piece] = make_float4(top.v, __int_as_float(top.at), sum, 0.f);
}

struct VerifyShared {
    Best top[VF_MAX_NEW];        // a node's largest logit
    float sum[VF_MAX_NEW];       // of its weights
    float w[VF_MAX_NEW];         // the weight of a node's token at its parent
    int token[VF_MAX_NEW];
    // a node's children, a bit each: all whose token is in the vocabulary, those whose token no
    // sibling before them has, those accepted if their turn comes, those that fp32 leaves open
    uint2 kids[VF_MAX_NEW], fresh[VF_MAX_NEW], taken[VF_MAX_NEW], open[VF_MAX_NEW];
    double w64[VF_MAX_NEW];
    int path[VF_MAX_NEW], len, stop;
    int gone[VF_MAX_NEW], n_gone;  // rejected tokens at the last node
    int last, turned_down;         // the rejected node of a chain, or 0
    float warp[VF_PICK / 32];
    float sure;        // of the block's places: the largest of what their ratios are at least
    int near, n_near;  // a place that may be the cluster's best, and how many there are
    // the exact pass
    float2 powers[128], scale;  // 2^(k / 128) and log2(e) / temperature, in two parts
    double part, total, warp64[VF_PICK / 32], best64;
    int warp_at[VF_PICK / 32], best_at;
};

// Four consecutive logits from an address that is a multiple of their size.
template <typename T>
__device__ __forceinline__ float4 verify_four(const T* p)
{
    return load4(p);
}

// The sum of a row's weights exp((x - m) / temperature) to 2^-38 of itself, by a cluster whose
// blocks have the places v0 .. v1 - 1 each; the same number in all of its threads.
// 2^t = 2^(k / 128) e^z with k = rint(128 t), |z| <= ln 2 / 256 (P. Tang's table method, 1989), where t,
// the table and the sums are pairs of fp32, whose sums and products are exact up to 2^-41 of a
// weight: 64-bit arithmetic has a sixty-fourth of fp32's rate here.
template <typename T>
__device__ __noinline__ double verify_sum64(VerifyShared& sh, const T* row, float m, double temperature, int v0, int v1)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x;
    if (tid < 128) {
        const double p = exp2(tid / 128.0);
        sh.powers[tid].x = static_cast<float>(p);
        sh.powers[tid].y = static_cast<float>(p - static_cast<float>(p));
    }
    if (tid == 128) {
        const double scale = 1.4426950408889634074 / temperature;
        sh.scale.x = static_cast<float>(scale);
        sh.scale.y = static_cast<float>(scale - static_cast<float>(scale));
    }
    __syncthreads();
    const float ch = sh.scale.x, cl = sh.scale.y;
    const bool infinite = isinf(m);
    constexpr int N = 8;  // places on their way
    float hi = 0.f, lo = 0.f;
    auto add = [&](float y) {  // and its rounding
        const float t = hi + y, z = t - hi;
        lo += (hi - (t - z)) + (y - z);
        hi = t;
    };
    for (int b0 = v0 + tid; b0 < v1; b0 += VF_PICK * N) {
        float x[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = b0 + i * VF_PICK < v1 ? verify_one(row + b0 + i * VF_PICK) : -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float dh = x[i] - m, back = dh - x[i], dl = (x[i] - (dh - back)) - (m + back);
            const float ph = dh * ch;
            if (!(ph > -125.f)) {  // less than 2^-125, or a NaN
                if (infinite && x[i] == m)
                    hi += 1.f;
                continue;
            }
            const float pl = fmaf(dl, ch, fmaf(dh, cl, fmaf(dh, ch, -ph)));
            const float k = rintf(128.f * ph), h = fmaf(k, -1.f / 128.f, ph);
            constexpr float LN2 = 0.6931471805599453f, REST = static_cast<float>(0.6931471805599453 - static_cast<double>(LN2));
            const float zh = h * LN2, zl = fmaf(pl, LN2, fmaf(h, REST, fmaf(h, LN2, -zh)));
            const float more = fmaf(zh * zh, fmaf(zh, fmaf(zh, 1.f / 24.f, 1.f / 6.f), 0.5f), zl);  // e^z - 1 - zh
            const int n = static_cast<int>(k);
            const float2 p = sh.powers[n & 127];
            const float power = __int_as_float(((n >> 7) + 127) << 23), w = p.x * power, wz = w * zh;
            add(w);
            add(wz);
            lo += fmaf(w, more, fmaf(w, zh, -wz)) + p.y * power * (1.f + zh);
        }
        const float rest = lo;  // the second part stays a rounding of the first
        lo = 0.f;
        add(rest);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float h2 = __shfl_xor_sync(0xffffffffu, hi, o);
        lo += __shfl_xor_sync(0xffffffffu, lo, o);
        add(h2);
    }
    if ((tid & 31) == 0)
        sh.warp64[tid >> 5] = static_cast<double>(hi) + lo;
    __syncthreads();
    if (tid == 0) {
        double part = 0.0;
        for (int w = 0; w < VF_PICK / 32; ++w)
            part += sh.warp64[w];
        sh.part = part;
    }
    cluster.sync();
    if (tid == 0) {
        double total = 0.0;
        for (int k = 0; k < static_cast<int>(cluster.num_blocks()); ++k)
            total += *cluster.map_shared_rank(&sh.part, k);
        sh.total = total;
    }
    cluster.sync();  // before a block writes its part again, or ends
    return sh.total;
}

// A set of nodes in shared memory: a node into it, by its half (64-bit atomics are loops that 63
// children of a node take turns in), and all of it.
__device__ __forceinline__ void verify_put(uint2& set, int node) { atomicOr(node < 32 ? &set.x : &set.y, 1u << (node & 31)); }
__device__ __forceinline__ unsigned long long verify_set(const uint2& set)
{
    return static_cast<unsigned long long>(set.y) << 32 | set.x;
}
// f of each node in `set`, ascending.
template <typename F>
__device__ __forceinline__ void verify_each(unsigned long long set, F f)
{
    for (; set; set &= set - 1)
        f(__ffsll(static_cast<long long>(set)) - 1);
}

// The next token by 64-bit ratios, of the places that fp32 left open: `near` of this thread's,
// one of which is `at`, or all of a cluster's if none was near.
template <typename T>
__device__ __noinline__ void verify_pick64(int* next, VerifyShared& sh, const T* row, const float* draft,
                                           const float* noise, Best top, float temp, int near, int at, int v0, int v1,
                                           int v4)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const double temperature = verify_temperature64(temp);
    const double z = draft ? verify_sum64(sh, row, top.v, temperature, v0, v1) : 0.0;
    double v64 = 0.0;
    int at64 = -1;
    auto larger = [&](double v, int place) {
        if (v > v64 || (v == v64 && place >= 0 && place < at64)) {
            v64 = v;
            at64 = place;
        }
    };
    auto look = [&](int v) {
        for (int k = 0; k < sh.n_gone; ++k)
            if (sh.gone[k] == v)
                return;
        const double w = verify_exp64(verify_clean(verify_one(row + v)), top.v, temperature);
        larger((draft ? fma(-z, static_cast<double>(draft[v]), w) : w) / noise[v], v);
    };
    if (near == 1) {
        look(at);
    } else if (near > 1 || sh.n_near == 0) {
        for (int b0 = v0 + 4 * tid; b0 < v4; b0 += 4 * VF_PICK)
            for (int i = 0; i < 4; ++i)
                look(b0 + i);
        for (int v = v4 + tid; v < v1; v += VF_PICK)
            look(v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        larger(__shfl_xor_sync(0xffffffffu, v64, o), __shfl_xor_sync(0xffffffffu, at64, o));
    if (lane == 0) {
        sh.warp64[warp] = v64;
        sh.warp_at[warp] = at64;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < VF_PICK / 32; ++w)
            larger(sh.warp64[w], sh.warp_at[w]);
        sh.best64 = v64;
        sh.best_at = at64;
    }
    cluster.sync();
    if (cluster.block_rank() == 0 && tid == 0) {
        for (int k = 1; k < static_cast<int>(cluster.num_blocks()); ++k)
            larger(*cluster.map_shared_rank(&sh.best64, k), *cluster.map_shared_rank(&sh.best_at, k));
        *next = at64 >= 0 ? at64 : top.at;  // nothing above 0: the largest logit
    }
    cluster.sync();  // no block ends while the first one reads
}

// From the last node that is known to be on the path as far as it is known; whether that is its end.
__device__ __forceinline__ bool verify_walk(VerifyShared& sh)
{
    if (threadIdx.x == 0) {
        int cur = sh.last, len = sh.len;
        unsigned long long next;
        while ((next = verify_set(sh.taken[cur]) | verify_set(sh.open[cur])) != 0 && !(verify_set(sh.open[cur]) & next & (0ull - next))) {
            cur = __ffsll(static_cast<long long>(next)) - 1;
            sh.path[len++] = cur;
        }
        sh.last = cur;
        sh.len = len;
        sh.stop = next == 0;
    }
    __syncthreads();
    return sh.stop;
}

// The path is known: it and the next token.
template <typename T>
__device__ __forceinline__ void verify_finish(const VerifyArgs& a, VerifyShared& sh, int s, int row0, int parent, int token,
                                              float temp, const VerifyScale& c, int v0, int v1)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int last = sh.last;
    if (parent == last) {  // the last node's children were all rejected
        if (a.draft)
            sh.turned_down = tid;  // a chain's one
        else if (token >= 0)
            sh.gone[atomicAdd(&sh.n_gone, 1)] = token;
    }
    if (rank == 0) {
        if (tid < a.max_new)
            a.path[static_cast<size_t>(s) * a.max_new + tid] = tid < sh.len ? sh.path[tid] : -1;
        if (tid == 0)
            a.n_path[s] = sh.len;
    }
    const Best top = sh.top[last];
    if (!(temp > 0.f) || top.at < 0) {
        if (rank == 0 && tid == 0)
            a.next[s] = top.at;
        return;
    }
    __syncthreads();
    const int n_gone = sh.n_gone, down = sh.turned_down;

    // ---- the next token
    const T* row = static_cast<const T*>(a.logits) + (row0 + last) * a.ld;
    const float* noise = a.noise + s * a.noise_ld;
    const float* draft = down ? a.draft + (row0 + down) * a.draft_ld : nullptr;
    const float z = sh.sum[last];
    const uint64_t minus = f2(-top.v, -top.v);
    const bool vec = !((reinterpret_cast<uintptr_t>(row) & (4 * sizeof(T) - 1)) | (reinterpret_cast<uintptr_t>(noise) & 15) |
                       (reinterpret_cast<uintptr_t>(draft) & 15));
    const int v4 = vec ? v0 + (max(0, v1 - v0) & ~3) : v0;
    // whether a rejected token is among this thread's places: few threads have to look each place up
    bool careful = false;
    for (int k = 0; k < n_gone; ++k) {
        const int v = sh.gone[k];
        careful |= v >= v0 && v < v1 && (v < v4 ? (v - v0) / 4 % VF_PICK == tid : (v - v4) % VF_PICK == tid);
    }
    // of this thread's places: the largest and the second largest of what a ratio may be, the
    // first one's place, and the largest of what a ratio is at least
    float first = 0.f, second = 0.f, sure = 0.f;
    int at = -1;
    auto place = [&](float most, float least, int v) {
        if (careful && (most > second || least > sure))
            for (int k = 0; k < n_gone; ++k)
                if (sh.gone[k] == v)
                    return;
        second = fmaxf(second, fminf(first, most));
        at = most > first ? v : at;
        first = fmaxf(first, most);
        sure = fmaxf(sure, least);
    };
    // Places that may not reach what one of the warp's is at least (bar) are passed over by a
    // cheap bound first: three of four pairs are.  Not with an infinite logit, whose weights that
    // bound does not have.
    float bar = isinf(top.v) ? -INFINITY : 0.f;
    constexpr float TINY = 1.1754944e-38f;  // 2^-126: weights that fp32 has as 0
    const float coarse = a.slack + 1.2e-5f, by_p = 1.f + coarse, by_q = -z * (1.f - coarse);
    auto close = [&](float x, float q, float inv, int v) {
        // r, and all that its numbers may be off by
        const float p = verify_exp(verify_clean(x), top.v, c), r = fmaf(-z, q, p);
        const float off = fmaf(p, verify_exp_off(x, top.v, c), fmaf(z * q, a.slack, TINY));
        // inv is infinite for a noise below 2^-128
        place((r + off) * inv, (r - off) * fminf(inv, 8.5070592e37f), v);
    };
    auto look = [&](float x, float y, float qx, float qy, float ex, float ey, int vx, int vy) {
        const uint64_t q = f2(qx, qy), inv = f2(__fdividef(1.f, ex), __fdividef(1.f, ey));
        const float2 u = un2(mul2(fma2(q, f2(by_q, by_q), fma2(verify_exp2(f2(x, y), minus, c), f2(by_p, by_p), f2(TINY, TINY))), inv));
        if (fmaxf(u.x, u.y) < bar)
            return;
        if (!(u.x < bar))
            close(x, qx, un2(inv).x, vx);
        if (!(u.y < bar))
            close(y, qy, un2(inv).y, vy);
    };
    constexpr int N = VF_BATCH / 4;
    for (int b = v0; b < v4; b += 4 * VF_PICK * N) {
        const int b0 = b + 4 * tid;
        float4 x[N], e[N], d[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int v = b0 + 4 * VF_PICK * i;
            x[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            e[i] = make_float4(INFINITY, INFINITY, INFINITY, INFINITY);  // a ratio of 0 is never taken
            d[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (v < v4) {
                x[i] = verify_four(row + v);
                e[i] = __ldcs(reinterpret_cast<const float4*>(noise + v));
                if (draft)
                    d[i] = __ldcs(reinterpret_cast<const float4*>(draft + v));
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int v = b0 + 4 * VF_PICK * i;
            look(x[i].x, x[i].y, d[i].x, d[i].y, e[i].x, e[i].y, v, v + 1);
            look(x[i].z, x[i].w, d[i].z, d[i].w, e[i].z, e[i].w, v + 2, v + 3);
            bar = isinf(top.v) ? bar : verify_warp_max(sure);
        }
    }
    // rows that do not begin alike, and what four do not divide
    for (int b = v4; b < v1; b += VF_PICK * VF_BATCH) {
        const int b0 = b + tid;
        float x[VF_BATCH], d[VF_BATCH], e[VF_BATCH];
#pragma unroll
        for (int i = 0; i < VF_BATCH; ++i) {
            const int v = b0 + i * VF_PICK;
            x[i] = v < v1 ? verify_one(row + v) : -INFINITY;
            e[i] = v < v1 ? __ldcs(noise + v) : INFINITY;
            d[i] = draft && v < v1 ? __ldcs(draft + v) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < VF_BATCH; i += 2)
            look(x[i], x[i + 1], d[i], d[i + 1], e[i], e[i + 1], b0 + i * VF_PICK, b0 + (i + 1) * VF_PICK);
        bar = isinf(top.v) ? bar : verify_warp_max(sure);
    }
    sure = verify_warp_max(sure);
    if (lane == 0)
        sh.warp[warp] = sure;
    __syncthreads();
    if (warp == 0) {
        sure = verify_warp_max(lane < VF_PICK / 32 ? sh.warp[lane] : 0.f);
        if (lane == 0) {
            sh.sure = sure;
            sh.n_near = 0;
        }
    }
    cluster.sync();
    float most = 0.f;
    for (int k = 0; k < blocks; ++k)
        most = fmaxf(most, *cluster.map_shared_rank(&sh.sure, k));
    const int near = (first > 0.f && first >= most) + (second > 0.f && second >= most);
    if (near)
        for (int k = 0; k < blocks; ++k) {
            VerifyShared* to = cluster.map_shared_rank(&sh, k);
            atomicAdd(&to->n_near, near);
            to->near = at;
        }
    cluster.sync();
    if (sh.n_near == 1 && most > 0.f) {
        if (rank == 0 && tid == 0)
            a.next[s] = sh.near;
        return;
    }
    verify_pick64(a.next + s, sh, row, draft, noise, top, temp, near, at, v0, v1, v4);
}

// The walk came to an open test, and does again: the last node's children once more, from the
// sum to 2^-38 and weights in 64 bits.  All blocks of the cluster have the same numbers, so they
// come here together.  A function of its own, which nothing follows, so that it takes no registers
// from the usual way.
template <typename T>
__device__ __noinline__ void verify_open(const VerifyArgs& a, VerifyShared& sh, int s, int row0, int parent, int token, bool mine,
                                         float own, float u, float q, float temp, int v0, int v1)
{
    const int tid = threadIdx.x;
    const unsigned long long me = 1ull << (tid & 63);
    const double temperature = verify_temperature64(temp);
    do {
        const int cur = sh.last;
        const float top = sh.top[cur].v;
        const double z = verify_sum64(sh, static_cast<const T*>(a.logits) + (row0 + cur) * a.ld, top, temperature, v0, v1);
        if (tid < VF_MAX_NEW && (verify_set(sh.fresh[cur]) & me))
            sh.w64[tid] = verify_exp64(own, top, temperature);
        if (tid == 0) {
            sh.sum[cur] = static_cast<float>(z);
            sh.taken[cur] = sh.open[cur] = make_uint2(0u, 0u);
        }
        __syncthreads();
        if (mine && parent == cur) {
            double left = z;
            verify_each(verify_set(sh.fresh[cur]) & (me - 1), [&](int i) { left -= sh.w64[i]; });
            if (static_cast<double>(u) * q * fmax(left, 0.0) < sh.w64[tid])
                verify_put(sh.taken[cur], tid);
        }
        __syncthreads();
    } while (!verify_walk(sh));
    verify_finish<T>(a, sh, s, row0, parent, token, temp, verify_scale(temp), v0, v1);
}

template <typename T>
__global__ void __launch_bounds__(VF_PICK, 2) verify_pick_kernel(const __grid_constant__ VerifyArgs a)
{
    namespace cg = cooperative_groups;
    __shared__ VerifyShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int s = blockIdx.x / blocks;
    const int tid = threadIdx.x, warp = tid >> 5;
    const float temp = a.temperature ? __ldg(a.temperature + s) : 1.f;
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
    const bool greedy = !(temp > 0.f);
    const VerifyScale c = verify_scale(greedy ? 1.f : temp);

    if (tid < VF_MAX_NEW)
        sh.kids[tid] = sh.fresh[tid] = sh.taken[tid] = sh.open[tid] = make_uint2(0u, 0u);
    // the tree's numbers and the random ones are on their way while the sums are still made
    int parent = -1, token = -1;
    float u = 0.f, q = 1.f;
    if (tid < n) {
        token = __ldg(a.tokens + row0 + tid);
        parent = tid == 0 ? -1 : a.parents ? __ldg(a.parents + row0 + tid) : tid - 1;
        u = __ldg(a.uniform + row0 + tid);
    }
    const int slice = ((a.vocab + blocks - 1) / blocks + 3) & ~3, v0 = rank * slice, v1 = min(a.vocab, v0 + slice);
    const float* noise = a.noise + s * a.noise_ld;
    if (!greedy)
        for (int v = v0 + 32 * tid; v < v1; v += 32 * VF_PICK)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + v));
    __syncthreads();
    pdl_wait();
    // eight threads a node join its pieces: the largest logit first, then the sums in two
    // parts (the second has what the first loses)
    const int node = tid >> 3;
    const float4* part = a.part + static_cast<size_t>(row0 + min(node, n - 1)) * a.pieces;
    constexpr int E = 5;  // pieces a thread has in registers: 40 a row
    float4 x[E];
    auto pieces = [&](int k0) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = k0 + (tid & 7) + 8 * e;
            x[e] = k < a.pieces ? __ldcg(part + k) : make_float4(-INFINITY, __int_as_float(-1), 0.f, 0.f);
        }
    };
    pieces(0);
    float own = -INFINITY;  // a node's token's logit at its parent
    if (tid < n) {
        if (tid > 0 && (parent < 0 || parent >= tid)) {
            parent = -1;
            if (rank == 0)
                set_error(a.err, DEVERR_BAD_ARG);
        }
        if (token < 0 || token >= a.vocab)
            token = -1;
        if (parent >= 0 && token >= 0) {
            verify_put(sh.kids[parent], tid);
            own = verify_clean(verify_one(logits + (row0 + parent) * a.ld + token));
            if (a.draft)
                q = __ldg(a.draft + (row0 + tid) * a.draft_ld + token);
        }
        sh.token[tid] = token;
    }
    if (warp < 4 * ((n + 15) / 16)) {
        Best top{-INFINITY, -1};
        auto largest = [&] {
#pragma unroll
            for (int e = 0; e < E; ++e)
                top = better(top, Best{x[e].x, __float_as_int(x[e].y)});
        };
        largest();
        for (int k = 8 * E; k < a.pieces; k += 8 * E) {
            pieces(k);
            largest();
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
            top = better(top, Best{__shfl_xor_sync(0xffffffffu, top.v, o), __shfl_xor_sync(0xffffffffu, top.at, o)});
        float hi = 0.f, lo = 0.f;
        auto add = [&](float v) {
            const float t = hi + v, z = t - hi;
            lo += (hi - (t - z)) + (v - z);
            hi = t;
        };
        for (int k = 0; k < a.pieces; k += 8 * E) {
            if (a.pieces > 8 * E)
                pieces(k);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (__float_as_int(x[e].y) >= 0)
                    add(x[e].z * verify_exp(x[e].x, top.v, c));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            const float h2 = __shfl_xor_sync(0xffffffffu, hi, o), l2 = __shfl_xor_sync(0xffffffffu, lo, o);
            add(h2);
            lo += l2;
        }
        if (node < n && (tid & 7) == 0) {
            sh.top[node] = top;
            sh.sum[node] = hi + lo;
        }
    }
    __syncthreads();
    const Best above = parent >= 0 ? sh.top[parent] : Best{-INFINITY, -1};
    const float w = parent < 0 || token < 0 || above.at < 0 || greedy ? 0.f : verify_exp(own, above.v, c);
    const unsigned long long me = 1ull << (tid & 63);
    bool mine = parent >= 0 && token >= 0;  // may be accepted
    if (mine)
        verify_each(verify_set(sh.kids[parent]) & (me - 1), [&](int i) { mine = mine && sh.token[i] != token; });
    if (mine)
        verify_put(sh.fresh[parent], tid);
    if (tid < n)
        sh.w[tid] = w;
    __syncthreads();

    // ---- each node's test, should its turn come: the children of a node are tried in ascending
    // order, so all its siblings before it were rejected; probabilities in units of 1 / the
    // node's sum.  Where the two sides are nearer than what fp32 may have rounded (rejected
    // siblings leave a difference of large numbers), the test is open.
    mine = mine && above.at >= 0 && own > -INFINITY;  // a weight of 0 is never accepted
    if (mine) {
        bool take, open = false;
        if (greedy) {
            take = token == above.at;
        } else {
            const float sum = sh.sum[parent], by = u * q;
            float left = sum;
            verify_each(verify_set(sh.fresh[parent]) & (me - 1), [&](int i) { left -= sh.w[i]; });
            const float gone = sum - left;
            left = by * fmaxf(left, 0.f);
            // the sum's and the weights' errors, and a rounding for each rejected one; 2^-126 for what
            // fp32 has as 0
            const float off = fmaf(a.slack, fmaf(by, sum + gone, w), fmaf(gone > 0.f ? 4e-6f : 0.f, by * sum, 1.1754944e-38f));
            take = left + off < w;
            open = !take && !(left - off >= w);
        }
        if (take)
            verify_put(sh.taken[parent], tid);
        if (open)
            verify_put(sh.open[parent], tid);
    }
    if (tid == 0) {
        sh.last = sh.path[0] = 0;
        sh.len = 1;
        sh.n_gone = sh.turned_down = 0;
    }
    __syncthreads();
    if (!verify_walk(sh)) {
        verify_open<T>(a, sh, s, row0, parent, token, mine, own, u, q, temp, v0, v1);
        return;
    }
    verify_finish<T>(a, sh, s, row0, parent, token, temp, c, v0, v1);
}

}  // namespace dq

namespace dqhost {

// More than eight blocks a cluster, allowed once per device.
template <typename K>
static cudaError_t verify_prepare(K kernel, bool (&done)[64])
{
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess && dev >= 0 && dev < 64)
            done[dev] = true;
    }
    return e;
}

// How the first kernel cuts a row (which may begin up to 7 elements into its first 16
// bytes): into the number of pieces whose rounds of blocks, four an SM with 16-bit logits
// and five with fp32 ones, take the fewest steps, a block's start and end counted as one and
// a half of them (405 rows of 100003 in bf16: 24.5 us; 27.5 with pieces of six steps, whose
// 2025 blocks are three rounds and a third).
struct VerifyCut {
    int pieces, steps;
    // What the fp32 sum of a row's weights may be off by, at most, relative to itself; more than a
    // weight of 2^-126 and up (verify_exp_off).  A weight 2^-t: ex2's 2^-22 and, of t, the three
    // roundings of verify_exp2, 3 t 2^-24 ln 2, where t averaged over a sum's weights is at most
    // log2(vocab) <= 24: 3.3e-6.  The joins of lanes, warps and pieces: 2e-6.  A step: an addition,
    // and another maximum's factor and its product: 6 2^-24.
    float slack() const { return 8e-6f + 3.6e-7f * static_cast<float>(steps); }
};
static VerifyCut verify_cut(int total_new, int vocab, bool wide)
{
    const int all = (vocab + 7 + dq::VF_STEP - 1) / dq::VF_STEP;
    const long long slots = (wide ? 5ll : 4ll) * sm_count();
    VerifyCut best{1, all};
    double least = 0.0;
    for (int p = 1; p <= std::min(all, 64); ++p) {
        const int steps = (all + p - 1) / p;
        if ((all + steps - 1) / steps != p)
            continue;  // as many steps as with fewer pieces
        const double cost = static_cast<double>((total_new * static_cast<long long>(p) + slots - 1) / slots) * (steps + 1.5);
        if (p == 1 || cost < least) {
            least = cost;
            best = {p, steps};
        }
    }
    return best;
}

}  // namespace dqhost

extern "C" {

DQ_API size_t dq_verify_draft_workspace_bytes(int total_new, int vocab)
{
    if (total_new < 1 || vocab < 1 || total_new > (1 << 24) || vocab > (1 << 24))
        return 0;
    const int pieces = std::max(dqhost::verify_cut(total_new, vocab, false).pieces, dqhost::verify_cut(total_new, vocab, true).pieces);
    return static_cast<size_t>(total_new) * pieces * sizeof(float4);
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
    const long long steps = (static_cast<long long>(v->vocab) + 7 + dq::VF_STEP - 1) / dq::VF_STEP;
    if (v->max_new > dq::VF_MAX_NEW || (v->draft_probs && v->parents) || v->vocab > (1 << 24) || v->total_new > (1 << 24) ||
        v->n_seq > (1 << 24) || v->total_new * steps > (1 << 30))
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
    const dqhost::VerifyCut cut = dqhost::verify_cut(v->total_new, v->vocab, v->type == DQ_TYPE_F32);
    const dq::VerifyArgs a{v->logits, v->logits_stride, v->draft_probs, v->draft_stride, v->noise, v->noise_stride,
                           v->tokens, v->parents, v->uniform, v->temperature, v->cu_new, v->path, v->n_path, v->next,
                           v->n_seq, v->total_new, v->max_new, v->vocab, cut.pieces, cut.steps, static_cast<float4*>(v->workspace),
                           cut.slack(), dqhost::device_error_flag()};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dqhost::with_type(v->type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const unsigned grid = static_cast<unsigned>(v->total_new) * cut.pieces;
        dq::verify_stats_kernel<T><<<grid, dq::VF_THREADS, 0, s>>>(a);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess)
            return err;
        // a dependent launch: it gathers the tree's numbers while the last pieces run
        static bool done[64] = {};
        const cudaError_t wide = dqhost::verify_prepare(dq::verify_pick_kernel<T>, done);
        if (wide != cudaSuccess)
            return wide;
        // as many blocks a sequence as are resident together, two an SM (1, 2, 4, 8 or 16)
        int blocks = dq::VF_CLUSTER;
        while (blocks > 1 && static_cast<long long>(v->n_seq) * blocks > 2 * dqhost::sm_count())
            blocks /= 2;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(v->n_seq) * blocks);
        cfg.blockDim = dim3(dq::VF_PICK);
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = blocks;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, dq::verify_pick_kernel<T>, a);
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
