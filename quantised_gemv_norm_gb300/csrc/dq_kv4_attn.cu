// dq_kv4_attn.cu -- single-token attention of a batch of sequences over the paged
// 4-bit cache (dq_attention_decode_kv4).
//
// A block takes a run of 16-key blocks of one sequence and one KV head; its warps
// take them in turn.  Each warp streams its cache blocks (2560 bytes, keys, values
// and scales together) into a ring of its own in shared memory with bulk copies and
// keeps its own running reference exponent, sum and output, all in registers;
// the block's warps meet once at the end, the blocks of one sequence in a second
// kernel.  The cache bytes bound it, so the arithmetic goes to the (warp-level)
// matrix instructions m16n8k16, whose 16 rows hold the group's up to 8 query heads
// twice: the fp16 part of a query in row h and the rest of it in row 8 + h, which
// gives 22 bits for the price of 11 with so few rows.  The codes c - 8 are exact in
// fp16 and need no scale before the product:
//   s_j   = sum_g d_jg (sum_{n in g} q_n (c_jn - 8)) + z_jg (sum_{n in g} q_n)
//   out_n = sum_j (p_j d_jg) (c_jn - 8) + sum_j p_j z_jg
// with g the groups of 32 dims; p_j d_jg is again two fp16 parts.
//
// p_j = 2^(s_j - r) with a reference r a head that follows the running maximum only
// when some s_j - r passes a cap: p_j d_jg stays in fp16's normal range on both
// sides, and the outputs are scaled only a few times a sequence.
#include <algorithm>

#include "dq_kv4.cuh"

namespace dq {

constexpr int KA_WARPS = 4;
constexpr int KA_NS = 4;       // ring stages a warp
constexpr int KA_PART = 132;   // floats of a partial result: r, l, two unused, 128 sums
constexpr float KA_CAP = 12.f;   // p_j <= 2^cap where every d <= 8
constexpr float KA_HEAD = 3.f;   // log2 that the maximum may grow before r follows it

struct Kv4AttnArgs {
    const void* q;
    void* out;
    const unsigned char* pool;
    const int* pages;
    const int* n_keys;
    float* part;       // [n_seq][n_kv][splits][8][KA_PART], or null: one block a sequence and KV head
    int n_seq, n_q, group, splits, chunk;  // chunk: 16-key blocks a thread block
    Kv4Shape s;
    int max_pages, max_keys;
    int* err;
};

__device__ __forceinline__ uint64_t f2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 un2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t half2_f2(uint32_t h)
{
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return f2(v.x, v.y);
}

__device__ __forceinline__ float ka_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four fp16 pairs c - 8 from a word: pair i has the codes at bits 4 i and 16 + 4 i.
// A code in mantissa bits 0-3 of 1024 is 1024 + c, in bits 4-7 of 64 it is 64 + c.
__device__ __forceinline__ void ka_codes(uint32_t w, uint32_t (&p)[4])
{
    const uint32_t w8 = w >> 8;
    const uint32_t a = (w & 0x000F000Fu) | 0x64006400u, b = (w & 0x00F000F0u) | 0x54005400u;
    const uint32_t c = (w8 & 0x000F000Fu) | 0x64006400u, d = (w8 & 0x00F000F0u) | 0x54005400u;
    // -1032 = 0xE408, -72 = 0xD480
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[0]) : "r"(a), "r"(0xE408E408u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[1]) : "r"(b), "r"(0xD480D480u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[2]) : "r"(c), "r"(0xE408E408u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[3]) : "r"(d), "r"(0xD480D480u));
}

__device__ __forceinline__ void ka_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x, y as an fp16 pair and what is left of them as another.
__device__ __forceinline__ void ka_split(uint64_t v, uint32_t& hi, uint32_t& lo)
{
    const float2 x = un2(v);
    hi = pack2(x.x, x.y, static_cast<const __half*>(nullptr));
    const float2 rest = un2(fma2(half2_f2(hi), f2(-1.f, -1.f), v));
    lo = pack2(rest.x, rest.y, static_cast<const __half*>(nullptr));
}

template <typename T>
__global__ void __launch_bounds__(32 * KA_WARPS, 3) kv4_attn_kernel(const Kv4AttnArgs a)
{
    __shared__ __align__(128) unsigned char ring[KA_WARPS][KA_NS][KV4_BYTES];
    __shared__ uint64_t full[KA_WARPS][KA_NS];
    __shared__ int skip[KA_WARPS][KA_NS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = lane >> 2, tq = lane & 3;  // this lane's head of the group, and quarter
    int x = blockIdx.x;
    const int c = x % a.splits;
    x /= a.splits;
    const int g = x % a.s.n_kv, b = x / a.s.n_kv;

    int n = __ldg(a.n_keys + b);
    if (n < 0 || n > a.max_keys) {
        if (threadIdx.x == 0 && c == 0 && g == 0)
            set_error(a.err, DEVERR_BAD_ARG);
        n = 0;
    }
    const int blk0 = c * a.chunk, blk1 = min(blk0 + a.chunk, (n + KV4_ROWS - 1) / KV4_ROWS);
    if (a.part && blk0 >= blk1)
        return;  // the join does not look at it
    const int cnt = blk0 + warp < blk1 ? (blk1 - blk0 - warp + KA_WARPS - 1) / KA_WARPS : 0;

    if (lane == 0) {
        for (int i = 0; i < KA_NS; ++i)
            mbar_init(&full[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();

    // ---- this warp's cache blocks: lane i has the page of the i-th of the next 32
    const int bpp = a.s.page_rows / KV4_ROWS;
    const int* pages = a.pages + static_cast<size_t>(b) * a.max_pages;
    auto block_at = [&](int i) { return blk0 + warp + KA_WARPS * i; };
    auto page_of = [&](int i) { return i < cnt ? __ldg(pages + block_at(i) / bpp) : 0; };
    int next_page = page_of(lane);
    long long off = 0;
    auto issue = [&](int i) {
        if ((i & 31) == 0) {
            off = next_page < 0 || next_page >= a.s.n_pages
                      ? -1
                      : ((static_cast<long long>(next_page) * a.s.n_kv + g) * bpp + block_at(i + lane) % bpp) * KV4_BYTES;
            next_page = page_of(i + 32 + lane);
        }
        const long long at = __shfl_sync(0xffffffffu, off, i & 31);
        if (lane == 0) {
            uint64_t* bar = &full[warp][i % KA_NS];
            skip[warp][i % KA_NS] = at < 0;
            if (at < 0) {
                set_error(a.err, DEVERR_BAD_ARG);
                mbar_arrive(bar);
            } else {
                mbar_arrive_expect_tx(bar, KV4_BYTES);
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                        smem_addr(ring[warp][i % KA_NS])),
                    "l"(a.pool + at), "r"(KV4_BYTES), "r"(smem_addr(bar))
                    : "memory");
            }
        }
        __syncwarp();
    };
    for (int i = 0; i < min(cnt, KA_NS); ++i)
        issue(i);

    // ---- queries: scaled by a power of two a head into fp16's range, in two parts
    uint32_t qa[8][4];
    float qsum[4], unscale;
    {
        float4 v[4][2];
        const T* q = static_cast<const T*>(a.q) + (static_cast<size_t>(b) * a.n_q + g * a.group + h) * ATT_HD + 8 * tq;
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                v[k][e] = h < a.group ? load4(q + 32 * k + 4 * e) : make_float4(0.f, 0.f, 0.f, 0.f);
                top = fmaxf(top, fmaxf(fmaxf(fabsf(v[k][e].x), fabsf(v[k][e].y)), fmaxf(fabsf(v[k][e].z), fabsf(v[k][e].w))));
            }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // largest |q| into [2^13, 2^14): the exponent field moves, nothing is rounded
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 13;
        e = max(-100, min(114, e));
        const float scale = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        unscale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * (0.08838834764831845f * 1.4426950408889634f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float sum = 0.f;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float4 w = v[k][m];
                const uint64_t p0 = f2(w.x * scale, w.y * scale), p1 = f2(w.z * scale, w.w * scale);
                ka_split(p0, qa[2 * k + m][0], qa[2 * k + m][1]);
                ka_split(p1, qa[2 * k + m][2], qa[2 * k + m][3]);
                const float2 s0 = un2(p0), s1 = un2(p1);
                sum += (s0.x + s0.y) + (s1.x + s1.y);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            qsum[k] = sum;
        }
    }

    uint64_t o[4][4];  // group g, i: head h, dims 32 g + 8 tq + i and + 4 + i
    uint64_t zacc[4], lacc = 0ull;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        zacc[k] = 0ull;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[k][i] = 0ull;
    }
    float r = -INFINITY, cap = KA_CAP;
    bool ok = true;
    for (int i = 0; i < cnt; ++i) {
        const int st = i % KA_NS;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[warp][st], (i / KA_NS) & 1))) {
            ok = false;
            break;
        }
        if (!skip[warp][st]) {
            unsigned char* kb = ring[warp][st];
            const int left = n - KV4_ROWS * block_at(i);
            if (left < KV4_ROWS) {
                // rows past the last key may hold anything: their value scales become zero
                // (their scores are masked below); the last block: nothing is copied over it
                const int u = lane >> 2;
                unsigned short* vs = reinterpret_cast<unsigned short*>(kb + KV4_VSCALES + 32 * u + 8 * (lane & 3));
                if (2 * u >= left)
                    vs[0] = vs[2] = 0;
                if (2 * u + 1 >= left)
                    vs[1] = vs[3] = 0;
                __syncwarp();
            }
            // scores of keys 8 nt + 2 tq, + 1 for head h
            uint64_t s[2];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const uint4 kw = lds128(kb + 64 * (8 * nt + h) + 16 * tq);
                const uint4 sc0 = lds128(kb + KV4_KSCALES + 32 * (4 * nt + tq));
                const uint4 sc1 = lds128(kb + KV4_KSCALES + 32 * (4 * nt + tq) + 16);
                const uint32_t words[4] = {kw.x, kw.y, kw.z, kw.w};
                const uint32_t dd[4] = {sc0.x, sc0.z, sc1.x, sc1.z}, zz[4] = {sc0.y, sc0.w, sc1.y, sc1.w};
                uint64_t acc = 0ull;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t p[4];
                    ka_codes(words[k], p);
                    float m[4] = {0.f, 0.f, 0.f, 0.f};
                    ka_mma(m, qa[2 * k][0], qa[2 * k][1], qa[2 * k][2], qa[2 * k][3], p[0], p[1]);
                    ka_mma(m, qa[2 * k + 1][0], qa[2 * k + 1][1], qa[2 * k + 1][2], qa[2 * k + 1][3], p[2], p[3]);
                    acc = fma2(add2(f2(m[0], m[1]), f2(m[2], m[3])), half2_f2(dd[k]), acc);
                    acc = fma2(half2_f2(zz[k]), f2(qsum[k], qsum[k]), acc);
                }
                s[nt] = mul2(acc, f2(unscale, unscale));
            }
            if (left < KV4_ROWS) {
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    float2 v = un2(s[nt]);
                    if (8 * nt + 2 * tq >= left)
                        v.x = -INFINITY;
                    if (8 * nt + 2 * tq + 1 >= left)
                        v.y = -INFINITY;
                    s[nt] = f2(v.x, v.y);
                }
            }
            uint32_t vd[2][4], vz[2][4];
            __half2 dmax = __half2half2(__ushort_as_half(0));
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const uint4 sc0 = lds128(kb + KV4_VSCALES + 32 * (4 * nt + tq));
                const uint4 sc1 = lds128(kb + KV4_VSCALES + 32 * (4 * nt + tq) + 16);
                vd[nt][0] = sc0.x, vz[nt][0] = sc0.y, vd[nt][1] = sc0.z, vz[nt][1] = sc0.w;
                vd[nt][2] = sc1.x, vz[nt][2] = sc1.y, vd[nt][3] = sc1.z, vz[nt][3] = sc1.w;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    dmax = __hmax2(dmax, *reinterpret_cast<const __half2*>(&vd[nt][k]));
            }
            const float2 s0 = un2(s[0]), s1 = un2(s[1]);
            const float top = fmaxf(fmaxf(s0.x, s0.y), fmaxf(s1.x, s1.y));
            // d <= 8 keeps p d below 2^15 under the cap; a larger one lowers the cap
            const bool wide = !__hble2(dmax, __half2half2(__ushort_as_half(0x4800)));
            if (__any_sync(0xffffffffu, top - r > cap || (wide && cap == KA_CAP))) {
                float d = fmaxf(__low2float(dmax), __high2float(dmax));
                float t = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                d = warp_max(d);
                if (d > 8.f)  // from now on for the largest scale there is
                    cap = 15.f - 16.f;
                if (t - r > cap) {
                    const float rn = t - (cap - KA_HEAD);
                    const float f = ka_ex2(r - rn);
                    r = rn;
                    lacc = mul2(lacc, f2(f, f));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        zacc[k] = mul2(zacc[k], f2(f, f));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            o[k][j] = mul2(o[k][j], f2(f, f));
                    }
                }
                __syncwarp();
            }
            const float rr = r == -INFINITY ? 0.f : r;
            const uint64_t p0 = f2(ka_ex2(s0.x - rr), ka_ex2(s0.y - rr)), p1 = f2(ka_ex2(s1.x - rr), ka_ex2(s1.y - rr));
            lacc = add2(lacc, add2(p0, p1));
            const uint4 va = lds128(kb + KV4_VCODES + 16 * lane), vb = lds128(kb + KV4_VCODES + 512 + 16 * lane);
            const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t h0, l0, h1, l1;
                ka_split(mul2(p0, half2_f2(vd[0][k])), h0, l0);
                ka_split(mul2(p1, half2_f2(vd[1][k])), h1, l1);
                zacc[k] = fma2(p0, half2_f2(vz[0][k]), zacc[k]);
                zacc[k] = fma2(p1, half2_f2(vz[1][k]), zacc[k]);
                uint32_t b0[4], b1[4];
                ka_codes(wa[k], b0);
                ka_codes(wb[k], b1);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // the sums over blocks are rounded adds: the matrix instruction's own
                    // accumulation cuts off (100001 keys: relative error 1.6e-6 with it)
                    float m[4] = {0.f, 0.f, 0.f, 0.f};
                    ka_mma(m, h0, l0, h1, l1, b0[j], b1[j]);
                    o[k][j] = add2(o[k][j], add2(f2(m[0], m[1]), f2(m[2], m[3])));
                }
            }
        }
        __syncwarp();  // every lane has read the stage
        if (i + KA_NS < cnt)
            issue(i + KA_NS);
    }
    if (!ok) {
        if (lane == 0) {
            set_error(a.err, DEVERR_TIMEOUT_FULL);
            for (int i = 0; i < min(cnt, KA_NS); ++i)
                if (!mbar_wait(&full[warp][i], 0) && !mbar_wait(&full[warp][i], 1))
                    set_error(a.err, DEVERR_TIMEOUT_DRAIN);
        }
    }
    __syncthreads();

    // ---- the warps' results meet in shared memory: r, l and 128 sums a head
    float* meet = reinterpret_cast<float*>(ring);
    static_assert(sizeof(ring) >= KA_WARPS * 8 * KA_PART * 4, "the ring holds the warps' results");
    {
        const float2 l2 = un2(lacc);
        float l = l2.x + l2.y;
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        float* mp = meet + (warp * 8 + h) * KA_PART;
        if (tq == 0) {
            mp[0] = r;
            mp[1] = l;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 z2 = un2(zacc[k]);
            float z = z2.x + z2.y;
            z += __shfl_xor_sync(0xffffffffu, z, 1);
            z += __shfl_xor_sync(0xffffffffu, z, 2);
            const float2 y0 = un2(o[k][0]), y1 = un2(o[k][1]), y2 = un2(o[k][2]), y3 = un2(o[k][3]);
            const float4 lo = make_float4(y0.x + z, y1.x + z, y2.x + z, y3.x + z);
            const float4 hi = make_float4(y0.y + z, y1.y + z, y2.y + z, y3.y + z);
            *reinterpret_cast<float4*>(mp + 4 + 32 * k + 8 * tq) = lo;
            *reinterpret_cast<float4*>(mp + 4 + 32 * k + 8 * tq + 4) = hi;
        }
    }
    __syncthreads();
    for (int hd = warp; hd < a.group; hd += KA_WARPS) {
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < KA_WARPS; ++w)
            m = fmaxf(m, meet[(w * 8 + hd) * KA_PART]);
        float l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KA_WARPS; ++w) {
            const float* mp = meet + (w * 8 + hd) * KA_PART;
            // a warp without keys has r = -infinity and sums of 0
            const float f = mp[0] == m ? 1.f : ka_ex2(mp[0] - m);
            const float4 y = *reinterpret_cast<const float4*>(mp + 4 + 4 * lane);
            l += f * mp[1];
            v.x += f * y.x;
            v.y += f * y.y;
            v.z += f * y.z;
            v.w += f * y.w;
        }
        if (a.part) {
            float* pp = a.part + (((static_cast<size_t>(b) * a.s.n_kv + g) * a.splits + c) * 8 + hd) * KA_PART;
            if (lane == 0) {
                pp[0] = m;
                pp[1] = l;
            }
            *reinterpret_cast<float4*>(pp + 4 + 4 * lane) = v;
        } else {
            const float inv = n > 0 && l != 0.f ? 1.0f / l : 0.f;
            store4(static_cast<T*>(a.out) + (static_cast<size_t>(b) * a.n_q + g * a.group + hd) * ATT_HD + 4 * lane,
                   make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        }
    }
}

// The splits' results of one sequence and query head: one warp, four dims a lane.
template <typename T>
__global__ void __launch_bounds__(32) kv4_join_kernel(const Kv4AttnArgs a)
{
    const int lane = threadIdx.x;
    const int b = blockIdx.x / a.n_q, hq = blockIdx.x % a.n_q, g = hq / a.group, h = hq % a.group;
    int n = __ldg(a.n_keys + b);
    if (n < 0 || n > a.max_keys)
        n = 0;
    const int blocks = (n + KV4_ROWS - 1) / KV4_ROWS, splits = (blocks + a.chunk - 1) / a.chunk;
    const float* base = a.part + ((static_cast<size_t>(b) * a.s.n_kv + g) * a.splits * 8 + h) * KA_PART;
    const size_t step = 8 * KA_PART;
    pdl_wait();
    float m = -INFINITY;
    for (int c = lane; c < splits; c += 32)
        m = fmaxf(m, __ldcg(base + c * step));
    m = warp_max(m);
    float l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < splits; ++c) {
        const float* pp = base + c * step;
        const float2 rl = __ldcg(reinterpret_cast<const float2*>(pp));
        const float4 y = __ldcg(reinterpret_cast<const float4*>(pp + 4) + lane);
        const float f = rl.x == m ? 1.f : ka_ex2(rl.x - m);
        l += f * rl.y;
        v.x += f * y.x;
        v.y += f * y.y;
        v.z += f * y.z;
        v.w += f * y.w;
    }
    const float inv = n > 0 && l != 0.f ? 1.0f / l : 0.f;
    store4(static_cast<T*>(a.out) + (static_cast<size_t>(b) * a.n_q + hq) * ATT_HD + 4 * lane,
           make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
}

}  // namespace dq

namespace dqhost {

// How a call is split: 16-key blocks a thread block, and thread blocks a sequence and
// KV head.
struct Kv4Split {
    int chunk, splits;
};

static Kv4Split kv4_split(int n_seq, int n_kv, int max_keys)
{
    const long long blocks = (static_cast<long long>(max_keys) + dq::KV4_ROWS - 1) / dq::KV4_ROWS;
    const long long all = blocks * n_seq * n_kv, room = 3ll * sm_count();
    long long chunk = (all + room - 1) / room;
    if (n_seq > 1)
        chunk = std::min(chunk, 64ll);
    chunk = std::max<long long>(chunk, dq::KA_WARPS);
    return {static_cast<int>(chunk), static_cast<int>((blocks + chunk - 1) / chunk)};
}

}  // namespace dqhost

extern "C" {

DQ_API size_t dq_attention_decode_kv4_workspace_bytes(int n_seq, int n_q, int n_kv, int max_keys)
{
    if (n_seq < 1 || n_q < 1 || n_kv < 1 || max_keys < 1)
        return 0;
    const dqhost::Kv4Split sp = dqhost::kv4_split(n_seq, n_kv, max_keys);
    return sp.splits > 1 ? static_cast<size_t>(n_seq) * n_kv * sp.splits * 8 * dq::KA_PART * sizeof(float) : 0;
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
    if (n_q / n_kv > 8)
        return DQ_ERR_UNSUPPORTED;
    if (!dqhost::aligned16(q) || !dqhost::aligned16(pool) || !dqhost::aligned16(out))
        return DQ_ERR_ALIGN;
    const dqhost::Kv4Split sp = dqhost::kv4_split(n_seq, n_kv, max_keys);
    const long long blocks = static_cast<long long>(n_seq) * n_kv * sp.splits;
    if (blocks > 0x7fffffffll || static_cast<long long>(n_seq) * n_q > 0x7fffffffll)
        return DQ_ERR_UNSUPPORTED;
    if (sp.splits > 1) {
        if (!workspace)
            return DQ_ERR_NULL;
        if (workspace_bytes < dq_attention_decode_kv4_workspace_bytes(n_seq, n_q, n_kv, max_keys))
            return DQ_ERR_SHAPE;
        if (!dqhost::aligned16(workspace))
            return DQ_ERR_ALIGN;
    }
    const dq::Kv4AttnArgs a{q, out, static_cast<const unsigned char*>(pool), pages, n_keys,
                            sp.splits > 1 ? static_cast<float*>(workspace) : nullptr, n_seq, n_q, n_q / n_kv, sp.splits,
                            sp.chunk, {n_kv, n_pages, page_size}, max_pages, max_keys, dqhost::device_error_flag()};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dqhost::with_type(type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        dq::kv4_attn_kernel<T><<<static_cast<unsigned>(blocks), 32 * dq::KA_WARPS, 0, s>>>(a);
        if (sp.splits > 1)
            dq::kv4_join_kernel<T><<<n_seq * n_q, 32, 0, s>>>(a);
        return cudaGetLastError();
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
