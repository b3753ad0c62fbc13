// dq_kv4_attn.cu -- single-token attention of a batch of sequences over the paged
// 4-bit cache (dq_attention_decode_kv4).
//
// A block takes a run of 16-key blocks of one sequence and one KV head; its warps
// take them in turn.  Each warp streams its cache blocks (2560 bytes, keys, values
// and scales together) into a ring of its own in shared memory with bulk copies and
// keeps its own running reference exponent, sum and output, all in registers;
// the block's warps meet once at the end, the blocks of one sequence in a second
// kernel.  Its floor is the cache's bytes, so the arithmetic goes to the
// (warp-level) matrix instructions m16n8k16, whose 16 rows hold the group's up to 8 query
// heads twice: the fp16 part of a query in row h and, for fp32 results, the rest of it in row
// 8 + h, which gives 22 bits for the price of 11 with so few rows.  The codes c - 8 are
// exact in fp16 and need no scale before the product:
//   s_j   = sum_g d_jg (sum_{n in g} q_n (c_jn - 8)) + z_jg (sum_{n in g} q_n)
//   out_n = sum_j (p_j d_jg) (c_jn - 8) + sum_j p_j z_jg
// with g the groups of 32 dims; p_j d_jg is again two fp16 parts for fp32 results and
// one for 16-bit ones.
//
// What bounds it is the latency of its chains of instructions: a cache block takes a warp
// 402 of them with one part (half of them codes and scales made into operands) and 451
// with two, each warp's largely in sequence, and the 12 warps an SM that 168 registers
// leave issue 0.59 (0.54) a clock and scheduler.  48 sequences of 1 to 12000 keys, 325 MB:
// 85 us (3.8 TB/s; 48 us at the memory's rate), one of 100001, 128 MB, two parts: 44 us
// (2.9 TB/s; 19 us).  A call of 64 keys takes 3.4 us in a graph.
//
// p_j = 2^(s_j - r) with a reference r a head that follows the running maximum only
// when some s_j - r passes a cap: p_j d_jg stays below fp16's largest number, and the
// outputs are scaled only a few times a sequence.  The cap is 12 where every value scale
// d is 8 or less and falls with the largest one seen, to -1; the largest p is within 2^3 of
// it.  Products below 2^-14 lose bits, each is off by half of fp16's smallest step (2^-25)
// at most: 2^-34 max(1, D / 4) of the largest p, D the largest scale.  s_j is rounded once
// more, to the unit of r, before r is subtracted (relative error at 100001 keys 8.5e-7, 8.4e-7
// in one fused step): the largest score is then the same number in both, where the fused
// step left out the rounding that r has and passed fp16's range at scores of 2^26.
#include <algorithm>

#include "dq_kv4.cuh"

namespace dq {

constexpr int KA_WARPS = 4;
constexpr int KA_STEP = 2;     // cache blocks a ring stage
constexpr int KA_NS = 2;       // ring stages a warp
constexpr int KA_RESIDENT = 3; // blocks an SM (4, at 128 registers: 96.5 against 94.0 us, 48 sequences)
constexpr int KA_PART = 132;   // floats of a partial result: r, l, two unused, 128 sums
constexpr float KA_CAP = 12.f;   // p_j <= 2^cap where every d <= 8 = 2^(15 - cap)
constexpr float KA_HEAD = 3.f;   // log2 that the maximum may grow before r follows it

struct Kv4AttnArgs {
    const void* q;
    void* out;
    const unsigned char* pool;
    const int* pages;
    const int* n_keys;
    float* part;       // [n_seq][n_kv][splits][group][KA_PART], or null: one block a sequence and KV head
    int n_seq, n_q, group, splits, chunk;  // chunk: 16-key blocks a thread block
    Kv4Shape s;
    int max_pages, max_keys;
    int* err;
};

// (w & m) | o as one instruction: with both constants immediate it would be two.
__device__ __forceinline__ uint32_t ka_and_or(uint32_t w, uint32_t m, uint32_t o)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(m), "r"(o));
    return r;
}
__device__ __forceinline__ uint32_t ka_opaque(uint32_t v)
{
    uint32_t r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Four fp16 pairs c - 8 from a word: pair i has the codes at bits 4 i and 16 + 4 i.
// A code in mantissa bits 0-3 of 1024 is 1024 + c, in bits 4-7 of 64 it is 64 + c.
__device__ __forceinline__ void ka_codes(uint32_t w, uint32_t k1024, uint32_t k64, uint32_t (&p)[4])
{
    const uint32_t w8 = w >> 8;
    const uint32_t a = ka_and_or(w, 0x000F000Fu, k1024), b = ka_and_or(w, 0x00F000F0u, k64);
    const uint32_t c = ka_and_or(w8, 0x000F000Fu, k1024), d = ka_and_or(w8, 0x00F000F0u, k64);
    // -1032 = 0xE408, -72 = 0xD480
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[0]) : "r"(a), "r"(0xE408E408u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[1]) : "r"(b), "r"(0xD480D480u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[2]) : "r"(c), "r"(0xE408E408u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[3]) : "r"(d), "r"(0xD480D480u));
}

// The same pairs without the 8, as fp16 numbers below the normal range: 2^-24 c for
// even pairs, 2^-20 c for odd ones.
__device__ __forceinline__ void ka_small_codes(uint32_t w, uint32_t (&p)[4])
{
    const uint32_t w8 = w >> 8;
    p[0] = w & 0x000F000Fu;
    p[1] = w & 0x00F000F0u;
    p[2] = w8 & 0x000F000Fu;
    p[3] = w8 & 0x00F000F0u;
}

__device__ __forceinline__ void ka_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1, float c0, float c1, float c2, float c3)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// The same from zero, and in place.
__device__ __forceinline__ void ka_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1)
{
    ka_mma(d, a0, a1, a2, a3, b0, b1, 0.f, 0.f, 0.f, 0.f);
}
__device__ __forceinline__ void ka_mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d += m, rounded.
__device__ __forceinline__ void ka_add(float (&d)[4], const float (&m)[4])
{
    const float2 x = un2(add2(f2(d[0], d[1]), f2(m[0], m[1]))), y = un2(add2(f2(d[2], d[3]), f2(m[2], m[3])));
    d[0] = x.x, d[1] = x.y, d[2] = y.x, d[3] = y.y;
}

// A row's result: the product of its first part and, with two, of its second.
template <bool TWO>
__device__ __forceinline__ uint64_t ka_both(const float (&d)[4])
{
    return TWO ? add2(f2(d[0], d[1]), f2(d[2], d[3])) : f2(d[0], d[1]);
}

// x, y as an fp16 pair and, with two parts, what is left of them as another.
template <bool TWO>
__device__ __forceinline__ void ka_split(uint64_t v, uint32_t& hi, uint32_t& lo)
{
    const float2 x = un2(v);
    hi = pack2(x.x, x.y, static_cast<const __half*>(nullptr));
    lo = 0u;
    if (!TWO)
        return;
    const float2 rest = un2(fma2(half2_f2(hi), f2(-1.f, -1.f), v));
    lo = pack2(rest.x, rest.y, static_cast<const __half*>(nullptr));
}

template <typename T>
__global__ void __launch_bounds__(32 * KA_WARPS, KA_RESIDENT) kv4_attn_kernel(const Kv4AttnArgs a)
{
    // two fp16 parts a query and probability, and centred key codes, where the result is
    // fp32; one part, as wide as the result's own mantissa or wider, where it has 16 bits
    constexpr bool TWO = std::is_same<T, float>::value;
    __shared__ __align__(128) unsigned char ring[KA_WARPS][KA_NS][KA_STEP][KV4_BYTES];
    __shared__ uint64_t full[KA_WARPS][KA_NS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = lane >> 2, tq = lane & 3;  // this lane's head of the group, and quarter
    pdl_trigger();
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
    // the warp's i-th cache block is blk0 + KA_STEP (warp + KA_WARPS (i / KA_STEP)) + i % KA_STEP
    const int first = blk0 + KA_STEP * warp;
    auto block_at = [&](int i) { return first + KA_STEP * KA_WARPS * (i / KA_STEP) + i % KA_STEP; };
    const int cnt = first < blk1 ? (blk1 - first + KA_STEP * KA_WARPS - 1) / (KA_STEP * KA_WARPS) : 0;  // stages

    if (lane == 0) {
        for (int i = 0; i < KA_NS; ++i)
            mbar_init(&full[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();

    // ---- lane i has the pool offset of the i-th of the next 32 cache blocks; a bad
    // page's bit is set in `bad` and its copy is page 0's, whose keys are then skipped
    const int bpp = a.s.page_rows / KV4_ROWS;
    const int* pages = a.pages + static_cast<size_t>(b) * a.max_pages;
    auto page_of = [&](int i) {
        const int blk = block_at(i);
        return blk < blk1 ? __ldg(pages + blk / bpp) : 0;
    };
    int next_page = page_of(lane);
    long long off = 0;
    unsigned bad = 0, bad_next = 0;
    auto issue = [&](int i) {  // stage i
        const int at = KA_STEP * i;
        if ((at & 31) == 0) {
            const bool wrong = next_page < 0 || next_page >= a.s.n_pages;
            bad_next = __ballot_sync(0xffffffffu, wrong);
            off = ((static_cast<long long>(wrong ? 0 : next_page) * a.s.n_kv + g) * bpp + block_at(at + lane) % bpp) *
                  KV4_BYTES;
            next_page = page_of(at + 32 + lane);
            if (bad_next && lane == 0)
                set_error(a.err, DEVERR_BAD_ARG);
        }
        const bool two = block_at(at) + 1 < blk1;
        if (lane == 0)
            mbar_arrive_expect_tx(&full[warp][i % KA_NS], two ? 2 * KV4_BYTES : KV4_BYTES);
        __syncwarp();
        const int k = lane - (at & 31);  // the lanes that have the stage's blocks copy them
        if (k == 0 || (k == 1 && two))
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    smem_addr(ring[warp][i % KA_NS][k])),
                "l"(a.pool + off), "r"(KV4_BYTES), "r"(smem_addr(&full[warp][i % KA_NS]))
                : "memory");
    };
    for (int i = 0; i < min(cnt, KA_NS); ++i)
        issue(i);

    // ---- queries: scaled by a power of two a head into fp16's range, in two parts;
    // the sums of a group's queries, for the codes' 8 and for z
    uint32_t qa[8][4];
    float unscale;
    // the two parts of the groups' sums of q as the operand of the z product, and -8 times
    // them for the d product that centres small codes: see below
    uint32_t qz, qd;
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
        // largest |q| into [2^6, 2^7), so that 8 * 32 of them stay below fp16's 2^16: the
        // exponent field moves, nothing is rounded
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 6;
        e = max(-100, min(121, e));
        const float scale = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        // to scores in powers of two; from small codes they come in units of 2^-24.  Queries
        // past the bound on e (2^95, 16-bit ones 2^71) take the bound's unit: two of their scores
        // differ by 2^-48 (2^-72) or more before it, by 2^13 after it, or not at all, and no
        // product with it passes fp32's range
        unscale = __uint_as_float(static_cast<uint32_t>(127 + min(e, TWO ? 88 : 64)) << 23) *
                  ((TWO ? 1.f : 16777216.f) * 0.08838834764831845f * 1.4426950408889634f);
        float qsum[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float sum = 0.f;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float4 w = v[k][m];
                const uint64_t p0 = f2(w.x * scale, w.y * scale), p1 = f2(w.z * scale, w.w * scale);
                ka_split<TWO>(p0, qa[2 * k + m][0], qa[2 * k + m][1]);
                // odd pairs of small codes are 2^-20 c
                ka_split<TWO>(TWO ? p1 : mul2(p1, f2(0.0625f, 0.0625f)), qa[2 * k + m][2], qa[2 * k + m][3]);
                const float2 s0 = un2(p0), s1 = un2(p1);
                sum += (s0.x + s0.y) + (s1.x + s1.y);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            qsum[k] = sum;
        }
        uint32_t h01, l01, h23, l23;
        ka_split<true>(f2(qsum[0], qsum[1]), h01, l01);
        ka_split<true>(f2(qsum[2], qsum[3]), h23, l23);
        qz = tq == 0 ? h01 : tq == 1 ? h23 : tq == 2 ? l01 : l23;
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(qd) : "r"(qz), "r"(0xC800C800u));  // -8
        if (TWO)
            qd = 0u;
    }
    const uint32_t k1024 = ka_opaque(0x64006400u), k64 = ka_opaque(0x54005400u);
    const uint32_t odd = (h & 1) ? 0x7632u : 0x5410u;  // the halves of key h of a pair

    // group k, pair j: dims 32 k + 4 h + 2 j of the group's heads 2 tq and 2 tq + 1, then
    // dims 32 k + 4 h + 2 j + 1 of the same
    float o[4][2][4];
    float zacc[4] = {0.f, 0.f, 0.f, 0.f};  // group h & 3 of heads 2 tq and 2 tq + 1, twice
    uint64_t lacc = 0ull;                  // head h
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[k][i >> 2][i & 3] = 0.f;
    float r = -INFINITY, cap = KA_CAP;
    uint32_t lim = 0x48004800u;  // 2^(15 - cap) as an fp16 pair: 8 at first

    // One cache block, `left` (1 or more) of its keys seen; all of them without TAIL.
    auto block = [&](auto tail, unsigned char* kb, int left) {
        constexpr bool TAIL = decltype(tail)::value;
        if (TAIL && left < KV4_ROWS) {
            // rows past the last key may hold anything: their value scales become zero (their
            // scores are masked below); the warp's last block: nothing is copied over it
            unsigned short* vs = reinterpret_cast<unsigned short*>(kb + KV4_VSCALES + 32 * h + 8 * tq);
            if (2 * h >= left)
                vs[0] = vs[2] = 0;
            if (2 * h + 1 >= left)
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
            // z (and d) of key 8 nt + h, groups 2 (tq & 1) and the next: B's rows 0-3 are the
            // groups' z against the sums' first parts, rows 4-7 against the second parts, rows
            // 8-15 the same with d
            const uint4 zs = lds128(kb + KV4_KSCALES + 32 * (4 * nt + (h >> 1)) + 16 * (tq & 1));
            const uint32_t words[4] = {kw.x, kw.y, kw.z, kw.w}, dd[4] = {sc0.x, sc0.z, sc1.x, sc1.z};
            float m[4];
            ka_mma(m, qz, 0u, qd, 0u, __byte_perm(zs.y, zs.w, odd), TWO ? 0u : __byte_perm(zs.x, zs.z, odd));
            const float u24 = 1.f / 16777216.f;
            uint64_t acc = TWO ? f2(m[0], m[1]) : mul2(f2(m[0], m[1]), f2(u24, u24));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // small codes cost five instructions fewer a word, but their sum with -8 sum q
                // cancels: a relative error of 1.4e-6 where centred ones give 2.9e-7
                uint32_t p[4];
                if (TWO)
                    ka_codes(words[k], k1024, k64, p);
                else
                    ka_small_codes(words[k], p);
                float t[4], t2[4];
                ka_mma(t, qa[2 * k][0], qa[2 * k][1], qa[2 * k][2], qa[2 * k][3], p[0], p[1]);
                ka_mma(t2, qa[2 * k + 1][0], qa[2 * k + 1][1], qa[2 * k + 1][2], qa[2 * k + 1][3], p[2], p[3], t[0], t[1],
                       t[2], t[3]);
                acc = fma2(ka_both<TWO>(t2), half2_f2(dd[k]), acc);
            }
            s[nt] = mul2(acc, f2(unscale, unscale));
        }
        if (TAIL) {
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
        uint32_t vd[2][4];
        __half2 dmax = __half2half2(__ushort_as_half(0));
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const uint4 sc0 = lds128(kb + KV4_VSCALES + 32 * (4 * nt + tq));
            const uint4 sc1 = lds128(kb + KV4_VSCALES + 32 * (4 * nt + tq) + 16);
            vd[nt][0] = sc0.x, vd[nt][1] = sc0.z, vd[nt][2] = sc1.x, vd[nt][3] = sc1.z;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                dmax = __hmax2(dmax, *reinterpret_cast<const __half2*>(&vd[nt][k]));
        }
        const float2 s0 = un2(s[0]), s1 = un2(s[1]);
        const float top = fmaxf(fmaxf(s0.x, s0.y), fmaxf(s1.x, s1.y));
        // d <= lim keeps p d at 2^15 or below under the cap.  A larger one lowers the cap, by no
        // more than it takes: the lower it is, the fewer bits p d has above fp16's smallest
        // number in groups with small scales (d of 1e-3 and the lowest cap: 2^-11 of them)
        const bool wide = !__hble2(dmax, *reinterpret_cast<const __half2*>(&lim));
        if (__any_sync(0xffffffffu, top - r > cap || wide)) {
            float t = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
            if (__any_sync(0xffffffffu, wide)) {
                // the power of two above the largest scale (an infinity counts as the largest)
                const uint32_t d2 = *reinterpret_cast<const uint32_t*>(&dmax);
                const uint32_t e = __reduce_max_sync(0xffffffffu, max(d2 & 0xffffu, d2 >> 16)) >> 10;
                cap = fmaxf(29.f - static_cast<float>(e), -1.f);  // 15 - (e - 15 + 1)
                lim = min(e + 1, 30u) << 10;
                lim = (e >= 30 ? 0x7C00u : lim) * 0x10001u;  // no scale is above an infinity
            }
            float f = 1.f;
            if (t - r > cap) {
                float rn = t - (cap - KA_HEAD);
                rn = t - rn > cap ? t : rn;  // a score of 2^27 and more: rounded past the cap
                f = ex2(r - rn);
                r = rn;
            }
            __syncwarp();
            lacc = mul2(lacc, f2(f, f));
            const float f0 = __shfl_sync(0xffffffffu, f, 8 * tq), f1 = __shfl_sync(0xffffffffu, f, 8 * tq + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                zacc[e] *= e & 1 ? f1 : f0;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    o[k >> 1][k & 1][e] *= e & 1 ? f1 : f0;
            }
        }
        const float2 e0 = un2(add2(s[0], f2(-r, -r)));
        const float2 e1 = un2(add2(s[1], f2(-r, -r)));
        const uint64_t p0 = f2(ex2(e0.x), ex2(e0.y)), p1 = f2(ex2(e1.x), ex2(e1.y));
        lacc = add2(lacc, add2(p0, p1));
        {
            // p z: A's row n is group n & 3 (rows 4-15 are not used)
            uint32_t h0, l0, h1, l1;
            ka_split<TWO>(p0, h0, l0);
            ka_split<TWO>(p1, h1, l1);
            const unsigned char* zs = kb + KV4_VSCALES + 32 * tq + 8 * (h & 3) + 4;
            const uint32_t z0 = lds32(zs), z1 = lds32(zs + 128);
            if (TWO) {
                float m[4], m2[4];
                ka_mma(m, z0, z0, z1, z1, h0, h1);
                ka_mma(m2, z0, z0, z1, z1, l0, l1, m[0], m[1], m[2], m[3]);
                ka_add(zacc, m2);
            } else {
                ka_mma_add(zacc, z0, z0, z1, z1, h0, h1);
            }
        }
        const uint4 va = lds128(kb + KV4_VCODES + 16 * lane), vb = lds128(kb + KV4_VCODES + 512 + 16 * lane);
        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t h0, l0, h1, l1;
            ka_split<TWO>(mul2(p0, half2_f2(vd[0][k])), h0, l0);
            ka_split<TWO>(mul2(p1, half2_f2(vd[1][k])), h1, l1);
            uint32_t b0[4], b1[4];
            ka_codes(wa[k], k1024, k64, b0);
            ka_codes(wb[k], k1024, k64, b1);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // 16 dims (i = 2 j in A's first 8 rows, 2 j + 1 in the others) by 16 keys, times
                // 16 keys by 8 heads.  For fp32 results the sums over blocks are rounded adds:
                // the matrix instruction's own accumulation cuts off (100001 keys: relative error
                // 1.6e-6 with it, 4.1e-7 so)
                if (TWO) {
                    float m[4], m2[4];
                    ka_mma(m, b0[2 * j], b0[2 * j + 1], b1[2 * j], b1[2 * j + 1], h0, h1);
                    ka_mma(m2, b0[2 * j], b0[2 * j + 1], b1[2 * j], b1[2 * j + 1], l0, l1, m[0], m[1], m[2], m[3]);
                    ka_add(o[k][j], m2);
                } else {
                    ka_mma_add(o[k][j], b0[2 * j], b0[2 * j + 1], b1[2 * j], b1[2 * j + 1], h0, h1);
                }
            }
        }
    };

    bool ok = true;
    for (int i = 0; i < cnt; ++i) {
        const int st = i % KA_NS;
        if ((KA_STEP * i & 31) == 0)
            bad = bad_next;  // the copies are ahead, but by less than 32 blocks
        if (!__all_sync(0xffffffffu, mbar_try_wait(&full[warp][st], (i / KA_NS) & 1)) &&
            !__all_sync(0xffffffffu, mbar_wait(&full[warp][st], (i / KA_NS) & 1))) {
            ok = false;
            break;
        }
        const int blk = block_at(KA_STEP * i), left = n - KV4_ROWS * blk;
        if (!bad && left >= KV4_ROWS * KA_STEP && blk + KA_STEP <= blk1) {
#pragma unroll
            for (int k = 0; k < KA_STEP; ++k)
                block(std::false_type{}, ring[warp][st][k], KV4_ROWS);
        } else {
#pragma unroll 1
            for (int k = 0; k < KA_STEP; ++k)
                if (blk + k < blk1 && !(bad >> (KA_STEP * i + k & 31) & 1))
                    block(std::true_type{}, ring[warp][st][k], left - KV4_ROWS * k);
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
        float* mp = meet + warp * 8 * KA_PART;
        if (tq == 0) {
            mp[h * KA_PART] = r;
            mp[h * KA_PART + 1] = l;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float za = __shfl_sync(0xffffffffu, zacc[0], 4 * k + tq), zb = __shfl_sync(0xffffffffu, zacc[1], 4 * k + tq);
            const float(&x)[4] = o[k][0], (&y)[4] = o[k][1];
            float* at = mp + 2 * tq * KA_PART + 4 + 32 * k + 4 * h;
            *reinterpret_cast<float4*>(at) = make_float4(x[0] + za, x[2] + za, y[0] + za, y[2] + za);
            *reinterpret_cast<float4*>(at + KA_PART) = make_float4(x[1] + zb, x[3] + zb, y[1] + zb, y[3] + zb);
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
            const float f = mp[0] == m ? 1.f : ex2(mp[0] - m);
            const float4 y = *reinterpret_cast<const float4*>(mp + 4 + 4 * lane);
            l += f * mp[1];
            v.x += f * y.x;
            v.y += f * y.y;
            v.z += f * y.z;
            v.w += f * y.w;
        }
        if (a.part) {
            float* pp = a.part + (((static_cast<size_t>(b) * a.s.n_kv + g) * a.splits + c) * a.group + hd) * KA_PART;
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

// The splits' results of one sequence and query head, four dims a lane: each warp adds
// up every JOIN-th split with a running maximum, four at a time so that their loads
// are in flight together, then the warps' sums meet.
template <typename T, int JOIN>
__global__ void __launch_bounds__(32 * JOIN) kv4_join_kernel(const Kv4AttnArgs a)
{
    __shared__ float ml[JOIN][2];
    __shared__ float4 sums[JOIN][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / a.n_q, hq = blockIdx.x % a.n_q, g = hq / a.group, h = hq % a.group;
    int n = __ldg(a.n_keys + b);
    if (n < 0 || n > a.max_keys)
        n = 0;
    const int blocks = (n + KV4_ROWS - 1) / KV4_ROWS, splits = (blocks + a.chunk - 1) / a.chunk;
    const float* base = a.part + ((static_cast<size_t>(b) * a.s.n_kv + g) * a.splits * a.group + h) * KA_PART;
    const size_t step = static_cast<size_t>(a.group) * KA_PART;
    pdl_wait();
    float m = -INFINITY, l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = warp; c0 < splits; c0 += 4 * JOIN) {
        float2 rl[4];
        float4 y[4];
        float top = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + JOIN * i;
            rl[i] = make_float2(-INFINITY, 0.f);
            y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < splits) {
                const float* pp = base + c * step;
                rl[i] = __ldcg(reinterpret_cast<const float2*>(pp));
                y[i] = __ldcg(reinterpret_cast<const float4*>(pp + 4) + lane);
            }
            top = fmaxf(top, rl[i].x);
        }
        // equal references (also two of -infinity) have the weight 1
        const float f = m == top ? 1.f : ex2(m - top);
        m = top;
        l *= f;
        v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w = rl[i].x == m ? 1.f : ex2(rl[i].x - m);
            l = fmaf(w, rl[i].y, l);
            v.x = fmaf(w, y[i].x, v.x);
            v.y = fmaf(w, y[i].y, v.y);
            v.z = fmaf(w, y[i].z, v.z);
            v.w = fmaf(w, y[i].w, v.w);
        }
    }
    if (lane == 0) {
        ml[warp][0] = m;
        ml[warp][1] = l;
    }
    sums[warp][lane] = v;
    __syncthreads();
    if (warp)
        return;
    float top = m;
#pragma unroll
    for (int w = 1; w < JOIN; ++w)
        top = fmaxf(top, ml[w][0]);
    l = 0.f;
    v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < JOIN; ++w) {
        const float f = ml[w][0] == top ? 1.f : ex2(ml[w][0] - top);
        const float4 y = sums[w][lane];
        l = fmaf(f, ml[w][1], l);
        v.x = fmaf(f, y.x, v.x);
        v.y = fmaf(f, y.y, v.y);
        v.z = fmaf(f, y.z, v.z);
        v.w = fmaf(f, y.w, v.w);
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

static bool kv4_counts_fit(int n_seq, int n_q, int n_kv, int max_keys)
{
    return n_q / n_kv <= 8 && n_kv <= (1 << 16) && max_keys <= (1 << 30) &&
           static_cast<long long>(n_seq) * n_q <= 0x7fffffffll;
}

// A thread block costs about two microseconds beside its keys, and a split's result
// is written and read back.  So: 16 blocks (256 keys) or fewer are not split (1 x 256
// keys: 5.5 us, 5.9 in two); where sequences and KV heads alone fill the card, splits
// hold 512 keys or more (32 x 500: 10.4 us, 16 with 128 keys); else the work is spread
// over two blocks an SM in splits of 128 to 512 keys (1 x 2000: 6.4 us, 9.8 with 512; 1
// x 16000: 13.1 us with 512, 14.4 with 288), and more than that over the three that are
// resident.  A batch's splits end at 1024 keys, so that sequences of different lengths
// share the card evenly; where its sequences and KV heads fill the card several times
// over, at as many times that, so that blocks and scratch go by max_keys and the card and
// not by the batch as well (256 sequences, 32 heads on 8, a bound of 131072 keys: 1000 keys
// each 332 -> 152 us, one of all 131072 among them 368 -> 182 us, scratch 1.1 GB -> 125 MB).
// The splits under either limit are of one size (100 x 2000 keys: 72 us, 81 with one of 1792
// and one of 208).
static Kv4Split kv4_split(int n_seq, int n_kv, int max_keys)
{
    const long long blocks = (static_cast<long long>(max_keys) + dq::KV4_ROWS - 1) / dq::KV4_ROWS;
    const long long pairs = static_cast<long long>(n_seq) * n_kv, all = blocks * pairs, sms = sm_count();
    if (blocks <= 16)
        return {static_cast<int>(blocks), 1};
    long long chunk = (all + 2 * sms - 1) / (2 * sms);
    if (chunk > 32)
        chunk = std::max((all + dq::KA_RESIDENT * sms - 1) / (dq::KA_RESIDENT * sms), 32ll);
    chunk = std::max(chunk, pairs >= sms ? 32ll : 8ll);
    const long long most = std::max(64ll, 64 * pairs / (dq::KA_RESIDENT * sms));
    if (n_seq > 1 && chunk > most) {
        const long long splits = (blocks + most - 1) / most;
        chunk = (blocks + splits - 1) / splits;
    }
    const long long round = dq::KA_WARPS * dq::KA_STEP;  // what the block's warps take at a time
    chunk = (chunk + round - 1) / round * round;
    return {static_cast<int>(chunk), static_cast<int>((blocks + chunk - 1) / chunk)};
}

}  // namespace dqhost

extern "C" {

DQ_API size_t dq_attention_decode_kv4_workspace_bytes(int n_seq, int n_q, int n_kv, int max_keys)
{
    if (n_seq < 1 || n_q < 1 || n_kv < 1 || n_q % n_kv || max_keys < 1 || !dqhost::kv4_counts_fit(n_seq, n_q, n_kv, max_keys))
        return 0;
    const dqhost::Kv4Split sp = dqhost::kv4_split(n_seq, n_kv, max_keys);
    return sp.splits > 1 ? static_cast<size_t>(n_seq) * n_q * sp.splits * dq::KA_PART * sizeof(float) : 0;
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
    if (!dqhost::kv4_counts_fit(n_seq, n_q, n_kv, max_keys))
        return DQ_ERR_UNSUPPORTED;
    if (!dqhost::aligned16(q) || !dqhost::aligned16(pool) || !dqhost::aligned16(out))
        return DQ_ERR_ALIGN;
    const dqhost::Kv4Split sp = dqhost::kv4_split(n_seq, n_kv, max_keys);
    const long long blocks = static_cast<long long>(n_seq) * n_kv * sp.splits;
    if (blocks > 0x7fffffffll)
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
        cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess || sp.splits == 1)
            return err;
        // a dependent launch: its blocks are there when the last of the first kernel's end
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(n_seq) * n_q);
        // many splits are those of few sequences, whose join has the card to itself (1 x 100001
        // keys: 45.2 -> 43.4 us with 8 warps; 48 x 6000, 12 splits: 88.0 -> 89.4)
        const int join = sp.splits > 16 ? 8 : 4;
        cfg.blockDim = dim3(32 * join);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, join == 8 ? dq::kv4_join_kernel<T, 8> : dq::kv4_join_kernel<T, 4>, a);
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
