// dq_prompt.cu -- causal attention of packed prompts (dq_attention_prompt) on the
// 5th-generation tensor cores.
//
// A block takes two tiles of 128 query rows of one sequence and one KV head.  A
// tile's rows are floor(128 / group) tokens times the `group` query heads that share
// the KV head, so the heads of a group read each key and value tile once.  Per tile
// of 128 keys, for each query tile:
//   S = Q K^T     tcgen05.mma, 128 x 128 fp32 in tensor memory, operands in shared
//                 memory (TMA, 128-byte swizzle);
//   P = 2^(c S - c m + b), c = log2(e) / sqrt(128), by four warps, one row a thread,
//                 with the row's running maximum m and sum l in fp32 registers; P goes
//                 back into tensor memory over S as 16-bit pairs;
//   O += P V      tcgen05.mma, P from tensor memory, V N-major from shared memory,
//                 128 x 128 fp32 in tensor memory.
// While the tensor cores work on one query tile, the other tile's warps do their
// exponentials.  m follows the true maximum only when that has grown by more than
// 2^8 (then l and O are scaled): the ratio P / l does not depend on which m and b are
// used and every sum is fp32, and the scaling of O, which would wait for the last
// product, is rare after the first tiles.  b is 7 in fp16, so that P fills its range up
// to 2^15 and a key is lost only below 2^-32 of the largest probability (with b = 0,
// 2^-25: 16000 keys of that size beside one key of value zero were gone); 0 in bf16.
//
// The running maximum and sum are M. Milakov and N. Gimelshein's online softmax (2018); the
// order of the work, tiles that take turns with a reference that moves rarely, follows what
// T. Dao, J. Shah and others have published on attention in one pass.
//
// 8192 tokens, 32 heads on 8 KV heads, fp16: 381 us, 1445 TFLOP/s (0.76 of the
// measured bf16 rate; 0.84 of the rate that the power limit leaves a library product
// over seconds, and the limit holds here too: 1.8 of 2.07 GHz at 1300 W; alone, from a
// rested card, 350 us); 350 GB/s of DRAM.  The products bound it, not the softmax: with
// P = S in place of the exponentials 382 of 385 us were left.  A round (both query tiles
// against one key tile, 32 products of 64 clocks: 1.02 us at 2 GHz) takes 1.22 us with no
// softmax at all and 1.31 whole: a product of 64 clocks reads 8 KB of shared memory for
// S and 4 KB for P V, and a round's copies write 64 KB; 256 KB are the 128 bytes a clock
// that shared memory has for as long as the products take.  A block's start and end (5
// us) come on top: a batch of twelve ragged prompts, 1432 blocks of 6 rounds on average,
// 142 us, 880 TFLOP/s; short prompts are nothing else: 256 of 40 tokens 121 us (bytes: 31),
// 1000 of 8 tokens 427 us (24).  Tried and not kept: blocks that fetch more work and copy the
// next tile during the end of one (ragged batch 158 us), one query tile a block and two
// blocks an SM (8192 tokens 419 us, ragged batch 147; 256 prompts of 40 tokens 121 ->
// 105, 1000 of 8 tokens 427 -> 257), two product warps taking turns (398 us), a product
// loop unrolled over the ring's slots (449 us), P handed over in quarters (16% more).
//
// Where the query tiles are too few for the card, the keys of each are split over
// several blocks and joined by a second kernel (64 queries over 16064 keys: 286 -> 26
// us; the keys' 66 MB take 10).  Above half the card's blocks nothing is split, and the
// last wave may be nearly empty: 1280 queries after 16000 keys are 160 equal blocks on 152
// SMs, 352 us (184 of products), 2048 queries 377 us (302).
//
// Key tiles that hold masked keys for some row (the diagonal's and a sequence's end)
// have their infinities and NaNs in V replaced by zero before the product, since a
// probability of 0 would not stop them; where such a key is seen by some row, the
// epilogue adds the values themselves to the rows that see them.
#include <algorithm>
#include <mutex>

#include "dq_tc.cuh"
#include "dq_tma_host.h"
#include "dq_types.cuh"

namespace dq {

constexpr int PR_HD = 128;
constexpr int PR_KEYS = 128;                  // keys a tile
constexpr int PR_STAGES = 5;                  // ring of key and value tiles, in turn
constexpr int PR_TILE = PR_KEYS * PR_HD * 2;  // bytes of a key, value or query tile
constexpr int PR_PANEL = PR_TILE / 2;         // 64 dims of it
// warps 0-7 softmax, then one that issues the products (of both query tiles: two warps
// let the tiles fall into step, products and exponentials in turn: 397 -> 505 us), one
// that copies and two that clean value tiles
constexpr int PR_MMA_WARP = 8, PR_TMA_WARP = 9, PR_CLEAN_WARP = 10;
constexpr int PR_CLEAN_BAR = 1;  // named barrier of the copying and the cleaning warps
constexpr int PR_THREADS = 384;
constexpr int PR_MAX_SPLITS = 64;
// A block's rows end within 256 keys of one another: at most this many key tiles
// are seen by some rows in part.
constexpr int PR_CLEAN = 3;
// registers a thread: 384 x 168 at the launch, moved to the softmax warps
constexpr int PR_SOFTMAX_REGS = 208, PR_OTHER_REGS = 88;
static_assert(256 * PR_SOFTMAX_REGS + 128 * PR_OTHER_REGS <= PR_THREADS * 168, "no more than the launch has");
constexpr int PR_SMEM = (2 + PR_STAGES) * PR_TILE + 1024 /* alignment */ + 512;
constexpr uint32_t PR_S0 = 0, PR_O0 = 256, PR_TCOLS = 512;  // tensor memory columns: S0 S1 O0 O1
constexpr float PR_C = 0.08838834764831845f * 1.4426950408889634f;
constexpr float PR_GROW = 8.0f;  // log2 of the growth of the maximum that is let pass
// c s - c m in one fused step has the rounding of c m in it, the same for a whole row until m
// moves: 2^-12 at this size of m, 2^13 at the largest that fp16 can give.  Past it m is
// subtracted from s first.
constexpr float PR_FAR = 32768.0f;
// b of a type: P <= 2^(b + PR_GROW)
template <typename T>
constexpr float PR_TOP = std::is_same<T, __nv_bfloat16>::value ? 0.f : 7.f;

struct PromptArgs {
    CUtensorMap tq, tk, tv;
    const void* v;
    void* out;
    long long v_row, v_head, o_row, o_head;
    const int* cu_q;
    const int* cu_k;
    int n_seq, total_q, total_k, n_kv, group, tq_tokens;  // tokens a query tile
    // the keys of a block tile shared by `splits` blocks: their unscaled outputs, by block
    // tile, KV head, split and query tile [32][128 rows][4], and maxima and sums [2][128]
    float* part;
    float* part_ml;
    int splits;
    FastDiv by_splits, by_kv, by_group, by_span;  // span: tokens a block tile
    int* err;
};

// One block's share: query tokens [t0, ...) of a sequence, its rows and keys.
struct PromptTile {
    int q0, k0, lq, lk, t0, live;
};

// Block tile `idx`, counted from the last sequence's last tile (a causal sequence's
// later tiles see more keys: they start first).  By one warp, four sequences a lane, so
// that the offsets of 128 are one wait for memory (256 sequences of 40 tokens: 162 us with
// two passes of 32 at a time, 121 us); `span` tokens a block.
__device__ __forceinline__ PromptTile prompt_find(const PromptArgs& a, int idx, int span, int lane)
{
    int q0 = 0, k0 = 0, rows = 0, keys = 0, t0 = 0, live = 0;
    int want = idx;  // tiles from the end of sequence s1 - 1
    for (int s1 = a.n_seq; s1 > 0 && (!live || idx == 0); s1 -= 128) {
        // sequences s1 - 1 - 4 lane - e; those below 0 have no rows
        int cq[5], ck[5];
#pragma unroll
        for (int e = 0; e < 5; ++e) {
            const int i = max(s1 - 4 * lane - e, 0);
            cq[e] = __ldg(a.cu_q + i);
            ck[e] = __ldg(a.cu_k + i);
        }
        int lq[4], n[4], sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // offsets that do not ascend within their totals: the first block reports them
            const bool ok = cq[e + 1] >= 0 && cq[e + 1] <= cq[e] && cq[e] <= a.total_q && ck[e + 1] >= 0 &&
                            ck[e + 1] <= ck[e] && ck[e] <= a.total_k;
            if (!ok && idx == 0)
                set_error(a.err, DEVERR_BAD_ARG);
            lq[e] = ok ? cq[e] - cq[e + 1] : 0;
            n[e] = fast_div(lq[e] + span - 1, a.by_span);
            sum += n[e];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += x;
        }
        int mine = want - (incl - sum);
        const unsigned hit = __ballot_sync(0xffffffffu, mine >= 0 && mine < sum);
        if (hit && !live) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool it = mine >= 0 && mine < n[e];
                q0 = it ? cq[e + 1] : q0;
                k0 = it ? ck[e + 1] : k0;
                rows = it ? lq[e] : rows;
                keys = it ? ck[e] - ck[e + 1] : keys;
                t0 = it ? (n[e] - 1 - mine) * span : t0;
                mine -= n[e];
            }
            const int src = __ffs(hit) - 1;
            q0 = __shfl_sync(0xffffffffu, q0, src);
            k0 = __shfl_sync(0xffffffffu, k0, src);
            rows = __shfl_sync(0xffffffffu, rows, src);
            keys = __shfl_sync(0xffffffffu, keys, src);
            t0 = __shfl_sync(0xffffffffu, t0, src);
            live = 1;
        }
        want -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return PromptTile{q0, k0, rows, keys, t0, live};
}

// Key tiles of each of a block's two query tiles, its tokens, and the keys that all of
// the block's rows see.
struct PromptSpan {
    int ntok[2], end[2], open;
};

__device__ __forceinline__ PromptSpan prompt_span(const PromptTile& tile, int tokens)
{
    PromptSpan p;
    p.open = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int ts = tile.t0 + t * tokens;
        p.ntok[t] = max(0, min(tokens, tile.lq - ts));
        const int hi = min(tile.lk, max(0, ts + p.ntok[t] + tile.lk - tile.lq));
        p.end[t] = p.ntok[t] ? (hi + PR_KEYS - 1) / PR_KEYS : 0;
        if (p.ntok[t])
            p.open = min(p.open, min(tile.lk, max(0, ts + 1 + tile.lk - tile.lq)));
    }
    return p;
}

// Key tiles [j0, j1) of split c.
__device__ __forceinline__ void prompt_split(const PromptSpan& p, int splits, int c, int& j0, int& j1)
{
    const int all = max(p.end[0], p.end[1]), per = splits == 1 ? all : (all + splits - 1) / splits;
    j0 = min(all, c * per);
    j1 = min(all, j0 + per);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Bits 15 and 31 set where the low and the high 16-bit value is an infinity or NaN.
template <typename T>
__device__ __forceinline__ uint32_t non_finite2(uint32_t w)
{
    constexpr bool half = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t mask = half ? 0x7C007C00u : 0x7F807F80u, one = half ? 0x04000400u : 0x00800080u;
    return ((w & mask) + one) & 0x80008000u;
}

template <typename T>
__device__ __forceinline__ float one16(uint32_t bits)
{
    if (std::is_same<T, __nv_bfloat16>::value)
        return bf16lo(bits);
    return half_bits_to_float(bits);
}

// The rest of a wait whose first poll found nothing.
__device__ __forceinline__ void prompt_wait_on(uint64_t* bar, uint32_t parity, volatile int* fail, int* err, int code)
{
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait_sleep(bar, parity, 20000u)) {
        if (*fail)
            return;
        if (globaltimer_ns() - t0 > WAIT_LIMIT_NS) {
            *fail = 1;
            set_error(err, code);
            return;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(PR_THREADS, 1) prompt_kernel(const __grid_constant__ PromptArgs a)
{
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    uint8_t* qs = sm;                    // two query tiles
    uint8_t* ring = sm + 2 * PR_TILE;    // PR_STAGES key and value tiles
    uint64_t* q_full = reinterpret_cast<uint64_t*>(ring + PR_STAGES * PR_TILE);  // [2]
    uint64_t* full = q_full + 2;             // [PR_STAGES] a ring tile landed
    uint64_t* freed = full + PR_STAGES;      // [PR_STAGES] its products are done
    // value tiles with masked keys, each with barriers of its own, used once: the ring's
    // phases go on without the warps that clean them
    uint64_t* v_full = freed + PR_STAGES;    // [PR_CLEAN] landed
    uint64_t* cleaned = v_full + PR_CLEAN;   // [PR_CLEAN] infinities and NaNs are out
    uint64_t* s_full = cleaned + PR_CLEAN;   // [2] S of a query tile written
    uint64_t* p_full = s_full + 2;           // [2][2] a half of P's keys written
    uint64_t* o_full = p_full + 4;           // [2] a product P V done
    uint64_t* drain = o_full + 2;
    PromptTile* shared_tile = reinterpret_cast<PromptTile*>(drain + 1);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(shared_tile + 1);
    volatile int* fail = reinterpret_cast<volatile int*>(tslot + 1);
    volatile int* poison = fail + 1;  // a seen value is an infinity or NaN

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int part = fast_div(blockIdx.x, a.by_splits), c = blockIdx.x - part * a.splits;
    const int idx = fast_div(part, a.by_kv), g = part - idx * a.n_kv;
    PromptTile tile{0, 0, 0, 0, 0, 0};
    PromptSpan sp;
    // this block's key tiles j0 + j, j < n, and j < end0 or end1 for query tile 0 or 1
    int j0 = 0, j1 = 0, n = 0, end0 = 0, end1 = 0;
    int jclean = 0;  // the first of them with a masked key for some row, may be below 0
    auto set_span = [&] {
        sp = prompt_span(tile, a.tq_tokens);
        prompt_split(sp, a.splits, c, j0, j1);
        n = j1 - j0;
        end0 = max(0, min(sp.end[0], j1) - j0);
        end1 = max(0, min(sp.end[1], j1) - j0);
        jclean = sp.open / PR_KEYS - j0;
    };
    // one copy of the ring: key tile 0, value tile 0, key tile 1, ...
    auto load_tile = [&](int i) {
        const int s = i % PR_STAGES, j = i >> 1;
        const bool clean = (i & 1) && j >= jclean;
        uint64_t* bar = clean ? &v_full[j - jclean] : &full[s];
        mbar_arrive_expect_tx(bar, PR_TILE);
        for (int p = 0; p < 2; ++p)
            tma_load_3d(ring + s * PR_TILE + p * PR_PANEL, (i & 1) ? &a.tv : &a.tk, 64 * p, tile.k0 + (j0 + j) * PR_KEYS,
                        g, bar);
        if (clean)
            mbar_arrive(&full[s]);  // the slot's phase goes on
    };
    pdl_trigger();
    if (warp == PR_TMA_WARP) {
        // the copying warp finds the block's tile and starts its copies while the others
        // are set up
        tile = prompt_find(a, idx, 2 * a.tq_tokens, lane);
        set_span();
        if (lane == 0) {
            *shared_tile = tile;
            for (int i = 0; i < 2; ++i) {
                mbar_init(&q_full[i], 1);
                mbar_init(&s_full[i], 1);
                mbar_init(&p_full[2 * i], 4);
                mbar_init(&p_full[2 * i + 1], 4);
                mbar_init(&o_full[i], 1);
            }
            for (int i = 0; i < PR_STAGES; ++i) {
                mbar_init(&full[i], 1);
                mbar_init(&freed[i], 1);
            }
            for (int i = 0; i < PR_CLEAN; ++i) {
                mbar_init(&v_full[i], 1);
                mbar_init(&cleaned[i], 2);
            }
            mbar_init(drain, 1);
            fence_mbar_init();
            *fail = 0;
            *poison = 0;
            for (int t = 0; t < 2; ++t) {
                if (!(t ? end1 : end0))
                    continue;
                mbar_arrive_expect_tx(&q_full[t], static_cast<uint32_t>(2 * a.tq_tokens * a.group * 128));
                for (int p = 0; p < 2; ++p)
                    tma_load_3d(qs + t * PR_TILE + p * PR_PANEL, &a.tq, 64 * p, g * a.group,
                                tile.q0 + tile.t0 + t * a.tq_tokens, &q_full[t]);
                if (t == 0 && n > 0)
                    load_tile(0);
            }
            for (int i = end0 ? 1 : 0; i < min(2 * n, PR_STAGES); ++i)
                load_tile(i);
        }
        __syncwarp();
    } else if (warp == PR_MMA_WARP) {
        tmem_alloc(tslot, PR_TCOLS);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp != PR_TMA_WARP) {
        tile = *shared_tile;
        set_span();
    }
    const uint32_t tbase = *tslot;

    // Bounded waits.  Once one has run out the block has given up: the others return at
    // once, every role runs to its end over whatever is there, and nothing is written.
    auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
        if (!mbar_try_wait(bar, parity))
            prompt_wait_on(bar, parity, fail, a.err, code);
    };

    if (tile.live && warp < PR_MMA_WARP) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PR_SOFTMAX_REGS));
        // ---- softmax and epilogue: warps 4 t .. 4 t + 3, thread r of them owns row r
        const int t = warp >> 2, r = tid & 127, end = t ? end1 : end0;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t ts = tbase + lanes + PR_S0 + 128 * t, to = tbase + lanes + PR_O0 + 128 * t;
        const int row_tok = fast_div(r, a.by_group);
        const int tok = tile.t0 + t * a.tq_tokens + row_tok;  // within the sequence
        const bool mine = row_tok < sp.ntok[t];
        const int lim = min(tile.lk, max(0, tok + 1 + tile.lk - tile.lq));  // keys this row sees
        float m = -INFINITY, l = 0.f, base = 0.f;
        bool far = false;  // |m| > PR_FAR for some row of the warp
        for (int j = 0; j < end; ++j) {
            wait(&s_full[t], j & 1, DEVERR_TIMEOUT_FULL);
            __syncwarp();
            tc_fence_after_sync();
            uint32_t s[128];
            // the maximum of the first half while the second is on its way
            float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            const int left = lim - (j0 + j) * PR_KEYS;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (q == 0) {
                    tmem_ld32(ts, s);
                    tmem_ld32(ts + 32, s + 32);
                }
                tmem_ld_wait();
                if (q == 0) {
                    tmem_ld32(ts + 64, s + 64);
                    tmem_ld32(ts + 96, s + 96);
                }
                if (j >= jclean) {
                    // a warp's rows end within 32 keys of one another: most runs of 16 are seen by
                    // all of them
#pragma unroll
                    for (int i0 = 64 * q; i0 < 64 * q + 64; i0 += 16)
                        if (__any_sync(0xffffffffu, left < i0 + 16)) {
#pragma unroll
                            for (int i = i0; i < i0 + 16; ++i)
                                if (i >= left)
                                    s[i] = 0xff800000u;  // -infinity
                        }
                }
#pragma unroll
                for (int i = 64 * q; i < 64 * q + 64; ++i)
                    top4[i & 3] = fmaxf(top4[i & 3], __uint_as_float(s[i]));
            }
            const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
            const bool grow = (top - m) * PR_C > PR_GROW;
            if (__any_sync(0xffffffffu, grow || far)) {
                const float mn = grow ? top : m;
                const float alpha = grow ? ex2((m - mn) * PR_C) : 1.0f;  // 0 from -infinity
                m = mn;
                l *= alpha;
                // a row's own m alone decides: its result is the same whatever the other rows hold
                const float ref = m == -INFINITY ? 0.f : m, off = fabsf(ref) > PR_FAR ? ref : 0.f;
                far = __any_sync(0xffffffffu, off != 0.f);
                base = fmaf(off - ref, PR_C, PR_TOP<T>);
                if (far) {
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        s[i] = __float_as_uint(__uint_as_float(s[i]) - off);
                }
                if (j > 0 && __any_sync(0xffffffffu, grow)) {
                    wait(&o_full[t], (j - 1) & 1, DEVERR_TIMEOUT_FULL);
                    __syncwarp();
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t o[32];
                        tmem_ld32(to + 32 * q, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(to + 32 * q, o);
                    }
                }
            }
            const uint64_t c2 = f2(PR_C, PR_C), b2 = f2(base, base);
            uint64_t sum0 = 0ull, sum1 = 0ull;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 x = un2(fma2(f2(__uint_as_float(s[64 * q + 2 * i]), __uint_as_float(s[64 * q + 2 * i + 1])),
                                              c2, b2));
                    const float y0 = ex2(x.x), y1 = ex2(x.y);
                    if (i & 1)
                        sum1 = add2(sum1, f2(y0, y1));
                    else
                        sum0 = add2(sum0, f2(y0, y1));
                    p[i] = pack2(y0, y1, static_cast<const T*>(nullptr));
                }
                // each half of the keys is multiplied while the next exponentials run
                tmem_st32(ts + 32 * q, p);
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[2 * t + q]);
            }
            const float2 sum = un2(add2(sum0, sum1));
            l += sum.x + sum.y;
        }
        if (end)
            wait(&o_full[t], (end - 1) & 1, DEVERR_TIMEOUT_FULL);
        const bool ok = __all_sync(0xffffffffu, !*fail);
        tc_fence_after_sync();
        const bool bad = *poison;
        if (ok && bad && end) {
            // the seen infinities and NaNs of V, which the products left out, added to the rows'
            // outputs (before these are scaled, which changes neither)
#pragma unroll 1
            for (int c32 = 0; c32 < 4; ++c32) {
                uint32_t o[32];
                tmem_ld32(to + 32 * c32, o);
                tmem_ld_wait();
                const int last = mine ? min(lim, j1 * PR_KEYS) : 0;
                for (int j = max(j0, j0 + jclean) * PR_KEYS; j < last; ++j) {
                    const uint4* vp = reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) +
                                                                     static_cast<long long>(tile.k0 + j) * a.v_row +
                                                                     static_cast<long long>(g) * a.v_head + 32 * c32);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 w = vp[i];
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t nf = non_finite2<T>(u[e]);
                            float& lo = reinterpret_cast<float&>(o[8 * i + 2 * e]);
                            float& hi = reinterpret_cast<float&>(o[8 * i + 2 * e + 1]);
                            if (nf & 0x8000u)
                                lo += one16<T>(u[e] & 0xffffu);
                            if (nf & 0x80000000u)
                                hi += one16<T>(u[e] >> 16);
                        }
                    }
                }
                __syncwarp();
                tmem_st32(to + 32 * c32, o);
            }
            tmem_st_wait();
        }
        if (ok && a.splits > 1) {
            if (end) {
                const size_t at = ((static_cast<size_t>(idx) * a.n_kv + g) * a.splits + c) * 2 + t;
                a.part_ml[at * 256 + r] = m;
                a.part_ml[at * 256 + 128 + r] = l;
                float4* po = reinterpret_cast<float4*>(a.part) + at * 32 * 128 + r;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t o[32];
                    tmem_ld32(to + 32 * q, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        po[(8 * q + i) * 128] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                            __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                }
            }
        } else if (ok && sp.ntok[t]) {
            // a row that sees no key is zero, one whose scores are all -infinity NaN (0 / 0)
            const float inv = lim > 0 ? 1.0f / l : 0.f;
            // The rows leave through the query tile's shared memory (its products are done), each
            // warp its own 32, 16-byte pieces in an order that spreads them over the banks: a
            // store then writes two whole rows and not 16 bytes of 32 (4-6 thousand clocks of a
            // block's end).
            uint8_t* stage = qs + t * PR_TILE + (r & ~31) * 256;
            uint32_t o[128];
            if (end) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(to + 32 * c, o + 32 * c);
                tmem_ld_wait();
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = __uint_as_float(o[8 * i + 2 * e]) * inv, y = __uint_as_float(o[8 * i + 2 * e + 1]) * inv;
                    w[e] = lim > 0 ? pack2(x, y, static_cast<const T*>(nullptr)) : 0u;
                }
                *reinterpret_cast<uint4*>(stage + lane * 256 + 16 * (i ^ (lane & 15))) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            const uint64_t at = mine ? reinterpret_cast<uint64_t>(
                                           static_cast<T*>(a.out) + static_cast<long long>(tile.q0 + tok) * a.o_row +
                                           static_cast<long long>(g * a.group + r - row_tok * a.group) * a.o_head)
                                     : 0ull;
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                const int row = 2 * i + (lane >> 4);
                const uint64_t to_row = __shfl_sync(0xffffffffu, at, row);
                const uint4 w = *reinterpret_cast<const uint4*>(stage + row * 256 + 16 * ((lane & 15) ^ (row & 15)));
                if (to_row)
                    *reinterpret_cast<uint4*>(to_row + 16 * (lane & 15)) = w;
            }
        }
    } else if (tile.live) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PR_OTHER_REGS));
        const int first_clean = 2 * max(0, jclean) + 1;  // the copy of the first value tile to be cleaned
        if (warp == PR_TMA_WARP) {
            int i = min(2 * n, PR_STAGES);
            bool called = first_clean >= 2 * n;  // the cleaning warps sleep until their first tile is on its way
            for (; i < 2 * n; ++i) {
                if (!called && first_clean < i) {
                    called = true;
                    named_bar_arrive(PR_CLEAN_BAR, 96);
                }
                wait(&freed[i % PR_STAGES], ((i / PR_STAGES) & 1) ^ 1, DEVERR_TIMEOUT_EMPTY);
                __syncwarp();
                if (__any_sync(0xffffffffu, *fail))
                    break;
                if (lane == 0)
                    load_tile(i);
            }
            if (!called)
                named_bar_arrive(PR_CLEAN_BAR, 96);
            // every copy has landed before the block ends
            if (lane == 0) {
                bool landed = true;
                for (int k = max(0, i - PR_STAGES); k < i; ++k)
                    landed = mbar_wait(&full[k % PR_STAGES], (k / PR_STAGES) & 1) && landed;
                for (int k = 0; k < PR_CLEAN && first_clean + 2 * k < i; ++k)
                    landed = mbar_wait(&v_full[max(0, -jclean) + k], 0) && landed;
                for (int t = 0; t < 2; ++t)
                    landed = (!(t ? end1 : end0) || mbar_wait(&q_full[t], 0)) && landed;
                if (!landed)
                    set_error(a.err, DEVERR_TIMEOUT_DRAIN);
            }
            __syncwarp();
        } else if (warp == PR_MMA_WARP) {
            if (n > 0) {
                constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
                constexpr uint32_t id_qk = umma_idesc_16bit(128, PR_KEYS, bf, false);
                constexpr uint32_t id_pv = umma_idesc_16bit(128, PR_HD, bf, true);
                const uint64_t qd0 = umma_desc_sw128(smem_addr(qs), 16, 1024);
                const uint64_t kd0 = umma_desc_sw128(smem_addr(ring), 16, 1024);
                const uint64_t vd0 = umma_desc_sw128(smem_addr(ring), PR_PANEL, 1024);
                // S_t = Q_t K^T: eight steps of 16 dims, four a panel
                auto qk = [&](int t, int slot) {
                    const uint64_t ad = qd0 + static_cast<uint64_t>(t * (PR_TILE >> 4));
                    const uint64_t bd = kd0 + static_cast<uint64_t>(slot * (PR_TILE >> 4));
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint64_t step = ((s >> 2) * PR_PANEL + (s & 3) * 32) >> 4;
                        umma_f16_warp(tbase + PR_S0 + 128 * t, ad + step, bd + step, id_qk, s > 0);
                    }
                    umma_commit_warp(&s_full[t]);
                };
                // O_t += P_t V: eight steps of 16 keys, four for each half of P
                auto pv = [&](int t, int slot, int half, bool first) {
                    const uint64_t bd = vd0 + static_cast<uint64_t>(slot * (PR_TILE >> 4));
#pragma unroll
                    for (int s = 4 * half; s < 4 * half + 4; ++s)
                        umma_f16_ta_warp(tbase + PR_O0 + 128 * t, tbase + PR_S0 + 128 * t + 8 * s,
                                         bd + static_cast<uint64_t>((s * 2048) >> 4), id_pv, !first || s > 0);
                };
                wait(&full[0], 0, DEVERR_TIMEOUT_FULL);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if ((t ? end1 : end0) > 0) {
                        wait(&q_full[t], 0, DEVERR_TIMEOUT_FULL);
                        qk(t, 0);
                    }
                umma_commit_warp(&freed[0]);
                // ring slots of value tile j and key tile j + 1, and their phases
                int sv = 1, sk = 2;
                uint32_t vphase = 0, kphase = 0;
                for (int j = 0; j < n; ++j) {
                    if (j >= jclean)
                        wait(&cleaned[j - jclean], 0, DEVERR_TIMEOUT_FULL);
                    else
                        wait(&full[sv], vphase, DEVERR_TIMEOUT_FULL);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (j >= (t ? end1 : end0))
                            continue;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            wait(&p_full[2 * t + half], j & 1, DEVERR_TIMEOUT_FULL);
                            tc_fence_after_sync();
                            pv(t, sv, half, j == 0);
                        }
                        umma_commit_warp(&o_full[t]);
                        if (j + 1 < (t ? end1 : end0)) {
                            if (t == 0 || end0 <= j + 1)
                                wait(&full[sk], kphase, DEVERR_TIMEOUT_FULL);
                            qk(t, sk);
                        }
                    }
                    umma_commit_warp(&freed[sv]);
                    if (j + 1 < n)
                        umma_commit_warp(&freed[sk]);
                    if ((sv += 2) >= PR_STAGES) {
                        sv -= PR_STAGES;
                        vphase ^= 1;
                    }
                    if ((sk += 2) >= PR_STAGES) {
                        sk -= PR_STAGES;
                        kphase ^= 1;
                    }
                }
                umma_commit_warp(drain);  // every product is done before the block ends
                if (!mbar_wait(drain, 0) && lane == 0)
                    set_error(a.err, DEVERR_TIMEOUT_DRAIN);
            }
            __syncwarp();
        } else if (first_clean < 2 * n) {
            named_bar_sync(PR_CLEAN_BAR, 96);
            // infinities and NaNs of the value tiles with masked keys become zero
            for (int j = max(0, jclean); j < n; ++j) {
                wait(&v_full[j - jclean], 0, DEVERR_TIMEOUT_FULL);
                uint8_t* vt = ring + (2 * j + 1) % PR_STAGES * PR_TILE;
                bool seen = false;
#pragma unroll 8
                for (int i = tid - 32 * PR_CLEAN_WARP; i < PR_TILE / 16; i += 64) {
                    uint4 w = *reinterpret_cast<const uint4*>(vt + 16 * i);
                    const uint32_t nx = non_finite2<T>(w.x), ny = non_finite2<T>(w.y), nz = non_finite2<T>(w.z),
                                   nw = non_finite2<T>(w.w);
                    if (nx | ny | nz | nw) {
                        // 0x8000 -> 0xffff per half: the halves to clear
                        w.x &= ~((nx >> 15) * 0xffffu);
                        w.y &= ~((ny >> 15) * 0xffffu);
                        w.z &= ~((nz >> 15) * 0xffffu);
                        w.w &= ~((nw >> 15) * 0xffffu);
                        *reinterpret_cast<uint4*>(vt + 16 * i) = w;
                        seen |= (j0 + j) * PR_KEYS + (i & 1023) / 8 < tile.lk;  // a panel's rows are 8 of these
                    }
                }
                if (seen)
                    *poison = 1;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&cleaned[j - jclean]);
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == PR_MMA_WARP)
        tmem_dealloc(tbase, PR_TCOLS);
}

// The splits of one block tile, KV head and query tile: a thread takes one row, 8 of its
// dims and every PR_JOIN-th split, then the threads of a row meet in shared memory.  A
// thread's maxima and sums are loaded together and then its outputs (two waits for
// memory in all, up to PR_BATCH splits at a time).
constexpr int PR_JOIN = 4, PR_BATCH = 8;

template <typename T>
__global__ void __launch_bounds__(128 * PR_JOIN) prompt_join_kernel(const __grid_constant__ PromptArgs a)
{
    __shared__ PromptTile shared_tile;
    __shared__ float2 meet_ml[PR_JOIN - 1][128];
    __shared__ float4 meet_o[PR_JOIN - 1][2][128];
    const int r = threadIdx.x & 127, part = threadIdx.x >> 7, q = blockIdx.y & 15, t = blockIdx.y >> 4;
    const int idx = fast_div(blockIdx.x, a.by_kv), g = blockIdx.x - idx * a.n_kv;
    if (threadIdx.x < 32) {
        const PromptTile x = prompt_find(a, idx, 2 * a.tq_tokens, threadIdx.x);
        if (threadIdx.x == 0)
            shared_tile = x;
    }
    __syncthreads();
    const PromptTile tile = shared_tile;
    const PromptSpan sp = prompt_span(tile, a.tq_tokens);
    const int row_tok = fast_div(r, a.by_group), tok = tile.t0 + t * a.tq_tokens + row_tok;
    const bool mine = tile.live && row_tok < sp.ntok[t];
    const size_t first = (static_cast<size_t>(idx) * a.n_kv + g) * a.splits;
    // the splits that have keys for this query tile are the first ones
    int j0, per;
    prompt_split(sp, a.splits, 0, j0, per);
    const int n = mine && per > 0 ? min(a.splits, (sp.end[t] + per - 1) / per) : 0;
    const float* ml = a.part_ml + (first * 2 + t) * 256 + r;
    const float4* po = reinterpret_cast<const float4*>(a.part) + (first * 2 + t) * 32 * 128 + 2 * q * 128 + r;
    pdl_wait();
    float m = -INFINITY, l = 0.f;
    float4 o[2] = {};
    for (int c0 = part; c0 < n; c0 += PR_JOIN * PR_BATCH) {
        float mc[PR_BATCH], lc[PR_BATCH], top = m;
        float4 x[PR_BATCH][2];
#pragma unroll
        for (int i = 0; i < PR_BATCH; ++i) {
            const int c = c0 + PR_JOIN * i;
            mc[i] = c < n ? __ldcg(ml + c * 512) : -INFINITY;
            lc[i] = c < n ? __ldcg(ml + c * 512 + 128) : 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x[i][h] = c < n ? __ldcg(po + static_cast<size_t>(c) * 2 * 32 * 128 + h * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < PR_BATCH; ++i)
            top = fmaxf(top, mc[i]);
        const float base = top == -INFINITY ? 0.f : top;
        const float f = ex2((m - base) * PR_C);
        m = top;
        l *= f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            o[h] = make_float4(o[h].x * f, o[h].y * f, o[h].z * f, o[h].w * f);
#pragma unroll
        for (int i = 0; i < PR_BATCH; ++i) {
            const float w = ex2((mc[i] - base) * PR_C);
            l = fmaf(w, lc[i], l);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                o[h].x = fmaf(w, x[i][h].x, o[h].x);
                o[h].y = fmaf(w, x[i][h].y, o[h].y);
                o[h].z = fmaf(w, x[i][h].z, o[h].z);
                o[h].w = fmaf(w, x[i][h].w, o[h].w);
            }
        }
    }
    if (part) {
        meet_ml[part - 1][r] = make_float2(m, l);
        meet_o[part - 1][0][r] = o[0];
        meet_o[part - 1][1][r] = o[1];
    }
    __syncthreads();
    if (part || !mine)
        return;
    float top = m;
#pragma unroll
    for (int i = 0; i < PR_JOIN - 1; ++i)
        top = fmaxf(top, meet_ml[i][r].x);
    const float base = top == -INFINITY ? 0.f : top, f = ex2((m - base) * PR_C);
    l *= f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        o[h] = make_float4(o[h].x * f, o[h].y * f, o[h].z * f, o[h].w * f);
#pragma unroll
    for (int i = 0; i < PR_JOIN - 1; ++i) {
        const float2 y = meet_ml[i][r];
        const float w = ex2((y.x - base) * PR_C);
        l = fmaf(w, y.y, l);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 x = meet_o[i][h][r];
            o[h].x = fmaf(w, x.x, o[h].x);
            o[h].y = fmaf(w, x.y, o[h].y);
            o[h].z = fmaf(w, x.z, o[h].z);
            o[h].w = fmaf(w, x.w, o[h].w);
        }
    }
    const bool sees = tok + 1 + tile.lk - tile.lq > 0 && tile.lk > 0;
    const float inv = sees ? 1.0f / l : 0.f;
    T* out = static_cast<T*>(a.out) + static_cast<long long>(tile.q0 + tok) * a.o_row +
             static_cast<long long>(g * a.group + r - row_tok * a.group) * a.o_head + 8 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        store4(out + 4 * h, sees ? make_float4(o[h].x * inv, o[h].y * inv, o[h].z * inv, o[h].w * inv)
                                 : make_float4(0.f, 0.f, 0.f, 0.f));
}

}  // namespace dq

namespace dqhost {

// How a call is cut into blocks: block tiles (at most, over all sequences) and the
// splits of each one's keys.
struct PromptCut {
    long long tiles;
    int splits;
};

static PromptCut prompt_cut(int n_seq, int total_q, int total_k, int n_q, int n_kv)
{
    const long long span = 2 * (128 / (n_q / n_kv)), seqs = std::min(n_seq, total_q);
    const long long tiles = (total_q - seqs) / span + seqs;
    const long long keys = (static_cast<long long>(total_k) + seqs * dq::PR_KEYS - 1) / (seqs * dq::PR_KEYS);
    // too few blocks for the card: the keys are split, into two key tiles at least
    const long long splits = std::min({sm_count() / (tiles * n_kv), keys / 2, static_cast<long long>(dq::PR_MAX_SPLITS)});
    return {tiles, static_cast<int>(std::max(1ll, splits))};
}

static size_t prompt_part_floats(const PromptCut& cut, int n_kv)
{
    return static_cast<size_t>(cut.tiles) * n_kv * cut.splits * 2 * 128;
}

// A 16-bit tensor [outer][middle][128] with the given strides (elements), copied in
// boxes of 64 dims with the 128-byte swizzle.
static bool prompt_map(EncodeTiled enc, CUtensorMap* m, int type, const void* p, int middle, long long middle_stride,
                       int outer, long long outer_stride, int box_middle, int box_outer)
{
    const cuuint64_t dims[3] = {dq::PR_HD, static_cast<cuuint64_t>(middle), static_cast<cuuint64_t>(outer)};
    // a stride of a dimension of one is never used, but has to be one that the encoder takes
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(middle > 1 ? middle_stride : dq::PR_HD) * 2,
                                   static_cast<cuuint64_t>(outer > 1 ? outer_stride : dq::PR_HD) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_middle), static_cast<cuuint32_t>(box_outer)};
    const cuuint32_t ones[3] = {1, 1, 1};
    return enc(m, type == DQ_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernel's shared memory, asked for once per device.
template <typename T>
static cudaError_t prompt_prepare()
{
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(dq::prompt_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, dq::PR_SMEM);
        if (e == cudaSuccess && dev >= 0 && dev < 64)
            done[dev] = true;
    }
    return e;
}

template <typename T>
static cudaError_t prompt_launch(const dq::PromptArgs& a, unsigned grid, const PromptCut& cut, cudaStream_t s)
{
    cudaError_t e = prompt_prepare<T>();
    if (e != cudaSuccess)
        return e;
    dq::prompt_kernel<T><<<grid, dq::PR_THREADS, dq::PR_SMEM, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess || cut.splits == 1)
        return e;
    // a dependent launch: it finds its tiles while the last blocks run
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cut.tiles * a.n_kv), 32);
    cfg.blockDim = dim3(128 * dq::PR_JOIN);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dq::prompt_join_kernel<T>, a);
}

}  // namespace dqhost

extern "C" {

DQ_API size_t dq_attention_prompt_workspace_bytes(int n_seq, int total_q, int total_k, int n_q, int n_kv)
{
    if (n_seq < 1 || total_q < 1 || total_k < 1 || n_q < 1 || n_kv < 1 || n_q % n_kv || n_q / n_kv > 128)
        return 0;
    const dqhost::PromptCut cut = dqhost::prompt_cut(n_seq, total_q, total_k, n_q, n_kv);
    return cut.splits > 1 ? dqhost::prompt_part_floats(cut, n_kv) * (dq::PR_HD + 2) * sizeof(float) : 0;
}

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
        if (((kv ? p->total_k : p->total_q) > 1 && rows[i] < dq::PR_HD) ||
            ((kv ? p->n_kv : p->n_q) > 1 && heads[i] < dq::PR_HD))
            return DQ_ERR_SHAPE;
    }
    if (p->head_dim != dq::PR_HD || p->n_q / p->n_kv > 128 || p->total_q > (1 << 30) || p->total_k > (1 << 30))
        return DQ_ERR_UNSUPPORTED;
    for (int i = 0; i < 4; ++i) {
        if (rows[i] % 8 || heads[i] % 8)
            return DQ_ERR_ALIGN;
        if (rows[i] >= (1ll << 38) || heads[i] >= (1ll << 38))  // the tensor maps' strides are below 2^40 bytes
            return DQ_ERR_UNSUPPORTED;
    }
    if (!dqhost::aligned16(p->q) || !dqhost::aligned16(p->k) || !dqhost::aligned16(p->v) || !dqhost::aligned16(p->out))
        return DQ_ERR_ALIGN;
    const int group = p->n_q / p->n_kv, tokens = 128 / group;
    const dqhost::PromptCut cut = dqhost::prompt_cut(p->n_seq, p->total_q, p->total_k, p->n_q, p->n_kv);
    const long long blocks = cut.tiles * p->n_kv * cut.splits;
    if (blocks > 0x7fffffffll)
        return DQ_ERR_UNSUPPORTED;
    if (cut.splits > 1) {
        if (!p->workspace)
            return DQ_ERR_NULL;
        if (p->workspace_bytes < dqhost::prompt_part_floats(cut, p->n_kv) * (dq::PR_HD + 2) * sizeof(float))
            return DQ_ERR_SHAPE;
        if (!dqhost::aligned16(p->workspace))
            return DQ_ERR_ALIGN;
    }
    dqhost::EncodeTiled enc = dqhost::encode_tiled();
    if (!enc)
        return DQ_ERR_UNSUPPORTED;
    dq::PromptArgs a{};
    if (!dqhost::prompt_map(enc, &a.tq, p->type, p->q, p->n_q, heads[0], p->total_q, rows[0], group, tokens) ||
        !dqhost::prompt_map(enc, &a.tk, p->type, p->k, p->total_k, rows[1], p->n_kv, heads[1], dq::PR_KEYS, 1) ||
        !dqhost::prompt_map(enc, &a.tv, p->type, p->v, p->total_k, rows[2], p->n_kv, heads[2], dq::PR_KEYS, 1))
        return DQ_ERR_UNSUPPORTED;
    a.v = p->v;
    a.out = p->out;
    a.v_row = rows[2];
    a.v_head = heads[2];
    a.o_row = rows[3];
    a.o_head = heads[3];
    a.cu_q = p->cu_q;
    a.cu_k = p->cu_k ? p->cu_k : p->cu_q;
    a.n_seq = p->n_seq;
    a.total_q = p->total_q;
    a.total_k = p->total_k;
    a.n_kv = p->n_kv;
    a.group = group;
    a.tq_tokens = tokens;
    a.splits = cut.splits;
    a.by_splits = dqhost::fast_divisor(cut.splits);
    a.by_kv = dqhost::fast_divisor(p->n_kv);
    a.by_group = dqhost::fast_divisor(group);
    a.by_span = dqhost::fast_divisor(2 * tokens);
    if (cut.splits > 1) {
        a.part = static_cast<float*>(p->workspace);
        a.part_ml = a.part + dqhost::prompt_part_floats(cut, p->n_kv) * dq::PR_HD;
    }
    a.err = dqhost::device_error_flag();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = static_cast<unsigned>(blocks);
    cudaError_t e = p->type == DQ_TYPE_F16 ? dqhost::prompt_launch<__half>(a, grid, cut, s)
                                           : dqhost::prompt_launch<__nv_bfloat16>(a, grid, cut, s);
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
