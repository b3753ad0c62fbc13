// dq_tree_tc.cu -- tree attention of many rows a KV head on the 5th-generation tensor
// cores.
//
// An item is one or two tiles of 128 query rows (as many whole tokens as fit, times the
// heads that share a KV head) of one sequence and KV head; blocks take equal stretches of
// all items' key tiles (dq_tree.cuh) and keep going from one item to the next.  Per tile of
// 128 keys, as in the prompt attention: S = Q K^T into tensor memory, P = 2^(c S - c m + b)
// by four warps, a row a thread, back over S in 16 bits, O += P V in tensor memory.  Two
// such chains t = 0, 1 run side by side, so that the products of one meet the exponentials
// of the other: with two query tiles (PAIR) a chain each, on the same keys; with one, the
// even and the odd key tiles, whose sums meet at the end of a segment.  A tile of 128 keys is
// 64 KB, 2900 clocks of a SM's share of the memory's rate; its products take 1024 clocks for
// one query tile, 2048 for two: the memory bounds both while the ring has enough on its way.
//
// One sequence of 16 tokens after 100001 keys, 410 MB: 73 us (floor 61: 4 us until the first
// scores, 3 for partial sums, 4 for their join); 32 sequences of up to 8 after up to 12000, 769
// MB: 137 us (115); 8 of 64 after up to 16000, 371 MB, 92 GFLOP: 86 us (56), DRAM 58% and
// matrix pipe 47% busy.  Beside starts and ends, each segment costs two query tiles a drain
// of the chains and 2.4 us to hand over partial sums (128 KB a block).  Tried and not kept:
// keys and values asked into L2 four tiles ahead (8 of 64: 93 -> 107 us), the next item's
// tiles copied before its queries (32 sequences 136 -> 138 us), ring tiles of one query tile in
// the order K0 V0 K1 V1 (84 us for the first case, 78 in the order of their use).
#include <mutex>

#include "dq_tc.cuh"
#include "dq_tree.cuh"

namespace dq {

constexpr int TT_KEYS = dqhost::TREE_TC_KEYS;
constexpr int TT_TILE = TT_KEYS * ATT_HD * 2;  // bytes of a tile of queries, keys or values
constexpr int TT_PANEL = TT_TILE / 2;          // 64 dims of it
// warps 0-3 and 4-7 softmax of chain 0 and 1, one that issues the products, one that copies,
// two that clean value tiles
constexpr int TT_MMA_WARP = 8, TT_TMA_WARP = 9, TT_CLEAN_WARP = 10, TT_THREADS = 384;
constexpr int TT_SOFTMAX_REGS = 208, TT_OTHER_REGS = 88;
static_assert(256 * TT_SOFTMAX_REGS + 128 * TT_OTHER_REGS <= TT_THREADS * 168, "no more than the launch has");
constexpr uint32_t TT_S0 = 0, TT_O0 = 256, TT_TCOLS = 512;  // tensor memory columns: S0 S1 O0 O1
// past this size of m it is subtracted from the scores before the product with c, whose
// rounding would otherwise show (the same bound as the prompt attention's)
constexpr float TT_FAR = 32768.0f;
constexpr int TT_MEET_BAR = 1;  // named barrier of the softmax warps

template <bool PAIR>
constexpr int TT_SLOTS = PAIR ? 5 : 6;  // ring of key and value tiles in turn, beside the query tiles
constexpr int TT_RING = 7 * TT_TILE;    // either way

using Cursor = TreeCursor<0, TT_KEYS>;  // items of whole tokens

struct TreeMiscT {
    uint64_t q_full, q_free;             // the segment's queries landed; its last S is done
    uint64_t full[6], freed[6];          // a ring tile landed; its products are done
    // value tiles with new tokens' keys land on barriers of their own, whose phases are those
    // tiles alone: the ring's go on without the warps that clean them
    uint64_t v_full[6], cleaned[6];
    uint64_t s_full[2], p_full[2][2], o_full[2];
    uint64_t drain;
    uint32_t absent[8];                  // of a key tile, by its number: runs of 16 keys whose page is outside the pool
    float ml[2][128][2];
    Cursor parked[8];  // the softmax warps' cursors while registers are short
    Cursor start;
    uint32_t tmem;
    int fail, poison;                    // poison: a new token's value is an infinity or NaN
};
constexpr int TT_SMEM = TT_RING + static_cast<int>(sizeof(TreeMiscT));
static_assert(TT_SMEM <= 232448, "a block's shared memory");

// Bits 32 w .. 32 w + 31 of the keys a row sees: those below `off` are past ones, bit off +
// t is that of new token t.
__device__ __forceinline__ uint32_t tree_word(uint64_t seen, int off, int w)
{
    const int sh = 32 * w - off;
    if (sh >= 64)
        return 0u;
    if (sh >= 0)
        return static_cast<uint32_t>(seen >> sh);
    if (sh <= -32)
        return 0xffffffffu;
    return static_cast<uint32_t>(seen << -sh) | ((1u << -sh) - 1);
}

// A place in the ring, and the parity of the phase that fills it.
template <int NS>
struct TreePlace {
    int s;
    uint32_t phase;
    __device__ __forceinline__ TreePlace after(int copies) const
    {
        const int at = s + copies;
        return TreePlace{at % NS, phase ^ (at / NS & 1)};
    }
};

// The order in which a segment of n tiles goes through the ring is the order of its use.
// PAIR: K0 V0 K1 V1 ...; one query tile, whose two chains have two tiles' scores under way:
// K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1).
template <bool PAIR>
__device__ __forceinline__ int tree_values_at(int j, int n)
{
    return PAIR ? 2 * j + 1 : min(2 * j + 2, 2 * n - 1);
}

template <typename T, bool PAIR>
__global__ void __launch_bounds__(TT_THREADS, 1) tree_tc_kernel(const __grid_constant__ TreeArgs a)
{
    constexpr int NS = TT_SLOTS<PAIR>, QT = PAIR ? 2 : 1, R = 128 * QT;
    constexpr float TOP = std::is_same<T, __half>::value ? 7.f : 0.f;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t* ring = sm + QT * TT_TILE;
    TreeMiscT& sh = *reinterpret_cast<TreeMiscT*>(sm + TT_RING);
    volatile int* fail = &sh.fail;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tokens = a.nodes / QT;  // a query tile
    if (warp == TT_TMA_WARP) {
        if (lane == 0) {
            mbar_init(&sh.q_full, 1);
            mbar_init(&sh.q_free, 1);
            for (int i = 0; i < NS; ++i) {
                mbar_init(&sh.full[i], 1);
                mbar_init(&sh.freed[i], 1);
                mbar_init(&sh.v_full[i], 1);
                mbar_init(&sh.cleaned[i], 2);
            }
            for (int t = 0; t < 2; ++t) {
                mbar_init(&sh.s_full[t], 1);
                mbar_init(&sh.p_full[t][0], 4);
                mbar_init(&sh.p_full[t][1], 4);
                mbar_init(&sh.o_full[t], 1);
            }
            mbar_init(&sh.drain, 1);
            fence_mbar_init();
            sh.fail = sh.poison = 0;
            tree_fetch_map(&a.map);
            tree_fetch_map(&a.tq);
        }
        pdl_wait();
        const Cursor first = tree_start<0, TT_KEYS>(a, lane);
        if (lane == 0)
            sh.start = first;
        __syncwarp();
    } else if (warp == TT_MMA_WARP) {
        tmem_alloc(&sh.tmem, TT_TCOLS);
    }
    pdl_wait();
    pdl_trigger();  // only now: the join reads lengths before this kernel ends
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const bool some = sh.start.left > 0;
    const uint32_t tbase = sh.tmem;
    TreeShared join{0, 0, 0, 0, -1};

    auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
        if (!mbar_try_wait(bar, parity))
            tree_wait_on(bar, parity, fail, a.err, code);
    };
    if (some && warp < TT_MMA_WARP) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TT_SOFTMAX_REGS));
        // ---- softmax and epilogue: thread r of chain t has row r of its query tile
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t ts = tbase + lanes + TT_S0 + 128 * t, to = tbase + lanes + TT_O0;
        const int token = static_cast<int>(fast_div(r, a.by_group)), head = r - token * a.group;
        uint32_t before = 0, mine = 0;  // key tiles of earlier segments, and of this chain so far
        for (Cursor c = sh.start; c.left > 0; c.next(a)) {
            if (lane == 0)
                sh.parked[warp] = c;
            const int n = c.end() - c.tile;
            int node = c.rt * a.nodes + (PAIR ? t * tokens : 0) + token;
            bool live = token < tokens && node < c.t.rows;
            int row = c.t.row0 + node;
            uint64_t seen = !live || c.t.keys == 0 ? 0ull : a.seen ? __ldcg(a.seen + row) : (2ull << node) - 1;
            if (c.t.rows < 64)
                seen &= (1ull << c.t.rows) - 1;
            const bool any = __any_sync(0xffffffffu, live);
            // of the segment's first tile: a new token's key in a tile, and the first tile with one
            const int past = c.t.past - c.tile * TT_KEYS, from_new = c.t.keys ? c.t.past / TT_KEYS - c.tile : -0x7fffffff;
            float m = -INFINITY, l = 0.f, base = 0.f;
            bool far = false;  // |m| > TT_FAR for some row of the warp
            for (int j = PAIR ? 0 : t; j < n; j += PAIR ? 1 : 2, ++mine) {
                const uint32_t parity = mine & 1;
                wait(&sh.s_full[t], parity, DEVERR_TIMEOUT_FULL);
                __syncwarp();
                tc_fence_after_sync();
                if (!any) {  // no row of this warp exists
                    if (lane == 0) {
                        mbar_arrive(&sh.p_full[t][0]);
                        mbar_arrive(&sh.p_full[t][1]);
                    }
                    continue;
                }
                const uint32_t absent = sh.absent[(before + j) & 7];
                const bool tail = j >= from_new || absent;
                uint32_t s[128];
                // the maximum of the first half while the second is on its way
                float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
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
                    if (tail) {
#pragma unroll
                        for (int w = 2 * q; w < 2 * q + 2; ++w) {
                            uint32_t word = from_new > -0x7fffffff ? tree_word(seen, past - j * TT_KEYS, w) : 0u;
                            if (absent >> (2 * w) & 1)
                                word &= 0xffff0000u;
                            if (absent >> (2 * w + 1) & 1)
                                word &= 0x0000ffffu;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(word >> i & 1))
                                    s[32 * w + i] = 0xff800000u;  // -infinity
                        }
                    }
#pragma unroll
                    for (int i = 64 * q; i < 64 * q + 64; ++i)
                        top4[i & 3] = fmaxf(top4[i & 3], __uint_as_float(s[i]));
                }
                const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                const bool grow = (top - m) * TR_C > TR_GROW;
                if (__any_sync(0xffffffffu, grow || far)) {
                    const float mn = grow ? top : m;
                    const float alpha = grow ? ex2((m - mn) * TR_C) : 1.0f;  // 0 from -infinity
                    m = mn;
                    l *= alpha;
                    // a row's own m alone decides: its result is the same whatever the other rows hold
                    const float ref = m == -INFINITY ? 0.f : m, off = fabsf(ref) > TT_FAR ? ref : 0.f;
                    far = __any_sync(0xffffffffu, off != 0.f);
                    base = fmaf(off - ref, TR_C, TOP);
                    if (far) {
#pragma unroll
                        for (int i = 0; i < 128; ++i)
                            s[i] = __float_as_uint(__uint_as_float(s[i]) - off);
                    }
                    if (j > (PAIR ? 0 : 1) && __any_sync(0xffffffffu, grow)) {
                        wait(&sh.o_full[t], parity ^ 1, DEVERR_TIMEOUT_FULL);
                        __syncwarp();
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            uint32_t o[32];
                            tmem_ld32(to + 128 * t + 32 * q, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st32(to + 128 * t + 32 * q, o);
                        }
                    }
                }
                const uint64_t c2 = f2(TR_C, TR_C), b2 = f2(base, base);
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
                        mbar_arrive(&sh.p_full[t][q]);
                }
                const float2 sum = un2(add2(sum0, sum1));
                l += sum.x + sum.y;
            }

            // ---- the segment's end
            __syncwarp();
            c = sh.parked[warp];
            const int g = c.g, rt = c.rt, end = c.tile + n;
            node = rt * a.nodes + (PAIR ? t * tokens : 0) + token;
            live = token < tokens && node < c.t.rows;
            row = c.t.row0 + node;
            if (n > (PAIR ? 0 : t))
                wait(&sh.o_full[t], (mine - 1) & 1, DEVERR_TIMEOUT_FULL);
            __syncwarp();
            float f0 = 1.f, f1 = 1.f;  // of the two chains' sums
            if (!PAIR) {
                sh.ml[t][r][0] = m;
                sh.ml[t][r][1] = l;
                named_bar_sync(TT_MEET_BAR, 256);
                const float m0 = sh.ml[0][r][0], l0 = sh.ml[0][r][1], m1 = sh.ml[1][r][0], l1 = sh.ml[1][r][1];
                m = fmaxf(m0, m1);
                f0 = m0 == m ? 1.f : ex2((m0 - m) * TR_C);
                f1 = m1 == m ? 1.f : ex2((m1 - m) * TR_C);
                l = l0 * f0 + l1 * f1;
            }
            tc_fence_after_sync();
            const bool whole = c.tile == 0 && end == c.tiles, ok = __all_sync(0xffffffffu, !*fail), bad = sh.poison;
            if (!whole && c.tile == 0)
                join = TreeShared{c.t.row0, c.t.rows, g, rt,
                                static_cast<int>(blockIdx.x) + (c.tiles - end + sh.start.left - 1) / sh.start.left};
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t at = static_cast<size_t>(blockIdx.x) * 2 + (c.tile == 0);
            const int rr = (PAIR ? 128 * t : 0) + r;
            if (!whole && live && ok && (PAIR || t == 0))
                a.part_ml[at * R + rr] = make_float2(m, l);
            if (any) {
                // the rows that this lane helps to write: those of its four, below
                uint64_t to_row[4];
                {
                    const uint64_t mine_at = live && ok ? reinterpret_cast<uint64_t>(static_cast<T*>(a.out) + static_cast<long long>(row) * a.o_row +
                                                                                     static_cast<long long>(g * a.group + head) * a.o_head)
                                                        : 0ull;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        to_row[i] = __shfl_sync(0xffffffffu, mine_at, (lane & ~3) + i);
                }
#pragma unroll 1
                for (int q = PAIR ? 0 : 2 * t; q < (PAIR ? 4 : 2 * t + 2); ++q) {
                    float o[32];
                    {
                        uint32_t x[32];
                        {
                            tmem_ld32(to + (PAIR ? 128 * t : 0) + 32 * q, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = PAIR ? __uint_as_float(x[i]) : __uint_as_float(x[i]) * f0;
                        }
                        if (!PAIR && n > 1) {
                            tmem_ld32(to + 128 + 32 * q, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = fmaf(__uint_as_float(x[i]), f1, o[i]);
                        }
                    }
                    if (bad) {
                        // new tokens' infinities and NaNs, which the products left out, to the rows that see them
                        const int last = min(c.t.keys, end * TT_KEYS);
                        for (int key = max(c.t.past, c.tile * TT_KEYS); key < last; ++key) {
                            const int page = __ldcg(a.pages + static_cast<size_t>(c.s) * a.max_pages + key / a.s.page_rows);
                            if (page < 0 || page >= a.s.n_pages || !(seen >> (key - c.t.past) & 1))
                                continue;
                            const uint4* vp = reinterpret_cast<const uint4*>(
                                static_cast<const T*>(a.pool) +
                                (kv16_row(a.s, page, 1, g) + key % a.s.page_rows) * ATT_HD + 32 * q);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint4 w = vp[i];
                                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t nf = tree_non_finite<T>(u[e]);
                                    if (nf & 0xffffu)
                                        o[8 * i + 2 * e] += tree_one<T>(u[e] & 0xffffu);
                                    if (nf >> 16)
                                        o[8 * i + 2 * e + 1] += tree_one<T>(u[e] >> 16);
                                }
                            }
                        }
                        __syncwarp();
                    }
                    if (whole) {
                        // 64 bytes of each row, in pieces of 16: four lanes trade theirs so that each has
                        // one piece of four rows and a store fills whole sectors (a piece a lane and row
                        // took four times the store's cycles)
                        uint32_t w[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[i][e] = l == 0.f ? 0u : pack2(o[8 * i + 2 * e] * inv, o[8 * i + 2 * e + 1] * inv, static_cast<const T*>(nullptr));
#pragma unroll
                        for (int d = 1; d < 4; d *= 2)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (i & d)
                                    continue;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & d ? w[i][e] : w[i + d][e], d);
                                    if (lane & d)
                                        w[i][e] = got;
                                    else
                                        w[i + d][e] = got;
                                }
                            }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (to_row[i])
                                *reinterpret_cast<uint4*>(to_row[i] + 64 * q + 16 * (lane & 3)) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
                    } else if (live && ok) {
                        float4* part = a.part + (at * 32 + 8 * q) * R + rr;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            part[i * R] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
            }
            tc_fence_before_sync();
            if (!PAIR)
                named_bar_sync(TT_MEET_BAR, 256);  // both chains' sums and numbers are read
            before += n;
        }
    } else if (some) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TT_OTHER_REGS));
        if (warp == TT_TMA_WARP) {
            // ---- copies: a lane takes one panel of one of a tile's boxes of rows
            const int box = a.box, boxes = TT_KEYS / box, ahead = 32 / boxes;
            const int u = lane & (boxes - 1), panel = lane / boxes;
            int slot = 0;
            uint32_t phase = 0, number = 0, segment = 0, v_phase = 0, v_used = 0;  // v_: a bit a slot
            long long issued = 0;
            for (Cursor c = sh.start; c.left > 0 && !__any_sync(0xffffffffu, *fail);
                 c.next(a), ++segment) {
                const int g = c.g, rt = c.rt;
                const int* pages = a.pages + static_cast<size_t>(c.s) * a.max_pages;
                // lane i has the page of box `first + i`, and of box `first + 32 + i`
                auto page_of = [&](int x) {
                    return static_cast<long long>(x) * box < c.t.keys ? __ldcg(pages + fast_div(x, a.by_boxes)) : 0;
                };
                const int from_new = c.t.keys ? c.t.past / TT_KEYS : 0;
                int first = c.tile, now = page_of(first * boxes + lane), then = page_of((first + ahead) * boxes + lane);
                wait(&sh.q_free, (segment & 1) ^ 1, DEVERR_TIMEOUT_EMPTY);
                __syncwarp();
                if (__any_sync(0xffffffffu, *fail))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.q_full, static_cast<uint32_t>(QT * 2 * tokens * a.group * 128));
                    for (int q = 0; q < QT; ++q)
                        for (int p = 0; p < 2; ++p)
                            tree_load(sm + q * TT_TILE + p * TT_PANEL, &a.tq, 64 * p, g * a.group,
                                      c.t.row0 + rt * a.nodes + q * tokens, &sh.q_full);
                }
                __syncwarp();
                // one tile of keys (kv = 0) or values; y: the lane's row of the pool, below 0 without one
                auto copy = [&](int kv, int k, int y, uint32_t bytes, uint32_t absent) {
                    wait(&sh.freed[slot], phase ^ 1, DEVERR_TIMEOUT_EMPTY);
                    __syncwarp();
                    if (__any_sync(0xffffffffu, *fail))
                        return;
                    uint8_t* to = ring + slot * TT_TILE;
                    if (absent && kv) {  // their probabilities are zero, so their values have to be finite
                        for (int i = lane; i < TT_TILE / 16; i += 32)
                            if (absent >> ((i & 1023) / 8 / 16) & 1)
                                *reinterpret_cast<uint4*>(to + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    const bool clean = kv && k >= from_new;
                    uint64_t* bar = clean ? &sh.v_full[slot] : &sh.full[slot];
                    if (lane == 0) {
                        if (kv == 0)
                            sh.absent[number & 7] = absent;
                        mbar_arrive_expect_tx(bar, bytes);
                        if (clean)
                            mbar_arrive(&sh.full[slot]);  // the slot's phase goes on
                    }
                    if (clean) {
                        v_phase ^= 1u << slot;
                        v_used |= 1u << slot;
                    }
                    __syncwarp();
                    if (y >= 0)
                        tree_load(to + panel * TT_PANEL + u * box * 128, &a.map, 0, y, panel, bar);
                    ++issued;
                    if (++slot == NS) {
                        slot = 0;
                        phase ^= 1;
                    }
                };
                const int end = c.end(), to_values = a.s.n_kv * a.s.page_rows;
                int y = -1, y_last = -1;
                uint32_t bytes = 0, absent = 0, bytes_last = 0, absent_last = 0;
                for (int k = c.tile; k < end; ++k, ++number) {
                    if (k - first == ahead) {
                        first = k;
                        now = then;
                        then = page_of((first + ahead) * boxes + lane);
                    }
                    const int page = __shfl_sync(0xffffffffu, now, ((k - first) * boxes + u) & 31);
                    const int x = k * boxes + u;
                    const bool mine = panel < 2 && static_cast<long long>(x) * box < c.t.keys;
                    const bool there = mine && page >= 0 && page < a.s.n_pages;
                    const unsigned have = __ballot_sync(0xffffffffu, there);
                    const unsigned lack = __ballot_sync(0xffffffffu, mine && !there && panel == 0);
                    absent = 0;
                    if (lack) {
                        for (int i = 0; i < boxes; ++i)
                            if (lack >> i & 1)
                                absent |= ((1u << (box / 16)) - 1) << (i * (box / 16));
                        if (lane == 0)
                            set_error(a.err, DEVERR_BAD_ARG);
                    }
                    bytes = static_cast<uint32_t>(__popc(have) * box * 128);
                    y = there ? static_cast<int>(kv16_row(a.s, page, 0, g)) +
                                    (x - static_cast<int>(fast_div(x, a.by_boxes) * a.by_boxes.d)) * box
                              : -1;
                    copy(0, k, y, bytes, absent);
                    if (PAIR)
                        copy(1, k, y < 0 ? y : y + to_values, bytes, absent);
                    else if (k > c.tile)
                        copy(1, k - 1, y_last < 0 ? y_last : y_last + to_values, bytes_last, absent_last);
                    y_last = y;
                    bytes_last = bytes;
                    absent_last = absent;
                }
                if (!PAIR)
                    copy(1, end - 1, y_last < 0 ? y_last : y_last + to_values, bytes_last, absent_last);
            }
            // every copy has landed before the block ends
            bool landed = true;
            for (long long i = max(0ll, issued - NS); i < issued; ++i)
                landed = mbar_wait(&sh.full[i % NS], static_cast<uint32_t>(i / NS) & 1) && landed;
            for (int i = 0; i < NS; ++i)
                if (v_used >> i & 1)
                    landed = mbar_wait(&sh.v_full[i], (v_phase >> i & 1) ^ 1) && landed;
            if (issued)  // of the last segment whose queries were asked for
                landed = mbar_wait(&sh.q_full, (segment & 1) ^ 1) && landed;
            if (!landed && lane == 0)
                set_error(a.err, DEVERR_TIMEOUT_DRAIN);
            __syncwarp();
        } else if (warp == TT_MMA_WARP) {
            constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
            constexpr uint32_t id_qk = umma_idesc_16bit(128, TT_KEYS, bf, false);
            constexpr uint32_t id_pv = umma_idesc_16bit(128, ATT_HD, bf, true);
            const uint64_t qd0 = umma_desc_sw128(smem_addr(sm), 16, 1024);
            const uint64_t kd0 = umma_desc_sw128(smem_addr(ring), 16, 1024);
            const uint64_t vd0 = umma_desc_sw128(smem_addr(ring), TT_PANEL, 1024);
            // S_t = Q K^T: eight steps of 16 dims, four a panel
            auto qk = [&](int t, int slot) {
                const uint64_t ad = qd0 + static_cast<uint64_t>((PAIR ? t : 0) * (TT_TILE >> 4));
                const uint64_t bd = kd0 + static_cast<uint64_t>(slot * (TT_TILE >> 4));
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint64_t step = ((s >> 2) * TT_PANEL + (s & 3) * 32) >> 4;
                    umma_f16_warp(tbase + TT_S0 + 128 * t, ad + step, bd + step, id_qk, s > 0);
                }
                umma_commit_warp(&sh.s_full[t]);
            };
            // O_t += P_t V: eight steps of 16 keys, four for each half of P
            auto pv = [&](int t, int slot, uint32_t parity, bool first) {
                const uint64_t bd = vd0 + static_cast<uint64_t>(slot * (TT_TILE >> 4));
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    wait(&sh.p_full[t][half], parity, DEVERR_TIMEOUT_FULL);
                    __syncwarp();
                    tc_fence_after_sync();
#pragma unroll
                    for (int s = 4 * half; s < 4 * half + 4; ++s)
                        umma_f16_ta_warp(tbase + TT_O0 + 128 * t, tbase + TT_S0 + 128 * t + 8 * s,
                                         bd + static_cast<uint64_t>((s * 2048) >> 4), id_pv, !first || s > 0);
                }
                umma_commit_warp(&sh.o_full[t]);
            };
            TreePlace<NS> at{0, 0};  // of the next tile in the ring
            uint32_t count0 = 0, count1 = 0, segment = 0, clean_phase = 0;  // tiles of the chains so far
            for (Cursor c = sh.start; c.left > 0; c.next(a), ++segment) {
                const int n = c.end() - c.tile, from_new = c.t.keys ? c.t.past / TT_KEYS : 0;
                auto landed = [&](const TreePlace<NS>& x) {
                    wait(&sh.full[x.s], x.phase, DEVERR_TIMEOUT_FULL);
                    __syncwarp();
                };
                wait(&sh.q_full, segment & 1, DEVERR_TIMEOUT_FULL);
                __syncwarp();
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!PAIR && t >= n)
                        continue;
                    if (!PAIR || t == 0)
                        landed(at);
                    qk(t, at.s);
                    if (!PAIR || t == 1) {
                        umma_commit_warp(&sh.freed[at.s]);
                        at = at.after(1);
                    }
                }
                if (n <= (PAIR ? 1 : 2))
                    umma_commit_warp(&sh.q_free);
                for (int j = 0; j < n; ++j) {
                    const TreePlace<NS> keys = at.after(1);  // the ones that come after these values
                    if (c.tile + j >= from_new) {
                        wait(&sh.cleaned[at.s], clean_phase >> at.s & 1, DEVERR_TIMEOUT_FULL);
                        clean_phase ^= 1u << at.s;
                        __syncwarp();
                    } else {
                        landed(at);
                    }
                    if (PAIR) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            pv(t, at.s, (count0 + j) & 1, j == 0);
                            if (j + 1 < n) {
                                if (t == 0)
                                    landed(keys);
                                qk(t, keys.s);
                            }
                        }
                        umma_commit_warp(&sh.freed[at.s]);
                        if (j + 1 < n)
                            umma_commit_warp(&sh.freed[keys.s]);
                        if (j + 2 == n)
                            umma_commit_warp(&sh.q_free);
                        at = j + 1 < n ? keys.after(1) : keys;
                    } else {
                        const int t = j & 1;
                        pv(t, at.s, ((t ? count1 : count0) + (j >> 1)) & 1, j < 2);
                        umma_commit_warp(&sh.freed[at.s]);
                        if (j + 2 < n) {
                            landed(keys);
                            qk(t, keys.s);
                            umma_commit_warp(&sh.freed[keys.s]);
                        }
                        if (j + 3 == n)
                            umma_commit_warp(&sh.q_free);
                        at = j + 2 < n ? keys.after(1) : keys;
                    }
                }
                count0 += PAIR ? n : (n + 1) / 2;
                count1 += PAIR ? n : n / 2;
            }
            umma_commit_warp(&sh.drain);  // every product is done before the block ends
            if (!mbar_wait(&sh.drain, 0) && lane == 0)
                set_error(a.err, DEVERR_TIMEOUT_DRAIN);
            __syncwarp();
        } else {
            // ---- infinities and NaNs of new tokens' values, and of what lies behind them, become zero
            TreePlace<NS> at{0, 0};
            uint32_t v_phase = 0;
            for (Cursor c = sh.start; c.left > 0; c.next(a)) {
                const int n = c.end() - c.tile, from_new = c.t.keys ? c.t.past / TT_KEYS : 0;
                for (int j = max(0, from_new - c.tile); j < n; ++j) {
                    const TreePlace<NS> here = at.after(tree_values_at<PAIR>(j, n));
                    wait(&sh.v_full[here.s], v_phase >> here.s & 1, DEVERR_TIMEOUT_FULL);
                    v_phase ^= 1u << here.s;
                    __syncwarp();
                    uint8_t* vt = ring + here.s * TT_TILE;
                    const int key0 = (c.tile + j) * TT_KEYS;
                    // 16-byte pieces of the rows from the first new key on, eight a row and panel
                    const int row0 = max(0, c.t.past - key0), each = 8 * (TT_KEYS - row0);
                    bool seen = false;
                    for (int i0 = tid - 32 * TT_CLEAN_WARP; i0 < 2 * each; i0 += 64 * 8) {
                        uint4 w[8];
                        int at[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int i = min(i0 + 64 * e, 2 * each - 1), second = i >= each;
                            at[e] = second * TT_PANEL + 16 * (8 * row0 + i - second * each);
                            w[e] = *reinterpret_cast<const uint4*>(vt + at[e]);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t nx = tree_non_finite<T>(w[e].x), ny = tree_non_finite<T>(w[e].y),
                                           nz = tree_non_finite<T>(w[e].z), nw = tree_non_finite<T>(w[e].w);
                            if (nx | ny | nz | nw) {
                                *reinterpret_cast<uint4*>(vt + at[e]) =
                                    make_uint4(w[e].x & ~nx, w[e].y & ~ny, w[e].z & ~nz, w[e].w & ~nw);
                                seen |= key0 + (at[e] % TT_PANEL) / 128 < c.t.keys;
                            }
                        }
                    }
                    if (seen)
                        *static_cast<volatile int*>(&sh.poison) = 1;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sh.cleaned[here.s]);
                }
                at = at.after(2 * n);
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == TT_MMA_WARP)
        tmem_dealloc(tbase, TT_TCOLS);
    if (tid == 0)
        a.join[blockIdx.x] = *fail ? TreeJoin{0, 0, 0, -1} : join.packed();
}

}  // namespace dq

namespace dqhost {

template <typename T, bool PAIR>
static cudaError_t tree_tc(const dq::TreeArgs& a, int blocks, cudaStream_t s)
{
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    {
        // the kernel's shared memory, asked for once per device
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !done[dev]) {
            e = cudaFuncSetAttribute(dq::tree_tc_kernel<T, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, dq::TT_SMEM);
            if (e != cudaSuccess)
                return e;
            if (dev >= 0 && dev < 64)
                done[dev] = true;
        }
    }
    return tree_dependent(dq::tree_tc_kernel<T, PAIR>, dim3(blocks), dq::TT_THREADS, dq::TT_SMEM, s, a);
}

cudaError_t tree_tc_launch(int type, bool pair, const dq::TreeArgs& a, int blocks, cudaStream_t s)
{
    return with_type16(type, [&](auto* p) {
        using T = std::remove_pointer_t<decltype(p)>;
        return pair ? tree_tc<T, true>(a, blocks, s) : tree_tc<T, false>(a, blocks, s);
    });
}

}  // namespace dqhost
