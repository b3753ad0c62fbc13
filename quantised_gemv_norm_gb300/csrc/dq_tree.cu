// dq_tree.cu -- attention of a few new tokens of each sequence, a drafted tree, a chain
// or one, over a paged 16-bit cache (dq_attention_tree): the kernel of up to 16 rows a KV
// head, the join of both kernels and the entry point.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(c (s_j - m) + b),  c = log2(e) / sqrt(128)
// over the keys that a row sees, in one pass: a row's running reference m follows its
// largest score only when that has grown by more than 2^8, sums are fp32, b is 7 in fp16 so
// that p fills the type's range up to 2^15 (0 in bf16).  The subtraction comes before the
// product with c, so scores of any size keep their differences.  The running maximum and sum
// are M. Milakov and N. Gimelshein's online softmax (2018).
//
// The floor is the cache: 512 bytes a key and KV head, read once for all query heads and new
// tokens that share it.  A block is four warps of matrix instructions (m16n8k16, 16 rows) and
// one that copies: tiles of 64 keys through a ring of six 16 KB slots by tensor copies with
// the 128-byte swizzle, which ldmatrix reads without conflicts.  Each warp takes 16 of a
// tile's keys with a reference, sum and output of its own; the four meet at an item's end.  Two
// blocks an SM keep 192 KB on their way, and one's meeting falls into the other's tiles.
// Blocks take equal stretches of all sequences' key tiles, worked out from the lengths on the
// device (dq_tree.cuh), so a batch of any lengths fills the card once; what an item's blocks
// have of it is joined by a second kernel.
//
// 64 sequences of one token after 1 to 12000 keys, 1.66 GB: 251 us, 6.6 TB/s, the measured
// copy rate; matrix pipe 18%, issue 15%.  One token after 100000 keys 68 us (floor 61), after
// 2000 keys 9.3 us, of which the start (lengths, pages, first keys: four waits for memory in a
// row) is three, a tile 0.6, the meeting and the join three.  On the 5th-generation tensor
// cores (dq_tree_tc.cu) the same three took 262, 71 and 12.3 us.  From 17 rows on those are
// used: a variant of this kernel with 32 rows a block, since removed, took 76 us for 8 tokens
// after 100000 keys where they take 73, 73 for 32 sequences of 5 after up to 4000 (67), 56 for
// 64 of 8 after 1000 (58).
#include <algorithm>
#include <mutex>

#include "dq_tree.cuh"

namespace dq {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void tree_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---- up to 16 rows a KV head: warp-level matrix instructions

constexpr int TM_ROWS = 16;                     // rows an item
constexpr int TM_KEYS = 64;                     // keys a tile
constexpr int TM_SLOT = TM_KEYS * ATT_HD * 2;   // bytes of a tile of keys or values
constexpr int TM_SLOTS = 6;                     // ring: keys, values, keys, ...
constexpr int TM_WARPS = 4, TM_THREADS = 32 * (TM_WARPS + 1), TM_RESIDENT = 2;
constexpr int TM_MEET = 2 * 16 * ATT_HD * 4;    // two warps' sums
constexpr int TM_SMEM = TM_SLOTS * TM_SLOT + TM_MEET + 512;

struct TreeMiscM {
    uint64_t full[TM_SLOTS], freed[TM_SLOTS];
    uint32_t absent[TM_SLOTS];  // runs of 16 keys whose page is outside the pool
    float ml[2][16][2];
    TreeCursor<TM_ROWS, TM_KEYS> start;
    int fail;
};
static_assert(sizeof(TreeMiscM) <= 512, "fits behind the ring");

template <typename T>
__global__ void __launch_bounds__(TM_THREADS, TM_RESIDENT) tree_mma_kernel(const __grid_constant__ TreeArgs a)
{
    constexpr int R = TM_ROWS, NK = TM_KEYS / TM_WARPS;  // keys a warp
    static_assert(NK == 16, "one step of the second product, two blocks of eight keys of the first");
    constexpr float TOP = std::is_same<T, __half>::value ? 7.f : 0.f;
    extern __shared__ __align__(1024) uint8_t ring[];
    float2* meet = reinterpret_cast<float2*>(ring + TM_SLOTS * TM_SLOT);
    TreeMiscM& sh = *reinterpret_cast<TreeMiscM*>(ring + TM_SLOTS * TM_SLOT + TM_MEET);
    volatile int* fail = &sh.fail;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == TM_WARPS) {
        if (lane == 0) {
            for (int i = 0; i < TM_SLOTS; ++i) {
                mbar_init(&sh.full[i], 1);
                mbar_init(&sh.freed[i], TM_WARPS);
            }
            fence_mbar_init();
            sh.fail = 0;
            tree_fetch_map(&a.map);
        }
        pdl_wait();
        const TreeCursor<TM_ROWS, TM_KEYS> first = tree_start<TM_ROWS, TM_KEYS>(a, lane);
        if (lane == 0)
            sh.start = first;
    }
    pdl_wait();
    pdl_trigger();  // only now: the join reads lengths before this kernel ends
    __syncthreads();
    TreeCursor<TM_ROWS, TM_KEYS> c = sh.start;
    const int each = c.left;
    TreeShared join{0, 0, 0, 0, -1};
    if (each > 0) {
        auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
            if (!mbar_try_wait(bar, parity))
                tree_wait_on(bar, parity, fail, a.err, code);
        };
        int slot = 0;
        uint32_t phase = 0;
        auto turn = [&] {
            if (++slot == TM_SLOTS) {
                slot = 0;
                phase ^= 1;
            }
        };
        if (warp == TM_WARPS) {
            // ---- copies: a lane takes one of a tile's boxes (16, 32 or 64 rows of a page)
            const int box = a.box, per_tile = TM_KEYS / box, ahead = 32 / per_tile;
            long long issued = 0;
            for (; c.left > 0 && !__any_sync(0xffffffffu, *fail); c.next(a)) {
                const int g = c.g;
                const int* pages = a.pages + static_cast<size_t>(c.s) * a.max_pages;
                // lane i has the page of box `first + i`, and of box `first + 32 + i`
                auto page_of = [&](int x) {
                    return static_cast<long long>(x) * box < c.t.keys ? __ldcg(pages + fast_div(x, a.by_boxes)) : 0;
                };
                int first = c.tile, now = page_of(first * per_tile + lane), then = page_of((first + ahead) * per_tile + lane);
                const int end = c.end();
                for (int k = c.tile; k < end; ++k) {
                    if (k - first == ahead) {
                        first = k;
                        now = then;
                        then = page_of((first + ahead) * per_tile + lane);
                    }
                    const int page = __shfl_sync(0xffffffffu, now, ((k - first) * per_tile + lane) & 31);
                    const int x = k * per_tile + lane;
                    const bool mine = lane < per_tile && static_cast<long long>(x) * box < c.t.keys;
                    const bool there = mine && page >= 0 && page < a.s.n_pages;
                    const unsigned have = __ballot_sync(0xffffffffu, there), lack = __ballot_sync(0xffffffffu, mine && !there);
                    uint32_t absent = 0;
                    if (lack) {
                        for (int i = 0; i < per_tile; ++i)
                            if (lack >> i & 1)
                                absent |= ((1u << (box / 16)) - 1) << (i * (box / 16));
                        if (lane == 0)
                            set_error(a.err, DEVERR_BAD_ARG);
                    }
                    const uint32_t bytes = static_cast<uint32_t>(__popc(have) * box * 256);
                    const int off = (x - static_cast<int>(fast_div(x, a.by_boxes) * a.by_boxes.d)) * box;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        wait(&sh.freed[slot], phase ^ 1, DEVERR_TIMEOUT_EMPTY);
                        __syncwarp();
                        if (__any_sync(0xffffffffu, *fail))
                            continue;
                        if (lane == 0) {
                            sh.absent[slot] = absent;
                            mbar_arrive_expect_tx(&sh.full[slot], bytes);
                        }
                        __syncwarp();
                        if (there)
                            tree_load(ring + slot * TM_SLOT + lane * box * 256, &a.map, 0,
                                      static_cast<int>(kv16_row(a.s, page, kv, g)) + off, 0, &sh.full[slot]);
                        ++issued;
                        turn();
                    }
                }
            }
            // every copy has landed before the block ends
            for (long long i = max(0ll, issued - TM_SLOTS); i < issued; ++i)
                if (!mbar_wait(&sh.full[i % TM_SLOTS], static_cast<uint32_t>(i / TM_SLOTS) & 1) && lane == 0)
                    set_error(a.err, DEVERR_TIMEOUT_DRAIN);
        } else {
            const int wk = warp, r8 = lane >> 2, q4 = lane & 3;
            const uint32_t panel = static_cast<uint32_t>(a.box) * 128;
            // byte offset of the warp's 16 keys in a slot
            const int box_of = wk * NK / a.box;
            const uint32_t keys_at = static_cast<uint32_t>(box_of * a.box * 256 + (wk * NK - box_of * a.box) * 128);
            // this lane's row and 16-byte piece of the four 8 x 8 matrices: of keys (two runs of 8,
            // two of dims), of values (the same, transposed)
            const uint32_t sw = lane & 7;
            const uint32_t k_at = ((lane >> 4) * 8 + sw) * 128 + (((lane >> 3 & 1) ^ sw) << 4);
            const uint32_t v_at = ((lane >> 3 & 1) * 8 + sw) * 128 + (((lane >> 4) ^ sw) << 4);
            const uint32_t base = smem_addr(ring);
            for (; c.left > 0; c.next(a)) {
                const int g = c.g, rt = c.rt;
                const TreeSeq t = c.t;
                // this lane's two rows
                const T* qp[2];
                uint64_t seen[2];
                bool live[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = rt * R + r8 + 8 * h, node = static_cast<int>(fast_div(r, a.by_group));
                    live[h] = node < t.rows;
                    const int row = t.row0 + (live[h] ? node : 0);
                    qp[h] = static_cast<const T*>(a.q) + static_cast<long long>(row) * a.q_row +
                            static_cast<long long>(g * a.group + r - node * a.group) * a.q_head;
                    seen[h] = !live[h] ? 0ull : a.seen ? __ldcg(a.seen + row) : (2ull << node) - 1;
                    if (t.rows < 64)
                        seen[h] &= (1ull << t.rows) - 1;
                }
                uint32_t q[8][4];
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            q[k][h + 2 * e] = live[h] ? __ldcg(reinterpret_cast<const uint32_t*>(qp[h] + 16 * k + 8 * e + 2 * q4)) : 0u;
                float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
                const int end = c.end();

                auto tile = [&](auto tail, int k) {
                    constexpr bool TAIL = decltype(tail)::value;
                    float s[NK / 8][4];
#pragma unroll
                    for (int i = 0; i < NK / 8; ++i)
                        s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
                    const uint32_t kb = base + slot * TM_SLOT;
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        uint32_t b[4];
                        ldsm4(b, ((kb + keys_at + k_at) ^ ((d & 3) * 32)) + (d >> 2) * panel);
                        tree_mma<T>(s[0], q[d], b[0], b[1]);
                        tree_mma<T>(s[1], q[d], b[2], b[3]);
                    }
                    const bool absent = TAIL && (!t.keys || (sh.absent[slot] >> wk & 1));  // the warp's 16 keys
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sh.freed[slot]);
                    turn();
                    // new token of this lane's first key
                    const int node0 = k * TM_KEYS + wk * NK + 2 * q4 - t.past;
                    if (TAIL) {
#pragma unroll
                        for (int i = 0; i < NK / 8; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int node = node0 + 8 * i + e;
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    if (absent || node >= 64 || (node >= 0 && !(seen[h] >> (node & 63) & 1)))
                                        s[i][2 * h + e] = -INFINITY;
                            }
                    }
                    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < NK / 8; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            top[h] = fmaxf(top[h], fmaxf(s[i][2 * h], s[i][2 * h + 1]));
                    if (__any_sync(0xffffffffu, (top[0] - m[0]) * TR_C > TR_GROW || (top[1] - m[1]) * TR_C > TR_GROW)) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float x = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                            float f = 1.f;
                            if ((x - m[h]) * TR_C > TR_GROW) {
                                f = ex2((m[h] - x) * TR_C);  // 0 from -infinity
                                m[h] = x;
                            }
                            l[h] *= f;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                o[i][2 * h] *= f;
                                o[i][2 * h + 1] *= f;
                            }
                        }
                    }
                    uint32_t p[4];
                    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
                    for (int i = 0; i < NK / 8; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float x = ex2(fmaf(s[i][2 * h] - ref[h], TR_C, TOP)), y = ex2(fmaf(s[i][2 * h + 1] - ref[h], TR_C, TOP));
                            l[h] += x + y;
                            p[2 * i + h] = pack2(x, y, static_cast<const T*>(nullptr));
                        }
                    wait(&sh.full[slot], phase, DEVERR_TIMEOUT_FULL);
                    __syncwarp();
                    const uint32_t vb = base + slot * TM_SLOT;
                    bool poison = false;
                    uint32_t keep[2], fresh[2];  // keys 2 q4, + 1 and 8 more: those that exist, those that are new
                    if (TAIL) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int node = node0 + 8 * e;
                            keep[e] = absent ? 0u : (node < t.rows ? 0xffffu : 0u) | (node + 1 < t.rows ? 0xffff0000u : 0u);
                            fresh[e] = (node >= 0 ? 0xffffu : 0u) | (node + 1 >= 0 ? 0xffff0000u : 0u);
                        }
                    }
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        uint32_t b[4];
                        ldsm4_trans(b, ((vb + keys_at + v_at) ^ ((d & 3) * 32)) + (d >> 2) * panel);
                        if (TAIL) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                b[e] &= keep[e & 1];
                                const uint32_t nf = tree_non_finite<T>(b[e]) & fresh[e & 1];
                                poison |= nf != 0;
                                b[e] &= ~nf;
                            }
                        }
                        tree_mma<T>(o[2 * d], p, b[0], b[1]);
                        tree_mma<T>(o[2 * d + 1], p, b[2], b[3]);
                    }
                    if (TAIL && __any_sync(0xffffffffu, poison)) {
                        // new tokens' infinities and NaNs, which the products left out: to the rows that see them
                        for (int key = 0; key < NK; ++key) {
                            const int node = k * TM_KEYS + wk * NK + key - t.past;
                            if (node < 0 || node >= t.rows || absent)
                                continue;
                            const uint32_t at = keys_at + key * 128;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const uint32_t w = *reinterpret_cast<const uint32_t*>(
                                    ring + slot * TM_SLOT + at + (i >> 3) * panel + (((i & 7) ^ (key & 7)) << 4) + 4 * q4);
                                const uint32_t nf = tree_non_finite<T>(w);
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    if (seen[h] >> node & 1) {
                                        if (nf & 0xffffu)
                                            o[i][2 * h] += tree_one<T>(w & 0xffffu);
                                        if (nf >> 16)
                                            o[i][2 * h + 1] += tree_one<T>(w >> 16);
                                    }
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sh.freed[slot]);
                    turn();
                };

                for (int k = c.tile; k < end; ++k) {
                    wait(&sh.full[slot], phase, DEVERR_TIMEOUT_FULL);
                    __syncwarp();
                    if ((k + 1) * TM_KEYS > t.past || sh.absent[slot])
                        tile(std::true_type{}, k);
                    else
                        tile(std::false_type{}, k);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                }
                // ---- the warps along the keys meet: half of them give, the others take
#pragma unroll
                for (int half = TM_WARPS / 2; half > 0; half /= 2) {
                    const int place = wk % half;
                    if (wk >= half && wk < 2 * half) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                meet[place * 1024 + (2 * i + h) * 32 + lane] = make_float2(o[i][2 * h], o[i][2 * h + 1]);
                        if (q4 == 0)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                sh.ml[place][r8 + 8 * h][0] = m[h];
                                sh.ml[place][r8 + 8 * h][1] = l[h];
                            }
                    }
                    named_bar_sync(1, 32 * TM_WARPS);
                    if (wk < half) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float m2 = sh.ml[place][r8 + 8 * h][0], l2 = sh.ml[place][r8 + 8 * h][1];
                            const float mn = fmaxf(m[h], m2);
                            const float f = m[h] == mn ? 1.f : ex2((m[h] - mn) * TR_C), f2 = m2 == mn ? 1.f : ex2((m2 - mn) * TR_C);
                            m[h] = mn;
                            l[h] = l[h] * f + l2 * f2;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 y = meet[place * 1024 + (2 * i + h) * 32 + lane];
                                o[i][2 * h] = o[i][2 * h] * f + y.x * f2;
                                o[i][2 * h + 1] = o[i][2 * h + 1] * f + y.y * f2;
                            }
                        }
                    }
                    named_bar_sync(1, 32 * TM_WARPS);
                }
                const bool whole = c.tile == 0 && end == c.tiles;
                if (!whole && c.tile == 0 && warp == 0) {
                    // the blocks that go on with the item: each has as many units as this one
                    join = TreeShared{t.row0, t.rows, g, rt,
                                    static_cast<int>(blockIdx.x) + (c.tiles - end + each - 1) / each};
                }
                if (wk == 0 && !*fail) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int rr = r8 + 8 * h, r = rt * R + rr, node = static_cast<int>(fast_div(r, a.by_group));
                        if (!live[h])
                            continue;
                        if (whole) {
                            const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];
                            T* out = static_cast<T*>(a.out) + static_cast<long long>(t.row0 + node) * a.o_row +
                                     static_cast<long long>(g * a.group + r - node * a.group) * a.o_head + 2 * q4;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                *reinterpret_cast<uint32_t*>(out + 8 * i) =
                                    l[h] == 0.f ? 0u : pack2(o[i][2 * h] * inv, o[i][2 * h + 1] * inv, static_cast<const T*>(nullptr));
                        } else {
                            const size_t at = static_cast<size_t>(blockIdx.x) * 2 + (c.tile == 0);
                            if (q4 == 0)
                                a.part_ml[at * R + rr] = make_float2(m[h], l[h]);
                            float2* part = reinterpret_cast<float2*>(a.part + (at * 32 + (q4 >> 1)) * R + rr) + (q4 & 1);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                part[4 * i * R] = make_float2(o[i][2 * h], o[i][2 * h + 1]);
                        }
                    }
                }
            }
        }
    }
    if (tid == 0)
        a.join[blockIdx.x] = *fail ? TreeJoin{0, 0, 0, -1} : join.packed();
}

// Items that several blocks had a part of.  A unit of work is 32 lanes' rows (of 16-row
// items: their rows twice, the next eight dims) and eight dims each, over all the blocks' sums.
// P = 1: one row of the grid a block of the first kernel, which has left the item that it
// began and did not end, and a warp a unit.  Where items are few and each had many blocks,
// one row an item, whose blocks are worked out while the first kernel still runs, and P warps
// a unit, each every P-th block's sums, which then meet.
constexpr int TJ_WARPS = 8, TJ_BATCH = 5;

template <typename T, int R, int KT, int P>
__global__ void __launch_bounds__(32 * TJ_WARPS) tree_join_kernel(const __grid_constant__ TreeArgs a, int per_seq)
{
    constexpr int ROWS = R < 32 ? R : 32;
    __shared__ float2 meet_ml[P > 1 ? TJ_WARPS : 1][32];
    __shared__ float4 meet_o[P > 1 ? TJ_WARPS : 1][2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    TreeShared j;
    int b = blockIdx.x;
    if (P == 1) {
        pdl_wait();
        const int4 x = __ldcg(reinterpret_cast<const int4*>(a.join + b));
        j = TreeShared{x.x, x.y >> 8, x.z, x.y & 0xff, x.w};
        if (j.last < 0)
            return;
    } else {
        // every warp for itself
        TreeCursor<(R < 128 ? R : 0), KT> c;
        const int s = blockIdx.x / per_seq, item = blockIdx.x - s * per_seq;
        int before = 0, total = 0;
        for (int s0 = 0; s0 < a.n_seq; s0 += 32) {
            int u = 0;
            if (s0 + lane < a.n_seq) {
                c.t = tree_seq(a, s0 + lane);
                u = c.units(a);
            }
            before += __reduce_add_sync(0xffffffffu, s0 + lane < s ? u : 0);
            total += __reduce_add_sync(0xffffffffu, u);
        }
        c.load(a, s);
        pdl_wait();  // before any return: this kernel ends after the first one
        if (item >= a.s.n_kv * c.row_tiles)
            return;
        const int each = tree_each(a, total), start = before + item * c.tiles;
        b = start / each;
        j = TreeShared{c.t.row0, c.t.rows, item / c.row_tiles, item % c.row_tiles, (start + c.tiles - 1) / each};
        if (j.last == b)
            return;
        if (__ldcg(&a.join[b].last) < 0)
            return;  // a wait ran out
    }
    const int n = j.last - b + 1, part = warp % P, u = blockIdx.y * (TJ_WARPS / P) + warp / P;
    const int rr = u % (R / ROWS) * ROWS + lane % ROWS, pair = u / (R / ROWS) * (32 / ROWS) + lane / ROWS;
    int node, head;
    if (R >= 128) {  // 128 rows for as many whole tokens as they hold
        const int in_tile = rr & 127, token = static_cast<int>(fast_div(in_tile, a.by_group)), tokens = a.nodes / (R < 128 ? 1 : R / 128);
        head = in_tile - token * a.group;
        node = token < tokens ? j.row_tile * a.nodes + (rr >> 7) * tokens + token : 0x7fffffff;
    } else {
        const int r = j.row_tile * R + rr;
        node = static_cast<int>(fast_div(r, a.by_group));
        head = r - node * a.group;
    }
    const bool live = node < j.rows;
    float m = -INFINITY, l = 0.f;
    float4 o[2] = {};
    auto add = [&](float2 ml, const float4 (&y)[2]) {
        const float top = fmaxf(m, ml.x), f = m == top ? 1.f : ex2((m - top) * TR_C), w = ml.x == top ? 1.f : ex2((ml.x - top) * TR_C);
        m = top;
        l = fmaf(w, ml.y, l * f);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            o[h] = make_float4(fmaf(w, y[h].x, o[h].x * f), fmaf(w, y[h].y, o[h].y * f), fmaf(w, y[h].z, o[h].z * f),
                               fmaf(w, y[h].w, o[h].w * f));
    };
    for (int k0 = part; k0 < n && live; k0 += P * TJ_BATCH) {
        float2 ml[TJ_BATCH];
        float4 y[TJ_BATCH][2];
#pragma unroll
        for (int e = 0; e < TJ_BATCH; ++e) {
            const int k = k0 + e * P;
            if (k < n) {
                const size_t at = static_cast<size_t>(b + k) * 2 + (k == 0);
                ml[e] = __ldcg(a.part_ml + at * R + rr);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    y[e][h] = __ldcg(a.part + (at * 32 + 2 * pair + h) * R + rr);
            }
        }
#pragma unroll
        for (int e = 0; e < TJ_BATCH; ++e)
            if (k0 + e * P < n)
                add(ml[e], y[e]);
    }
    if (P > 1) {
        meet_ml[warp][lane] = make_float2(m, l);
        meet_o[warp][0][lane] = o[0];
        meet_o[warp][1][lane] = o[1];
        __syncthreads();
        if (part)
            return;
#pragma unroll
        for (int w = 1; w < P; ++w) {
            const float4 y[2] = {meet_o[warp + w][0][lane], meet_o[warp + w][1][lane]};
            add(meet_ml[warp + w][lane], y);
        }
    }
    if (live) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[2 * h] = l == 0.f ? 0u : pack2(o[h].x * inv, o[h].y * inv, static_cast<const T*>(nullptr));
            w[2 * h + 1] = l == 0.f ? 0u : pack2(o[h].z * inv, o[h].w * inv, static_cast<const T*>(nullptr));
        }
        *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + static_cast<long long>(j.row0 + node) * a.o_row +
                                  static_cast<long long>(j.kv * a.group + head) * a.o_head + 8 * pair) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace dq

namespace dqhost {

// Rows a block and blocks: two of 16 rows an SM, or one of 128 or 256 on the tensor
// cores of the 5th generation.
struct TreeCut {
    int rows, blocks;
    bool tc() const { return rows >= 128; }
    // tokens an item where it has whole ones, else 0; row tiles of that many new tokens
    int nodes(int group) const { return tc() ? 128 / group * (rows / 128) : 0; }
    int row_tiles(int n, int group) const
    {
        return tc() ? (n + nodes(group) - 1) / nodes(group) : (n * group + rows - 1) / rows;
    }
};

static TreeCut tree_cut(int max_new, int group)
{
    const int rows = max_new * group;
    if (rows > dq::TM_ROWS)
        return {(max_new + 128 / group - 1) / (128 / group) > 1 ? 256 : 128, sm_count()};
    return {dq::TM_ROWS, dq::TM_RESIDENT * sm_count()};
}

static size_t tree_bytes(const TreeCut& c)
{
    const size_t rows = static_cast<size_t>(c.blocks) * 2 * c.rows;
    return rows * (dq::ATT_HD + 2) * sizeof(float) + (c.blocks * sizeof(dq::TreeJoin) + 15) / 16 * 16;
}

// A kernel's attribute, set once per device.
template <typename K>
static cudaError_t tree_prepare(K kernel, cudaFuncAttribute what, int value, bool (&done)[64])
{
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(kernel, what, value);
        if (e == cudaSuccess && dev >= 0 && dev < 64)
            done[dev] = true;
    }
    return e;
}

template <typename T>
static cudaError_t tree_launch(const dq::TreeArgs& a, const TreeCut& cut, cudaStream_t s)
{
    static bool done[64] = {};
    cudaError_t e = tree_prepare(dq::tree_mma_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, dq::TM_SMEM, done);
    if (e != cudaSuccess)
        return e;
    return tree_dependent(dq::tree_mma_kernel<T>, dim3(cut.blocks), dq::TM_THREADS, dq::TM_SMEM, s, a);
}

// The join: a dependent launch.
template <typename T, int R, int KT>
static cudaError_t tree_join(const dq::TreeArgs& a, const TreeCut& cut, cudaStream_t s)
{
    const int per_seq = a.s.n_kv * cut.row_tiles(a.max_new, a.group);
    const long long items = static_cast<long long>(a.n_seq) * per_seq;
    // warps a unit: an item has about blocks / items blocks' sums
    int parts = 1;
    if (items * 8 <= cut.blocks)
        while (parts < 8 && items * parts * dq::TJ_BATCH < cut.blocks)
            parts *= 2;
    return tree_dependent(parts == 1   ? dq::tree_join_kernel<T, R, KT, 1>
                          : parts == 2 ? dq::tree_join_kernel<T, R, KT, 2>
                          : parts == 4 ? dq::tree_join_kernel<T, R, KT, 4>
                                       : dq::tree_join_kernel<T, R, KT, 8>,
                          dim3(static_cast<unsigned>(parts == 1 ? cut.blocks : items), static_cast<unsigned>(R / 2 * parts / dq::TJ_WARPS)),
                          32 * dq::TJ_WARPS, 0, s, a, per_seq);
}

}  // namespace dqhost

extern "C" {

DQ_API size_t dq_attention_tree_workspace_bytes(int n_seq, int max_new, int n_q, int n_kv)
{
    if (n_seq < 1 || max_new < 1 || max_new > dq::TR_MAX_NEW || n_q < 1 || n_kv < 1 || n_q % n_kv ||
        n_q / n_kv > dq::TR_MAX_GROUP)
        return 0;
    return dqhost::tree_bytes(dqhost::tree_cut(max_new, n_q / n_kv));
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
    const int group = t->n_q / t->n_kv;
    const dqhost::TreeCut cut = dqhost::tree_cut(t->max_new, group);
    // units of work, at most, as the kernels count them in 32 bits
    const long long tile = cut.tc() ? dqhost::TREE_TC_KEYS : dq::TM_KEYS, tiles = (static_cast<long long>(t->max_pages) * t->page_size + tile - 1) / tile;
    if (tiles * cut.row_tiles(t->max_new, group) * t->n_seq * t->n_kv >= (1 << 30))
        return DQ_ERR_UNSUPPORTED;
    if (t->workspace_bytes < dq_attention_tree_workspace_bytes(t->n_seq, t->max_new, t->n_q, t->n_kv))
        return DQ_ERR_SHAPE;
    int box = cut.tc() ? dqhost::TREE_TC_KEYS : dq::TM_KEYS;  // rows of a copy: what divides a tile and a page
    while (t->page_size % box)
        box /= 2;
    dq::TreeArgs a{};
    if (!dqhost::tree_map(&a.map, t->type, t->pool, {64, 2ll * t->n_pages * t->n_kv * t->page_size, 2}, {dq::ATT_HD * 2, 128},
                          box, cut.tc() ? 1 : 2))
        return DQ_ERR_UNSUPPORTED;
    if (cut.tc()) {
        const int tokens = 128 / group;
        a.nodes = cut.nodes(group);
        // a stride of a dimension of one is never used, but has to be one that the encoder takes
        if (!dqhost::tree_map(&a.tq, t->type, t->q, {dq::ATT_HD, t->n_q, t->total_new},
                              {2 * (t->n_q > 1 ? heads[0] : dq::ATT_HD), 2 * (t->total_new > 1 ? rows[0] : dq::ATT_HD)}, group,
                              tokens))
            return DQ_ERR_UNSUPPORTED;
    }
    a.pool = t->pool;
    a.q = t->q;
    a.out = t->out;
    a.q_row = rows[0];
    a.q_head = heads[0];
    a.o_row = rows[1];
    a.o_head = heads[1];
    a.pages = t->pages;
    a.n_past = t->n_past;
    a.cu_new = t->cu_new;
    a.seen = t->seen;
    const size_t part_rows = static_cast<size_t>(cut.blocks) * 2 * cut.rows;
    a.part = static_cast<float4*>(t->workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part + part_rows * (dq::ATT_HD / 4));
    a.join = reinterpret_cast<dq::TreeJoin*>(a.part_ml + part_rows);
    a.room = static_cast<long long>(t->max_pages) * t->page_size;
    a.n_seq = t->n_seq;
    a.total_new = t->total_new;
    a.max_new = t->max_new;
    a.group = group;
    a.max_pages = t->max_pages;
    a.box = box;
    // a block's units where there are few: a tile costs less than starting a block and joining
    // its sums, but they run side by side (one token after 2000 keys: 8.8 us with 1 or 2, 9.2
    // with 4; 64 tokens: 17.4 us with 1, 20.3 with 2, 23.6 with 4)
    a.least = cut.tc() ? 1 : 2;
    a.s = {t->n_kv, t->n_pages, t->page_size};
    a.by_group = dqhost::fast_divisor(group);
    a.by_nodes = dqhost::fast_divisor(std::max(1, a.nodes));
    a.by_blocks = dqhost::fast_divisor(cut.blocks);
    a.by_boxes = dqhost::fast_divisor(t->page_size / box);
    a.err = dqhost::device_error_flag();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dqhost::with_type16(t->type, [&](auto* p) {
        using T = std::remove_pointer_t<decltype(p)>;
        cudaError_t err = cut.tc() ? dqhost::tree_tc_launch(t->type, cut.rows == 256, a, cut.blocks, s)
                                   : dqhost::tree_launch<T>(a, cut, s);
        if (err != cudaSuccess)
            return err;
        return !cut.tc()         ? dqhost::tree_join<T, dq::TM_ROWS, dq::TM_KEYS>(a, cut, s)
               : cut.rows == 128 ? dqhost::tree_join<T, 128, dqhost::TREE_TC_KEYS>(a, cut, s)
                                 : dqhost::tree_join<T, 256, dqhost::TREE_TC_KEYS>(a, cut, s);
    });
    return e == cudaSuccess ? DQ_OK : dqhost::set_cuda_error(e);
}

}  // extern "C"
