// dq_tree.cuh -- tree attention over the paged 16-bit cache: arguments, how the work is
// spread over the blocks, and what its two kernels share.
#pragma once

#include "dq_kv16.cuh"
#include "dq_tma_host.h"

namespace dq {

constexpr float TR_C = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(128)
constexpr int TR_MAX_NEW = 64, TR_MAX_GROUP = 64;
// log2 of the growth of a row's maximum that is let pass before its sums are scaled: a
// probability is up to 2^8 (fp16: of 2^7 at the maximum, up to 2^15)
constexpr float TR_GROW = 8.f;

struct TreeJoin;

struct TreeArgs {
    CUtensorMap map;  // the pool as [2 halves of a row][rows][64]
    CUtensorMap tq;   // the queries as [rows][heads][128]
    const void* pool;
    const void* q;
    void* out;
    long long q_row, q_head, o_row, o_head;
    const int* pages;
    const int* n_past;
    const int* cu_new;
    const unsigned long long* seen;
    // unscaled sums, and their maxima and sums of probabilities, of each block's first and last
    // segment: [blocks][2][32 fours of dims][rows a block], [blocks][2][rows a block]
    float4* part;
    float2* part_ml;
    TreeJoin* join;   // [blocks]
    long long room;   // rows that max_pages pages hold
    int n_seq, total_new, max_new, group, max_pages, box, least;
    int nodes;        // tokens an item where it has whole ones, else 0
    Kv16Shape s;
    FastDiv by_group, by_boxes, by_nodes, by_blocks;  // boxes of a page; blocks of the first kernel
    int* err;
};

// A sequence's new rows, and the keys before them; no rows where cu_new is not in order,
// no keys where n_past does not fit.
struct TreeSeq {
    int row0, rows, past, keys;
    bool bad;
};

// Loads of inputs go past L1, here and in the kernels: a dependent launch may have started
// before they were written.
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int s)
{
    TreeSeq t;
    int r1;
    if (a.cu_new) {
        t.row0 = __ldcg(a.cu_new + s);
        r1 = __ldcg(a.cu_new + s + 1);
    } else {
        t.row0 = s * a.max_new;
        r1 = t.row0 + a.max_new;
    }
    t.past = __ldcg(a.n_past + s);
    const bool in_order = t.row0 >= 0 && r1 >= t.row0 && r1 <= a.total_new && r1 - t.row0 <= a.max_new;
    t.rows = in_order ? r1 - t.row0 : 0;
    const bool fits = t.past >= 0 && static_cast<long long>(t.past) + t.rows <= a.room;
    t.bad = !in_order || !fits;
    if (!fits)
        t.past = 0;
    t.keys = fits ? t.past + t.rows : 0;
    return t;
}

// Units a block.
__device__ __forceinline__ int tree_each(const TreeArgs& a, int total)
{
    const int each = static_cast<int>(fast_div(total, a.by_blocks));
    return max(a.least, each + (each * static_cast<int>(a.by_blocks.d) < total));
}

// The work is counted in units: one key tile of one item, an item being a row tile of one
// sequence and KV head.  Sequence by sequence, item by item, tile by tile they are one
// long row, of which every block takes an equal stretch; a stretch is cut into segments
// where items change.  The host has seen that the units are fewer than 2^30.
template <int R, int KT>
struct TreeCursor {
    TreeSeq t;
    int s, row_tiles, tiles;  // of the sequence
    int g, rt, tile;          // the item's KV head and row tile, the segment's first key tile
    int left;                 // units of the block's stretch

    __device__ __forceinline__ int units(const TreeArgs& a)
    {
        // R rows whatever tokens they are of, or (R = 0) a.nodes whole tokens
        row_tiles = R ? (t.rows * a.group + R - 1) / (R ? R : 1) : static_cast<int>(fast_div(t.rows + a.nodes - 1, a.by_nodes));
        tiles = max(1, (t.keys + KT - 1) / KT);
        return a.s.n_kv * row_tiles * tiles;
    }
    __device__ __forceinline__ void load(const TreeArgs& a, int seq)
    {
        s = seq;
        t = tree_seq(a, seq);
        units(a);
    }
    __device__ __forceinline__ int end() const { return min(tiles, tile + left); }
    // to the next segment
    __device__ __forceinline__ void next(const TreeArgs& a)
    {
        left -= end() - tile;
        tile = 0;
        if (left <= 0 || ++rt < row_tiles)
            return;
        rt = 0;
        if (++g < a.s.n_kv)
            return;
        g = 0;
        do
            load(a, s + 1);
        while (row_tiles == 0);  // there are units left, so there is a sequence with some
    }
};

// Where the block's stretch begins, by one warp; left = 0: it has none.  A lane has four
// consecutive sequences at a time, so that the lengths of 128 are one wait for memory.
template <int R, int KT>
__device__ __forceinline__ TreeCursor<R, KT> tree_start(const TreeArgs& a, int lane)
{
    constexpr int E = 4;
    TreeCursor<R, KT> c;
    int u[E], mine = 0, incl = 0, total = 0;
    // sequences s0 ..: the lane's units, and those of all lanes up to it
    auto round = [&](int s0, bool report) {
        mine = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int s = s0 + E * lane + e;
            u[e] = 0;
            if (s < a.n_seq) {
                c.t = tree_seq(a, s);
                u[e] = c.units(a);
                if (report && c.t.bad)
                    set_error(a.err, DEVERR_BAD_ARG);
            }
            mine += u[e];
        }
        incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += x;
        }
    };
    for (int s0 = 0; s0 < a.n_seq; s0 += 32 * E) {
        round(s0, blockIdx.x == 0);
        total += __shfl_sync(0xffffffffu, incl, 31);
    }
    const int each = tree_each(a, total);
    int want = each * static_cast<int>(blockIdx.x);
    const int left = min(each, total - want);
    c.left = 0;
    if (left <= 0)
        return c;
    for (int s0 = 0; s0 < a.n_seq; s0 += 32 * E) {
        if (a.n_seq > 32 * E)
            round(s0, false);
        const unsigned hit = __ballot_sync(0xffffffffu, want >= incl - mine && want < incl);
        if (hit) {
            int off = want - (incl - mine), s = 0;
#pragma unroll
            for (int e = 0; e < E - 1; ++e)
                if (s == e && off >= u[e]) {
                    off -= u[e];
                    ++s;
                }
            const int src = __ffs(hit) - 1;
            off = __shfl_sync(0xffffffffu, off, src);
            s = s0 + E * src + __shfl_sync(0xffffffffu, s, src);
            c.load(a, s);
            const int item = off / c.tiles;
            c.g = c.row_tiles > 1 ? item / c.row_tiles : item;
            c.rt = item - c.g * c.row_tiles;
            c.tile = off - item * c.tiles;
            c.left = left;
            return c;
        }
        want -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return c;  // not reached: want is below the total
}

// What a block leaves for the join: its last segment began an item that later blocks go
// on with, the last of them `last`; -1: nothing to join.
struct __align__(16) TreeJoin {
    int row0, rows_tile, kv, last;
};
struct TreeShared {
    int row0, rows, kv, row_tile, last;
    __device__ __forceinline__ TreeJoin packed() const { return TreeJoin{row0, rows << 8 | row_tile, kv, last}; }
};
static_assert(TR_MAX_NEW <= 128 && TR_MAX_GROUP * TR_MAX_NEW / 16 <= 256, "a row tile's number has eight bits");

__device__ __forceinline__ void tree_fetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void tree_load(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

template <typename T>
__device__ __forceinline__ float tree_one(uint32_t bits)
{
    return std::is_same<T, __half>::value ? half_bits_to_float(bits) : bf16lo(bits);
}

// 0xffff in the halves of a pair that are an infinity or NaN.
template <typename T>
__device__ __forceinline__ uint32_t tree_non_finite(uint32_t w)
{
    constexpr bool half = std::is_same<T, __half>::value;
    constexpr uint32_t mask = half ? 0x7C007C00u : 0x7F807F80u, one = half ? 0x04000400u : 0x00800080u;
    return ((((w & mask) + one) & 0x80008000u) >> 15) * 0xffffu;
}

// The rest of a wait whose first poll found nothing; once one has run out the others
// return at once and the block writes nothing.
__device__ __forceinline__ void tree_wait_on(uint64_t* bar, uint32_t parity, volatile int* fail, int* err, int code)
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

}  // namespace dq

namespace dqhost {

// 3-D boxes of a 16-bit tensor with the 128-byte swizzle; strides in bytes.
inline bool tree_map(CUtensorMap* m, int type, const void* p, const long long (&dim)[3], const long long (&stride)[2],
                     int box1, int box2)
{
    const EncodeTiled enc = encode_tiled();
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim[0]), static_cast<cuuint64_t>(dim[1]), static_cast<cuuint64_t>(dim[2])};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride[0]), static_cast<cuuint64_t>(stride[1])};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2)};
    const cuuint32_t ones[3] = {1, 1, 1};
    return enc && enc(m, type == DQ_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                      const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A dependent launch: the kernel sets itself up while the one before it ends.
template <typename... P, typename... A>
cudaError_t tree_dependent(void (*kernel)(P...), dim3 grid, int threads, int shared, cudaStream_t s, const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(shared);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The tensor-core kernel (dq_tree_tc.cu): one query tile of 128 rows a block, or two.
constexpr int TREE_TC_KEYS = 128;  // keys a tile
cudaError_t tree_tc_launch(int type, bool pair, const dq::TreeArgs& a, int blocks, cudaStream_t s);

}  // namespace dqhost
