// dq_kv4.cuh -- the 4-bit cache's block: places of codes and scales
// (include/dq.h defines the layout), shared by its store, read and attention.
#pragma once

#include "dq_attn.cuh"
#include "dq_types.cuh"

namespace dq {

constexpr int KV4_ROWS = DQ_KV4_BLOCK_ROWS;
constexpr int KV4_BYTES = DQ_KV4_BLOCK_BYTES;
constexpr int KV4_VCODES = 1024, KV4_KSCALES = 2048, KV4_VSCALES = 2304;

// Byte offset of the 32-bit word with the 8 key codes of row j, dims 32 g + 8 t ...
__device__ __forceinline__ int kv4_key_word(int j, int t, int g) { return 64 * j + 4 * (4 * t + g); }
// Byte offset of the 16-bit half with the 4 value codes of row j, dims 32 g + 8 t ...
// (r = 2 t); the half of the next 4 dims is 64 bytes further.
__device__ __forceinline__ int kv4_value_half(int j, int t, int g)
{
    return KV4_VCODES + 512 * (j >> 3) + 16 * (8 * t + ((j >> 1) & 3)) + 4 * g + 2 * (j & 1);
}
// Byte offset of row j's d for dims 32 g ...; z is 4 bytes further.
__device__ __forceinline__ int kv4_scale(int base, int j, int g) { return base + 32 * (j >> 1) + 8 * g + 2 * (j & 1); }

struct Kv4Shape {
    int n_kv, n_pages, page_rows;  // page_rows: rows a page, a multiple of 16
};

}  // namespace dq

namespace dqhost {

// The checks that the 4-bit cache's entry points share.
inline int kv4_check_shape(int n_kv, int head_dim, int n_pages, int page_size)
{
    if (n_kv < 1 || n_pages < 1 || page_size < dq::KV4_ROWS || page_size % dq::KV4_ROWS)
        return DQ_ERR_SHAPE;
    if (head_dim != dq::ATT_HD || static_cast<long long>(n_pages) * page_size > 0x7fffffffll || n_kv > (1 << 16))
        return DQ_ERR_UNSUPPORTED;
    return DQ_OK;
}

}  // namespace dqhost
