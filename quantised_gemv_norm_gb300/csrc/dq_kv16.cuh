// dq_kv16.cuh -- the paged 16-bit cache (include/dq.h defines the layout): what its
// store, its row moves and its attention share.
#pragma once

#include "dq_attn.cuh"
#include "dq_types.cuh"

namespace dq {

constexpr int KV16_ROWS = 16;  // a page is a multiple of this many rows

struct Kv16Shape {
    int n_kv, n_pages, page_rows;
};

// Row 0 of a page's keys (which = 0) or values (1) of one head, in rows of 128 from the
// pool's start.
__device__ __forceinline__ long long kv16_row(const Kv16Shape& s, int page, int which, int g)
{
    return ((2ll * page + which) * s.n_kv + g) * s.page_rows;
}

}  // namespace dq

namespace dqhost {

// The checks that the 16-bit cache's entry points share.  Rows of the pool are counted in
// 31 bits (a tensor map's coordinate).
inline int kv16_check_shape(int type, int n_kv, int head_dim, int n_pages, int page_size)
{
    if (n_kv < 1 || n_pages < 1 || page_size < dq::KV16_ROWS || page_size % dq::KV16_ROWS ||
        (type != DQ_TYPE_F16 && type != DQ_TYPE_BF16))
        return DQ_ERR_SHAPE;
    if (head_dim != dq::ATT_HD || n_kv > (1 << 16) || static_cast<long long>(n_pages) * page_size > 0x7fffffffll ||
        static_cast<long long>(n_pages) * page_size * 2 * n_kv > 0x7fffffffll)
        return DQ_ERR_UNSUPPORTED;
    return DQ_OK;
}

// f(pointer of the type) for one of the two 16-bit types.
template <typename F>
cudaError_t with_type16(int type, F f)
{
    if (type == DQ_TYPE_F16)
        return f(static_cast<__half*>(nullptr));
    return f(static_cast<__nv_bfloat16*>(nullptr));
}

}  // namespace dqhost
