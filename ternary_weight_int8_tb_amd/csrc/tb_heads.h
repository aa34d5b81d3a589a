// tb_heads.h -- argument checks of the calls around the paged cache (host code).
#pragma once

#include "tb_host.h"

namespace tbh {

// bytes from the first to the last element of `rows` rows of heads; 0 for strides or a type that are refused
inline size_t heads_bytes(const tb_heads &h, long long rows, int dim)
{
    const size_t eb = dtype_bytes(h.dtype);
    const long long rs = rows > 1 ? h.row_stride : 0, hs = h.heads > 1 ? h.head_stride : 0;
    // so far apart, the last element lies past any address
    constexpr long long kFar = 1ll << 56;
    if (!eb || h.heads < 1 || h.heads > 65536 || rs < 0 || hs < 0 || rs % 8 || hs % 8 || rs > kFar / rows || hs > kFar / h.heads)
        return 0;
    return (size_t)((rows - 1) * rs + (h.heads - 1) * hs + dim) * eb;
}

inline bool page_ok(int page) { return page >= 16 && page <= 256 && (page & (page - 1)) == 0; }

inline bool cache_ok(const tb_kv_cache &c)
{
    return c.pages >= 1 && c.kv_heads >= 1 && c.kv_heads <= 65536 && page_ok(c.page) && (long long)c.pages * c.page < (1ll << 31) && c.dim >= 16 && c.dim <= 512 &&
           c.dim % 16 == 0 && (c.dtype == TB_BF16 || c.dtype == TB_F16);
}
// bytes of each of its two arrays
inline size_t cache_bytes(const tb_kv_cache &c) { return (size_t)c.pages * c.page * c.dim * 2 * (size_t)c.kv_heads; }

inline int log2_of(int page) { return page <= 16 ? 4 : page <= 32 ? 5 : page <= 64 ? 6 : page <= 128 ? 7 : 8; }

}  // namespace tbh
