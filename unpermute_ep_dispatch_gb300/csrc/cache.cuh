// cache.cuh -- the paged key-value cache as its writer and its reader see it.
#pragma once

#include "epd_math.cuh"

namespace epd {

constexpr int kMaxHeadDim = 256;

// The largest number of positions that a sequence's pages hold.
__host__ __device__ inline int64_t cache_positions(const epd_cache_t &c) { return (int64_t)c.max_pages * c.page_size; }

inline epd_status_t check_cache(const epd_cache_t *c) {
    if (!c || (c->dtype != EPD_BF16 && c->dtype != EPD_FP8_E4M3)) return EPD_ERR_INVALID_ARG;
    const bool fp8 = c->dtype == EPD_FP8_E4M3;
    const int unit = fp8 ? 16 : 8;  // elements of 16 bytes
    if (c->num_kv_heads < 1 || c->head_dim < unit || c->head_dim % unit || c->page_size < 1) return EPD_ERR_INVALID_ARG;
    if (c->num_pages < 0 || c->num_pages > INT32_MAX || c->num_seqs < 0 || c->max_pages < 0) return EPD_ERR_INVALID_ARG;
    if (cache_positions(*c) > INT32_MAX || c->table_stride < c->max_pages) return EPD_ERR_INVALID_ARG;
    if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0 || c->page_stride % unit ||
        c->token_stride % unit || c->head_stride % unit)
        return EPD_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->k_scale) || !aligned4(c->v_scale) ||
        !aligned4(c->page_table))
        return EPD_ERR_INVALID_ARG;
    if (c->num_pages > 0 && (!c->k || !c->v || (fp8 && (!c->k_scale || !c->v_scale)))) return EPD_ERR_INVALID_ARG;
    if (!fp8 && (c->k_scale || c->v_scale)) return EPD_ERR_INVALID_ARG;
    if (c->num_seqs > 0 && c->max_pages > 0 && !c->page_table) return EPD_ERR_INVALID_ARG;
    if (c->head_dim > kMaxHeadDim) return EPD_ERR_UNSUPPORTED;
    return EPD_OK;
}

}  // namespace epd
