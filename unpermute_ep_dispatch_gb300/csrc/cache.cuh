// cache.cuh -- the paged key-value cache as its writer and its reader see it.
#pragma once

#include "epd_math.cuh"

namespace epd {

constexpr int kMaxHeadDim = 256;

// t / d for t < 2^31 by a product: mul = ceil(2^(31 + shift) / d), 2^shift >= d.
struct Divisor {
    uint32_t mul, shift, d;
};
inline Divisor divisor(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return {(uint32_t)(((1ull << (31 + s)) + d - 1) / d), s, d};
}
__device__ __forceinline__ uint32_t divide(uint32_t t, const Divisor &v) { return __umulhi(2 * t, v.mul) >> v.shift; }

// The largest number of positions that a sequence's pages hold.
__host__ __device__ inline int64_t cache_positions(const epd_cache_t &c) { return (int64_t)c.max_pages * c.page_size; }

inline epd_status_t check_cache(const epd_cache_t *c) {
    if (!c || (c->dtype != EPD_BF16 && c->dtype != EPD_FP8_E4M3)) return EPD_ERR_INVALID_ARG;
    const bool fp8 = c->dtype == EPD_FP8_E4M3;
    const int unit = fp8 ? 16 : 8;  // elements of 16 bytes
    if (c->num_kv_heads < 1 || c->head_dim < unit || c->head_dim % unit || c->page_size < 1) return EPD_ERR_INVALID_ARG;
    if (c->num_pages < 0 || c->num_pages > INT32_MAX || c->num_seqs < 0 || c->max_pages < 0) return EPD_ERR_INVALID_ARG;
    if (cache_positions(*c) > INT32_MAX || (c->table_stride != 0 && c->table_stride < c->max_pages)) return EPD_ERR_INVALID_ARG;
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

// Whether every position and head of the cache is one of its own, as its writer needs it (the reader
// takes rows that several share).
inline bool rows_apart(const epd_cache_t &c) {
    const bool fp8 = c.dtype == EPD_FP8_E4M3;
    auto apart = [&](int64_t n, int64_t stride, int64_t scale_stride) { return n <= 1 || (stride > 0 && (!fp8 || scale_stride > 0)); };
    return apart(c.num_pages, c.page_stride, c.scale_page_stride) && apart(c.page_size, c.token_stride, c.scale_token_stride) &&
           apart(c.num_kv_heads, c.head_stride, c.scale_head_stride);
}

}  // namespace epd
