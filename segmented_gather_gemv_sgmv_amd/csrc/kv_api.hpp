// kv_api.hpp -- checks of a cache that its entry points and attention's share.
#pragma once

#include "kv_format.hpp"

namespace sgmv {

inline int kv_check_sizes(int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                          int32_t kind) {
    if (num_pages < 1 || page_size < kKvBlock || page_size % kKvBlock || kv_heads < 1 || head_dim < 1 ||
        (kind != SGMV_KV_FP8 && kind != SGMV_KV_FP4))
        return SGMV_ERR_BAD_SHAPE;
    // Heads are a grid's second dimension; blocks of 16 tokens are counted in 31 bits.
    if (head_dim > kKvMaxDim || kv_heads > 65535 ||
        (long long)num_pages * (page_size / kKvBlock) > 0x7FFFFFFFll)
        return SGMV_ERR_UNSUPPORTED;
    return SGMV_OK;
}

inline int kv_check(const sgmv_kv_cache* c) {
    if (!c) return SGMV_ERR_NULL_PTR;
    if (const int e = kv_check_sizes(c->num_pages, c->page_size, c->kv_heads, c->head_dim, c->kind))
        return e;
    if (!c->k || !c->v || !c->k_scales || !c->v_scales) return SGMV_ERR_NULL_PTR;
    if ((((uintptr_t)c->k | (uintptr_t)c->v | (uintptr_t)c->k_scales | (uintptr_t)c->v_scales) & 15u) != 0)
        return SGMV_ERR_UNSUPPORTED;
    return SGMV_OK;
}

}  // namespace sgmv
