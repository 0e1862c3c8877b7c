// kv_cache.cuh -- the paged NVFP4 cache as its kernels see it.
#pragma once

#include "common.cuh"

namespace nvfp4 {

// Codes [2][pages][kv_heads][page_size][dim / 2] and scale bytes [2][pages][kv_heads]
// [page_size][dim / 16], keys first: the tokens of one page and head lie together.
struct CacheView {
    uint8_t* q;
    uint8_t* sf;
    const float* amax;  // of the keys, of the values
    int64_t pages;
    int kv_heads;
    int page_shift;     // log2 of the page size
    int64_t half;       // tokens x heads of the keys: where the values begin
};

constexpr int kMinPage = 16, kMaxPage = 1024;

inline nvfp4_status check_cache(const nvfp4_kv_cache* c, CacheView* v)
{
    if (!c || !c->q || !c->sf || !c->amax) return NVFP4_ERR_INVALID_ARG;
    if (c->dim != 64 && c->dim != 128 && c->dim != 256) return NVFP4_ERR_SHAPE;
    if (c->page_size < kMinPage || c->page_size > kMaxPage || (c->page_size & (c->page_size - 1))) return NVFP4_ERR_SHAPE;
    // (pages and places in a table are 32-bit numbers; offsets into the cache are 64-bit)
    if (c->pages < 1 || c->pages > 0x7fffffffll || c->kv_heads < 1 || c->kv_heads > 1024) return NVFP4_ERR_SHAPE;
    if (off16(c->q) || off16(c->sf) || (reinterpret_cast<uintptr_t>(c->amax) & 3u)) return NVFP4_ERR_ALIGN;
    v->q = c->q, v->sf = c->sf, v->amax = c->amax, v->pages = c->pages, v->kv_heads = c->kv_heads;
    v->page_shift = 0;
    while ((1 << v->page_shift) < c->page_size) ++v->page_shift;
    v->half = c->pages * c->kv_heads * c->page_size;
    return NVFP4_OK;
}

}  // namespace nvfp4
