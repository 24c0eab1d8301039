// paged.cuh -- the paged coded cache on the device: its record and the
// host-side conversion (include/hqmq.h, hqmq_kv_pages).
#pragma once

#include "hqmq_device.cuh"

namespace hqmq {

constexpr int PG_CHUNKS = 32;                 // chunks of a token of a head (D = 128)
constexpr uint32_t PG_MAX_S = 48;             // 24 S ids fit 12 bits; tables fit shared memory

struct PagesDev {
    uint32_t *words;
    uint16_t *radius;
    uint32_t *flags;                          // NULL: no outliers
    uint16_t *val;
    const float4 *cb;
    const float *thr;
    const uint4 *table;
    uint32_t S, b;
    int n_pages, page_size, page_shift, heads, cap;

    // flat index of row `row` of (page, head): words at * b, radii at * 32, flags at * 1
    __device__ __forceinline__ size_t at(int page, int head, int row) const {
        return ((size_t)page * heads + head) * page_size + row;
    }
    __device__ __forceinline__ uint2 *slots(int page, int head) const {
        return reinterpret_cast<uint2 *>(val) + ((size_t)page * heads + head) * cap;
    }
};

inline PagesDev pages_dev(const hqmq_kv_pages *p, uint32_t b) {
    PagesDev d;
    d.words = p->idx_words;
    d.radius = p->radius;
    d.flags = p->flags;
    d.val = p->out_val;
    d.cb = reinterpret_cast<const float4 *>(p->codebook);
    d.thr = p->thr;
    d.table = reinterpret_cast<const uint4 *>(p->table);
    d.S = p->S;
    d.b = b;
    d.n_pages = p->n_pages;
    d.page_size = p->page_size;
    d.page_shift = 0;
    while ((1 << d.page_shift) < p->page_size) ++d.page_shift;
    d.heads = p->heads;
    d.cap = p->flags ? p->out_cap : 0;
    return d;
}

// Flagged chunks in rows [0, row) of a (page, head): one warp, all lanes get
// the sum.
__device__ __forceinline__ uint32_t flags_before(const uint32_t *f, int row, int lane) {
    uint32_t n = 0;
    for (int u = lane; u < row; u += 32) n += __popc(f[u]);
    return __reduce_add_sync(FULL, n);
}

}  // namespace hqmq
