// paged_read.cu -- the dense K or V of a paged cache's tokens
// (include/hqmq.h, hqmq_paged_read).
#include "paged.cuh"

namespace hqmq {

constexpr int PR_WARPS = 8;

struct ReadArgs {
    PagesDev p;
    const int *len, *table;
    int max_pages, T;
    void *y;
    DevStatus *st;
};

__device__ __forceinline__ void store_chunk(float *y, float4 v) {
    *reinterpret_cast<float4 *>(y) = v;
}
__device__ __forceinline__ void store_chunk(__nv_bfloat16 *y, float4 v) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(y) = make_uint2(*reinterpret_cast<uint32_t *>(&a),
                                               *reinterpret_cast<uint32_t *>(&b));
}

// A warp takes one token of one head, a lane one chunk.
template <typename E> __global__ void __launch_bounds__(PR_WARPS * 32) k_paged_read(ReadArgs a) {
    pdl_wait();
    const PagesDev &p = a.p;
    const int lane = threadIdx.x & 31;
    const int head = blockIdx.y, seq = blockIdx.z;
    const int t = blockIdx.x * PR_WARPS + (threadIdx.x >> 5);
    if (t >= min(a.len[seq], a.T)) return;
    const int col = t >> p.page_shift, row = t & (p.page_size - 1);
    const int page = col < a.max_pages ? a.table[(size_t)seq * a.max_pages + col] : -1;
    if (page < 0 || page >= p.n_pages) {
        if (lane == 0 && a.st) atomicOr(&a.st->flags, HQMQ_FLAG_BAD_PAGE);
        return;
    }
    const size_t at = p.at(page, head, row);
    const uint32_t idx = token_index(p.words + at * p.b, p.b, lane);
    const float r = f16_bits_to_f32(p.radius[at * PG_CHUNKS + lane]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (idx < 24u * p.S) {
        const float4 c = codeword((int)(idx % 24u), __ldg(p.cb + (size_t)head * p.S + idx / 24u));
        v = make_float4(__fmul_rn(r, c.x), __fmul_rn(r, c.y), __fmul_rn(r, c.z), __fmul_rn(r, c.w));
    } else if (a.st) {
        atomicOr(&a.st->flags, HQMQ_FLAG_BAD_INDEX);
    }
    if (p.flags) {
        const uint32_t f = p.flags[at];
        const uint32_t slot = flags_before(p.flags + at - row, row, lane) + __popc(f & ((1u << lane) - 1u));
        if (((f >> lane) & 1u) && slot < (uint32_t)p.cap) {
            const uint2 h = p.slots(page, head)[slot];
            v = make_float4(f16_bits_to_f32(h.x & 0xFFFFu), f16_bits_to_f32(h.x >> 16),
                            f16_bits_to_f32(h.y & 0xFFFFu), f16_bits_to_f32(h.y >> 16));
        }
    }
    E *y = reinterpret_cast<E *>(a.y) + (((size_t)seq * p.heads + head) * a.T + t) * 128 + 4 * lane;
    store_chunk(y, v);
}

}  // namespace hqmq

extern "C" int hqmq_launch_paged_read(const hqmq_kv_pages *c, uint32_t b, int n_seqs,
                                      const int32_t *len, const int32_t *table, int max_pages, int T,
                                      void *y, int out_dtype, hqmq_status *st, cudaStream_t stream) {
    using namespace hqmq;
    ReadArgs a;
    a.p = pages_dev(c, b);
    a.len = len;
    a.table = table;
    a.max_pages = max_pages;
    a.T = T;
    a.y = y;
    a.st = reinterpret_cast<DevStatus *>(st);
    const dim3 grid((unsigned)((T + PR_WARPS - 1) / PR_WARPS), (unsigned)c->heads, (unsigned)n_seqs);
    const cudaError_t e = out_dtype == HQMQ_BF16
        ? launch_pdl(k_paged_read<__nv_bfloat16>, grid, dim3(PR_WARPS * 32), 0, stream, a)
        : launch_pdl(k_paged_read<float>, grid, dim3(PR_WARPS * 32), 0, stream, a);
    return e == cudaSuccess ? HQMQ_OK : HQMQ_ERR_CUDA;
}
