// paged_attention.cu -- decode-phase attention over paged coded caches with a
// prefix shared by the whole batch (include/hqmq.h, hqmq_attention_paged).
//
//   o = sum_t softmax_t(scale <q, K^_t>) V^_t
// over the prefix's tokens and the sequence's own.  The token ranges are
// split; each part gives its rows' running maximum m (base 2), sum l and
// unnormalised output, which a last kernel joins:
//   M = max m_i,  o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// The prefix's parts take all B G rows of a KV head, so its codes are
// decoded once per part for every sequence.
#include "paged.cuh"

namespace hqmq {

constexpr int PA_D = 128;
constexpr int PA_PART = PA_D + 2;             // floats of a partial result: m, l, O[D]
constexpr int PA_SMS = 148;                   // the split of the token ranges aims at one B200

struct AttnPlan {
    int prefix_parts, prefix_len;             // parts of the prefix and tokens in each
    int own_parts, own_len;                   // the same for the sequences' own tokens
};

constexpr int PA_ROWS = 64;                   // rows of a prefix CTA
constexpr int PA_TILE = 32;                   // tokens decoded at a time
constexpr int PA_MIN_PART = 256;              // fewest tokens worth a part of their own

inline void split_range(int tokens, int64_t ctas_per_part, int &parts, int &len) {
    parts = 0;
    len = 0;
    if (tokens <= 0) return;
    int64_t want = (2 * PA_SMS + ctas_per_part - 1) / ctas_per_part;
    const int64_t most = ((int64_t)tokens + PA_MIN_PART - 1) / PA_MIN_PART;
    if (want > most) want = most;
    if (want < 1) want = 1;
    len = (int)(((tokens + want - 1) / want + PA_TILE - 1) / PA_TILE * PA_TILE);
    parts = (tokens + len - 1) / len;
}

inline AttnPlan attn_plan_paged(int B, int Hq, int Hk, int max_tokens, int prefix_len) {
    AttnPlan p;
    const int64_t rows = (int64_t)B * (Hq / Hk);
    split_range(prefix_len, Hk * ((rows + PA_ROWS - 1) / PA_ROWS), p.prefix_parts, p.prefix_len);
    split_range(max_tokens, (int64_t)Hk * B, p.own_parts, p.own_len);
    return p;
}

struct PagedAttnArgs {
    const uint16_t *q;
    PagesDev k, v;
    int B, Hk, G;
    const int *seq_len, *table, *prefix_table;
    int max_pages, prefix_len;
    AttnPlan plan;
    float sl2;
    float *part;                              // [B Hq][prefix_parts + own_parts][PA_PART]
    DevStatus *st;
};

// One chunk of a token as bf16 values.
__device__ __forceinline__ float4 chunk_value(const PagesDev &p, int page, int head, int row,
                                              uint32_t before, int c) {
    const size_t at = p.at(page, head, row);
    const uint32_t idx = token_index(p.words + at * p.b, p.b, c);
    const float r = f16_bits_to_f32(p.radius[at * PG_CHUNKS + c]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (idx < 24u * p.S) {
        const float4 w = codeword((int)(idx % 24u), __ldg(p.cb + (size_t)head * p.S + idx / 24u));
        v = make_float4(__fmul_rn(r, w.x), __fmul_rn(r, w.y), __fmul_rn(r, w.z), __fmul_rn(r, w.w));
    }
    if (p.flags) {
        const uint32_t f = p.flags[at];
        const uint32_t slot = before + __popc(f & ((1u << c) - 1u));
        if (((f >> c) & 1u) && slot < (uint32_t)p.cap) {
            const uint2 h = p.slots(page, head)[slot];
            v = make_float4(f16_bits_to_f32(h.x & 0xFFFFu), f16_bits_to_f32(h.x >> 16),
                            f16_bits_to_f32(h.y & 0xFFFFu), f16_bits_to_f32(h.y >> 16));
        }
    }
    v.x = __bfloat162float(__float2bfloat16_rn(v.x));
    v.y = __bfloat162float(__float2bfloat16_rn(v.y));
    v.z = __bfloat162float(__float2bfloat16_rn(v.z));
    v.w = __bfloat162float(__float2bfloat16_rn(v.w));
    return v;
}

// 4 warps; a warp takes every fourth row, a lane one token of the tile for
// the scores and four dimensions for the output.
template <bool PREFIX>
__global__ void __launch_bounds__(128) k_paged_attn(PagedAttnArgs a) {
    constexpr int RW = PREFIX ? PA_ROWS / 4 : 4;
    __shared__ float s_k[PA_TILE][PA_D + 1];
    __shared__ float4 s_v[PA_TILE][PA_D / 4];
    __shared__ int s_ok[PA_TILE];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int split = blockIdx.x, hk = blockIdx.y;
    const int rows = PREFIX ? a.B * a.G : a.G, row0 = PREFIX ? (int)blockIdx.z * PA_ROWS : 0;
    const int nparts = a.plan.prefix_parts + a.plan.own_parts;
    const int *table = PREFIX ? a.prefix_table : a.table + (size_t)blockIdx.z * a.max_pages;
    const int cap = PREFIX ? a.prefix_len : a.max_pages << a.k.page_shift;
    const int len = PREFIX ? a.prefix_len : min(max(a.seq_len[blockIdx.z], 0), cap);
    const int plen = PREFIX ? a.plan.prefix_len : a.plan.own_len;
    const int t_end = (int)min((int64_t)len, (int64_t)(split + 1) * plen);
    float m[RW], l[RW];
    float4 o[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int t0 = split * plen; t0 < t_end; t0 += PA_TILE) {
        __syncthreads();
        for (int i = warp; i < PA_TILE; i += 4) {
            const int t = t0 + i;
            int page = -1;
            if (t < t_end) {
                page = table[t >> a.k.page_shift];
                if (page < 0 || page >= a.k.n_pages || page >= a.v.n_pages) {
                    page = -1;
                    if (lane == 0 && a.st) atomicOr(&a.st->flags, HQMQ_FLAG_BAD_PAGE);
                }
            }
            float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
            if (page >= 0) {
                const int row = t & (a.k.page_size - 1);
                const size_t f0 = a.k.at(page, hk, 0);
                const uint32_t kb = a.k.flags ? flags_before(a.k.flags + f0, row, lane) : 0u;
                const uint32_t vb = a.v.flags ? flags_before(a.v.flags + f0, row, lane) : 0u;
                kv = chunk_value(a.k, page, hk, row, kb, lane);
                vv = chunk_value(a.v, page, hk, row, vb, lane);
            }
            s_k[i][4 * lane] = kv.x;
            s_k[i][4 * lane + 1] = kv.y;
            s_k[i][4 * lane + 2] = kv.z;
            s_k[i][4 * lane + 3] = kv.w;
            s_v[i][lane] = vv;
            if (lane == 0) s_ok[i] = page >= 0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int r = row0 + warp + 4 * i;
            if (r >= rows) continue;
            const int b = PREFIX ? r / a.G : (int)blockIdx.z, g = PREFIX ? r % a.G : r;
            const uint32_t *q = reinterpret_cast<const uint32_t *>(a.q) +
                                ((size_t)b * a.Hk * a.G + hk * a.G + g) * (PA_D / 2);
            float s = 0.f;
            for (int d = 0; d < PA_D / 2; ++d) {
                const uint32_t w = __ldg(q + d);
                s = fmaf(__uint_as_float(w << 16), s_k[lane][2 * d], s);
                s = fmaf(__uint_as_float(w & 0xFFFF0000u), s_k[lane][2 * d + 1], s);
            }
            s = s_ok[lane] ? s * a.sl2 : -INFINITY;
            float mt = s;
#pragma unroll
            for (int k = 16; k; k >>= 1) mt = fmaxf(mt, __shfl_xor_sync(FULL, mt, k));
            const float mn = fmaxf(m[i], mt);
            if (mn == -INFINITY) continue;
            const float f = exp2f(m[i] - mn), pr = s_ok[lane] ? exp2f(s - mn) : 0.f;
            float sum = pr;
#pragma unroll
            for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(FULL, sum, k);
            l[i] = l[i] * f + sum;
            m[i] = mn;
            o[i].x *= f; o[i].y *= f; o[i].z *= f; o[i].w *= f;
            for (int t = 0; t < PA_TILE; ++t) {
                const float pt = __shfl_sync(FULL, pr, t);
                const float4 v = s_v[t][lane];
                o[i].x = fmaf(pt, v.x, o[i].x);
                o[i].y = fmaf(pt, v.y, o[i].y);
                o[i].z = fmaf(pt, v.z, o[i].z);
                o[i].w = fmaf(pt, v.w, o[i].w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int r = row0 + warp + 4 * i;
        if (r >= rows) continue;
        const int b = PREFIX ? r / a.G : (int)blockIdx.z, g = PREFIX ? r % a.G : r;
        float *p = a.part + (((size_t)b * a.Hk * a.G + hk * a.G + g) * nparts +
                             (PREFIX ? split : a.plan.prefix_parts + split)) * PA_PART;
        if (lane == 0) {
            p[0] = m[i];
            p[1] = l[i];
        }
        p[2 + 4 * lane] = o[i].x;
        p[3 + 4 * lane] = o[i].y;
        p[4 + 4 * lane] = o[i].z;
        p[5 + 4 * lane] = o[i].w;
    }
}

// Joins a row's parts; one warp per row.
__global__ void __launch_bounds__(128)
k_paged_join(const float *part, int rows, int nparts, void *o, int out_dtype, float *lse) {
    pdl_wait();
    const int lane = threadIdx.x & 31, row = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const float *p = part + (size_t)row * nparts * PA_PART;
    float m = -INFINITY;
    for (int i = lane; i < nparts; i += 32) m = fmaxf(m, p[(size_t)i * PA_PART]);
#pragma unroll
    for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, k));
    const float mu = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < nparts; ++i) {
        const float *pi = p + (size_t)i * PA_PART;
        if (pi[1] == 0.f) continue;                          // (no token)
        const float f = exp2f(pi[0] - mu);
        l += pi[1] * f;
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] += pi[2 + 4 * lane + k] * f;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float v = acc[k] * inv;
        const size_t at = (size_t)row * PA_D + 4 * lane + k;
        if (out_dtype == HQMQ_BF16) reinterpret_cast<__nv_bfloat16 *>(o)[at] = __float2bfloat16_rn(v);
        else reinterpret_cast<float *>(o)[at] = v;
    }
    if (lse && lane == 0) lse[row] = l == 0.f ? -INFINITY : (mu + log2f(l)) * 0.69314718056f;
}

}  // namespace hqmq

extern "C" uint64_t hqmq_paged_attn_workspace_bytes(int B, int Hq, int Hk, int max_tokens,
                                                    int prefix_len) {
    using namespace hqmq;
    const AttnPlan p = attn_plan_paged(B, Hq, Hk, max_tokens, prefix_len);
    const uint64_t n = (uint64_t)B * Hq * (p.prefix_parts + p.own_parts) * PA_PART * sizeof(float);
    return ((n + 255) & ~255ull) + 256;
}

extern "C" int hqmq_launch_attention_paged(const uint16_t *q, const hqmq_kv_pages *k,
                                           const hqmq_kv_pages *v, uint32_t bk, uint32_t bv, int B, int Hq,
                                           const int32_t *seq_len, const int32_t *table, int max_pages,
                                           const int32_t *prefix_table, int prefix_len, float scale,
                                           void *o, int out_dtype, float *lse, void *ws,
                                           hqmq_status *st, cudaStream_t stream) {
    using namespace hqmq;
    PagedAttnArgs a;
    a.q = q;
    a.k = pages_dev(k, bk);
    a.v = pages_dev(v, bv);
    a.B = B;
    a.Hk = k->heads;
    a.G = Hq / k->heads;
    a.seq_len = seq_len;
    a.table = table;
    a.prefix_table = prefix_table;
    a.max_pages = max_pages;
    a.prefix_len = prefix_len;
    a.plan = attn_plan_paged(B, Hq, k->heads, max_pages * k->page_size, prefix_len);
    a.sl2 = (float)((double)scale * 1.4426950408889634);
    a.part = reinterpret_cast<float *>(ws);
    a.st = reinterpret_cast<DevStatus *>(st);
    const int nparts = a.plan.prefix_parts + a.plan.own_parts, rows = B * Hq;
    cudaError_t e = cudaSuccess;
    if (a.plan.prefix_parts)
        e = launch_pdl(k_paged_attn<true>, dim3(a.plan.prefix_parts, a.Hk, (B * a.G + PA_ROWS - 1) / PA_ROWS),
                       dim3(128), 0, stream, a);
    if (e == cudaSuccess && a.plan.own_parts)
        e = launch_pdl(k_paged_attn<false>, dim3(a.plan.own_parts, a.Hk, B), dim3(128), 0, stream, a);
    if (e == cudaSuccess)
        e = launch_pdl(k_paged_join, dim3((rows + 3) / 4), dim3(128), 0, stream, (const float *)a.part, rows,
                       nparts, o, out_dtype, lse);
    return e == cudaSuccess ? HQMQ_OK : HQMQ_ERR_CUDA;
}
