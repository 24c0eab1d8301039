// paged_read.cu -- the dense K or V of a paged cache's tokens
// (include/hqmq.h, hqmq_paged_read).
//
// A CTA takes up to 256 tokens of one sequence and head: the head's codewords
// go to shared memory, the tokens' flag words become slots (a scan that starts
// anew with every page), then each warp decodes its tokens, a lane two chunks
// (bf16) or one (fp32), so that every store is 16 bytes and a token's row is
// contiguous.  A token's addresses are worked out once, by the thread that
// looked its page up, and the loads of four steps are issued without a branch
// before the first is used.  32768 tokens of 8 heads, S = 32, to bf16 (97 MB)
// take 26.7 us, 3.6 TB/s (to fp32, 164 MB, 39.4 us; 131072 tokens 99 and 134 us,
// 3.9 and 4.9 TB/s): half the rate of a copy and more.  The chain length -> page
// -> flags -> codes of a CTA's start and the shared-memory pipe (a codeword per
// chunk, with bank conflicts) share the rest; other numbers of table copies
// (4: 32 us, they take L1's room; 1: 26.7), eight steps in flight (30) and CTAs
// that stay for several rounds (27) gained nothing.
#include <type_traits>

#include "paged.cuh"

namespace hqmq {

constexpr int PR_WARPS = 8;
constexpr int PR_THREADS = PR_WARPS * 32;
constexpr int PR_COPIES = 2;                  // of the codeword table

struct ReadArgs {
    PagesDev p;
    const int *len, *table;
    int max_pages, T, span;                   // span: tokens of a CTA, 32 .. 256
    void *y;
    DevStatus *st;
};

// A token, ready for its decoders: no address arithmetic is left to them.
struct __align__(16) ReadTok {
    const uint32_t *words;                    // (of some row, if this one is left alone)
    const uint16_t *radius;
    const uint2 *val;                         // its first value
    uint32_t flags;
    int left;                                 // slots of the page from there; < 0: the row is left alone
};

__device__ __forceinline__ float4 half4(uint2 h) {
    return make_float4(f16_bits_to_f32(h.x & 0xFFFFu), f16_bits_to_f32(h.x >> 16), f16_bits_to_f32(h.y & 0xFFFFu),
                       f16_bits_to_f32(h.y >> 16));
}

// CPL: chunks a lane takes (2: bf16, 1: fp32); a warp's step covers CPL tokens.
// (Index widths known to the compiler gain nothing: 26.9 us.)
template <int CPL> __global__ void __launch_bounds__(PR_THREADS, 4) k_paged_read(ReadArgs a) {
    extern __shared__ float4 s_tab[];         // [24 S + 1][PR_COPIES]
    __shared__ ReadTok s_tok[PR_THREADS];
    __shared__ uint32_t s_sum[PR_WARPS];
    pdl_wait();
    pdl_trigger();
    const PagesDev &p = a.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = blockIdx.y, seq = blockIdx.z, t0 = blockIdx.x * a.span;
    const int n = min(min(a.len[seq], a.T) - t0, a.span);
    if (n <= 0) return;

    // this thread's token: its page, flags and the slot of its first value
    const int me = t0 + threadIdx.x;
    ReadTok tok = {p.words, p.radius, nullptr, 0u, -1};
    int page = -1;
    if ((int)threadIdx.x < n) {
        const int col = me >> p.page_shift;
        page = col < a.max_pages ? a.table[(size_t)seq * a.max_pages + col] : -1;
        if (page < 0 || page >= p.n_pages) {
            page = -1;
            if (a.st) atomicOr(&a.st->flags, HQMQ_FLAG_BAD_PAGE);
        }
    }
    const int row = me & (p.page_size - 1);
    if (page >= 0) {
        const size_t at = p.at(page, head, row);
        tok.words = p.words + at * p.b;
        tok.radius = p.radius + at * PG_CHUNKS;
        tok.left = 0;
    }
    if (p.flags) {
        uint32_t before = 0;                  // flagged chunks in the rows of the first page before t0
        if (page >= 0) tok.flags = p.flags[p.at(page, head, row)];
        const int row0 = t0 & (p.page_size - 1);
        if (row0 > 0) {
            const int col = t0 >> p.page_shift;
            const int pg = col < a.max_pages ? a.table[(size_t)seq * a.max_pages + col] : -1;
            if (pg >= 0 && pg < p.n_pages) before = flags_before(p.flags + p.at(pg, head, 0), row0, lane);
        }
        const uint32_t c = __popc(tok.flags);
        uint32_t inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) s_sum[warp] = inc;
        // sums of the page's earlier rows: within the warp, then of the warps between
        uint32_t start = inc - c;
        const int first = (int)threadIdx.x - row;          // the thread of the page's row 0 (< 0: before t0)
        const int from = max(first, warp * 32) - warp * 32;  // its lane, if it is in this warp
        start -= __shfl_sync(FULL, inc - c, from & 31);
        __syncthreads();
        for (int w = max(first, 0) >> 5; w < warp; ++w) start += s_sum[w];
        if (first < 0) start += before;
        if (page >= 0) {
            tok.left = max(p.cap - (int)start, 0);
            tok.val = reinterpret_cast<const uint2 *>(p.slots(page, head)) + start;
        }
    }
    s_tok[threadIdx.x] = tok;
    const uint32_t words = 24u * p.S;
    for (uint32_t e = threadIdx.x; e <= words; e += PR_THREADS) {
        float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < words) c = codeword((int)(e % 24u), __ldg(p.cb + (size_t)head * p.S + e / 24u));
#pragma unroll
        for (int r = 0; r < PR_COPIES; ++r) s_tab[e * PR_COPIES + ((r + e) & (PR_COPIES - 1))] = c;
    }
    __syncthreads();

    constexpr int STEPS = 4;                  // loads in flight: STEPS tokens a lane
    const uint32_t b = p.b;
    const int sub = CPL == 2 ? lane >> 4 : 0, c0 = CPL == 2 ? 2 * (lane & 15) : lane;
    const uint32_t bit = (uint32_t)c0 * b, wi = bit >> 5, sh = bit & 31u, mask = (1u << b) - 1u;
    const bool two = wi + 1 < b;              // (CPL b bits lie in one or two words: b <= 11)
    const uint32_t below = (1u << c0) - 1u;
    const float4 *tab = s_tab + (lane & (PR_COPIES - 1));
    using Out = typename std::conditional<CPL == 2, uint16_t, float>::type;
    Out *const y0 = reinterpret_cast<Out *>(a.y) + (((size_t)seq * p.heads + head) * a.T + t0 + sub) * 128 + 4 * c0;
    bool bad = false;
    for (int i0 = warp * STEPS * CPL; i0 < n; i0 += PR_WARPS * STEPS * CPL) {
        uint32_t lo[STEPS], hi[STEPS], rad[STEPS], own[STEPS];       // own: which of the lane's chunks have values
        uint2 val[STEPS];                     // the first of them
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const ReadTok &k = s_tok[i0 + s * CPL + sub];
            const uint32_t *w = k.words + wi;
            lo[s] = __ldcs(w);
            hi[s] = two ? __ldcs(w + 1) : 0u;
            if (CPL == 2) rad[s] = __ldcs(reinterpret_cast<const uint32_t *>(k.radius + c0));
            else rad[s] = __ldcs(k.radius + c0);
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const ReadTok &k = s_tok[i0 + s * CPL + sub];
            const uint32_t flags = k.flags;
            const int room = k.left - __popc(flags & below);         // slots from the lane's first value
            own[s] = room <= 0 ? 0u : (flags >> c0) & (CPL == 2 ? 3u : 1u);
            if (CPL == 2 && room == 1 && own[s] == 3u) own[s] = 1u;
            if (own[s]) val[s] = __ldcs(k.val + __popc(flags & below));
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            if (s_tok[i0 + s * CPL + sub].left < 0) continue;
            const uint32_t v = __funnelshift_r(lo[s], hi[s], sh);
            float4 y[CPL];
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const uint32_t idx = (v >> (c * b)) & mask;
                const float r = f16_bits_to_f32(c ? rad[s] >> 16 : rad[s] & 0xFFFFu);
                const float4 w = tab[min(idx, words) * PR_COPIES];
                y[c] = make_float4(__fmul_rn(r, w.x), __fmul_rn(r, w.y), __fmul_rn(r, w.z), __fmul_rn(r, w.w));
                if (idx >= words) {           // (not r 0: r may be infinite)
                    y[c] = w;
                    bad = true;
                }
            }
            if (own[s]) {
                y[CPL == 2 && own[s] == 2u ? CPL - 1 : 0] = half4(val[s]);
                if (CPL == 2 && own[s] == 3u) {
                    const ReadTok &k = s_tok[i0 + s * CPL + sub];
                    y[CPL - 1] = half4(__ldcs(k.val + __popc(k.flags & below) + 1));
                }
            }
            Out *const out = y0 + (i0 + s * CPL) * 128;
            if (CPL == 2) {
                uint32_t h[4];
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    const __nv_bfloat162 p0 = __floats2bfloat162_rn(y[c].x, y[c].y),
                                         p1 = __floats2bfloat162_rn(y[c].z, y[c].w);
                    h[2 * c] = *reinterpret_cast<const uint32_t *>(&p0);
                    h[2 * c + 1] = *reinterpret_cast<const uint32_t *>(&p1);
                }
                *reinterpret_cast<uint4 *>(out) = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
                *reinterpret_cast<float4 *>(out) = y[0];
            }
        }
    }
    if (bad && a.st) atomicOr(&a.st->flags, HQMQ_FLAG_BAD_INDEX);
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
    // 256 tokens a CTA, so that its codeword table is a small part of the work (32768 tokens, 8 heads, S = 32:
    // 27 us, with 32 tokens 63), fewer where that would leave SMs idle (5 sequences of 203 tokens, 4 heads: 3.6
    // us, with 256 tokens 6.6)
    a.span = 256;
    while (a.span > 32 && (int64_t)((T + a.span - 1) / a.span) * c->heads * n_seqs < 2 * 148) a.span /= 2;
    const size_t smem = (size_t)(24 * c->S + 1) * PR_COPIES * sizeof(float4);
    auto kern = out_dtype == HQMQ_BF16 ? k_paged_read<2> : k_paged_read<1>;
    const dim3 grid((unsigned)((T + a.span - 1) / a.span), (unsigned)c->heads, (unsigned)n_seqs);
    return launch_pdl(kern, grid, dim3(PR_THREADS), smem, stream, a) == cudaSuccess ? HQMQ_OK : HQMQ_ERR_CUDA;
}
