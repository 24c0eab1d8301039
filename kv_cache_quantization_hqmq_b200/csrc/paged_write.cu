// paged_write.cu -- quantising new K and V tokens straight into the pages of
// a paged cache (include/hqmq.h, hqmq_paged_write).
//
// A unit of work is the run of new tokens of one sequence that fall in one
// page, for one head of K or of V: one CTA.  Inside it the outlier slots
// follow from the page's flag words alone (the popcounts of the rows before),
// so no counter is stored, nothing depends on the order in which CTAs run,
// and a row can be written again.
#include "paged.cuh"

#include "search.cuh"

namespace hqmq {

constexpr int PW_WARPS = 8;
constexpr int PW_MAX_PAGE = 256;

struct WriteArgs {
    PagesDev p[2];
    const void *x[2];
    int64_t st[2], sh[2];
    int n_tokens, n_seqs, max_pages;
    const int *cu, *pos0, *table;
    DevStatus *st_out;
};

// A run of new tokens in one page.
struct Run {
    int token0, n;                            // rows of x
    int seq, col, row0;                       // block-table entry, first row in the page
    bool bad;                                 // the sequence's positions start below 0
};

__device__ __forceinline__ int clamp_tok(int v, int n) { return min(max(v, 0), n); }

// The run number `item` of the call, in sequence and page order; n = 0 if
// there are fewer.  Warp-collective.
__device__ __forceinline__ Run find_run(const WriteArgs &a, int item, int lane) {
    Run r = {0, 0, 0, 0, 0, false};
    const int shift = a.p[0].page_shift, P = a.p[0].page_size;
    int left = item;
    for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
        const int b = b0 + lane;
        int t0 = 0, n = 0, pos = 0;
        if (b < a.n_seqs) {
            t0 = clamp_tok(a.cu[b], a.n_tokens);
            n = max(clamp_tok(a.cu[b + 1], a.n_tokens) - t0, 0);
            pos = a.pos0[b];
        }
        // positions below 0 make one bad run of the whole sequence
        const bool bad = pos < 0;
        const int first = (bad ? 0 : pos) & (P - 1);
        int runs = n == 0 ? 0 : bad ? 1 : (int)(((int64_t)first + n - 1) >> shift) + 1;
        int inc = runs;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += u;
        }
        const unsigned hit = __ballot_sync(FULL, left < inc);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int k = left - __shfl_sync(FULL, inc - runs, src);
            t0 = __shfl_sync(FULL, t0, src);
            n = __shfl_sync(FULL, n, src);
            pos = __shfl_sync(FULL, pos, src);
            r.seq = b0 + src;
            r.bad = pos < 0;
            if (r.bad) {
                r.token0 = t0;
                r.n = n;
                return r;
            }
            const int f = pos & (P - 1);
            const int skip = k == 0 ? 0 : k * P - f;          // tokens in the runs before
            r.token0 = t0 + skip;
            r.row0 = k == 0 ? f : 0;
            r.n = min(P - r.row0, n - skip);
            r.col = (pos >> shift) + k;
            return r;
        }
        left -= __shfl_sync(FULL, inc, 31);
    }
    return r;
}

// The argmax of <x, q_p q_s> over the S codewords of a head: fp32 scores, and
// fp64 where fp32 cannot tell.  y = x conj(q_s) errs by at most 4 u |x| per
// component (u = 2^-24) and twice the score, max(2 max |y_i|, sum |y_i|), by
// 22 u |x|; the best one is at least sqrt(2) |x| (no direction is farther
// than 45 degrees from the 24 directions of 2T).  Two scores whose order
// fp32 could have wrong thus lie within 44 u / sqrt(2) = 1.9e-6 of each
// other, relative; 4e-6 is used.
constexpr float NEAR_TIE = 1.0f - 4e-6f;

struct Score64 {
    double y[4];
    double score;
    __device__ __forceinline__ Score64(float x0, float x1, float x2, float x3, float4 q) {
        const double a = x0, b = x1, c = x2, d = x3;
        const double w = q.x, i = q.y, j = q.z, k = q.w;
        y[0] = a * w + b * i + c * j + d * k;
        y[1] = b * w - a * i - c * k + d * j;
        y[2] = c * w - a * j + b * k - d * i;
        y[3] = d * w - a * k - b * j + c * i;
        const double m = fmax(fmax(fabs(y[0]), fabs(y[1])), fmax(fabs(y[2]), fabs(y[3])));
        const double sum = fabs(y[0]) + fabs(y[1]) + fabs(y[2]) + fabs(y[3]);
        score = fmax(2.0 * m, sum);
    }
    __device__ __forceinline__ int closest() const {
        const double a0 = fabs(y[0]), a1 = fabs(y[1]), a2 = fabs(y[2]), a3 = fabs(y[3]);
        const double m = fmax(fmax(a0, a1), fmax(a2, a3));
        if (2.0 * m >= a0 + a1 + a2 + a3) {
            const int ax = a0 == m ? 0 : a1 == m ? 1 : a2 == m ? 2 : 3;
            return 2 * ax + (y[ax] < 0.0 ? 1 : 0);
        }
        return 8 + (y[0] < 0.0 ? 1 : 0) + (y[1] < 0.0 ? 2 : 0) + (y[2] < 0.0 ? 4 : 0) +
               (y[3] < 0.0 ? 8 : 0);
    }
};

__device__ __forceinline__ uint32_t best_index(float x0, float x1, float x2, float x3,
                                               const float4 *s_cb, uint32_t S) {
    float best = -1.0f, second = -1.0f;
    uint32_t bs = 0;
    for (uint32_t s = 0; s < S; ++s) {
        float y0, y1, y2, y3;
        const float sc = dot_conj_score2(x0, x1, x2, x3, s_cb[s], y0, y1, y2, y3);
        second = fmaxf(second, fminf(sc, best));
        if (sc > best) { best = sc; bs = s; }
    }
    if (second >= best * NEAR_TIE) {
        double b64 = -1.0;
        for (uint32_t s = 0; s < S; ++s) {
            float y0, y1, y2, y3;
            if (dot_conj_score2(x0, x1, x2, x3, s_cb[s], y0, y1, y2, y3) < best * NEAR_TIE) continue;
            const Score64 e(x0, x1, x2, x3, s_cb[s]);
            if (e.score > b64) { b64 = e.score; bs = s; }
        }
    }
    return bs * 24u + (uint32_t)Score64(x0, x1, x2, x3, s_cb[bs]).closest();
}

template <int DT>
__global__ void __launch_bounds__(PW_WARPS * 32) k_paged_write(WriteArgs a) {
    __shared__ Run s_run;
    __shared__ float4 s_cb[PG_MAX_S];
    __shared__ uint32_t s_mask[PW_MAX_PAGE];  // outlier masks of the run's rows
    __shared__ int s_slot[PW_MAX_PAGE];       // first slot of each row
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = blockIdx.y, role = blockIdx.z;
    const PagesDev p = a.p[role];
    if (warp == 0) {
        const Run r = find_run(a, blockIdx.x, lane);
        if (lane == 0) s_run = r;
    }
    for (uint32_t i = threadIdx.x; i < p.S; i += blockDim.x) s_cb[i] = __ldg(p.cb + (size_t)head * p.S + i);
    __syncthreads();
    const Run r = s_run;
    if (r.n == 0) return;
    int page = -1;
    if (!r.bad && r.col < a.max_pages) page = a.table[(size_t)r.seq * a.max_pages + r.col];
    if (page < 0 || page >= p.n_pages) {
        if (threadIdx.x == 0 && a.st_out) atomicOr(&a.st_out->flags, HQMQ_FLAG_BAD_PAGE);
        return;
    }
    const size_t at0 = p.at(page, head, r.row0);
    const size_t esz = DT == HQMQ_BF16 ? 2 : 4;
    const char *x = reinterpret_cast<const char *>(a.x[role]) + head * a.sh[role] * (int64_t)esz;
    const bool med3 = p.flags != nullptr;
    unsigned n_out = 0, n_over = 0, n_sat = 0, n_nf = 0;
    if (med3) {
        const float th = p.thr[head];
        for (int t = warp; t < r.n; t += PW_WARPS) {
            float x0, x1, x2, x3;
            load_chunk<DT>(x + (r.token0 + t) * a.st[role] * (int64_t)esz, lane, x0, x1, x2, x3);
            const uint32_t m = __ballot_sync(FULL, chunk_norm(x0, x1, x2, x3) > th);
            if (lane == 0) s_mask[t] = m;
        }
        __syncthreads();
        if (warp == 0) {
            int slot = (int)flags_before(p.flags + at0 - r.row0, r.row0, lane);
            for (int t0 = 0; t0 < r.n; t0 += 32) {
                const int t = t0 + lane;
                const int c = t < r.n ? __popc(s_mask[t]) : 0;
                int inc = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(FULL, inc, o);
                    if (lane >= o) inc += u;
                }
                if (t < r.n) s_slot[t] = slot + inc - c;
                slot += __shfl_sync(FULL, inc, 31);
            }
        }
        __syncthreads();
    }
    for (int t = warp; t < r.n; t += PW_WARPS) {
        float x0, x1, x2, x3;
        load_chunk<DT>(x + (r.token0 + t) * a.st[role] * (int64_t)esz, lane, x0, x1, x2, x3);
        const size_t at = at0 + t;
        if (med3) {
            const uint32_t m = s_mask[t];
            const int slot = s_slot[t] + __popc(m & ((1u << lane) - 1u));
            const bool out = (m >> lane) & 1u;
            const bool kept = out && slot < p.cap;
            const uint32_t f = __ballot_sync(FULL, kept);
            if (lane == 0) p.flags[at] = f;
            if (kept) {
                int sv = 0;
                const uint32_t h01 = f32x2_to_f16x2_sat(x0, x1, sv);
                const uint32_t h23 = f32x2_to_f16x2_sat(x2, x3, sv);
                n_sat += sv;
                p.slots(page, head)[slot] = make_uint2(h01, h23);
                x0 = x1 = x2 = x3 = 0.f;
            }
            n_out += out;
            n_over += out && !kept;
        }
        const float nr = chunk_norm(x0, x1, x2, x3);
        const bool finite = nr == nr && nr != __int_as_float(0x7F800000);
        uint32_t idx = 0;
        uint16_t rh = 0x7E00u;
        if (finite) {
            int sat = 0;
            rh = radius_to_f16(nr, sat);
            n_sat += sat;
            if (nr > 0.f) idx = best_index(x0, x1, x2, x3, s_cb, p.S);
        } else {
            ++n_nf;
        }
        __syncwarp();
        p.radius[at * PG_CHUNKS + lane] = rh;
        pack_group32<0>(idx, p.b, lane, pack_const(p.b, lane), p.words + at * p.b);
    }
    if (a.st_out) {
        const unsigned o = __reduce_add_sync(FULL, n_out), ov = __reduce_add_sync(FULL, n_over);
        const unsigned sa = __reduce_add_sync(FULL, n_sat), nf = __reduce_add_sync(FULL, n_nf);
        if (lane == 0) {
            if (o) atomicAdd(&a.st_out->n_outliers, (unsigned long long)o);
            if (ov) atomicOr(&a.st_out->flags, HQMQ_FLAG_OUTLIER_OVERFLOW);
            status_add(a.st_out, HQMQ_FLAG_SATURATED, &a.st_out->n_saturated, sa);
            status_add(a.st_out, HQMQ_FLAG_NONFINITE, &a.st_out->n_nonfinite, nf);
        }
    }
}

}  // namespace hqmq

extern "C" int hqmq_launch_paged_write(const hqmq_kv_pages *k, const hqmq_kv_pages *v,
                                       uint32_t bk, uint32_t bv, const void *xk, const void *xv,
                                       int dtype, int64_t kst, int64_t ksh, int64_t vst, int64_t vsh,
                                       int n_tokens, int n_seqs, const int32_t *cu,
                                       const int32_t *pos0, const int32_t *table, int max_pages,
                                       hqmq_status *st, cudaStream_t stream) {
    using namespace hqmq;
    WriteArgs a = {};
    a.p[0] = pages_dev(k, bk);
    a.x[0] = xk;
    a.st[0] = kst;
    a.sh[0] = ksh;
    if (v) {
        a.p[1] = pages_dev(v, bv);
        a.x[1] = xv;
        a.st[1] = vst;
        a.sh[1] = vsh;
    }
    a.n_tokens = n_tokens;
    a.n_seqs = n_seqs;
    a.max_pages = max_pages;
    a.cu = cu;
    a.pos0 = pos0;
    a.table = table;
    a.st_out = reinterpret_cast<DevStatus *>(st);
    // a sequence's n tokens touch at most (n - 1) / P + 2 pages, and no more than n
    int64_t runs = (int64_t)n_tokens / k->page_size + 2ll * n_seqs;
    if (runs > n_tokens) runs = n_tokens;
    const dim3 grid((unsigned)runs, (unsigned)k->heads, v ? 2u : 1u);
    const cudaError_t e = dtype == HQMQ_BF16
        ? launch_pdl(k_paged_write<HQMQ_BF16>, grid, dim3(PW_WARPS * 32), 0, stream, a)
        : launch_pdl(k_paged_write<HQMQ_F32>, grid, dim3(PW_WARPS * 32), 0, stream, a);
    return e == cudaSuccess ? HQMQ_OK : HQMQ_ERR_CUDA;
}
