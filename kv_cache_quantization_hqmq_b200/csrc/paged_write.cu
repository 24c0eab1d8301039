// paged_write.cu -- quantising new K and V tokens straight into the pages of
// a paged cache (include/hqmq.h, hqmq_paged_write).
//
// A unit of work is the run of new tokens of one sequence that fall in one
// page, for one head of K or of V.  Inside it the outlier slots follow from
// the page's flag words alone (the popcounts of the rows before), so no
// counter is stored, nothing depends on the order in which CTAs run, and a
// row can be written again.
//
// The index is the argmax of the exact scores <x, q_p q_s>: fp32 scores decide
// unless the two best lie within rounding of each other; then fp64 does.
//   * k_paged_write<SEARCH = 1> (prefill): the search table of the head names
//     up to 8 candidates per chunk; their codewords sit in shared memory.  A
//     warp keeps four tokens' table records in flight.
//   * k_paged_write<SEARCH = 0> (decode steps, and heads without tables): the
//     loop over the S secondary codewords, y = x conj(q_s) scoring the 24
//     primaries at once.  A run of few tokens shares each token's loop among
//     the CTA's warps.
#include "paged.cuh"

#include "search.cuh"

namespace hqmq {

constexpr int PW_WARPS = 8;
constexpr int PW_THREADS = PW_WARPS * 32;
constexpr int PW_MAX_PAGE = 256;
constexpr int PW_COPIES = 4;                  // of the codeword table
constexpr int PW_BATCH = 4;                   // tokens a warp searches at once
constexpr int PW_SEARCH_FROM = 8;             // tokens of a sequence, on average

struct WriteArgs {
    PagesDev p[2];
    const void *x[2];
    int64_t st[2], sh[2];
    int n_tokens, n_seqs, max_pages, runs;    // runs: more there cannot be
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

// Two fp32 scores whose order rounding could have turned lie within this
// factor of each other.  u = 2^-24.  Loop: y = x conj(q_s) errs by at most
// 4 u |x| per component, twice the score, max(2 max |y_i|, sum |y_i|), by
// 22 u |x|; the best is at least sqrt(2) |x| (no direction is farther than 45
// degrees from the 24 directions of 2T): 44 u / sqrt(2) = 1.9e-6, relative.
// Candidates: a codeword component carries three roundings and the dot product
// four, at most 10 u |x| of a best score of at least |x| / sqrt(2): 1.7e-6.
constexpr float NEAR_TIE = 1.0f - 4e-6f;

struct Score64 {
    double y0, y1, y2, y3, score;
    __device__ __forceinline__ Score64(float x0, float x1, float x2, float x3, float4 q) {
        const double a = x0, b = x1, c = x2, d = x3;
        const double w = q.x, i = q.y, j = q.z, k = q.w;
        y0 = a * w + b * i + c * j + d * k;
        y1 = b * w - a * i - c * k + d * j;
        y2 = c * w - a * j + b * k - d * i;
        y3 = d * w - a * k - b * j + c * i;
        const double m = fmax(fmax(fabs(y0), fabs(y1)), fmax(fabs(y2), fabs(y3)));
        score = fmax(2.0 * m, fabs(y0) + fabs(y1) + fabs(y2) + fabs(y3));
    }
    // the 2T element of that score, ties to the lowest index
    __device__ __forceinline__ int closest() const {
        const double a0 = fabs(y0), a1 = fabs(y1), a2 = fabs(y2), a3 = fabs(y3);
        const double m = fmax(fmax(a0, a1), fmax(a2, a3));
        if (2.0 * m >= a0 + a1 + a2 + a3) {
            const int ax = a0 == m ? 0 : a1 == m ? 1 : a2 == m ? 2 : 3;
            const double y = ax == 0 ? y0 : ax == 1 ? y1 : ax == 2 ? y2 : y3;
            return 2 * ax + (y < 0.0 ? 1 : 0);
        }
        return 8 + (y0 < 0.0 ? 1 : 0) + (y1 < 0.0 ? 2 : 0) + (y2 < 0.0 ? 4 : 0) + (y3 < 0.0 ? 8 : 0);
    }
};

// The best and the second best of secondaries [s0, s1) in fp32.
struct Best {
    float best, second;
    uint32_t s;
};
__device__ __forceinline__ Best scan_secondaries(float x0, float x1, float x2, float x3, const float4 *s_cb,
                                                 uint32_t s0, uint32_t s1) {
    Best b = {-1.0f, -1.0f, s0};
    for (uint32_t s = s0; s < s1; ++s) {
        float y0, y1, y2, y3;
        const float sc = dot_conj_score2(x0, x1, x2, x3, s_cb[s], y0, y1, y2, y3);
        b.second = fmaxf(b.second, fminf(sc, b.best));
        if (sc > b.best) {
            b.best = sc;
            b.s = s;
        }
    }
    return b;
}
// The index, from the best of all S secondaries.
__device__ __forceinline__ uint32_t settle_index(float x0, float x1, float x2, float x3, const float4 *s_cb,
                                                 uint32_t S, Best b) {
    if (b.second >= b.best * NEAR_TIE) {
        double b64 = -1.0;
        for (uint32_t s = 0; s < S; ++s) {
            float y0, y1, y2, y3;
            if (dot_conj_score2(x0, x1, x2, x3, s_cb[s], y0, y1, y2, y3) < b.best * NEAR_TIE) continue;
            const Score64 e(x0, x1, x2, x3, s_cb[s]);
            if (e.score > b64) {
                b64 = e.score;
                b.s = s;
            }
        }
    }
    return b.s * 24u + (uint32_t)Score64(x0, x1, x2, x3, s_cb[b.s]).closest();
}

// The table record of a chunk (finite, not 0): search.cuh.
__device__ __forceinline__ const uint4 *record_of(const uint4 *tb, float x0, float x1, float x2, float x3) {
    const float a0 = fabsf(x0), a1 = fabsf(x1), a2 = fabsf(x2), a3 = fabsf(x3);
    const float m = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
    const bool e0 = a0 == m, e01 = e0 || a1 == m, e012 = e01 || a2 == m;
    const int ax = e0 ? 0 : e01 ? 1 : e012 ? 2 : 3;
    const float xa = e0 ? x0 : e01 ? x1 : e012 ? x2 : x3;
    const float c1 = e0 ? x1 : x0, c2 = e01 ? x2 : x1, c3 = e012 ? x3 : x2;
    const float inv = __fdividef(1.0f, m);    // (cells are widened by far more than its error)
    const int cell = (cell_coord(c1 * inv) * LUT_G + cell_coord(c2 * inv)) * LUT_G + cell_coord(c3 * inv);
    return tb + (2 * ax + (xa < 0.0f ? 1 : 0)) * LUT_CELLS + cell;
}

__device__ __forceinline__ double exact_score(float x0, float x1, float x2, float x3, uint32_t id, const float4 *s_cb) {
    const float4 q = s_cb[id / 24u];
    float p0, p1, p2, p3;
    element_2t((int)(id % 24u), p0, p1, p2, p3);
    const double a = p0, b = p1, c = p2, d = p3, w = q.x, i = q.y, j = q.z, k = q.w;
    return x0 * (a * w - b * i - c * j - d * k) + x1 * (a * i + b * w + c * k - d * j) +
           x2 * (a * j - b * k + c * w + d * i) + x3 * (a * k + b * j - c * i + d * w);
}

// The index among the record's candidates (kmax: the longest list of the warp).
__device__ __forceinline__ uint32_t pick_candidate(float x0, float x1, float x2, float x3, uint4 rec, uint32_t kmax,
                                                   const float4 *tab, const float4 *s_cb) {
    const uint32_t sl[4] = {rec.x, rec.y, rec.z, rec.w};
    float best = -INFINITY, second = -INFINITY;
    uint32_t bid = 0;
#pragma unroll
    for (int k = 0; k < LUT_SLOTS; ++k) {
        if ((uint32_t)k >= kmax) break;       // (warp-uniform)
        const uint32_t id = (sl[k >> 1] >> ((k & 1) * 16)) & LUT_ID_MASK;
        const float4 c = tab[id * PW_COPIES];
        const float sc = fmaf(x3, c.w, fmaf(x2, c.z, fmaf(x1, c.y, x0 * c.x)));
        second = fmaxf(second, fminf(sc, best));
        if (sc > best) {
            best = sc;
            bid = id;
        }
    }
    if (second >= best * NEAR_TIE && best > 0.f) {            // (0: nothing to search)
        double b64 = -1.0;
        const uint32_t n = (rec.x >> 12) & 0xFu;
        for (uint32_t k = 0; k < n; ++k) {
            const uint32_t w = k < 2 ? sl[0] : k < 4 ? sl[1] : k < 6 ? sl[2] : sl[3];
            const uint32_t id = (w >> ((k & 1u) * 16)) & LUT_ID_MASK;
            const double e = exact_score(x0, x1, x2, x3, id, s_cb);
            if (e > b64) {
                b64 = e;
                bid = id;
            }
        }
    }
    return bid;
}

// One token of a warp, a lane one chunk: flags, values and radius; what is
// left to search (0 if nothing is).
struct Token {
    float x0, x1, x2, x3;
    bool search;
};
struct Tally {
    unsigned out, over, sat, nf;
};
__device__ __forceinline__ void store_token(Token &t, const PagesDev &p, size_t at, uint2 *slots, bool med3,
                                            uint32_t mask, int slot0, int lane, Tally &n) {
    if (med3) {
        const int slot = slot0 + __popc(mask & ((1u << lane) - 1u));
        const bool out = (mask >> lane) & 1u, kept = out && slot < p.cap;
        const uint32_t f = __ballot_sync(FULL, kept);
        if (lane == 0) p.flags[at] = f;
        if (kept) {
            int sv = 0;
            const uint32_t h01 = f32x2_to_f16x2_sat(t.x0, t.x1, sv);
            const uint32_t h23 = f32x2_to_f16x2_sat(t.x2, t.x3, sv);
            n.sat += sv;
            slots[slot] = make_uint2(h01, h23);
            t.x0 = t.x1 = t.x2 = t.x3 = 0.f;
        }
        n.out += out;
        n.over += out && !kept;
    }
    const float r = chunk_norm(t.x0, t.x1, t.x2, t.x3);
    const bool finite = r == r && r != __int_as_float(0x7F800000);
    uint16_t rh = 0x7E00u;
    if (finite) {
        int sat = 0;
        rh = radius_to_f16(r, sat);
        n.sat += sat;
    } else {
        ++n.nf;
    }
    t.search = finite && r > 0.f;
    p.radius[at * PG_CHUNKS + lane] = rh;
}

template <int DT, int SEARCH>
__global__ void __launch_bounds__(PW_THREADS, SEARCH ? 3 : 5) k_paged_write(WriteArgs a) {
    extern __shared__ float4 s_tab[];         // SEARCH: [24 S + 1][PW_COPIES] codewords
    __shared__ Run s_run;
    __shared__ float4 s_cb[PG_MAX_S];
    __shared__ uint32_t s_mask[PW_MAX_PAGE];  // outlier masks of the run's rows
    __shared__ int s_slot[PW_MAX_PAGE];       // first slot of each row
    __shared__ Best s_best[SEARCH ? 1 : PW_THREADS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = blockIdx.y, role = blockIdx.z;
    const PagesDev &p = a.p[role];
    pdl_wait();
    pdl_trigger();
    const bool med3 = p.flags != nullptr;
    const float th = med3 ? p.thr[head] : 0.f;
    for (uint32_t i = threadIdx.x; i < p.S; i += PW_THREADS) s_cb[i] = __ldg(p.cb + (size_t)head * p.S + i);
    if (SEARCH) {
        const uint32_t words = 24u * p.S;
        for (uint32_t e = threadIdx.x; e <= words; e += PW_THREADS) {
            float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
            if (e < words) c = codeword((int)(e % 24u), __ldg(p.cb + (size_t)head * p.S + e / 24u));
#pragma unroll
            for (int r = 0; r < PW_COPIES; ++r) s_tab[e * PW_COPIES + ((r + e) & (PW_COPIES - 1))] = c;
        }
    }
    const size_t esz = DT == HQMQ_BF16 ? 2 : 4;
    const char *x = reinterpret_cast<const char *>(a.x[role]) + head * a.sh[role] * (int64_t)esz;
    const int64_t xt = a.st[role] * (int64_t)esz;
    const PackConst pc = pack_const(p.b, lane);
    Tally n = {0, 0, 0, 0};

    for (int item = blockIdx.x; item < a.runs; item += gridDim.x) {
        if (warp == 0) {
            const Run r = find_run(a, item, lane);
            if (lane == 0) s_run = r;
        }
        __syncthreads();
        const Run r = s_run;
        if (r.n == 0) break;                  // (there are no more)
        int page = -1;
        if (!r.bad && r.col < a.max_pages) page = a.table[(size_t)r.seq * a.max_pages + r.col];
        if (page < 0 || page >= p.n_pages) {
            if (threadIdx.x == 0 && a.st_out) atomicOr(&a.st_out->flags, HQMQ_FLAG_BAD_PAGE);
            __syncthreads();                  // (s_run)
            continue;
        }
        const size_t at0 = p.at(page, head, r.row0);
        uint2 *slots = p.slots(page, head);
        const char *x0p = x + r.token0 * xt;
        if (med3) {
            for (int t = warp; t < r.n; t += PW_WARPS) {
                float x0, x1, x2, x3;
                load_chunk<DT>(x0p + t * xt, lane, x0, x1, x2, x3);
                const uint32_t m = __ballot_sync(FULL, chunk_norm(x0, x1, x2, x3) > th);
                if (lane == 0) s_mask[t] = m;
            }
            uint32_t before = 0;
            if (warp == 0) before = flags_before(p.flags + at0 - r.row0, r.row0, lane);
            __syncthreads();
            if (warp == 0) {
                int slot = (int)before;
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
        }
        __syncthreads();
        if (SEARCH) {
            const uint4 *tb = p.table + (size_t)head * LUT_ENTRIES;
            for (int t0 = warp * PW_BATCH; t0 < r.n; t0 += PW_WARPS * PW_BATCH) {
                Token k[PW_BATCH];
                uint4 rec[PW_BATCH];
#pragma unroll
                for (int i = 0; i < PW_BATCH; ++i) {
                    k[i] = {0.f, 0.f, 0.f, 0.f, false};
                    if (t0 + i < r.n) load_chunk<DT>(x0p + (t0 + i) * xt, lane, k[i].x0, k[i].x1, k[i].x2, k[i].x3);
                }
#pragma unroll
                for (int i = 0; i < PW_BATCH; ++i) {
                    rec[i] = make_uint4(1u << 12, 0u, 0u, 0u);
                    if (t0 + i >= r.n) continue;              // (warp-uniform)
                    store_token(k[i], p, at0 + t0 + i, slots, med3, med3 ? s_mask[t0 + i] : 0u,
                                med3 ? s_slot[t0 + i] : 0, lane, n);
                    if (k[i].search) rec[i] = __ldg(record_of(tb, k[i].x0, k[i].x1, k[i].x2, k[i].x3));
                }
#pragma unroll
                for (int i = 0; i < PW_BATCH; ++i) {
                    if (t0 + i >= r.n) continue;
                    const uint32_t cnt = (rec[i].x >> 12) & 0xFu;
                    const uint32_t kmax = __reduce_max_sync(FULL, cnt);
                    uint32_t idx = pick_candidate(k[i].x0, k[i].x1, k[i].x2, k[i].x3, rec[i], kmax,
                                                  s_tab + (lane & (PW_COPIES - 1)), s_cb);
                    if (!k[i].search) idx = 0;
                    else if (cnt == 0)        // a cell with more candidates than a record holds
                        idx = settle_index(k[i].x0, k[i].x1, k[i].x2, k[i].x3, s_cb, p.S,
                                           scan_secondaries(k[i].x0, k[i].x1, k[i].x2, k[i].x3, s_cb, 0, p.S));
                    __syncwarp();
                    pack_group32<0>(idx, p.b, lane, pc, p.words + (at0 + t0 + i) * p.b);
                }
            }
        } else {
            // warps of a token: 8, 4, 2 or 1, each with a share of the secondaries
            const int wpt = r.n == 1 ? 8 : r.n == 2 ? 4 : r.n <= 4 ? 2 : 1;
            const int share = warp & (wpt - 1);
            const uint32_t s0 = p.S * share / wpt, s1 = p.S * (share + 1) / wpt;
            const int per = PW_WARPS / wpt;   // tokens at a time
            for (int t0 = 0; t0 < r.n; t0 += per) {
                const int t = t0 + warp / wpt;
                Token k = {0.f, 0.f, 0.f, 0.f, false};
                Best b = {-1.0f, -1.0f, 0};
                if (t < r.n) {
                    load_chunk<DT>(x0p + t * xt, lane, k.x0, k.x1, k.x2, k.x3);
                    if (share == 0) {
                        store_token(k, p, at0 + t, slots, med3, med3 ? s_mask[t] : 0u, med3 ? s_slot[t] : 0, lane, n);
                    } else if (med3) {
                        const uint32_t m = s_mask[t];
                        const int slot = s_slot[t] + __popc(m & ((1u << lane) - 1u));
                        if (((m >> lane) & 1u) && slot < p.cap) k.x0 = k.x1 = k.x2 = k.x3 = 0.f;
                    }
                    b = scan_secondaries(k.x0, k.x1, k.x2, k.x3, s_cb, s0, s1);
                }
                if (wpt > 1) {
                    s_best[SEARCH ? 0 : threadIdx.x] = b;
                    __syncthreads();
                    if (share == 0) {
                        for (int w = 1; w < wpt; ++w) {       // in order of s: the lowest of equal scores stays
                            const Best o = s_best[SEARCH ? 0 : threadIdx.x + 32 * w];
                            b.second = fmaxf(fmaxf(b.second, o.second), fminf(b.best, o.best));
                            if (o.best > b.best) {
                                b.best = o.best;
                                b.s = o.s;
                            }
                        }
                    }
                }
                if (share == 0 && t < r.n) {
                    const uint32_t idx = k.search ? settle_index(k.x0, k.x1, k.x2, k.x3, s_cb, p.S, b) : 0u;
                    __syncwarp();
                    pack_group32<0>(idx, p.b, lane, pc, p.words + (at0 + t) * p.b);
                }
                if (wpt > 1) __syncthreads(); // (s_best)
            }
        }
        __syncthreads();                      // (s_run, s_mask, s_slot)
    }
    if (a.st_out) {
        const unsigned o = __reduce_add_sync(FULL, n.out), ov = __reduce_add_sync(FULL, n.over);
        const unsigned sa = __reduce_add_sync(FULL, n.sat), nf = __reduce_add_sync(FULL, n.nf);
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
    a.runs = (int)runs;
    const int roles = v ? 2 : 1;
    // the tables pay from runs of a few tokens on (their codewords have to be brought to shared memory)
    const bool search = k->table && (!v || v->table) && n_tokens >= PW_SEARCH_FROM * n_seqs;
    const uint32_t S = v && v->S > k->S ? v->S : k->S;
    const size_t smem = search ? (size_t)(24 * S + 1) * PW_COPIES * sizeof(float4) : 0;
    // with tables a CTA goes through several runs of its head; 3 CTAs to an SM
    int64_t gx = runs;
    if (search) {
        const int64_t fill = (3 * 148 + k->heads * roles - 1) / (k->heads * roles);
        if (gx > fill) gx = fill;
    }
    const dim3 grid((unsigned)gx, (unsigned)k->heads, (unsigned)roles);
    auto kern = dtype == HQMQ_BF16 ? (search ? k_paged_write<HQMQ_BF16, 1> : k_paged_write<HQMQ_BF16, 0>)
                                   : (search ? k_paged_write<HQMQ_F32, 1> : k_paged_write<HQMQ_F32, 0>);
    if (smem > 32 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return HQMQ_ERR_CUDA;
    return launch_pdl(kern, grid, dim3(PW_THREADS), smem, stream, a) == cudaSuccess ? HQMQ_OK : HQMQ_ERR_CUDA;
}
