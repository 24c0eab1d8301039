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
//   * k_paged_write_table (prefill): the search table of the head names up to 8
//     candidates per chunk; their codewords sit in shared memory.  A warp
//     counts the outliers of its eight tokens, then searches them one by one, the
//     next one's record under way.  L1 has to hold records and tokens, and
//     warps to hide their latency: one copy of the codewords (its bank
//     conflicts cost less than the space; 4 copies, 3 CTAs an SM: 59 us for 4096
//     tokens, 8 heads, K and V, S = 32) and 64 registers (eight tokens in
//     registers, two records in flight, 80 registers: 61 us) take 52.5 us,
//     40 G chunks/s.
//   * k_paged_write_loop (decode steps, small codebooks, heads without
//     tables): the loop over the S secondary codewords, y = x conj(q_s)
//     scoring the 24 primaries at once.  A run of one or two tokens shares each
//     token's loop among the CTA's warps.
#include "paged.cuh"

#include "search.cuh"

namespace hqmq {

constexpr int PW_LOOP_WARPS = 4, PW_TABLE_WARPS = 8;
constexpr int PW_TOKENS = 8;                  // tokens of a warp of the table kernel, at most
constexpr uint32_t PW_SEARCH_S = 8;           // the smallest codebook that is searched through its tables
constexpr int PW_RUNS_FROM = 4;               // tokens of a sequence, on average

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
// The 2T element of the best score of y, or -1 where fp32 cannot tell: the two families, the two largest
// axes or the sign of a half unit's component within rounding.
__device__ __forceinline__ int closest_clear(float y0, float y1, float y2, float y3) {
    const float a0 = fabsf(y0), a1 = fabsf(y1), a2 = fabsf(y2), a3 = fabsf(y3);
    const float h0 = fmaxf(a0, a1), l0 = fminf(a0, a1), h1 = fmaxf(a2, a3), l1 = fminf(a2, a3);
    const float m = fmaxf(h0, h1), next = fmaxf(fminf(h0, h1), h0 >= h1 ? l0 : l1);
    const float sum = (a0 + a1) + (a2 + a3), axis = m + m, near = 4e-6f * fmaxf(axis, sum);
    if (fabsf(axis - sum) <= near) return -1;
    if (axis > sum) {
        if (2.0f * (m - next) <= near) return -1;
        const int ax = a0 == m ? 0 : a1 == m ? 1 : a2 == m ? 2 : 3;
        const float y = ax == 0 ? y0 : ax == 1 ? y1 : ax == 2 ? y2 : y3;
        return 2 * ax + (y < 0.0f ? 1 : 0);
    }
    if (fminf(l0, l1) <= near) return -1;
    return 8 + (y0 < 0.0f ? 1 : 0) + (y1 < 0.0f ? 2 : 0) + (y2 < 0.0f ? 4 : 0) + (y3 < 0.0f ? 8 : 0);
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
    float y0, y1, y2, y3;
    dot_conj_score2(x0, x1, x2, x3, s_cb[b.s], y0, y1, y2, y3);
    int c = closest_clear(y0, y1, y2, y3);
    if (c < 0) c = Score64(x0, x1, x2, x3, s_cb[b.s]).closest();
    return b.s * 24u + (uint32_t)c;
}

// The largest r2 whose rounded root is not above th: r = RN(sqrt(r2)) > th exactly where r2 > this (the
// root is monotone).  th NaN or infinite: nothing is above it.
__device__ __forceinline__ float square_threshold(float th) {
    if (!(th >= 0.f)) return th < 0.f ? -1.f : INFINITY;
    float c = th * th;
    while (__fsqrt_rn(c) > th) c = __uint_as_float(__float_as_uint(c) - 1u);
    while (c < INFINITY && __fsqrt_rn(__uint_as_float(__float_as_uint(c) + 1u)) <= th) c = __uint_as_float(__float_as_uint(c) + 1u);
    return c;
}
__device__ __forceinline__ float square_norm(float x0, float x1, float x2, float x3) {
    return __fmaf_rn(x3, x3, __fmaf_rn(x2, x2, __fmaf_rn(x1, x1, __fmul_rn(x0, x0))));
}

// One coordinate's cell as the mantissa of 2^23 + cell: the map of search.cuh, shrunk by 2^-20 and moved
// by 2^-17 so that t = +-1 (up to rounding) stay inside the grid, which moves a cell's border by 3.2e-6 at
// most; cells list what can win up to 1e-5 beyond their borders.
__device__ __forceinline__ uint32_t cell_bits(float t) {
    constexpr float HG = 0.5f * LUT_G, SHRINK = 1.0f - 1.0f / 1048576.0f;
    const float v = fmaf(t, fmaf(MAP_B * HG * SHRINK, t * t, MAP_A * HG * SHRINK), HG + 1.0f / 131072.0f);
    return __float_as_uint(__fadd_rz(v, 8388608.0f));
}
// The table record of a chunk (finite, not 0): search.cuh.
__device__ __forceinline__ uint32_t record_of(float x0, float x1, float x2, float x3) {
    const float a0 = fabsf(x0), a1 = fabsf(x1), a2 = fabsf(x2), a3 = fabsf(x3);
    const float m = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
    const bool e0 = a0 == m, e01 = e0 || a1 == m, e012 = e01 || a2 == m;
    const uint32_t ax = e0 ? 0u : e01 ? 2u : e012 ? 4u : 6u;
    const float xa = e0 ? x0 : e01 ? x1 : e012 ? x2 : x3;
    const float c1 = e0 ? x1 : x0, c2 = e01 ? x2 : x1, c3 = e012 ? x3 : x2;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(m));
    constexpr uint32_t BASE = 0x4B000000u * (LUT_G * LUT_G + LUT_G + 1u);
    const uint32_t cell = cell_bits(c1 * inv) * (LUT_G * LUT_G) + cell_bits(c2 * inv) * LUT_G + cell_bits(c3 * inv) - BASE;
    return (ax + (__float_as_uint(xa) >> 31)) * LUT_CELLS + cell;
}

// One token of a warp, a lane one chunk.
struct Token {
    float x0, x1, x2, x3;
    bool search;                              // an index has to be found (else it is 0)
};

// The index among the record's candidates (kmax: the longest list of the warp), `clear` unless another
// score is as near as rounding.  A score's bits, the last three replaced by 7 - slot, order scores and
// then slots as integers (the best score is above 0); 128 units of 2^-23 or 2^-24, relative, are 7.6e-6 at
// least: NEAR_TIE's 4e-6 and twice the 2^-20 that the replaced bits can be worth.
__device__ __forceinline__ uint32_t pick_candidate(const Token &t, uint4 rec, uint32_t kmax, const float4 *tab,
                                                   bool &clear) {
    const uint32_t sl[4] = {rec.x, rec.y, rec.z, rec.w};
    int best = -1, second = -1;
#pragma unroll
    for (int k = 0; k < LUT_SLOTS; ++k) {
        if ((uint32_t)k >= kmax) break;       // (warp-uniform)
        const uint32_t id = (sl[k >> 1] >> ((k & 1) * 16)) & LUT_ID_MASK;
        const float4 c = tab[id];
        const float sc = fmaf(t.x3, c.w, fmaf(t.x2, c.z, fmaf(t.x1, c.y, t.x0 * c.x)));
        const int key = (int)((__float_as_uint(sc) & ~7u) | (7u - k));
        second = max(second, min(key, best));
        best = max(best, key);
    }
    const int k = 7 - (best & 7);
    const uint32_t w = k < 4 ? (k < 2 ? sl[0] : sl[1]) : (k < 6 ? sl[2] : sl[3]);
    const uint32_t id = (w >> ((k & 1) * 16)) & LUT_ID_MASK;
    clear = !t.search || (best - second > 128 && (rec.x & 0xF000u) != 0u);
    return t.search ? id : 0u;
}

// A stored token's index words again, by the loop over the codebook: for what the table's candidates in
// fp32 could not tell, and for cells with more candidates than a record holds.  Out of line and after the
// warp's other tokens, so that it costs them no registers.
template <int DT>
__device__ __noinline__ void settle_token(const PagesDev &p, const char *x, size_t at, const float4 *s_cb, int lane) {
    RawChunk<DT> c;
    c.load(x, lane);
    Token t = {c.e(0), c.e(1), c.e(2), c.e(3), false};
    if (p.flags && ((p.flags[at] >> lane) & 1u)) t.x0 = t.x1 = t.x2 = t.x3 = 0.f;
    const float r = chunk_norm(t.x0, t.x1, t.x2, t.x3);
    uint32_t idx = 0;
    if (r > 0.f && r < INFINITY)
        idx = settle_index(t.x0, t.x1, t.x2, t.x3, s_cb, p.S,
                           scan_secondaries(t.x0, t.x1, t.x2, t.x3, s_cb, 0, p.S));
    __syncwarp();
    pack_group32<0>(idx, p.b, lane, pack_const(p.b, lane), p.words + at * p.b);
}

struct Tally {
    unsigned out, over, sat, nf;
    __device__ __forceinline__ void add_to(DevStatus *st, int lane) const {
        if (!st) return;
        const unsigned o = __reduce_add_sync(FULL, out), ov = __reduce_add_sync(FULL, over);
        const unsigned sa = __reduce_add_sync(FULL, sat), f = __reduce_add_sync(FULL, nf);
        if (lane == 0) {
            if (o) atomicAdd(&st->n_outliers, (unsigned long long)o);
            if (ov) atomicOr(&st->flags, HQMQ_FLAG_OUTLIER_OVERFLOW);
            status_add(st, HQMQ_FLAG_SATURATED, &st->n_saturated, sa);
            status_add(st, HQMQ_FLAG_NONFINITE, &st->n_nonfinite, f);
        }
    }
};

// Where a run goes.
struct Place {
    size_t at0;                               // flat index of its first row
    uint2 *slots;
    const char *x;                            // its first token's chunks of this head
};
template <int DT>
__device__ __forceinline__ bool find_place(const WriteArgs &a, const PagesDev &p, const Run &r, int head, int role,
                                           Place &pl) {
    int page = -1;
    if (!r.bad && r.col < a.max_pages) page = a.table[(size_t)r.seq * a.max_pages + r.col];
    if (page < 0 || page >= p.n_pages) {
        if (threadIdx.x == 0 && a.st_out) atomicOr(&a.st_out->flags, HQMQ_FLAG_BAD_PAGE);
        return false;
    }
    pl.at0 = p.at(page, head, r.row0);
    pl.slots = p.slots(page, head);
    pl.x = reinterpret_cast<const char *>(a.x[role]) +
           (head * a.sh[role] + r.token0 * a.st[role]) * (int64_t)(DT == HQMQ_BF16 ? 2 : 4);
    return true;
}

// Flags, values and radius of a token (mask: chunks above the threshold; slot0: the first one's slot).
__device__ __forceinline__ void store_token(Token &t, const PagesDev &p, size_t at, uint2 *slots, uint32_t mask,
                                            int slot0, int lane, Tally &n) {
    if (p.flags) {
        uint32_t f = 0;
        if (mask) {                           // (warp-uniform)
            const int slot = slot0 + __popc(mask & ((1u << lane) - 1u));
            const bool out = (mask >> lane) & 1u, kept = out && slot < p.cap;
            f = __ballot_sync(FULL, kept);
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
        if (lane == 0) p.flags[at] = f;
    }
    const float r = chunk_norm(t.x0, t.x1, t.x2, t.x3);
    const bool finite = r < INFINITY;         // (false for NaN)
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

template <int DT>
__global__ void __launch_bounds__(PW_TABLE_WARPS * 32, 4) k_paged_write_table(const __grid_constant__ WriteArgs a) {
    constexpr int WARPS = PW_TABLE_WARPS, THREADS = WARPS * 32;
    extern __shared__ float4 s_tab[];         // 24 S + 1 codewords
    __shared__ Run s_run;
    __shared__ float4 s_cb[PG_MAX_S];
    __shared__ uint32_t s_cnt[WARPS + 1];     // outliers of each warp's tokens, and before the block
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = blockIdx.y, role = blockIdx.z;
    const PagesDev &p = a.p[role];
    pdl_wait();
    pdl_trigger();
    const float th2 = p.flags ? square_threshold(p.thr[head]) : INFINITY;
    const uint32_t words = 24u * p.S;
    for (uint32_t i = threadIdx.x; i < p.S; i += THREADS) s_cb[i] = __ldg(p.cb + (size_t)head * p.S + i);
    for (uint32_t e = threadIdx.x; e <= words; e += THREADS)
        s_tab[e] = e < words ? codeword((int)(e % 24u), __ldg(p.cb + (size_t)head * p.S + e / 24u))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t xt = a.st[role] * (int64_t)(DT == HQMQ_BF16 ? 2 : 4);
    const uint4 *tb = p.table + (size_t)head * LUT_ENTRIES;
    const PackConst pc = pack_const(p.b, lane);
    Tally n = {0, 0, 0, 0};

    if (warp == 0) {
        const Run r = find_run(a, blockIdx.x, lane);
        if (lane == 0) s_run = r;
    }
    __syncthreads();
    const Run r = s_run;
    if (r.n == 0) return;
    Place pl;
    if (!find_place<DT>(a, p, r, head, role, pl)) return;
    // blocks of 64 tokens, 8 to a warp; shorter runs in equal shares
    const int per = min((r.n + WARPS - 1) / WARPS, PW_TOKENS);
    for (int b0 = 0; b0 < r.n; b0 += WARPS * per) {
        const int t0 = b0 + warp * per, mine = min(max(r.n - t0, 0), per);
        const char *xw = pl.x + t0 * xt;
        int slot = 0;
        if (p.flags) {
            int cnt = 0;
            RawChunk<DT> x[PW_TOKENS];
#pragma unroll
            for (int i = 0; i < PW_TOKENS; ++i) {
                x[i].zero();
                if (i < mine) x[i].load(xw + i * xt, lane);
            }
#pragma unroll
            for (int i = 0; i < PW_TOKENS; ++i) {         // (a threshold below 0 is passed by zeros)
                const bool out = square_norm(x[i].e(0), x[i].e(1), x[i].e(2), x[i].e(3)) > th2;
                cnt += __popc(__ballot_sync(FULL, i < mine && out));
            }
            if (lane == 0) s_cnt[warp] = cnt;
            if (warp == 0) {              // (a later block: the rows before are this call's, counted in slots)
                const uint32_t f = b0 == 0 ? flags_before(p.flags + pl.at0 - r.row0, r.row0, lane) : s_cnt[WARPS];
                if (lane == 0) s_cnt[WARPS] = f;
            }
            __syncthreads();
            slot = (int)s_cnt[WARPS];
            for (int w = 0; w < warp; ++w) slot += (int)s_cnt[w];
            uint32_t all = s_cnt[WARPS];
            for (int w = 0; w < WARPS; ++w) all += s_cnt[w];
            __syncthreads();
            if (threadIdx.x == 0) s_cnt[WARPS] = all;
        }
        uint32_t unclear = 0;             // tokens of the warp
        // a token's record is under way while the one before is searched
        RawChunk<DT> next;
        next.zero();
        if (mine > 0) next.load(xw, lane);
        Token k = {0.f, 0.f, 0.f, 0.f, false};
        uint4 rec = make_uint4(1u << 12, 0u, 0u, 0u);
        size_t at = pl.at0 + t0;
#pragma unroll 1
        for (int i = 0; i <= mine; ++i, ++at) {
            const Token ks = k;
            const uint4 rs = rec;
            if (i < mine) {
                k = {next.e(0), next.e(1), next.e(2), next.e(3), false};
                if (i + 1 < mine) next.load(xw + (i + 1) * xt, lane);
                uint32_t mask = 0;
                if (p.flags) mask = __ballot_sync(FULL, square_norm(k.x0, k.x1, k.x2, k.x3) > th2);
                store_token(k, p, at, pl.slots, mask, slot, lane, n);
                slot += __popc(mask);
                rec = make_uint4(1u << 12, 0u, 0u, 0u);
                if (k.search) rec = __ldg(tb + record_of(k.x0, k.x1, k.x2, k.x3));
            }
            if (i > 0) {
                const uint32_t kmax = __reduce_max_sync(FULL, (rs.x >> 12) & 0xFu);
                bool clear;
                const uint32_t idx = pick_candidate(ks, rs, kmax, s_tab, clear);
                if (!__all_sync(FULL, clear)) unclear |= 1u << (i - 1);
                pack_group32<0>(idx, p.b, lane, pc, p.words + (at - 1) * p.b);
            }
        }
        __syncwarp();
        for (; unclear; unclear &= unclear - 1u) {
            const int i = __ffs(unclear) - 1;
            settle_token<DT>(p, pl.x + (t0 + i) * xt, pl.at0 + t0 + i, s_cb, lane);
        }
    }
    n.add_to(a.st_out, lane);
}

// CTAS: resident on an SM.  Steps of one token want many short CTAs (64 sequences, 8 heads: 8.0 us at 7, 10.2
// at 5), longer runs the registers for more chunks' arithmetic at once (runs of 16, S = 8: 14.6 and 11.5 us).
template <int DT, int BB, int CTAS>
__global__ void __launch_bounds__(PW_LOOP_WARPS * 32, CTAS) k_paged_write_loop(const __grid_constant__ WriteArgs a) {
    constexpr int WARPS = PW_LOOP_WARPS, THREADS = WARPS * 32;
    __shared__ float4 s_cb[PG_MAX_S];
    __shared__ uint32_t s_cnt[WARPS];
    __shared__ Best s_best[THREADS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = blockIdx.y, role = blockIdx.z;
    const PagesDev &p = a.p[role];
    pdl_wait();
    pdl_trigger();
    // (every warp finds the run by itself: no one waits for another)
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
    if (threadIdx.x < p.S) q = __ldg(p.cb + (size_t)head * p.S + threadIdx.x);
    const float thr = p.flags ? __ldg(p.thr + head) : 0.f;
    const Run r = find_run(a, blockIdx.x, lane);
    if (r.n == 0) return;
    Place pl;
    if (!find_place<DT>(a, p, r, head, role, pl)) return;
    const int64_t xt = a.st[role] * (int64_t)(DT == HQMQ_BF16 ? 2 : 4);
    // warps of a token: 4, 2 or 1, each with a share of the secondaries
    const int wpt = r.n == 1 ? 4 : r.n == 2 ? 2 : 1, per = WARPS / wpt;
    const int share = warp & (wpt - 1), own = warp / wpt;
    RawChunk<DT> next;
    next.zero();
    if (own < r.n) next.load(pl.x + own * xt, lane);
    uint32_t before = 0;                      // flagged chunks before the tokens of this turn
    if (p.flags) before = flags_before(p.flags + pl.at0 - r.row0, r.row0, lane);
    if (threadIdx.x < p.S) s_cb[threadIdx.x] = q;
    const float th2 = p.flags ? square_threshold(thr) : INFINITY;
    const uint32_t s0 = p.S * share / wpt, s1 = p.S * (share + 1) / wpt;
    const PackConst pc = pack_const(p.b, lane);
    Tally n = {0, 0, 0, 0};
    for (int t0 = 0; t0 < r.n; t0 += per) {
        const int t = t0 + own;
        const RawChunk<DT> c = next;
        if (t + per < r.n) next.load(pl.x + (t + per) * xt, lane);
        Token k = {c.e(0), c.e(1), c.e(2), c.e(3), false};
        uint32_t mask = 0;
        if (p.flags && t < r.n) mask = __ballot_sync(FULL, square_norm(k.x0, k.x1, k.x2, k.x3) > th2);
        if (lane == 0) s_cnt[warp] = __popc(mask);
        __syncthreads();
        int slot = (int)before;
        for (int w = 0; w < own; ++w) slot += (int)s_cnt[w * wpt];
        for (int w = 0; w < per; ++w) before += s_cnt[w * wpt];
        if (t < r.n) {
            if (share == 0) {
                store_token(k, p, pl.at0 + t, pl.slots, mask, slot, lane, n);
            } else if (((mask >> lane) & 1u) && slot + __popc(mask & ((1u << lane) - 1u)) < p.cap) {
                k.x0 = k.x1 = k.x2 = k.x3 = 0.f;
            }
        }
        Best b = {-1.0f, -1.0f, 0};
        if (t < r.n) b = scan_secondaries(k.x0, k.x1, k.x2, k.x3, s_cb, s0, s1);
        if (share) s_best[threadIdx.x] = b;
        __syncthreads();
        if (share == 0 && t < r.n) {
            for (int w = 1; w < wpt; ++w) {   // in order of s: the lowest of equal scores stays
                const Best o = s_best[threadIdx.x + 32 * w];
                b.second = fmaxf(fmaxf(b.second, o.second), fminf(b.best, o.best));
                if (o.best > b.best) {
                    b.best = o.best;
                    b.s = o.s;
                }
            }
            const uint32_t idx = k.search ? settle_index(k.x0, k.x1, k.x2, k.x3, s_cb, p.S, b) : 0u;
            __syncwarp();
            pack_group32<BB>(idx, p.b, lane, pc, p.words + (pl.at0 + t) * p.b);
        }
    }
    n.add_to(a.st_out, lane);
}

using WriteKernel = void (*)(WriteArgs);
template <int DT, int BB> WriteKernel write_kernel_b(bool search, bool runs_of_some) {
    return search ? k_paged_write_table<DT> : runs_of_some ? k_paged_write_loop<DT, BB, 5> : k_paged_write_loop<DT, BB, 7>;
}
// bb: bits of the indices of K and V where the loop is compiled for them (S = 6 .. 10 and 22 .. 42), else 0.
// Steps of one token of 64 sequences, 8 heads, fp32, with the width at run time and compiled in: S = 32 8.4
// and 7.8 us, S = 8 6.1 and 5.8; the table kernel gains nothing by it (4096 tokens 52.4 and 52.8 us).
template <int DT> WriteKernel write_kernel(uint32_t bb, bool search, bool runs_of_some) {
    return bb == 8    ? write_kernel_b<DT, 8>(search, runs_of_some)
           : bb == 10 ? write_kernel_b<DT, 10>(search, runs_of_some)
                      : write_kernel_b<DT, 0>(search, runs_of_some);
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
    const int roles = v ? 2 : 1;
    const uint32_t S = v && v->S > k->S ? v->S : k->S;
    // the tables pay for runs of some tokens (their codewords have to be brought to shared memory) and
    // codebooks of some size (the loop costs about 25 instructions a secondary).  8 heads, K and V, loop and
    // table, us: 4096 tokens, pages of 64: S = 32 131 and 51, S = 8 69 and 41; 768 tokens in sequences of
    //            pages of 16, 8 tokens  16 tokens  24 tokens   of 64, 8 tokens  16 tokens  24 tokens
    //   S = 8          23.3 31.2  21.3 23.1  19.6 20.3          21.1 26.8  20.4 19.0  18.4 18.2
    //   S = 16         27.4 33.7  25.6 24.4  24.5 21.9          24.9 29.3  25.1 21.6  23.5 19.5
    //   S = 32         35.2 40.1  34.9 30.2  33.1 26.4          32.8 35.8  33.9 25.4  33.0 23.5
    // One kernel takes the whole call, by the average: lengths stay on the device.  A batch that mixes single
    // tokens with a long run pays for it (S = 32, pages of 64, tables; the two parts as calls of their own): 64
    // single tokens and a run of 512 take 38 us (8 + 20), 256 and a run of 1024 106 us (27 + 25).
    const int search_from = S < 16 ? 24 : 16;
    const bool search = k->table && (!v || v->table) && S >= PW_SEARCH_S && n_tokens >= search_from * n_seqs;
    const size_t smem = search ? (size_t)(24 * S + 1) * sizeof(float4) : 0;
    const dim3 grid((unsigned)runs, (unsigned)k->heads, (unsigned)roles);
    const uint32_t bb = v && bv != bk ? 0 : bk;
    const bool runs_of_some = n_tokens >= PW_RUNS_FROM * n_seqs;
    auto kern = dtype == HQMQ_BF16 ? write_kernel<HQMQ_BF16>(bb, search, runs_of_some)
                                   : write_kernel<HQMQ_F32>(bb, search, runs_of_some);
    const dim3 block((search ? PW_TABLE_WARPS : PW_LOOP_WARPS) * 32);
    return launch_pdl(kern, grid, block, smem, stream, a) == cudaSuccess ? HQMQ_OK : HQMQ_ERR_CUDA;
}
