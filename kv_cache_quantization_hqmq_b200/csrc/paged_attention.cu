// paged_attention.cu -- decode-phase attention over paged coded caches with a
// prefix shared by the whole batch (include/hqmq.h, hqmq_attention_paged).
//
//   o = sum_t softmax_t(scale <q, K^_t>) V^_t
// over the prefix's tokens and the sequence's own.
//
// Work.  Tokens are taken in tiles of 32.  A KV head has these segments: the
// prefix, once for every 128 MT rows (row = query head of the group of one
// sequence; all B G of them), then each sequence's own tokens (G rows).  The
// tiles of all heads form one list, which the CTAs (one per SM) share out
// evenly in contiguous ranges, so lengths may differ as they like and the
// lengths stay on the device.  A CTA's piece of a segment gives a partial
// result per row, running maximum m (base 2), sum l and unnormalised output;
// k_paged_join joins a row's partials:
//   M = max m_i,  o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
//
// k_paged_attn, warps by role:
//   * 8 producer warps, 4 for K and 4 for V, decode a tile's codes from
//     global memory (fetched two tiles ahead, page ids four) through the
//     head's codeword table in shared memory into bf16 tiles [32 tokens][128]
//     in the tensor core's 128-byte swizzle: K is the K-major B operand of
//     S = Q K^T, V, in the same layout, the MN-major B operand of O += P V;
//   * one thread issues the products (tcgen05.mma, 128 rows, accumulators
//     and the A operands Q and P in tensor memory);
//   * 4 MT softmax warps, a thread per row: scores from tensor memory, online
//     softmax in base 2, P back as two bf16 terms P_hi + P_lo (about 16
//     significant bits).  The reference maximum moves only when a row's
//     maximum has grown by more than 2^8 (then O is rescaled in tensor
//     memory): weights up to 2^8 lose nothing in floating point.
// Segments with at most 32 rows put the same rows into each of the four
// 32-lane quarters; quarter w takes columns 8 w .. 8 w + 7 of every tile (the
// others get weight 0) and keeps a partial of its own.
//
// Every wait is bounded; one that runs out sets HQMQ_FLAG_TIMEOUT.
#include "paged.cuh"
#include "tcgen05.cuh"

namespace hqmq {

constexpr int PA_D = 128;
constexpr int PA_TILE = 32;                   // tokens of a tile
constexpr int PA_PART = 132;                  // floats of a row's partial: m, l, -, -, O[128]
constexpr int PA_CTAS = 148;                  // one per SM of a B200
constexpr int PA_MIN_TILES = 2;               // fewest tiles worth a CTA
constexpr int PA_REP_ROWS = 32;               // segments up to this many rows are replicated
constexpr float PA_RESCALE = 8.0f;
constexpr int TILE_BYTES = PA_TILE * PA_D * 2;
constexpr int MASK_RING = 8;
constexpr int PROD_WARPS = 8;

struct PagedAttnArgs {
    const uint16_t *q;
    PagesDev k, v;
    int B, Hk, G, rows;                       // rows = B G of a KV head over the prefix
    const int *seq_len, *table, *prefix_table;
    int max_pages, prefix_len;
    int row_tiles, prefix_tiles;              // segments of the prefix, tiles in each
    float sl2;                                // |scale| log2(e)
    uint32_t q_flip;                          // sign bits to flip in q (scale < 0)
    float *part_prefix, *part_own;            // [segment + CTA][rows][PA_PART]
    int prefix_slot_rows, own_slot_rows;
    DevStatus *st;
};

// Own tokens of sequence b, and their tiles.
__device__ __forceinline__ int own_len(const PagedAttnArgs &a, int b) {
    return min(max(__ldg(a.seq_len + b), 0), a.max_pages << a.k.page_shift);
}
__device__ __forceinline__ int own_tiles(const PagedAttnArgs &a, int b) {
    return a.max_pages ? (own_len(a, b) + PA_TILE - 1) / PA_TILE : 0;
}
// Tiles of the sequences before b and of all of them; warp-collective.
__device__ __forceinline__ int64_t tiles_before(const PagedAttnArgs &a, int b_end, int64_t *all) {
    const int lane = threadIdx.x & 31;
    int64_t before = 0, total = 0;
    if (a.max_pages) {
        for (int b = lane; b < a.B; b += 32) {
            const int n = own_tiles(a, b);
            total += n;
            if (b < b_end) before += n;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(FULL, before, o);
        total += __shfl_xor_sync(FULL, total, o);
    }
    *all = total;
    return before;
}

// How the list of all heads' tiles is shared out.
struct Shares {
    int64_t per_head, total;
    int ctas;
    __device__ __forceinline__ Shares(const PagedAttnArgs &a, int64_t own_total) {
        per_head = (int64_t)a.row_tiles * a.prefix_tiles + own_total;
        total = per_head * a.Hk;
        ctas = (int)min((int64_t)PA_CTAS, max(total / PA_MIN_TILES, (int64_t)1));
    }
    __device__ __forceinline__ int64_t begin(int c) const { return c * total / ctas; }
    __device__ __forceinline__ int owner(int64_t tile) const {
        return (int)(((tile + 1) * ctas - 1) / total);
    }
};

// A place in the list: tile `tile` of segment `seg` of `head`.
struct Cursor {
    int head, seg, tile, n_tiles, left;       // tiles of the segment, tiles left of the CTA's share
    __device__ __forceinline__ void settle(const PagedAttnArgs &a) {
        while (left > 0 && tile >= n_tiles) {
            tile = 0;
            if (++seg == a.row_tiles + a.B) {
                seg = 0;
                ++head;
            }
            n_tiles = seg < a.row_tiles ? a.prefix_tiles : own_tiles(a, seg - a.row_tiles);
        }
    }
    __device__ __forceinline__ int piece() const { return min(n_tiles - tile, left); }
    __device__ __forceinline__ void skip(const PagedAttnArgs &a, int n) {
        tile += n;
        left -= n;
        settle(a);
    }
    __device__ __forceinline__ bool prefix(const PagedAttnArgs &a) const { return seg < a.row_tiles; }
};

// Rows of a segment, whether they are replicated, and its softmax groups.
template <int MT> struct Rows {
    int n, base;
    bool rep;
    __device__ __forceinline__ Rows(const PagedAttnArgs &a, const Cursor &c) {
        if (c.prefix(a)) {
            base = c.seg * 128 * MT;
            n = min(a.rows - base, 128 * MT);
            rep = a.rows <= PA_REP_ROWS;
        } else {
            base = 0;
            n = a.G;
            rep = true;
        }
    }
    __device__ __forceinline__ int groups() const { return rep ? 1 : (n + 127) / 128; }
};

template <int MT> struct Shared {
    static constexpr int NB = MT == 1 ? 2 : 1;          // S and P buffers of a group
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full[MT], s_full[MT][NB], s_empty[MT][NB], p_full[MT][NB], p_empty[MT][NB];
    uint64_t heads;                                     // the producers, at a change of heads
    uint64_t drain;
    uint32_t mask[MASK_RING];                           // valid tokens of the last tiles
    Cursor start;
    uint32_t tmem;
    int failed;
};

// Tensor memory columns: O and Q of every group, then its S and P buffers.
template <int MT> struct Tmem {
    static constexpr int NB = Shared<MT>::NB;
    static constexpr uint32_t COLS = 512;
    __device__ __forceinline__ static uint32_t o(int g) { return g * 128; }
    __device__ __forceinline__ static uint32_t q(int g) { return MT * 128 + g * 64; }
    __device__ __forceinline__ static uint32_t s(int g, int i) { return MT * 192 + (g * NB + i) * 32; }
    __device__ __forceinline__ static uint32_t p(int g, int i) { return MT * 192 + (MT * NB + g * NB + i) * 32; }
    static_assert(MT * 192 + 2 * MT * NB * 32 <= 512, "tensor memory");
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}
// (r a, r b), each the IEEE fp32 product.
__device__ __forceinline__ float2 mul_pair(float r, float a, float b) {
    float2 o;
    asm("{.reg .b64 t, s;\n\tmov.b64 t, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\t"
        "mul.rn.f32x2 t, t, s;\n\tmov.b64 {%0, %1}, t;}"
        : "=f"(o.x), "=f"(o.y) : "f"(a), "f"(b), "f"(r));
    return o;
}
__device__ __forceinline__ float4 lds128(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------

// Codeword table of a head: entry i, copy r at byte (i R + r) 16, so that the
// 8 lanes of a 16-byte phase, reading copies lane % R, meet in no bank (R = 8)
// or in pairs (R = 4).  Entry 24 S is zero, for indices out of range.
template <int R> __host__ __device__ constexpr uint32_t table_bytes(uint32_t S) { return (24u * S + 1u) * R * 16u; }

template <int R>
__device__ __forceinline__ void build_table(const PagesDev &p, int head, uint32_t base, int thread) {
    const uint32_t n = 24u * p.S;
    for (uint32_t e = thread; e <= n; e += 128) {
        float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < n) c = codeword((int)(e % 24u), __ldg(p.cb + (size_t)head * p.S + e / 24u));
#pragma unroll
        for (int r = 0; r < R; ++r)
            sts128(base + (e * R + ((r + e) & (R - 1))) * 16, __float_as_uint(c.x), __float_as_uint(c.y),
                   __float_as_uint(c.z), __float_as_uint(c.w));
    }
}

// Words that hold a lane's 8 indices (bits 8 q b .. 8 q b + 8 b - 1).
template <int BT> struct RunWords { static constexpr int N = BT == 8 ? 2 : BT == 10 ? 3 : 4; };

// One tile on its way: lane (q, token) = (lane / 8, 8 sub + lane % 8) decodes
// chunks 8 q .. 8 q + 7 of that token; for the flags lane = token.
template <int BT> struct Slot {
    int t0, head;                             // tile whose page ids are under way
    bool first;                               // first tile of a piece
    int page;                                 // raw page id of token t0 + lane
    int d_t0, d_head;                         // tile whose codes are under way
    bool d_first;
    int d_page, l_page;                       // page of the decoded token, of token t0 + lane
    uint4 rad;
    uint32_t w[RunWords<BT>::N];
    uint32_t flags;                           // of token t0 + lane
    uint32_t mask;                            // valid tokens
    uint32_t f8;                              // flagged chunks among this lane's
    int slot;                                 // slot of the first of them
    uint2 val;                                // and its value
};

template <int BT, int R> struct Producer {
    const PagedAttnArgs &a;
    const PagesDev &p;
    const int lane, sub, q;
    const bool is_k;
    int base;                                 // flagged chunks before the next tile of the page

    __device__ __forceinline__ Producer(const PagedAttnArgs &a_, bool k, int sub_, int lane_)
        : a(a_), p(k ? a_.k : a_.v), lane(lane_), sub(sub_), q(lane_ >> 3), is_k(k), base(0) {}

    // Page ids of the cursor's tile.
    __device__ __forceinline__ void fetch_pages(Slot<BT> &s, Cursor &c, bool &first) {
        s.head = -1;
        if (c.left <= 0) return;
        s.head = c.head;
        s.t0 = c.tile * PA_TILE;
        s.first = first;
        const bool pre = c.prefix(a);
        const int b = c.seg - a.row_tiles;
        const int len = pre ? a.prefix_len : own_len(a, b);
        const int *tab = pre ? a.prefix_table : a.table + (size_t)b * a.max_pages;
        const int t = s.t0 + lane;
        s.page = -2;                          // no token
        if (t < len) s.page = __ldg(tab + (t >> p.page_shift));
        const int seg = c.seg, head = c.head;
        c.skip(a, 1);
        first = c.seg != seg || c.head != head;
    }

    // Codes of the tile whose page ids have arrived.
    __device__ __forceinline__ void fetch_codes(Slot<BT> &s) {
        s.d_head = s.head;
        if (s.head < 0) return;
        s.d_t0 = s.t0;
        s.d_first = s.first;
        int pg = s.page;
        if (pg != -2 && (pg < 0 || pg >= a.k.n_pages || pg >= a.v.n_pages)) {
            if (a.st) atomicOr(&a.st->flags, HQMQ_FLAG_BAD_PAGE);
            pg = -1;
        }
        s.mask = __ballot_sync(FULL, pg >= 0);
        s.l_page = pg;
        s.d_page = __shfl_sync(FULL, pg, sub * 8 + (lane & 7));
        s.rad = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < RunWords<BT>::N; ++i) s.w[i] = 0u;
        if (s.d_page >= 0) {
            const size_t at = p.at(s.d_page, s.head, (s.t0 + sub * 8 + (lane & 7)) & (p.page_size - 1));
            s.rad = __ldg(reinterpret_cast<const uint4 *>(p.radius + at * PG_CHUNKS) + q);
            const uint32_t *w = p.words + at * p.b;
            const uint32_t wo = (8u * q * p.b) >> 5;
#pragma unroll
            for (int i = 0; i < RunWords<BT>::N; ++i)
                if (BT || wo + i < p.b) s.w[i] = __ldg(w + wo + i);
        }
        s.flags = 0u;
        if (p.flags && pg >= 0) s.flags = __ldg(p.flags + p.at(pg, s.head, (s.t0 + lane) & (p.page_size - 1)));
    }

    // Slots of the flagged chunks and the first value, once the flags are there.
    __device__ __forceinline__ void fetch_values(Slot<BT> &s) {
        s.f8 = 0u;
        if (s.d_head < 0 || !p.flags) return;
        const int row = (s.d_t0 + lane) & (p.page_size - 1);
        const int row0 = __shfl_sync(FULL, row, 0);
        if (row0 == 0) base = 0;
        else if (s.d_first) {                 // a piece that starts inside a page
            const int pg = __shfl_sync(FULL, s.l_page, 0);
            base = pg >= 0 ? (int)flags_before(p.flags + p.at(pg, s.d_head, 0), row0, lane) : 0;
        }
        const int n = __popc(s.flags);
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += u;
        }
        int start = base + inc - n;
        if (p.page_size == 16 && lane >= 16) start -= __shfl_sync(0xFFFF0000u, inc - n, 16);
        base += __shfl_sync(FULL, inc, 31);
        const int tok = sub * 8 + (lane & 7);
        start = __shfl_sync(FULL, start, tok);
        const uint32_t f = __shfl_sync(FULL, s.flags, tok);
        s.f8 = (f >> (8 * q)) & 0xFFu;
        s.slot = start + __popc(f & ((1u << (8 * q)) - 1u));
        if (s.f8 && s.slot < p.cap) s.val = __ldg(p.slots(s.d_page, s.d_head) + s.slot);
    }

    // The lane's 8 chunks to the tile, then the flagged ones over them.
    __device__ __forceinline__ void decode(const Slot<BT> &s, uint32_t table, uint32_t tile) {
        constexpr int N = RunWords<BT>::N, LG = R == 8 ? 7 : 6;
        const uint32_t b = BT ? BT : p.b, sh = (8u * q * b) & 31u;
        uint32_t x[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = BT == 8 ? s.w[i] : i + 1 < N ? __funnelshift_r(s.w[i], s.w[i + 1], sh) : s.w[i] >> sh;
        const uint32_t copy = (uint32_t)(lane & (R - 1)) * 16u;
        const uint32_t zero = ((24u * p.S) << LG) | copy;
        const int tok = sub * 8 + (lane & 7);
        const uint32_t row = tile + (q >> 1) * (TILE_BYTES / 2) + (tok >> 3) * 1024 + (tok & 7) * 128;
        const uint32_t u0 = (q & 1) * 4, swz = tok & 7;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t v;                       // index << LG, other bits around it
            if (BT) {
                constexpr int BB = BT ? BT : 1;
                const int pos = j * BB, wi = pos >> 5, s5 = pos & 31;
                if (s5 + BB > 32 && wi + 1 < N) v = __funnelshift_r(x[wi], x[wi + 1 < N ? wi + 1 : wi], s5 - LG);
                else v = s5 >= LG ? x[wi] >> (s5 - LG) : x[wi] << (LG - s5);
            } else {
                const uint32_t pos = j * b, wi = pos >> 5, s5 = pos & 31u;
                uint32_t lo = x[0], hi = x[1];
#pragma unroll
                for (int i = 1; i < N; ++i)
                    if (wi == (uint32_t)i) {
                        lo = x[i];
                        hi = i + 1 < N ? x[i + 1] : 0u;
                    }
                v = __funnelshift_r(lo, hi, s5) << LG;
            }
            v = min((v & (((1u << b) - 1u) << LG)) | copy, zero);
            const float4 c = lds128(table + v);
            const uint32_t rw = j < 2 ? s.rad.x : j < 4 ? s.rad.y : j < 6 ? s.rad.z : s.rad.w;
            const float r = f16_bits_to_f32((j & 1) ? rw >> 16 : rw & 0xFFFFu);
            const float2 y01 = mul_pair(r, c.x, c.y), y23 = mul_pair(r, c.z, c.w);
            o[2 * (j & 1)] = bf16x2(y01.x, y01.y);
            o[2 * (j & 1) + 1] = bf16x2(y23.x, y23.y);
            if (j & 1) sts128(row + ((u0 + (j >> 1)) ^ swz) * 16, o[0], o[1], o[2], o[3]);
        }
        if (__any_sync(FULL, s.f8 != 0u)) {
            uint32_t f8 = s.f8;
            uint2 h = s.val;
            int slot = s.slot;
            while (f8) {
                if (slot >= p.cap) break;
                const int j = __ffs(f8) - 1;
                f8 &= f8 - 1u;
                sts64(row + ((u0 + (j >> 1)) ^ swz) * 16 + (j & 1) * 8,
                      bf16x2(f16_bits_to_f32(h.x & 0xFFFFu), f16_bits_to_f32(h.x >> 16)),
                      bf16x2(f16_bits_to_f32(h.y & 0xFFFFu), f16_bits_to_f32(h.y >> 16)));
                ++slot;
                if (f8 && slot < p.cap) h = __ldg(p.slots(s.d_page, s.d_head) + slot);
            }
        }
    }
};

// The producer warps wait for one another; false if one does not come.
__device__ __forceinline__ bool meet(uint64_t &bar, int &times, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar);
    return mbar_wait(&bar, times++ & 1);
}

template <int BT, int R, int MT>
__device__ __forceinline__ void produce(const PagedAttnArgs &a, Shared<MT> &sh, uint32_t tables, uint32_t tiles,
                                        int warp, int lane) {
    const bool is_k = warp < 4;
    const int sub = warp & 3;
    Producer<BT, R> pr(a, is_k, sub, lane);
    const uint32_t table = tables + (is_k ? 0u : table_bytes<R>(a.k.S));
    const uint32_t my_tiles = tiles + (is_k ? 0u : 2u * TILE_BYTES);
    uint64_t *full = is_k ? sh.k_full : sh.v_full, *empty = is_k ? sh.k_empty : sh.v_empty;
    Cursor c = sh.start;
    const int total = c.left;
    bool first = true;
    Slot<BT> s[2];
    pr.fetch_pages(s[0], c, first);
    pr.fetch_pages(s[1], c, first);
    pr.fetch_codes(s[0]);
    pr.fetch_codes(s[1]);
    pr.fetch_pages(s[0], c, first);
    pr.fetch_pages(s[1], c, first);
    pr.fetch_values(s[0]);
    int head = -1, meetings = 0;
    for (int n = 0; n < total; n += 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (n + i >= total) break;
            Slot<BT> &x = s[i];
            pr.fetch_values(s[1 - i]);
            if (x.d_head != head) {           // (all producers change heads at the same tile)
                if (!meet(sh.heads, meetings, lane)) {
                    sh.failed = 1;
                    return;
                }
                head = x.d_head;
                build_table<R>(pr.p, head, table, sub * 32 + lane);
                if (!meet(sh.heads, meetings, lane)) {
                    sh.failed = 1;
                    return;
                }
            }
            const int use = (n + i) >> 1;     // times this buffer has been filled
            if (use > 0 && !mbar_wait(empty + i, (use - 1) & 1)) {
                sh.failed = 1;
                return;
            }
            pr.decode(x, table, my_tiles + i * TILE_BYTES);
            if (warp == 0 && lane == 0) sh.mask[(n + i) & (MASK_RING - 1)] = x.mask;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full + i);
            pr.fetch_codes(x);
            pr.fetch_pages(x, c, first);
        }
    }
}

// ---------------------------------------------------------------------------
// the matrix products: one thread
// ---------------------------------------------------------------------------
template <int MT>
__device__ __forceinline__ bool issue_products(const PagedAttnArgs &a, Shared<MT> &sh, uint32_t tiles) {
    constexpr int NB = Shared<MT>::NB;
    const uint32_t tmem = sh.tmem;
    constexpr uint32_t id_s = mma_idesc(128, PA_TILE, false), id_o = mma_idesc(128, PA_D, true);
    Cursor c = sh.start;
    int tile_no = 0, cnt[MT], pieces[MT];
#pragma unroll
    for (int g = 0; g < MT; ++g) cnt[g] = pieces[g] = 0;
    while (c.left > 0) {
        const int n = c.piece();
        const int groups = Rows<MT>(a, c).groups();
#pragma unroll
        for (int g = 0; g < MT; ++g) {
            if (g >= groups) continue;
            if (!mbar_wait(&sh.q_full[g], pieces[g] & 1)) return false;
            ++pieces[g];
        }
        tc_fence_after();
        for (int i = 0; i <= n; ++i) {
            if (i < n) {                      // S = Q K^T of tile i
                const int st = (tile_no + i) & 1, use = (tile_no + i) >> 1;
                if (!mbar_wait(&sh.k_full[st], use & 1)) return false;
#pragma unroll
                for (int g = 0; g < MT; ++g) {
                    if (g >= groups) continue;
                    const int no = cnt[g] + i, buf = no % NB, u = no / NB;
                    if (u > 0 && !mbar_wait(&sh.s_empty[g][buf], (u - 1) & 1)) return false;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t b = tiles + st * TILE_BYTES + (k >> 2) * (TILE_BYTES / 2) + (k & 3) * 32;
                        mma_ts(tmem + Tmem<MT>::s(g, buf), tmem + Tmem<MT>::q(g) + k * 8, smem_desc(b, 16, 1024),
                               id_s, k > 0);
                    }
                    mma_commit(&sh.s_full[g][buf]);
                }
                mma_commit(&sh.k_empty[st]);
            }
            if (i > 0) {                      // O += P V of tile i - 1
                const int j = i - 1, st = (tile_no + j) & 1, use = (tile_no + j) >> 1;
                if (!mbar_wait(&sh.v_full[st], use & 1)) return false;
#pragma unroll
                for (int g = 0; g < MT; ++g) {
                    if (g >= groups) continue;
                    const int no = cnt[g] + j, buf = no % NB, u = no / NB;
                    if (!mbar_wait(&sh.p_full[g][buf], u & 1)) return false;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t b = tiles + 2 * TILE_BYTES + st * TILE_BYTES + k * 2048;
                        const uint64_t d = smem_desc(b, TILE_BYTES / 2, 1024);
                        mma_ts(tmem + Tmem<MT>::o(g), tmem + Tmem<MT>::p(g, buf) + k * 8, d, id_o, j > 0 || k > 0);
                        mma_ts(tmem + Tmem<MT>::o(g), tmem + Tmem<MT>::p(g, buf) + 16 + k * 8, d, id_o, 1u);
                    }
                    mma_commit(&sh.p_empty[g][buf]);
                }
                mma_commit(&sh.v_empty[st]);
            }
        }
        tile_no += n;
#pragma unroll
        for (int g = 0; g < MT; ++g)
            if (g < groups) cnt[g] += n;
        c.skip(a, n);
    }
    return true;
}

// ---------------------------------------------------------------------------
// softmax
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// N scores of a row (columns col0 ..), their weights relative to 2^ref as two
// bf16 terms in p[0 .. N/2) and p[16 .. 16 + N/2); returns their sum.
template <int N>
__device__ __forceinline__ float weights(const uint32_t (&s)[N], uint32_t mask, float sl2, float ref,
                                         uint32_t *hi, uint32_t *lo) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const float x0 = fmaf(__uint_as_float(s[j]), sl2, -ref), x1 = fmaf(__uint_as_float(s[j + 1]), sl2, -ref);
        const float p0 = (mask >> j) & 1u ? ex2(x0) : 0.f, p1 = (mask >> (j + 1)) & 1u ? ex2(x1) : 0.f;
        sum += p0 + p1;
        const uint32_t h = bf16x2(p0, p1);
        hi[j / 2] = h;
        lo[j / 2] = bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xFFFF0000u));
    }
    return sum;
}
template <int N> __device__ __forceinline__ float row_max(const uint32_t (&s)[N], uint32_t mask) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, (mask >> j) & 1u ? __uint_as_float(s[j]) : -INFINITY);
    return m;
}

template <int MT>
__device__ __forceinline__ bool softmax(const PagedAttnArgs &a, Shared<MT> &sh, int warp, int lane) {
    constexpr int NB = Shared<MT>::NB;
    const int g = warp >> 2, quad = warp & 3;
    const uint32_t tmem = sh.tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t t_o = tmem + Tmem<MT>::o(g), t_q = tmem + Tmem<MT>::q(g);
    Cursor c = sh.start;
    int tile_no = 0, cnt = 0;
    while (c.left > 0) {
        const int n = c.piece();
        const Rows<MT> rows(a, c);
        if (g >= rows.groups()) {
            tile_no += n;
            c.skip(a, n);
            continue;
        }
        // the rows' queries
        const int r = rows.rep ? lane : g * 128 + quad * 32 + lane;
        const bool live = r < rows.n;
        const bool pre = c.prefix(a);
        {
            const int gr = rows.base + r;
            const size_t qr = pre ? ((size_t)(gr / a.G) * a.Hk + c.head) * a.G + gr % a.G
                                  : ((size_t)(c.seg - a.row_tiles) * a.Hk + c.head) * a.G + r;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (live) v = __ldg(reinterpret_cast<const uint4 *>(a.q + qr * PA_D) + hf * 8 + i);
                    w[4 * i] = v.x ^ a.q_flip;
                    w[4 * i + 1] = v.y ^ a.q_flip;
                    w[4 * i + 2] = v.z ^ a.q_flip;
                    w[4 * i + 3] = v.w ^ a.q_flip;
                }
                tmem_st32(t_q + hf * 32, w);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full[g]);
        }
        float ref = -INFINITY, l = 0.f;       // exponents are relative to ref
        float m = -INFINITY;                  // largest score so far (times sl2)
        for (int i = 0; i < n; ++i, ++cnt) {
            const int buf = cnt % NB, u = cnt / NB;
            if (!mbar_wait(&sh.s_full[g][buf], u & 1)) return false;
            tc_fence_after();
            const uint32_t mask = sh.mask[(tile_no + i) & (MASK_RING - 1)];
            uint32_t p[32], s[32], s8[8];
            float mt;
            if (rows.rep) {
                tmem_ld8(tmem + Tmem<MT>::s(g, buf) + 8 * quad, s8);
                tmem_wait_ld();
                mt = row_max(s8, mask >> (8 * quad));
            } else {
                tmem_ld32(tmem + Tmem<MT>::s(g, buf), s);
                tmem_wait_ld();
                mt = row_max(s, mask);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.s_empty[g][buf]);
            m = fmaxf(m, mt * a.sl2);
            if (__any_sync(FULL, m > ref + PA_RESCALE)) {
                if (i > 0) {                  // O holds tiles before this one
                    const int pb = (cnt - 1) % NB, pu = (cnt - 1) / NB;
                    if (!mbar_wait(&sh.p_empty[g][pb], pu & 1)) return false;
                    tc_fence_after();
                    const float f = ref == -INFINITY ? 0.f : exp2f(ref - m);
                    l *= f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[32];
                        tmem_ld32(t_o + 32 * k, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(t_o + 32 * k, o);
                    }
                    tmem_wait_st();
                }
                ref = m;
            }
            const float rf = ref == -INFINITY ? 0.f : ref;
            if (rows.rep) {
                uint32_t h[4], lo[4];
                l += weights(s8, mask >> (8 * quad), a.sl2, rf, h, lo);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const bool mine = (e >> 2) == quad;
                    p[e] = mine ? h[e & 3] : 0u;
                    p[16 + e] = mine ? lo[e & 3] : 0u;
                }
            } else {
                l += weights(s, mask, a.sl2, rf, p, p + 16);
            }
            if (u > 0 && !mbar_wait(&sh.p_empty[g][buf], (u - 1) & 1)) return false;
            tc_fence_after();
            tmem_st32(tmem + Tmem<MT>::p(g, buf), p);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[g][buf]);
        }
        // the piece's partial
        const int pb = (cnt - 1) % NB, pu = (cnt - 1) / NB;
        if (!mbar_wait(&sh.p_empty[g][pb], pu & 1)) return false;
        tc_fence_after();
        const int seg = pre ? c.head * a.row_tiles + c.seg : c.head * a.B + c.seg - a.row_tiles;
        const int slot_rows = pre ? a.prefix_slot_rows : a.own_slot_rows;
        const int srow = rows.rep ? quad * rows.n + lane : r;
        float *dst = (pre ? a.part_prefix : a.part_own) +
                     (((size_t)seg + blockIdx.x) * slot_rows + srow) * PA_PART;
        if (live) *reinterpret_cast<float2 *>(dst) = make_float2(ref, l);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t o[32];
            tmem_ld32(t_o + 32 * k, o);
            tmem_wait_ld();
            if (live) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<uint4 *>(dst + 4 + 32 * k + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
        }
        tc_fence_before();
        tile_no += n;
        c.skip(a, n);
    }
    return true;
}

template <int BT, int R, int MT>
__global__ void __launch_bounds__((4 * MT + PROD_WARPS + 1) * 32, 1) k_paged_attn(PagedAttnArgs a) {
    constexpr int NB = Shared<MT>::NB;
    extern __shared__ uint8_t dyn[];
    __shared__ Shared<MT> sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (smem_addr(dyn) + 1023u) & ~1023u;         // the swizzle's period
    const uint32_t tiles = base, tables = base + 4 * TILE_BYTES;
    if (warp == 4 * MT + PROD_WARPS) {
        tmem_alloc(&sh.tmem, Tmem<MT>::COLS);
        if (lane == 0) {
            sh.failed = 0;
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh.k_full[i], 4);
                mbar_init(&sh.v_full[i], 4);
                mbar_init(&sh.k_empty[i], 1);
                mbar_init(&sh.v_empty[i], 1);
            }
            for (int g = 0; g < MT; ++g) {
                mbar_init(&sh.q_full[g], 4);
                for (int i = 0; i < NB; ++i) {
                    mbar_init(&sh.s_full[g][i], 1);
                    mbar_init(&sh.s_empty[g][i], 4);
                    mbar_init(&sh.p_full[g][i], 4);
                    mbar_init(&sh.p_empty[g][i], 1);
                }
            }
            mbar_init(&sh.heads, PROD_WARPS);
            mbar_init(&sh.drain, 1);
            mbar_init_fence();
        }
    }
    pdl_wait();
    if (warp == 0) {                          // this CTA's share of the list
        int64_t own_total;
        tiles_before(a, 0, &own_total);
        const Shares w(a, own_total);
        Cursor c = {0, 0, 0, 0, 0};
        if (w.total > 0 && (int)blockIdx.x < w.ctas) {
            const int64_t t0 = w.begin(blockIdx.x);
            c.left = (int)(w.begin(blockIdx.x + 1) - t0);
            c.head = (int)(t0 / w.per_head);
            int64_t rem = t0 - c.head * w.per_head;
            const int64_t pre = (int64_t)a.row_tiles * a.prefix_tiles;
            if (rem < pre) {
                c.seg = (int)(rem / a.prefix_tiles);
                c.tile = (int)(rem % a.prefix_tiles);
                c.n_tiles = a.prefix_tiles;
            } else {
                rem -= pre;
                for (int b0 = 0; b0 < a.B; b0 += 32) {
                    const int n = b0 + lane < a.B ? own_tiles(a, b0 + lane) : 0;
                    int64_t inc = n;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int64_t u = __shfl_up_sync(FULL, inc, o);
                        if (lane >= o) inc += u;
                    }
                    const unsigned hit = __ballot_sync(FULL, rem < inc);
                    if (hit) {
                        const int src = __ffs(hit) - 1;
                        c.seg = a.row_tiles + b0 + src;
                        c.n_tiles = __shfl_sync(FULL, n, src);
                        c.tile = (int)(rem - __shfl_sync(FULL, inc - n, src));
                        break;
                    }
                    rem -= __shfl_sync(FULL, inc, 31);
                }
            }
        }
        if (lane == 0) sh.start = c;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    if (warp < 4 * MT) {
        if (!softmax<MT>(a, sh, warp, lane)) sh.failed = 1;
    } else if (warp < 4 * MT + PROD_WARPS) {
        produce<BT, R, MT>(a, sh, tables, tiles, warp - 4 * MT, lane);
    } else if (lane == 0) {
        if (!issue_products<MT>(a, sh, tiles)) sh.failed = 1;
        mma_commit(&sh.drain);                // nothing may be in flight when tensor memory goes
        if (!mbar_wait(&sh.drain, 0)) sh.failed = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4 * MT + PROD_WARPS) {
        tc_fence_after();
        tmem_free(sh.tmem, Tmem<MT>::COLS);
    }
    if (threadIdx.x == 0 && sh.failed && a.st) atomicOr(&a.st->flags, HQMQ_FLAG_TIMEOUT);
}

// Joins the partials of every row; one warp per row.
template <int MT>
__global__ void __launch_bounds__(128)
k_paged_join(PagedAttnArgs a, void *o, int out_dtype, float *lse) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)a.B * a.Hk * a.G) return;
    const int g = (int)(row % a.G), head = (int)(row / a.G % a.Hk), b = (int)(row / a.G / a.Hk);
    int64_t own_total;
    const int64_t before = tiles_before(a, b, &own_total);
    const Shares w(a, own_total);
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // the partials of one segment: `copies` rows `stride` apart in each slot
    auto take = [&](int64_t first_tile, int n_tiles, const float *part, int64_t seg, int slot_rows, int srow,
                    int copies, int stride) {
        if (n_tiles == 0) return;
        const int c1 = w.owner(first_tile + n_tiles - 1);
        for (int c = w.owner(first_tile); c <= c1; ++c) {
            for (int k = 0; k < copies; ++k) {
                const float *p = part + ((seg + c) * slot_rows + srow + k * stride) * PA_PART;
                const float2 ml = *reinterpret_cast<const float2 *>(p);
                const float4 v = *reinterpret_cast<const float4 *>(p + 4 + 4 * lane);
                if (ml.x == -INFINITY) continue;             // no token
                const float mn = fmaxf(m, ml.x);
                const float f0 = exp2f(m - mn), f1 = exp2f(ml.x - mn);
                m = mn;
                l = l * f0 + ml.y * f1;
                acc.x = acc.x * f0 + v.x * f1;
                acc.y = acc.y * f0 + v.y * f1;
                acc.z = acc.z * f0 + v.z * f1;
                acc.w = acc.w * f0 + v.w * f1;
            }
        }
    };
    if (a.prefix_tiles) {
        const int r = b * a.G + g;
        const bool rep = a.rows <= PA_REP_ROWS;
        const int rt = r / (128 * MT);
        take(head * w.per_head + (int64_t)rt * a.prefix_tiles, a.prefix_tiles, a.part_prefix,
             (int64_t)head * a.row_tiles + rt, a.prefix_slot_rows, rep ? r : r % (128 * MT), rep ? 4 : 1, a.rows);
    }
    take(head * w.per_head + (int64_t)a.row_tiles * a.prefix_tiles + before, own_tiles(a, b), a.part_own,
         (int64_t)head * a.B + b, a.own_slot_rows, g, 4, a.G);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const size_t at = (size_t)row * PA_D + 4 * lane;
    if (out_dtype == HQMQ_BF16)
        *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(o) + at) =
            make_uint2(bf16x2(acc.x * inv, acc.y * inv), bf16x2(acc.z * inv, acc.w * inv));
    else
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(o) + at) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (lse && lane == 0) lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
}

// Workspace: partials of the prefix's segments, then of the sequences'.
struct PartPlan {
    int mt, row_tiles, prefix_slot_rows, own_slot_rows;
    uint64_t prefix_bytes, own_bytes;
};
inline PartPlan part_plan(int B, int Hq, int Hk, int max_tokens, int prefix_len) {
    PartPlan p;
    const int64_t rows = (int64_t)B * (Hq / Hk);
    p.mt = prefix_len > 0 && rows > 128 ? 2 : 1;
    p.row_tiles = prefix_len > 0 ? (int)((rows + 128 * p.mt - 1) / (128 * p.mt)) : 0;
    p.prefix_slot_rows = rows <= PA_REP_ROWS ? (int)(4 * rows) : 128 * p.mt;
    p.own_slot_rows = 4 * (Hq / Hk);
    p.prefix_bytes = prefix_len > 0 ? ((uint64_t)p.row_tiles * Hk + PA_CTAS) * p.prefix_slot_rows * PA_PART * 4 : 0;
    p.own_bytes = max_tokens > 0 ? ((uint64_t)B * Hk + PA_CTAS) * p.own_slot_rows * PA_PART * 4 : 0;
    return p;
}

template <int BT, int R, int MT>
static int launch_paged_attn(const PagedAttnArgs &a, int ctas, void *o, int out_dtype, float *lse,
                             cudaStream_t stream) {
    const size_t smem = 1024 + 4 * TILE_BYTES + table_bytes<R>(a.k.S) + table_bytes<R>(a.v.S);
    auto kern = k_paged_attn<BT, R, MT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return HQMQ_ERR_CUDA;
    const int64_t rows = (int64_t)a.B * a.Hk * a.G;
    if (ctas > 0 && launch_pdl(kern, dim3(ctas), dim3((4 * MT + PROD_WARPS + 1) * 32), smem, stream, a) != cudaSuccess)
        return HQMQ_ERR_CUDA;
    return launch_pdl(k_paged_join<MT>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, a, o, out_dtype,
                      lse) == cudaSuccess
               ? HQMQ_OK : HQMQ_ERR_CUDA;
}

template <int MT>
static int launch_paged_attn_mt(const PagedAttnArgs &a, int ctas, void *o, int out_dtype, float *lse,
                                cudaStream_t stream) {
    // the index widths of S = 8 and S = 32; 8 table copies (no bank conflicts) where both tables fit
    const bool same = a.k.b == a.v.b;
    if (same && a.k.b == 8) return launch_paged_attn<8, 8, MT>(a, ctas, o, out_dtype, lse, stream);
    const bool r8 = 1024 + 4 * TILE_BYTES + table_bytes<8>(a.k.S) + table_bytes<8>(a.v.S) + sizeof(Shared<MT>) <=
                    227 * 1024;
    if (same && a.k.b == 10)
        return r8 ? launch_paged_attn<10, 8, MT>(a, ctas, o, out_dtype, lse, stream)
                  : launch_paged_attn<10, 4, MT>(a, ctas, o, out_dtype, lse, stream);
    return launch_paged_attn<0, 4, MT>(a, ctas, o, out_dtype, lse, stream);
}

}  // namespace hqmq

extern "C" uint64_t hqmq_paged_attn_workspace_bytes(int B, int Hq, int Hk, int max_tokens,
                                                    int prefix_len) {
    const hqmq::PartPlan p = hqmq::part_plan(B, Hq, Hk, max_tokens, prefix_len);
    return ((p.prefix_bytes + p.own_bytes + 255) & ~255ull) + 256;
}

extern "C" int hqmq_launch_attention_paged(const uint16_t *q, const hqmq_kv_pages *k,
                                           const hqmq_kv_pages *v, uint32_t bk, uint32_t bv, int B, int Hq,
                                           const int32_t *seq_len, const int32_t *table, int max_pages,
                                           const int32_t *prefix_table, int prefix_len, float scale,
                                           void *o, int out_dtype, float *lse, void *ws,
                                           hqmq_status *st, cudaStream_t stream) {
    using namespace hqmq;
    const PartPlan p = part_plan(B, Hq, k->heads, max_pages * k->page_size, prefix_len);
    PagedAttnArgs a;
    a.q = q;
    a.k = pages_dev(k, bk);
    a.v = pages_dev(v, bv);
    a.B = B;
    a.Hk = k->heads;
    a.G = Hq / k->heads;
    a.rows = B * a.G;
    a.seq_len = seq_len;
    a.table = table;
    a.prefix_table = prefix_table;
    a.max_pages = max_pages;
    a.prefix_len = prefix_len;
    a.row_tiles = p.row_tiles;
    a.prefix_tiles = (prefix_len + PA_TILE - 1) / PA_TILE;
    const double sl2 = (double)scale * 1.4426950408889634;
    a.sl2 = (float)(sl2 < 0 ? -sl2 : sl2);
    a.q_flip = scale < 0 ? 0x80008000u : 0u;
    a.part_prefix = reinterpret_cast<float *>(ws);
    a.part_own = reinterpret_cast<float *>(reinterpret_cast<char *>(ws) + p.prefix_bytes);
    a.prefix_slot_rows = p.prefix_slot_rows;
    a.own_slot_rows = p.own_slot_rows;
    a.st = reinterpret_cast<DevStatus *>(st);
    // tiles there can be at most
    const int64_t most = a.Hk * ((int64_t)a.row_tiles * a.prefix_tiles +
                                 (int64_t)B * (((int64_t)max_pages * k->page_size + PA_TILE - 1) / PA_TILE));
    const int64_t want = most == 0 ? 0 : most / PA_MIN_TILES < 1 ? 1 : most / PA_MIN_TILES;
    const int ctas = (int)(want < PA_CTAS ? want : PA_CTAS);
    return p.mt == 2 ? launch_paged_attn_mt<2>(a, ctas, o, out_dtype, lse, stream)
                     : launch_paged_attn_mt<1>(a, ctas, o, out_dtype, lse, stream);
}
