// paged_attention.cu -- decode-phase attention over paged coded caches with a
// prefix shared by the whole batch (include/hqmq.h, hqmq_attention_paged).
//
//   o = sum_t softmax_t(scale <q, K^_t>) V^_t
// over the prefix's tokens and the sequence's own.
//
// Work.  Tokens are taken in tiles of 64.  A KV head has these segments: the
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
//   * scout warps look the tiles' pages and flag words up and tell the
//     producers where each token's codes and flagged values lie;
//   * 16 producer warps decode codes from global memory (fetched two tiles
//     ahead) through the head's codeword table in shared memory into bf16
//     tiles [64 tokens][128]
//     in the tensor core's 128-byte swizzle: K is the K-major B operand of
//     S = Q K^T, V, in the same layout, the MN-major B operand of O += P V;
//   * two warps issue the products (tcgen05.mma, 128 rows, accumulators
//     and the A operands Q and P in tensor memory);
//   * 4 MT softmax warps, a thread per row: scores from tensor memory, online
//     softmax in base 2, P back as bf16: two terms for bf16 outputs (they leave
//     2^-17 of a weight, so that the output's own half step, 2^-8, is all that
//     shows; one term leaves as much as that step), three for fp32 outputs
//     (2^-24, so that fp32 outputs are fp32 accurate).  The sum is
//     taken in fp32 before the rounding.  The reference maximum moves only when a row's
//     maximum has grown by more than 2^8 (then O is rescaled in tensor
//     memory): weights up to 2^8 lose nothing in floating point.
// Segments with at most 32 rows put the same rows into each of the four
// 32-lane quarters; quarter w takes columns 16 w .. 16 w + 15 of every tile
// (the others get weight 0) and keeps a partial of its own.
//
// MT = 2 (bf16 outputs, more than 128 rows over the prefix) decodes a tile once
// for 256 rows instead of twice: what bounds it is not the products (1536
// clocks a tile at 4096 multiply-adds a clock) but the chain scores -> softmax
// -> P V -> next scores of its two half-tile buffers, beside which the
// producers' decoding fits.  Measured (device time, calls back to back; bf16, S = 32, 8 KV heads, pages of
// 64): 32 sequences of up to 1000 tokens behind 131072: 230 us, 138 GFLOP at
// 600 TFLOP/s, 272 MB of codes (269 us as a call with cold caches).  With one
// term a weight it takes 204 us, and of the variants tried at that stage a score
// step of 64 tokens without double buffers took 235 us, one warp for all
// products 259 us.  One group of 128 rows (MT = 1) spends its time on the
// pieces' ends and the decoding: 16 sequences of up to 500 tokens behind 8191:
// 32 us.
//
// Every wait is bounded; one that runs out sets HQMQ_FLAG_TIMEOUT.
#include "paged.cuh"
#include "tcgen05.cuh"

namespace hqmq {

constexpr int PA_D = 128;
constexpr int PA_TILE = 64;                   // tokens of a tile
constexpr int PA_PART = 132;                  // floats of a row's partial: m, l, -, -, O[128]
constexpr int PA_CTAS = 148;                  // one per SM of a B200
// Segments up to this many rows are replicated (prefix of 4096, 8 rows a head, 32 heads, own parts of up to
// 1111 tokens: 52 us; 54 with the prefix's rows in one quarter only).
constexpr int PA_REP_ROWS = 32;
constexpr float PA_RESCALE = 8.0f;
constexpr int TILE_BYTES = PA_TILE * PA_D * 2;
constexpr int META_RING = 4;                  // tiles
constexpr int MASK_RING = 16;                 // the scouts are at most 10 tiles ahead of the softmax
constexpr int PROD_WARPS = 16;

struct PagedAttnArgs {
    const uint16_t *q;
    PagesDev k, v;
    uint32_t copies_k, copies_v;              // of their codeword tables
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

// a / b for a >= 0, b > 0 (a 64-bit division costs some 500 clocks).
__device__ __forceinline__ int quotient(int64_t a, int64_t b) {
    return (a | b) < (1ll << 32) ? (int)((uint32_t)a / (uint32_t)b) : (int)(a / b);
}

// How the list of all heads' tiles is shared out: CTA c takes the tiles
// [c len, (c + 1) len).
struct Shares {
    int64_t per_head, total;
    uint32_t len;
    __device__ __forceinline__ Shares(const PagedAttnArgs &a, int64_t own_total) {
        per_head = (int64_t)a.row_tiles * a.prefix_tiles + own_total;
        total = per_head * a.Hk;
        len = (uint32_t)max((total + PA_CTAS - 1) / PA_CTAS, (int64_t)1);
    }
    __device__ __forceinline__ int owner(int64_t tile) const { return quotient(tile, len); }
};

// A place in the list: tile `tile` of segment `seg` of `head`.
struct Cursor {
    int head, seg, tile, n_tiles, left;       // tiles of the segment, tiles left of the CTA's share
    __device__ __forceinline__ bool prefix(const PagedAttnArgs &a) const { return seg < a.row_tiles; }
    __device__ __forceinline__ int piece() const { return min(left, n_tiles - tile); }
    __device__ __forceinline__ void skip(const PagedAttnArgs &a, int n);
};
// Over the segments that have no tiles left.
__device__ __forceinline__ Cursor settled(const PagedAttnArgs &a, Cursor c) {
    while (c.left > 0 && c.tile >= c.n_tiles) {
        c.tile = 0;
        if (++c.seg == a.row_tiles + a.B) {
            c.seg = 0;
            ++c.head;
        }
        c.n_tiles = c.seg < a.row_tiles ? a.prefix_tiles : own_tiles(a, c.seg - a.row_tiles);
    }
    return c;
}
__device__ __forceinline__ void Cursor::skip(const PagedAttnArgs &a, int n) {
    tile += n;
    left -= n;
    if (tile >= n_tiles) *this = settled(a, *this);
}

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

// Warps: 4 MT softmax, 16 producers, two scouts, two for the products.  The
// block is launched with REGS a thread, and each group of four warps takes what it
// needs of their sum.  (The compiler spills at REGS: 24 to 28 bytes with three terms a weight, 8 to 32 with two
// groups, none or 4 with one group and two terms.)
template <int MT> struct Roles {
    static constexpr int SCOUT = 4 * MT + PROD_WARPS, SCOUTS = 2, PRODUCTS = SCOUT + SCOUTS;
    static constexpr int THREADS = (PRODUCTS + 2) * 32;
    static constexpr int REGS = MT == 1 ? 80 : 72;
    static constexpr int SOFTMAX = MT == 1 ? 128 : 80, PRODUCER = 72, REST = MT == 1 ? 64 : 56;
    static_assert(REGS * THREADS <= 65536, "registers of an SM");
    static_assert(128 * MT * SOFTMAX + 32 * PROD_WARPS * PRODUCER + 128 * REST <= REGS * THREADS, "register shares");
};

// What a scout warp finds out about a tile.
struct Meta {
    long long page[PA_TILE / 16];             // page * heads + head of every 16 tokens
    int row0, head;                           // row of the first token in its page
    uint32_t mask[2];                         // valid tokens
    uint2 flags[2][PA_TILE / 2];              // flag words of K and V
    uint32_t start[2][PA_TILE / 2];           // slots of their first values, 16 bits each
};

template <int MT> struct Shared {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full[MT], s_full[MT][2], s_empty[MT][2], p_full[MT][2], p_empty[MT][2];
    uint64_t meta_full[META_RING], meta_empty[META_RING];
    uint64_t pair_done;                                 // the second group has left a piece of two groups
    uint64_t heads;                                     // the producers, at a change of heads
    uint64_t drain[2];
    Meta meta[META_RING];
    uint2 mask[MASK_RING];                              // valid tokens of the last tiles
    Cursor start;
    int total, last_head;                               // tiles of the share, and the last one's head
    uint32_t tmem;
    int failed;
};

// Tensor memory columns.  One group of rows: O, Q, two S buffers, two P
// buffers.  Two groups: O and Q of both, and per group two buffers of 32
// columns for the scores of half a tile, which their weights then replace;
// replicated rows, which use one group only, take all four for two S buffers
// and the second group's O for their P buffers.  All 512 columns are allocated, so they start at address 0,
// a constant in every product.
template <int MT, int NT> struct Tmem {
    static constexpr uint32_t COLS = 512, P_COLS = 32 * NT;
    __host__ __device__ static constexpr uint32_t o(int g) { return g * 128; }
    __host__ __device__ static constexpr uint32_t q(int g) { return MT * 128 + g * 64; }
    __host__ __device__ static constexpr uint32_t s(int i) { return MT * 192 + i * 64; }
    __host__ __device__ static constexpr uint32_t half(int g, int h) { return MT * 192 + g * 64 + h * 32; }
    __host__ __device__ static constexpr uint32_t p(int i) { return MT == 1 ? 320 + i * P_COLS : 128 + i * 64; }
    static_assert(MT == 1 ? 320 + 2 * P_COLS <= 512 : P_COLS <= 64, "tensor memory");
};
// Where term t of the weights of tokens 16 k .. 16 k + 15 lies in P.
template <int NT> __host__ __device__ constexpr uint32_t p_col(int k, int t) { return (k >> 1) * 16 * NT + t * 16 + (k & 1) * 8; }

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
// scouts: warp s of N takes every N-th tile, lane l = its tokens 2 l and 2 l + 1
// ---------------------------------------------------------------------------
// A tile's page ids are fetched two of the warp's tiles before it is handed
// on, its flag words one.
template <int SCOUTS> struct Scout {
    const PagedAttnArgs &a;
    const int lane;
    Cursor c;
    int len;                                  // tokens of the cursor's segment
    const int *tab;                           // and its pages

    struct Tile {
        int head, t0, n, page;                // head < 0: none; n tokens
        uint2 fk, fv;
        uint32_t before;                      // flagged chunks in the page's earlier rows, this lane's, K | V << 16
    };

    __device__ __forceinline__ Scout(const PagedAttnArgs &a_, const Cursor &c_, int lane_, int first)
        : a(a_), lane(lane_), c(c_) {
        segment();
        step(first);
    }
    __device__ __forceinline__ void segment() {
        const bool pre = c.prefix(a);
        const int b = c.seg - a.row_tiles;
        len = c.left <= 0 ? 0 : pre ? a.prefix_len : own_len(a, b);
        tab = pre ? a.prefix_table : a.table + (size_t)b * a.max_pages;
    }
    __device__ __forceinline__ void step(int n) {
        for (; n > 0 && c.left > 0; --n) {
            --c.left;
            if (++c.tile >= c.n_tiles) {
                c = settled(a, c);
                segment();
            }
        }
    }

    __device__ __forceinline__ void pages(Tile &x) {
        x.head = -1;
        if (c.left <= 0) return;
        x.head = c.head;
        x.t0 = c.tile * PA_TILE;
        x.n = min(len - x.t0, PA_TILE);
        x.page = -2;                          // no token
        if (2 * lane < x.n) x.page = __ldg(tab + ((x.t0 + 2 * lane) >> a.k.page_shift));
        step(SCOUTS);
    }
    __device__ __forceinline__ void flags(Tile &x) {
        x.fk = x.fv = make_uint2(0u, 0u);
        x.before = 0u;
        if (x.head < 0) return;
        if (x.page != -2 && (x.page < 0 || x.page >= a.k.n_pages || x.page >= a.v.n_pages)) {
            if (a.st) atomicOr(&a.st->flags, HQMQ_FLAG_BAD_PAGE);
            x.page = -1;
        }
        const int row0 = x.t0 & (a.k.page_size - 1);
        const int pg0 = __shfl_sync(FULL, x.page, 0);
        if (x.page >= 0) {
            const size_t at = a.k.at(x.page, x.head, (x.t0 + 2 * lane) & (a.k.page_size - 1));
            if (a.k.flags) x.fk = __ldg(reinterpret_cast<const uint2 *>(a.k.flags + at));
            if (a.v.flags) x.fv = __ldg(reinterpret_cast<const uint2 *>(a.v.flags + at));
            if (2 * lane + 1 >= x.n) x.fk.y = x.fv.y = 0u;
        }
        if (row0 > 0 && pg0 >= 0) {           // pages of 128 or 256 tokens: the rows before the tile's
            const size_t at = a.k.at(pg0, x.head, 2 * lane);
            for (int r = 0; r < row0; r += PA_TILE) {
                uint2 k = make_uint2(0u, 0u), v = k;
                if (a.k.flags) k = __ldg(reinterpret_cast<const uint2 *>(a.k.flags + at + r));
                if (a.v.flags) v = __ldg(reinterpret_cast<const uint2 *>(a.v.flags + at + r));
                x.before += (__popc(k.x) + __popc(k.y)) | ((__popc(v.x) + __popc(v.y)) << 16);
            }
        }
    }
    __device__ __forceinline__ void hand_on(const Tile &x, Meta &m, uint2 *mask) {
        const int row0 = x.t0 & (a.k.page_size - 1);
        const uint32_t base = row0 > 0 ? __reduce_add_sync(FULL, x.before) : 0u;
        const uint32_t n0 = __popc(x.fk.x) | (__popc(x.fv.x) << 16);
        const uint32_t n = n0 + (__popc(x.fk.y) | (__popc(x.fv.y) << 16));
        uint32_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += u;
        }
        // slots start anew with every page: 8, 16 or more lanes
        const uint32_t before = __shfl_sync(FULL, inc - n, lane & ~((a.k.page_size >> 1) - 1) & 31);
        const uint32_t start = base + (inc - n) - before;
        m.flags[0][lane] = x.fk;
        m.flags[1][lane] = x.fv;
        m.start[0][lane] = (start & 0xFFFFu) | ((start + n0) << 16);
        m.start[1][lane] = (start >> 16) | ((start + n0) & 0xFFFF0000u);
        if ((lane & 7) == 0) m.page[lane >> 3] = (long long)x.page * a.k.heads + x.head;
        const uint32_t ok = __ballot_sync(FULL, x.page >= 0);
        if (lane < 2) {                       // half of the mask: two groups of 16 tokens
            const uint32_t g = ok >> (16 * lane);
            const int rest = x.n - 32 * lane;
            uint32_t w = ((g & 1u) ? 0xFFFFu : 0u) | ((g & 0x100u) ? 0xFFFF0000u : 0u);
            if (rest < 32) w &= rest <= 0 ? 0u : (1u << rest) - 1u;
            m.mask[lane] = w;
            reinterpret_cast<uint32_t *>(mask)[lane] = w;
        }
        if (lane == 0) {
            m.row0 = row0;
            m.head = x.head;
        }
    }
};

template <int MT>
__device__ __forceinline__ bool scout(const PagedAttnArgs &a, Shared<MT> &sh, int which, int lane) {
    constexpr int SCOUTS = Roles<MT>::SCOUTS;
    Scout<SCOUTS> s(a, sh.start, lane, which);
    const int total = sh.total;
    typename Scout<SCOUTS>::Tile now, next;   // (flag words under way; page ids under way)
    next.head = -1;
    // the first two rounds only fill the pipeline
#pragma unroll 1
    for (int t = which - 2 * SCOUTS; t < total; t += SCOUTS) {
        const typename Scout<SCOUTS>::Tile x = now;
        now = next;
        s.flags(now);
        s.pages(next);
        if (t < which) continue;
        const int slot = t % META_RING;
        if (!mbar_wait(&sh.meta_empty[slot], ((t / META_RING) & 1) ^ 1)) return false;
        s.hand_on(x, sh.meta[slot], &sh.mask[t % MASK_RING]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.meta_full[slot]);
    }
    return true;
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------

// Codeword table of a head: entry i, copy r at byte (i R + r) 16, so that the
// 8 lanes of a 16-byte phase, reading copies lane % R, meet in no bank (R = 8)
// or in pairs (R = 4).  Entry 24 S is zero, for indices out of range.
__host__ __device__ constexpr uint32_t table_bytes(uint32_t S, uint32_t R) { return (24u * S + 1u) * R * 16u; }
// Shared memory: two K and two V tiles, the tables, then Shared.
__host__ __device__ constexpr uint32_t attn_table_end(uint32_t sk, uint32_t rk, uint32_t sv, uint32_t rv) {
    return 4u * TILE_BYTES + ((table_bytes(sk, rk) + table_bytes(sv, rv) + 127u) & ~127u);
}

__device__ __forceinline__ void build_table(const PagesDev &p, uint32_t R, int head, uint32_t base, int thread) {
    const uint32_t n = 24u * p.S;
    for (uint32_t e = thread; e <= n; e += PROD_WARPS * 16) {
        float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < n) c = codeword((int)(e % 24u), __ldg(p.cb + (size_t)head * p.S + e / 24u));
#pragma unroll 1
        for (uint32_t r = 0; r < R; ++r)
            sts128(base + (e * R + ((r + e) & (R - 1))) * 16, __float_as_uint(c.x), __float_as_uint(c.y),
                   __float_as_uint(c.z), __float_as_uint(c.w));
    }
}

// Words that hold a lane's 16 indices (bits 16 h b .. 16 h b + 16 b - 1).
template <int BT> struct RunWords { static constexpr int N = BT == 8 ? 4 : BT == 10 ? 5 : 6; };

// One tile's codes on their way: lane (h, token) = (lane / 16, 16 sub + lane
// % 16) decodes chunks 16 h .. 16 h + 15 of that token.
template <int BT> struct Slot {
    int head;
    uint4 rad[2];
    uint32_t w[RunWords<BT>::N];
    uint32_t flagged;                         // flagged chunks among this lane's
    int slot;                                 // slot of the first of them
    uint2 val;                                // and its value
    const uint2 *slots;
};

template <int BT> struct Producer {
    const PagesDev &p;
    const int lane, h, tok, which;
    const uint32_t stride, copy;              // bytes of a table entry, this lane's copy in the table
    const uint32_t row;                       // this lane's 128 bytes in a tile, its swizzle in bits 4 - 6

    __device__ __forceinline__ Producer(const PagesDev &p_, int which_, int sub, int lane_, uint32_t R, uint32_t table)
        : p(p_), lane(lane_), h(lane_ >> 4), tok(sub * 16 + (lane_ & 15)), which(which_), stride(R * 16u),
          copy(table + (lane_ & (R - 1u)) * 16u),
          row(h * (TILE_BYTES / 2) + (tok >> 3) * 1024 + (tok & 7) * 128 + (tok & 7) * 16) {}

    __device__ __forceinline__ void fetch(Slot<BT> &s, const Meta &m) {
        s.head = m.head;
        s.rad[0] = s.rad[1] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < RunWords<BT>::N; ++i) s.w[i] = 0u;
        s.flagged = 0u;
        if (!((m.mask[tok >> 5] >> (tok & 31)) & 1u)) return;
        const long long ph = m.page[tok >> 4];
        const size_t at = ((size_t)ph << p.page_shift) + ((m.row0 + tok) & (p.page_size - 1));
        const uint4 *rad = reinterpret_cast<const uint4 *>(p.radius + at * PG_CHUNKS) + 2 * h;
        s.rad[0] = __ldg(rad);
        s.rad[1] = __ldg(rad + 1);
        const uint32_t b = BT ? BT : p.b, wo = (h * b) >> 1;
        const uint32_t *w = p.words + at * b + wo;
#pragma unroll
        for (int i = 0; i < RunWords<BT>::N; ++i)
            if (BT || wo + i < b) s.w[i] = __ldg(w + i);
        const uint32_t f = reinterpret_cast<const uint32_t *>(m.flags[which])[tok];
        s.flagged = (f >> (16 * h)) & 0xFFFFu;
        s.slot = reinterpret_cast<const uint16_t *>(m.start[which])[tok] + (h ? __popc(f & 0xFFFFu) : 0);
        s.slots = reinterpret_cast<const uint2 *>(p.val) + (size_t)ph * p.cap;
        if (s.flagged && s.slot < p.cap) s.val = __ldg(s.slots + s.slot);
    }

    // The lane's 16 chunks to the tile, then the flagged ones over them.
    __device__ __forceinline__ void decode(const Slot<BT> &s, uint32_t tile) {
        constexpr int N = RunWords<BT>::N;
        const uint32_t b = BT ? BT : p.b, sh = BT ? 0u : ((h * b) & 1u) * 16u;
        uint32_t x[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = BT ? s.w[i] : i + 1 < N ? __funnelshift_r(s.w[i], s.w[i + 1], sh) : s.w[i] >> sh;
        const uint32_t zero = 24u * p.S, to = tile + row;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float4 c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = 4 * g + k;
                uint32_t v;                   // the index, other bits above it
                if (BT) {
                    constexpr int BB = BT ? BT : 1;
                    const int pos = j * BB, wi = pos >> 5, s5 = pos & 31;
                    if (s5 + BB > 32) v = __funnelshift_r(x[wi], x[wi + 1 < N ? wi + 1 : wi], s5);
                    else v = x[wi] >> s5;
                } else {
                    const uint32_t pos = j * b, wi = pos >> 5, s5 = pos & 31u;
                    uint32_t lo = x[0], hi = x[1];
#pragma unroll
                    for (int i = 1; i < N; ++i)
                        if (wi == (uint32_t)i) {
                            lo = x[i];
                            hi = i + 1 < N ? x[i + 1] : 0u;
                        }
                    v = __funnelshift_r(lo, hi, s5);
                }
                c[k] = lds128(min(v & ((1u << b) - 1u), zero) * stride + copy);
            }
            const uint4 r4 = s.rad[g >> 1];
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                const uint32_t rw = g & 1 ? (k ? r4.w : r4.z) : (k ? r4.y : r4.x);
                const float r0 = f16_bits_to_f32(rw & 0xFFFFu), r1 = f16_bits_to_f32(rw >> 16);
                const float2 y0 = mul_pair(r0, c[k].x, c[k].y), y1 = mul_pair(r0, c[k].z, c[k].w);
                const float2 y2 = mul_pair(r1, c[k + 1].x, c[k + 1].y), y3 = mul_pair(r1, c[k + 1].z, c[k + 1].w);
                sts128(to ^ ((2 * g + (k >> 1)) * 16), bf16x2(y0.x, y0.y), bf16x2(y1.x, y1.y), bf16x2(y2.x, y2.y),
                       bf16x2(y3.x, y3.y));
            }
        }
        uint32_t f = s.flagged;
        uint2 v = s.val;
        int slot = s.slot;
        while (f && slot < p.cap) {
            const int j = __ffs(f) - 1;
            f &= f - 1u;
            sts64((to ^ ((j >> 1) * 16)) + (j & 1) * 8,
                  bf16x2(f16_bits_to_f32(v.x & 0xFFFFu), f16_bits_to_f32(v.x >> 16)),
                  bf16x2(f16_bits_to_f32(v.y & 0xFFFFu), f16_bits_to_f32(v.y >> 16)));
            ++slot;
            if (f && slot < p.cap) v = __ldg(s.slots + slot);
        }
    }
};

// The producer warps wait for one another; false if one does not come.
__device__ __forceinline__ bool meet(uint64_t &bar, int &times, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar);
    return mbar_wait(&bar, times++ & 1);
}

// Warps 0-7 take the even tiles, 8-15 the odd ones; of each eight, four
// decode K and four V, sixteen tokens each.  A tile's codes are fetched before
// the warp's last one is decoded.
template <int BT, int MT>
__device__ __forceinline__ bool produce(const PagedAttnArgs &a, Shared<MT> &sh, uint32_t tables, uint32_t tiles,
                                        int warp, int lane) {
    const int st = warp >> 3, which = (warp >> 2) & 1, sub = warp & 3;
    const PagesDev &p = which ? a.v : a.k;
    const uint32_t R = which ? a.copies_v : a.copies_k;
    const uint32_t table = tables + (which ? table_bytes(a.k.S, a.copies_k) : 0u);
    Producer<BT> pr(p, which, sub, lane, R, table);
    const uint32_t tile = tiles + (which ? 2u * TILE_BYTES : 0u) + st * TILE_BYTES;
    uint64_t *full = (which ? sh.v_full : sh.k_full) + st, *empty = (which ? sh.v_empty : sh.k_empty) + st;
    const int total = sh.total, last_head = sh.last_head;
    int head = sh.start.head, meetings = 0;
    uint32_t par = 1;                         // phase of `empty` to wait for
    Slot<BT> x, next;

    // (the first head's tables while the scouts look the first tiles up)
    if (total > 0) {
        build_table(p, R, head, table, (st * 4 + sub) * 32 + lane);
        if (!meet(sh.heads, meetings, lane)) return false;
    }
    next.head = head;
    // the first round only fetches; one round past the end meets the heads that are left
#pragma unroll 1
    for (int n = st - 2; n < total + 2; n += 2) {
        x = next;
        next.head = last_head;
        if (n + 2 < total) {
            const int r = (n + 2) % META_RING;
            if (!mbar_wait(&sh.meta_full[r], ((n + 2) / META_RING) & 1)) return false;
            pr.fetch(next, sh.meta[r]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.meta_empty[r]);
        }
        // every producer passes through every head: they meet, build its tables and meet again
        while (n >= 0 && head < x.head) {
            if (!meet(sh.heads, meetings, lane)) return false;
            ++head;
            build_table(p, R, head, table, (st * 4 + sub) * 32 + lane);
            if (!meet(sh.heads, meetings, lane)) return false;
        }
        if (n < 0 || n >= total) continue;
        if (!mbar_wait(empty, par)) return false;
        par ^= 1u;
        pr.decode(x, tile);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
    }
    return true;
}

// ---------------------------------------------------------------------------
// the matrix products: a warp for the scores, one for P V
// ---------------------------------------------------------------------------
// Steps are tiles (buffer = stage) or, for two groups, half tiles (buffer =
// half).  Each step of a group goes scores -> softmax -> P V; where P replaces
// S, the next scores in that buffer wait for P V.  Under the producers' load on
// shared memory a look at a barrier takes some 250 clocks, so the two products
// have a warp each (of which one lane issues), the softmax looks ahead, and one
// copy of code serves every stage, buffer and group (instruction fetch, too, is
// a limit of a kernel with so many roles).  Weights in columns of their own,
// so that the next scores need not wait for P V, take one more barrier in the
// softmax: 224 us for 207 (131072 tokens, 256 rows).
struct Operands {
    static constexpr uint32_t HI = (1024u >> 4) | (1u << 14) | (2u << 29);    // descriptor: sbo, version, swizzle
    uint32_t k_lo, v_lo;
    __device__ __forceinline__ Operands(uint32_t tiles)
        : k_lo((tiles >> 4) | (1u << 16)), v_lo(((tiles + 2 * TILE_BYTES) >> 4) | ((TILE_BYTES / 2 / 16) << 16)) {}
};

template <int MT, int NT>
__device__ __forceinline__ bool issue_scores(const PagedAttnArgs &a, Shared<MT> &sh, uint32_t tiles, bool leader) {
    using TM = Tmem<MT, NT>;
    const Operands op(tiles);
    Cursor c = sh.start;
    int no = 0;                               // tiles so far: stage no % 2, phase no / 2
    uint32_t ph = 0, pq = 0;                  // phases of the groups' two buffers (bit 2 g + b), and of q_full
    while (c.left > 0) {
        const int n = c.piece();
        const Rows<MT> rows(a, c);
        const int groups = rows.groups();
        const bool two = MT == 1 || rows.rep;
        for (int g = 0; g < groups; ++g) {
            if (!mbar_wait(&sh.q_full[g], (pq >> g) & 1)) return false;
            pq ^= 1u << g;
        }
        const uint32_t idesc = two ? mma_idesc(128, PA_TILE, false) : mma_idesc(128, PA_TILE / 2, false);
        const int steps = two ? 1 : 2 * groups;               // of a tile: half, then group
        for (const int end = no + n; no < end; ++no) {
            const int st = no & 1;
            if (!mbar_wait(&sh.k_full[st], (no >> 1) & 1)) return false;
#pragma unroll 1
            for (int i = 0; i < steps; ++i) {
                const int h = i >= groups ? 1 : 0, g = i - h * groups, b = two ? st : h;
                if (!mbar_wait(two ? &sh.s_empty[g][b] : &sh.p_empty[g][b], ((ph >> (2 * g + b)) & 1) ^ 1)) return false;
                ph ^= 1u << (2 * g + b);
                tc_fence_after();
                const uint32_t d = two ? TM::s(b) : TM::half(g, h), q = TM::q(g);
                const uint32_t lo = op.k_lo + st * (TILE_BYTES >> 4) + h * (32 * 128 / 16);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)   // 32 bytes of a row; the second 64 elements in the next block
                        mma_ts(d, q + k * 8, lo + (k >> 2) * (TILE_BYTES / 2 / 16) + (k & 3) * 2, op.HI, idesc, k > 0);
                    mma_commit(&sh.s_full[g][b]);
                }
            }
            if (leader) mma_commit(&sh.k_empty[st]);
        }
        c.skip(a, n);
    }
    return true;
}

template <int MT, int NT>
__device__ __forceinline__ bool issue_outputs(const PagedAttnArgs &a, Shared<MT> &sh, uint32_t tiles, bool leader) {
    using TM = Tmem<MT, NT>;
    constexpr uint32_t idesc = mma_idesc(128, PA_D, true);
    const Operands op(tiles);
    Cursor c = sh.start;
    int no = 0;
    uint32_t ph = 0;
    while (c.left > 0) {
        const int n = c.piece();
        const Rows<MT> rows(a, c);
        const int groups = rows.groups();
        const bool two = MT == 1 || rows.rep;
        const int steps = two ? 1 : 2 * groups;
        uint32_t add = 0;                     // bit g: O of the group holds earlier steps
        for (const int end = no + n; no < end; ++no) {
            const int st = no & 1;
            if (!mbar_wait(&sh.v_full[st], (no >> 1) & 1)) return false;
#pragma unroll 1
            for (int i = 0; i < steps; ++i) {
                const int h = i >= groups ? 1 : 0, g = i - h * groups, b = two ? st : h;
                if (!mbar_wait(&sh.p_full[g][b], (ph >> (2 * g + b)) & 1)) return false;
                ph ^= 1u << (2 * g + b);
                tc_fence_after();
                const uint32_t acc = (add >> g) & 1u;
                add |= 1u << g;
                const uint32_t o = TM::o(g), pc = two ? TM::p(b) : TM::half(g, h);
                const uint32_t lo = op.v_lo + st * (TILE_BYTES >> 4) + h * (32 * 128 / 16);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < PA_TILE / 16; ++k) {
                        if (k == 2 && !two) break;
#pragma unroll
                        for (int x = 0; x < NT; ++x)
                            mma_ts(o, pc + p_col<NT>(k, x), lo + k * 128, op.HI, idesc, k || x ? 1u : acc);
                    }
                    mma_commit(&sh.p_empty[g][b]);
                }
            }
            if (leader) mma_commit(&sh.v_empty[st]);
        }
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
// (a0, a1) m + c, and (a0, a1) + (b0, b1), as packed operations.
__device__ __forceinline__ float2 fma_pair(float a0, float a1, float m, float c) {
    float2 o;
    asm("{.reg .b64 t, u, v;\n\tmov.b64 t, {%2, %3};\n\tmov.b64 u, {%4, %4};\n\tmov.b64 v, {%5, %5};\n\t"
        "fma.rn.f32x2 t, t, u, v;\n\tmov.b64 {%0, %1}, t;}"
        : "=f"(o.x), "=f"(o.y) : "f"(a0), "f"(a1), "f"(m), "f"(c));
    return o;
}
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) {
    float2 o;
    asm("{.reg .b64 t, u;\n\tmov.b64 t, {%2, %3};\n\tmov.b64 u, {%4, %5};\n\t"
        "add.rn.f32x2 t, t, u;\n\tmov.b64 {%0, %1}, t;}"
        : "=f"(o.x), "=f"(o.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return o;
}
__device__ __forceinline__ float2 sub_pair(float2 a, float2 b) {     // a + (-1) b: no sign flips beside it
    float2 o;
    asm("{.reg .b64 t, u, v;\n\tmov.b64 t, {%2, %3};\n\tmov.b64 u, {%4, %5};\n\tmov.b64 v, {%6, %6};\n\t"
        "fma.rn.f32x2 t, u, v, t;\n\tmov.b64 {%0, %1}, t;}"
        : "=f"(o.x), "=f"(o.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(-1.0f));
    return o;
}
__device__ __forceinline__ float2 bf16_pair(uint32_t h) {
    return make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
}

// Weights 2^(s sl2 - ref) of 16 scores as NT bf16 terms (term t of pair j in
// out[t][j]); sum gets them added.
template <int NT>
__device__ __forceinline__ void weights(const uint32_t *s, float sl2, float ref, float2 &sum, uint32_t (&out)[NT][8]) {
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        const float2 x = fma_pair(__uint_as_float(s[j]), __uint_as_float(s[j + 1]), sl2, -ref);
        float2 p = make_float2(ex2(x.x), ex2(x.y));
        sum = add_pair(sum, p);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t h = bf16x2(p.x, p.y);
            out[t][j / 2] = h;
            if (t + 1 < NT) {
                const float2 f = bf16_pair(h);
                p = sub_pair(p, f);
            }
        }
    }
}
template <int N> __device__ __forceinline__ float row_max(const uint32_t *s) {
    float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        m0 = fmaxf(fmaxf(m0, __uint_as_float(s[j])), __uint_as_float(s[j + 1]));
        m1 = fmaxf(fmaxf(m1, __uint_as_float(s[j + 2])), __uint_as_float(s[j + 3]));
    }
    return fmaxf(m0, m1);
}
// Scores of columns that are not in the mask become -inf (weight 0: sl2 > 0).
template <int N> __device__ __forceinline__ void hide(uint32_t (&s)[N], uint32_t mask) {
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (!((mask >> j) & 1u)) s[j] = 0xFF800000u;
}

template <int MT, int NT> struct Softmax {
    using TM = Tmem<MT, NT>;
    const PagedAttnArgs &a;
    Shared<MT> &sh;
    const int g, quad, lane;
    const uint32_t lanes;                     // tensor memory address of this warp's lanes
    float ref, m;                             // exponents are relative to ref; largest score so far (times sl2)
    float2 l;
    uint32_t ph;                              // phases of the group's two buffers
    uint32_t there;                           // the next step's scores are there

    __device__ __forceinline__ void arrive(uint64_t *bar) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    }

    // Moves ref to m if some row's maximum has outgrown it; `done` completes (phase `par`) with the
    // products of the tiles before, which O then holds (nullptr: there are none).
    __device__ __forceinline__ bool rescale(float mt, uint64_t *done, uint32_t par) {
        m = fmaxf(m, mt * a.sl2);
        if (!__any_sync(FULL, m > ref + PA_RESCALE)) return true;
        if (done) {
            if (!mbar_wait(done, par)) return false;
            tc_fence_after();
            const float f = ref == -INFINITY ? 0.f : exp2f(ref - m);
            l.x *= f;
            l.y *= f;
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
                uint32_t o[8];
                tmem_ld8(lanes + TM::o(g) + 8 * k, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st8(lanes + TM::o(g) + 8 * k, o);
            }
            tmem_wait_st();
        }
        ref = m;
        return true;
    }
    // The weights of 16 scores to their columns of P.
    __device__ __forceinline__ void put(const uint32_t *s, float rf, uint32_t p) {
        uint32_t w[NT][8];
        weights<NT>(s, a.sl2, rf, l, w);
#pragma unroll
        for (int t = 0; t < NT; ++t) tmem_st8(p + 16 * t, w[t]);
    }

    // Replicated rows: 16 of the columns of the piece's tile i, in buffer b.
    __device__ __forceinline__ bool tile_rep(int i, int b, const uint2 &valid) {
        const uint32_t p_there = mbar_test(&sh.p_empty[0][b], ((ph >> b) & 1) ^ 1);
        if (!there && !mbar_wait(&sh.s_full[0][b], (ph >> b) & 1)) return false;
        tc_fence_after();
        const uint32_t mask = ((quad & 2 ? valid.y : valid.x) >> (16 * (quad & 1))) & 0xFFFFu;
        uint32_t s[16];
        tmem_ld16(lanes + TM::s(b) + 16 * quad, s);
        tmem_wait_ld();
        arrive(&sh.s_empty[0][b]);
        if (mask != 0xFFFFu) hide(s, mask);
        if (!rescale(row_max<16>(s), i > 0 ? &sh.p_empty[0][b ^ 1] : nullptr, ((ph >> (b ^ 1)) & 1) ^ 1)) return false;
        if (!p_there && !mbar_wait(&sh.p_empty[0][b], ((ph >> b) & 1) ^ 1)) return false;
        tc_fence_after();
        put(s, ref == -INFINITY ? 0.f : ref, lanes + TM::p(b) + p_col<NT>(quad, 0));
        there = mbar_test(&sh.s_full[0][b ^ 1], (ph >> (b ^ 1)) & 1);
        tmem_wait_st();
        arrive(&sh.p_full[0][b]);
        ph ^= 1u << b;
        return true;
    }
    // A row per thread, one group: all 64 columns of tile i, in buffer b.
    __device__ __forceinline__ bool tile_full(int i, int b, const uint2 &valid) {
        const uint32_t p_there = mbar_test(&sh.p_empty[g][b], ((ph >> b) & 1) ^ 1);
        if (!there && !mbar_wait(&sh.s_full[g][b], (ph >> b) & 1)) return false;
        tc_fence_after();
        const uint2 mask = valid;
        uint32_t s0[32], s1[32];
        tmem_ld32(lanes + TM::s(b), s0);
        tmem_ld32(lanes + TM::s(b) + 32, s1);
        tmem_wait_ld();
        arrive(&sh.s_empty[g][b]);
        if (mask.x != FULL) hide(s0, mask.x);
        if (mask.y != FULL) hide(s1, mask.y);
        if (!rescale(fmaxf(row_max<32>(s0), row_max<32>(s1)), i > 0 ? &sh.p_empty[g][b ^ 1] : nullptr,
                     ((ph >> (b ^ 1)) & 1) ^ 1))
            return false;
        if (!p_there && !mbar_wait(&sh.p_empty[g][b], ((ph >> b) & 1) ^ 1)) return false;
        tc_fence_after();
        const float rf = ref == -INFINITY ? 0.f : ref;
        const uint32_t tp = lanes + TM::p(b);
        put(s0, rf, tp + p_col<NT>(0, 0));
        put(s0 + 16, rf, tp + p_col<NT>(1, 0));
        put(s1, rf, tp + p_col<NT>(2, 0));
        put(s1 + 16, rf, tp + p_col<NT>(3, 0));
        there = mbar_test(&sh.s_full[g][b ^ 1], (ph >> (b ^ 1)) & 1);
        tmem_wait_st();
        arrive(&sh.p_full[g][b]);
        ph ^= 1u << b;
        return true;
    }
    // A row per thread, two groups: half h of a tile, its weights in the place of its scores.
    __device__ __forceinline__ bool half_tile(bool first, int h, const uint32_t &valid) {
        if (!there && !mbar_wait(&sh.s_full[g][h], (ph >> h) & 1)) return false;
        tc_fence_after();
        const uint32_t mask = valid, ts = lanes + TM::half(g, h);
        uint32_t s[32];
        tmem_ld32(ts, s);
        tmem_wait_ld();
        if (mask != FULL) hide(s, mask);
        if (!rescale(row_max<32>(s), first ? nullptr : &sh.p_empty[g][h ^ 1], ((ph >> (h ^ 1)) & 1) ^ 1)) return false;
        const float rf = ref == -INFINITY ? 0.f : ref;
        put(s, rf, ts);
        put(s + 16, rf, ts + 8);
        there = mbar_test(&sh.s_full[g][h ^ 1], (ph >> (h ^ 1)) & 1);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&sh.s_empty[g][h]);   // (for the replicated pieces, which wait for it)
            mbar_arrive(&sh.p_full[g][h]);
        }
        ph ^= 1u << h;
        return true;
    }
};

// This thread's row of the piece at c: 16-byte loads of its query, all of a half at once.
template <int MT, int NT>
__device__ __forceinline__ void load_query(const PagedAttnArgs &a, Shared<MT> &sh, Softmax<MT, NT> &sm, const Cursor &c,
                                           const Rows<MT> &rows, int r) {
    const int gr = rows.base + r;
    const size_t qr = c.prefix(a) ? ((size_t)(gr / a.G) * a.Hk + c.head) * a.G + gr % a.G
                                  : ((size_t)(c.seg - a.row_tiles) * a.Hk + c.head) * a.G + r;
    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + qr * PA_D);
    constexpr int N = MT == 1 ? 8 : 4;        // 16 bytes at once
#pragma unroll 1
    for (int i = 0; i < 16; i += N) {
        uint4 v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = r < rows.n ? __ldg(src + i + k) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t f = a.q_flip;
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const uint32_t w[8] = {v[k].x ^ f, v[k].y ^ f, v[k].z ^ f, v[k].w ^ f,
                                   v[k + 1].x ^ f, v[k + 1].y ^ f, v[k + 1].z ^ f, v[k + 1].w ^ f};
            tmem_st8(sm.lanes + Tmem<MT, NT>::q(sm.g) + 4 * (i + k), w);
        }
    }
    tmem_wait_st();
    sm.arrive(&sh.q_full[sm.g]);
}

template <int MT, int NT>
__device__ __forceinline__ bool softmax(const PagedAttnArgs &a, Shared<MT> &sh, int warp, int lane) {
    using TM = Tmem<MT, NT>;
    const int quad = warp & 3;
    Softmax<MT, NT> sm = {a, sh, warp >> 2, quad, lane, (uint32_t)(quad * 32) << 16, 0.f, 0.f,
                          make_float2(0.f, 0.f), 0u, 0u};
    const int g = sm.g;
    Cursor c = sh.start;
    int no = 0, pairs = 0;                    // tiles, and pieces of two groups, so far
    bool cleared = false;                     // P is zero outside this quarter's columns
    bool loaded = false;                      // the piece's queries are there
    while (c.left > 0) {
        const int n = c.piece();
        const Rows<MT> rows(a, c);
        const Cursor at = c;
        const int t0 = no;                    // the piece's first tile
        no += n;
        c.skip(a, n);
        if (g >= rows.groups()) continue;
        const int r = rows.rep ? lane : g * 128 + quad * 32 + lane;
        const bool live = r < rows.n;
        const bool pre = at.prefix(a);
        if (!loaded) {
            // (replicated rows keep P where the second group had O)
            if (MT == 2 && rows.rep && pairs > 0 && !mbar_wait(&sh.pair_done, (pairs - 1) & 1)) return false;
            if (rows.rep && !cleared) {
                const uint32_t z[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll 1
                for (int i = 0; i < (int)TM::P_COLS / 8; ++i) {
                    tmem_st8(sm.lanes + TM::p(0) + 8 * i, z);
                    tmem_st8(sm.lanes + TM::p(1) + 8 * i, z);
                }
            }
            cleared = rows.rep;
            load_query<MT, NT>(a, sh, sm, at, rows, r);
        }
        sm.there = 0;
        sm.ref = sm.m = -INFINITY;
        sm.l = make_float2(0.f, 0.f);
        if (rows.rep) {
            for (int i = 0; i < n; ++i)
                if (!sm.tile_rep(i, (t0 + i) & 1, sh.mask[(t0 + i) % MASK_RING])) return false;
        } else if (MT == 1) {
            for (int i = 0; i < n; ++i)
                if (!sm.tile_full(i, (t0 + i) & 1, sh.mask[(t0 + i) % MASK_RING])) return false;
        } else {
#pragma unroll 1
            for (int i = 0; i < 2 * n; ++i)
                if (!sm.half_tile(i == 0, i & 1, reinterpret_cast<const uint32_t *>(sh.mask)[(2 * t0 + i) % (2 * MASK_RING)]))
                    return false;
        }
        // the next piece's queries, so that its first scores are under way while this one's output is read
        // (Q is free: its last scores have come; a change of the rows' kind moves other columns, and waits)
        loaded = false;
        if (c.left > 0) {
            const Rows<MT> to(a, c);
            if (to.rep == rows.rep && g < to.groups()) {
                load_query<MT, NT>(a, sh, sm, c, to, to.rep ? lane : g * 128 + quad * 32 + lane);
                loaded = true;
            }
        }
        // the piece's partial
        const int lb = MT == 1 || rows.rep ? (no - 1) & 1 : 1;
        if (!mbar_wait(&sh.p_empty[g][lb], ((sm.ph >> lb) & 1) ^ 1)) return false;
        tc_fence_after();
        const int seg = pre ? at.head * a.row_tiles + at.seg : at.head * a.B + at.seg - a.row_tiles;
        const int slot_rows = pre ? a.prefix_slot_rows : a.own_slot_rows;
        const int srow = rows.rep ? quad * rows.n + lane : r;
        float *dst = (pre ? a.part_prefix : a.part_own) +
                     (((size_t)seg + blockIdx.x) * slot_rows + srow) * PA_PART;
        const float l = sm.l.x + sm.l.y;      // (NaN scores alone leave ref at -inf: not "no token")
        if (live) *reinterpret_cast<float2 *>(dst) = make_float2(sm.ref == -INFINITY && l != 0.f ? 0.f : sm.ref, l);
#pragma unroll 2
        for (int k = 0; k < 16; ++k) {
            uint32_t o[8];
            tmem_ld8(sm.lanes + TM::o(g) + 8 * k, o);
            tmem_wait_ld();
            if (live) {
                *reinterpret_cast<uint4 *>(dst + 4 + 8 * k) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4 *>(dst + 8 + 8 * k) = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
        tc_fence_before();
        if (MT == 2 && rows.groups() == 2) {
            ++pairs;
            if (g == 1) sm.arrive(&sh.pair_done);
        }
    }
    return true;
}

template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <int BT, int MT, int NT>
__global__ void __launch_bounds__(Roles<MT>::THREADS, 1) k_paged_attn(const __grid_constant__ PagedAttnArgs a) {
    constexpr int SCOUT = Roles<MT>::SCOUT, PRODUCTS = Roles<MT>::PRODUCTS;
    extern __shared__ __align__(1024) uint8_t dyn[];   // (the swizzle's period)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t tiles = smem_addr(dyn), tables = tiles + 4 * TILE_BYTES;
    Shared<MT> &sh = *reinterpret_cast<Shared<MT> *>(dyn + attn_table_end(a.k.S, a.copies_k, a.v.S, a.copies_v));
    if (warp == PRODUCTS) {
        tmem_alloc(&sh.tmem, Tmem<MT, NT>::COLS);
        if (lane == 0) {
            sh.failed = 0;
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh.k_full[i], PROD_WARPS / 4);
                mbar_init(&sh.v_full[i], PROD_WARPS / 4);
                mbar_init(&sh.k_empty[i], 1);
                mbar_init(&sh.v_empty[i], 1);
            }
            for (int g = 0; g < MT; ++g) {
                mbar_init(&sh.q_full[g], 4);
                for (int i = 0; i < 2; ++i) {
                    mbar_init(&sh.s_full[g][i], 1);
                    mbar_init(&sh.s_empty[g][i], 4);
                    mbar_init(&sh.p_full[g][i], 4);
                    mbar_init(&sh.p_empty[g][i], 1);
                }
            }
            for (int i = 0; i < META_RING; ++i) {
                mbar_init(&sh.meta_full[i], 1);
                mbar_init(&sh.meta_empty[i], PROD_WARPS / 2);
            }
            mbar_init(&sh.pair_done, 4);
            mbar_init(&sh.heads, PROD_WARPS);
            mbar_init(&sh.drain[0], 1);
            mbar_init(&sh.drain[1], 1);
            mbar_init_fence();
        }
    }
    pdl_wait();
    if (warp == 0) {                          // this CTA's share of the list
        int64_t own_total;
        tiles_before(a, 0, &own_total);
        const Shares w(a, own_total);
        Cursor c = {0, 0, 0, 0, 0};
        const int64_t from = (int64_t)blockIdx.x * w.len;
        if (from < w.total) {
            c.left = (int)min((int64_t)w.len, w.total - from);
            c.head = quotient(from, w.per_head);
            int64_t rem = from - c.head * w.per_head;
            const int64_t pre = (int64_t)a.row_tiles * a.prefix_tiles;
            if (rem < pre) {
                c.seg = quotient(rem, a.prefix_tiles);
                c.n_tiles = a.prefix_tiles;
                c.tile = (int)(rem - (int64_t)c.seg * a.prefix_tiles);
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
        if (lane == 0) {
            sh.total = c.left;
            sh.last_head = c.left > 0 ? quotient(from + c.left - 1, w.per_head) : 0;
        }
        if (lane == 0) sh.start = c;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    bool ok = true;
    if (warp < 4 * MT) {
        regs_up<Roles<MT>::SOFTMAX>();
        ok = softmax<MT, NT>(a, sh, warp, lane);
    } else if (warp < SCOUT) {
        regs_down<Roles<MT>::PRODUCER>();
        ok = produce<BT, MT>(a, sh, tables, tiles, warp - 4 * MT, lane);
    } else {
        regs_down<Roles<MT>::REST>();
        if (warp < PRODUCTS) {
            ok = scout<MT>(a, sh, warp - SCOUT, lane);
        } else {
            const bool leader = elect_one();
            ok = sh.tmem == 0u && (warp == PRODUCTS ? issue_scores<MT, NT>(a, sh, tiles, leader)
                                                    : issue_outputs<MT, NT>(a, sh, tiles, leader));
            if (leader) mma_commit(&sh.drain[warp - PRODUCTS]);   // nothing may be in flight when tensor memory goes
            if (!mbar_wait(&sh.drain[warp - PRODUCTS], 0)) ok = false;
            __syncwarp();
        }
    }
    if (!ok) sh.failed = 1;
    tc_fence_before();
    __syncthreads();
    if (warp == PRODUCTS) {
        tc_fence_after();
        tmem_free(sh.tmem, Tmem<MT, NT>::COLS);
    }
    if (threadIdx.x == 0 && sh.failed && a.st) atomicOr(&a.st->flags, HQMQ_FLAG_TIMEOUT);
}

// Joins the partials of a row, a CTA each.  Its four warps take every fourth
// partial, four at a time, all of whose loads are issued at once (a lane four
// elements), and join their four results in shared memory; where the partials
// are is worked out while the last CTAs of k_paged_attn still run (the lengths
// were written before that kernel began).  Latency is the bound: 1024 rows of
// about 16 partials take 4.5 us after the last CTA.
constexpr int PJ_BATCH = 4;
template <int MT>
__global__ void __launch_bounds__(128)
k_paged_join(const __grid_constant__ PagedAttnArgs a, void *o, int out_dtype, float *lse) {
    __shared__ float s_acc[4][PA_D];
    __shared__ float2 s_ml[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x, rg = (int)((unsigned)row / (unsigned)a.G), g = row - rg * a.G;
    const int b = (int)((unsigned)rg / (unsigned)a.Hk), head = rg - b * a.Hk;
    int64_t own_total;
    const int64_t before = tiles_before(a, b, &own_total);
    const Shares w(a, own_total);
    // where the row's partials are: those of the prefix, then those of its own tokens
    int n_pre = 0, n_own = 0, copies = 1, stride = 0;
    const float *pre = nullptr, *own = nullptr;
    size_t pre_step = 0, own_step = 0;        // from one CTA's slot to the next
    const int64_t head0 = head * w.per_head;
    if (a.prefix_tiles) {
        const int r = b * a.G + g, rt = r / (128 * MT);
        const bool rep = a.rows <= PA_REP_ROWS;
        const int64_t at = head0 + (int64_t)rt * a.prefix_tiles;
        const int c0 = w.owner(at), c1 = w.owner(at + (a.prefix_tiles - 1));
        copies = rep ? 4 : 1;
        stride = a.rows * PA_PART;
        n_pre = (c1 - c0 + 1) * copies;
        pre_step = (size_t)a.prefix_slot_rows * PA_PART;
        pre = a.part_prefix + ((size_t)head * a.row_tiles + rt + c0) * pre_step + (rep ? r : r % (128 * MT)) * PA_PART;
    }
    if (const int n = own_tiles(a, b)) {
        const int64_t at = head0 + (int64_t)a.row_tiles * a.prefix_tiles + before;
        const int c0 = w.owner(at), c1 = w.owner(at + (n - 1));
        n_own = (c1 - c0 + 1) * 4;
        own_step = (size_t)a.own_slot_rows * PA_PART;
        own = a.part_own + ((size_t)head * a.B + b + c0) * own_step + g * PA_PART;
    }
    pdl_wait();
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = warp; i0 < n_pre + n_own; i0 += 4 * PJ_BATCH) {
        float2 ml[PJ_BATCH];                  // (-inf: no token, and O may be anything)
        float4 v[PJ_BATCH];
#pragma unroll
        for (int k = 0; k < PJ_BATCH; ++k) {
            const int i = i0 + 4 * k, j = i - n_pre;
            ml[k] = make_float2(-INFINITY, 0.f);
            if (i >= n_pre + n_own) continue;
            const float *p = j < 0 ? pre + (size_t)(copies == 4 ? i >> 2 : i) * pre_step + (copies == 4 ? (i & 3) * stride : 0)
                                   : own + (size_t)(j >> 2) * own_step + (j & 3) * a.G * PA_PART;
            ml[k] = *reinterpret_cast<const float2 *>(p);
            v[k] = *reinterpret_cast<const float4 *>(p + 4 + 4 * lane);
        }
        float mn = m;
#pragma unroll
        for (int k = 0; k < PJ_BATCH; ++k) mn = fmaxf(mn, ml[k].x);
        if (mn == -INFINITY) continue;
        const float f0 = exp2f(m - mn);
        m = mn;
        l *= f0;
        acc.x *= f0; acc.y *= f0; acc.z *= f0; acc.w *= f0;
#pragma unroll
        for (int k = 0; k < PJ_BATCH; ++k) {
            if (ml[k].x == -INFINITY) continue;
            const float f = exp2f(ml[k].x - mn);
            l += ml[k].y * f;
            acc.x += v[k].x * f;
            acc.y += v[k].y * f;
            acc.z += v[k].z * f;
            acc.w += v[k].w * f;
        }
    }
    *reinterpret_cast<float4 *>(&s_acc[warp][4 * lane]) = acc;
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    m = fmaxf(fmaxf(s_ml[0].x, s_ml[1].x), fmaxf(s_ml[2].x, s_ml[3].x));
    l = 0.f;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (s_ml[k].x == -INFINITY) continue;
        const float f = exp2f(s_ml[k].x - m);
        l += s_ml[k].y * f;
        y += s_acc[k][threadIdx.x] * f;
    }
    y = l == 0.f ? 0.f : y * (1.f / l);
    const size_t at = (size_t)row * PA_D + threadIdx.x;
    if (out_dtype == HQMQ_BF16) reinterpret_cast<__nv_bfloat16 *>(o)[at] = __float2bfloat16_rn(y);
    else reinterpret_cast<float *>(o)[at] = y;
    if (lse && threadIdx.x == 0) lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
}

// Workspace: partials of the prefix's segments, then of the sequences'.  The
// size covers both output types.
struct PartPlan {
    int mt, row_tiles, prefix_slot_rows, own_slot_rows;
    uint64_t prefix_bytes, own_bytes;
};
inline PartPlan part_plan(int B, int Hq, int Hk, int max_tokens, int prefix_len, int out_dtype) {
    PartPlan p;
    const int64_t rows = (int64_t)B * (Hq / Hk);
    // fp32 outputs take three terms of P, which leaves tensor memory for one group of rows.  (256 rows of 32
    // sequences with up to 1000 own tokens, bf16, two groups at once and one after the other: behind 131072
    // tokens 234 and 302 us, behind 32768 100 and 106, behind 8191 62 and 57.)
    p.mt = prefix_len > 0 && rows > 128 && out_dtype == HQMQ_BF16 ? 2 : 1;
    p.row_tiles = prefix_len > 0 ? (int)((rows + 128 * p.mt - 1) / (128 * p.mt)) : 0;
    p.prefix_slot_rows = rows <= PA_REP_ROWS ? (int)(4 * rows) : 128 * p.mt;
    p.own_slot_rows = 4 * (Hq / Hk);
    p.prefix_bytes = prefix_len > 0 ? ((uint64_t)p.row_tiles * Hk + PA_CTAS) * p.prefix_slot_rows * PA_PART * 4 : 0;
    p.own_bytes = max_tokens > 0 ? ((uint64_t)B * Hk + PA_CTAS) * p.own_slot_rows * PA_PART * 4 : 0;
    return p;
}

template <int BT, int MT, int NT>
static int launch_paged_attn_b(const PagedAttnArgs &a, int ctas, void *o, int out_dtype, float *lse,
                               cudaStream_t stream) {
    const size_t smem = attn_table_end(a.k.S, a.copies_k, a.v.S, a.copies_v) + sizeof(Shared<MT>);
    auto kern = k_paged_attn<BT, MT, NT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return HQMQ_ERR_CUDA;
    const int64_t rows = (int64_t)a.B * a.Hk * a.G;
    if (ctas > 0 && launch_pdl(kern, dim3(ctas), dim3(Roles<MT>::THREADS), smem, stream, a) != cudaSuccess)
        return HQMQ_ERR_CUDA;
    return launch_pdl(k_paged_join<MT>, dim3((unsigned)rows), dim3(128), 0, stream, a, o, out_dtype,
                      lse) == cudaSuccess
               ? HQMQ_OK : HQMQ_ERR_CUDA;
}

template <int MT, int NT>
static int launch_paged_attn(PagedAttnArgs &a, int ctas, void *o, int out_dtype, float *lse, cudaStream_t stream) {
    // 8 table copies (no bank conflicts) where they fit, K's first (S = 8, 32 heads: 52 us; 57 with 4 of each)
    const auto fits = [&](uint32_t rk, uint32_t rv) {
        return attn_table_end(a.k.S, rk, a.v.S, rv) + sizeof(Shared<MT>) <= 227 * 1024;
    };
    a.copies_k = fits(8, 4) ? 8 : 4;
    a.copies_v = fits(a.copies_k, 8) ? 8 : 4;
    // the index widths of S = 8 and S = 32 (6 .. 10, 22 .. 42) are compiled in; others, and K and V that differ,
    // pick an index's words by selects (S = 32 compiled in and not: 131072 tokens, 256 rows 233 and 276 us; 8191
    // tokens, 128 rows 32.0 and 35.4)
    if (a.k.b == a.v.b && a.k.b == 8) return launch_paged_attn_b<8, MT, NT>(a, ctas, o, out_dtype, lse, stream);
    if (a.k.b == a.v.b && a.k.b == 10) return launch_paged_attn_b<10, MT, NT>(a, ctas, o, out_dtype, lse, stream);
    return launch_paged_attn_b<0, MT, NT>(a, ctas, o, out_dtype, lse, stream);
}

}  // namespace hqmq

extern "C" uint64_t hqmq_paged_attn_workspace_bytes(int B, int Hq, int Hk, int max_tokens,
                                                    int prefix_len) {
    uint64_t n = 0;
    for (int dt : {HQMQ_BF16, HQMQ_F32}) {
        const hqmq::PartPlan p = hqmq::part_plan(B, Hq, Hk, max_tokens, prefix_len, dt);
        if (p.prefix_bytes + p.own_bytes > n) n = p.prefix_bytes + p.own_bytes;
    }
    return ((n + 255) & ~255ull) + 256;
}

extern "C" int hqmq_launch_attention_paged(const uint16_t *q, const hqmq_kv_pages *k,
                                           const hqmq_kv_pages *v, uint32_t bk, uint32_t bv, int B, int Hq,
                                           const int32_t *seq_len, const int32_t *table, int max_pages,
                                           const int32_t *prefix_table, int prefix_len, float scale,
                                           void *o, int out_dtype, float *lse, void *ws,
                                           hqmq_status *st, cudaStream_t stream) {
    using namespace hqmq;
    const PartPlan p = part_plan(B, Hq, k->heads, max_pages * k->page_size, prefix_len, out_dtype);
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
    a.sl2 = fmaxf((float)(sl2 < 0 ? -sl2 : sl2), 1.2e-38f);  // (above 0, so that -inf stays -inf)
    a.q_flip = scale < 0 ? 0x80008000u : 0u;
    a.part_prefix = reinterpret_cast<float *>(ws);
    a.part_own = reinterpret_cast<float *>(reinterpret_cast<char *>(ws) + p.prefix_bytes);
    a.prefix_slot_rows = p.prefix_slot_rows;
    a.own_slot_rows = p.own_slot_rows;
    a.st = reinterpret_cast<DevStatus *>(st);
    // tiles there can be at most
    const int64_t most = a.Hk * ((int64_t)a.row_tiles * a.prefix_tiles +
                                 (int64_t)B * (((int64_t)max_pages * k->page_size + PA_TILE - 1) / PA_TILE));
    const int ctas = (int)(most < PA_CTAS ? most : PA_CTAS);
    if (out_dtype == HQMQ_F32) return launch_paged_attn<1, 3>(a, ctas, o, out_dtype, lse, stream);
    return p.mt == 2 ? launch_paged_attn<2, 2>(a, ctas, o, out_dtype, lse, stream)
                     : launch_paged_attn<1, 2>(a, ctas, o, out_dtype, lse, stream);
}
