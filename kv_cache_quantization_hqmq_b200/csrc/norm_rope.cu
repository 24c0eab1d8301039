// norm_rope.cu -- RMS norm of query and key head vectors with the position
// rotation, in one pass (include/hqmq.h, hqmq_qk_norm_rope).
//
// A CTA takes one or a few tokens; their R / 2 angles are computed once, in
// fp64, into shared memory and serve all heads.  The first vectors are loaded
// before the angles, so that both latencies run at the same time.
//
// k_norm_rope: a lane takes 16 elements of a vector as two runs of 8 that are
// rotated with each other (or 16 neighbours, when pairs are neighbours or
// pass through), LPV lanes a vector: 16-byte accesses, the partner of every
// element in the same lane, log2(LPV) shuffles for the norm.  It needs R and
// D - R to be multiples of 16 (a lane's 16 elements rotate or pass through as
// a whole, in two runs of 8) and 16-byte aligned vectors; k_norm_rope_any
// (a warp per vector, element by element) takes every other call, four times
// slower: 8192 tokens of 40 bf16 heads of 128 take 31 us in the first, 129 in
// the second; heads of 96 28 us with all 96 elements rotated, 104 with 24;
// heads of 80 25 us with 32 rotated, 98 with 40 (fp32 42 and 109).  A third
// kernel with runs of 4 would bring those back; none is built.
#include "hqmq_device.cuh"

namespace hqmq {

constexpr int NR_MAX_D = 512;
constexpr int NR_ANY_WARPS = 8;
constexpr int NR_THREADS = 512;
constexpr int NR_MAX_ANGLES = 1024;           // of the tokens of a CTA

struct NormRopeArgs {
    const void *in[2];
    void *out[2];
    int64_t ib[2], it[2], ih[2], ob[2], ot[2], oh[2];
    int heads[2];
    const void *w[2];
    int w_f32;
    int T, D, R, interleaved;
    float eps;
    const int *pos;
    const double *inv_freq;
};

// cos and sin of pos * inv_freq: the turns in fp64, their fraction in fp32.
__device__ __forceinline__ float2 angle_cs(int pos, double inv_freq) {
    const double turns = (double)pos * inv_freq * 0.15915494309189533577;
    const float f = (float)(2.0 * (turns - rint(turns)));
    float2 cs;
    sincospif(f, &cs.y, &cs.x);
    return cs;
}

template <typename E> __device__ __forceinline__ float to_f32(E v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E> __device__ __forceinline__ E from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// Eight neighbouring elements, 16-byte aligned.
template <typename E> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const void *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float *f) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void store(void *p, const float *f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float *f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    static __device__ __forceinline__ void store(void *p, const float *f) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// A CTA takes a span of tokens and blockDim.x / LPV heads (blockIdx.y: which);
// a thread stays with its 16 elements of its head and walks the tokens, loading
// the next one's elements before it works on the current one's.
// Bandwidth is the bound, so what counts is loads in flight: weights and
// angles come from shared memory, which leaves 64 registers a thread, and the
// span is chosen so that the last round of CTAs is nearly full (8192 tokens of
// 40 heads of 128, bf16, 168 MB: 31 us, 5.4 TB/s; weights in registers and
// spans of 8: 41 us).  fp32 elements take twice the registers: those instances
// spill 16 to 28 bytes at 64 (the same tokens in fp32, 336 MB: 57 us, 5.8 TB/s).
template <typename E, int LPV, bool PAIRS>
__global__ void __launch_bounds__(NR_THREADS, 2) k_norm_rope(const __grid_constant__ NormRopeArgs a, unsigned tokens,
                                                             int span) {
    // A part's eight angles, and its 16 weights, as four float4 each that lie LPV (of those that rotate: R / 16)
    // apart: neighbouring lanes read neighbouring words.
    __shared__ __align__(16) float2 s_cs[NR_MAX_ANGLES];
    __shared__ __align__(16) float4 s_w[2][4 * LPV];
    pdl_wait();
    pdl_trigger();
    const unsigned t0 = blockIdx.x * span;
    const int n_tok = (int)min((unsigned)span, tokens - t0);
    const int half = a.R / 2, total = a.heads[0] + a.heads[1];
    const int part = threadIdx.x & (LPV - 1);     // which 16 elements
    // element offsets of the two runs of 8
    const bool rot = part * 16 < a.R, split = rot && !PAIRS;
    const int e0 = split ? part * 8 : part * 16, e1 = split ? half + part * 8 : part * 16 + 8;
    const int hh = blockIdx.y * (blockDim.x / LPV) + threadIdx.x / LPV;
    const bool on = hh < total && part * 16 < a.D;
    const bool is_k = hh >= a.heads[0];
    const int h = is_k ? hh - a.heads[0] : hh;
    const int64_t it = is_k ? a.it[1] : a.it[0], ot = is_k ? a.ot[1] : a.ot[0];
    const int64_t ib = is_k ? a.ib[1] : a.ib[0], ob = is_k ? a.ob[1] : a.ob[0];
    unsigned bb = t0 / (unsigned)a.T, tt = t0 - bb * (unsigned)a.T;
    const E *in = reinterpret_cast<const E *>(is_k ? a.in[1] : a.in[0]) + h * (is_k ? a.ih[1] : a.ih[0]) + bb * ib + tt * it;
    E *out = reinterpret_cast<E *>(is_k ? a.out[1] : a.out[0]) + h * (is_k ? a.oh[1] : a.oh[0]) + bb * ob + tt * ot;
    const void *w = is_k ? a.w[1] : a.w[0];

    Raw8<E> r0 = {}, r1 = {};
    if (on) {
        r0.load(in + e0);
        r1.load(in + e1);
    }
    // (all these loads are on their way before the first is waited for)
    const int angles = n_tok * half;
    int pos = 0;
    double freq = 0.0;
    if ((int)threadIdx.x < angles) {
        const int k = threadIdx.x / half;
        pos = a.pos[t0 + k];
        freq = a.inv_freq[threadIdx.x - k * half];
    }
#pragma unroll 2
    for (int i = threadIdx.x; i < 2 * a.D; i += blockDim.x) {
        const int side = i >= a.D, e = i - side * a.D;
        // element e is number m of part p
        const bool er = e < a.R && !PAIRS, up = er && e >= half;
        const int p = er ? (up ? e - half : e) >> 3 : e >> 4, m = er ? (e & 7) + (up ? 8 : 0) : e & 15;
        const void *sw = a.w[side];
        if (sw)
            reinterpret_cast<float *>(s_w[side])[((m >> 2) * LPV + p) * 4 + (m & 3)] =
                a.w_f32 ? reinterpret_cast<const float *>(sw)[e]
                        : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(sw)[e]);
    }
    const int rot_parts = half / 8;
    for (int i = threadIdx.x; i < angles;) {
        const int k = i / half, j = i - k * half;
        s_cs[k * half + ((((j >> 1) & 3) * rot_parts + (j >> 3)) << 1) + (j & 1)] = angle_cs(pos, freq);
        i += blockDim.x;
        if (i < angles) {
            pos = a.pos[t0 + i / half];
            freq = a.inv_freq[i % half];
        }
    }
    __syncthreads();
    const float inv_d = 1.0f / (float)a.D;
    for (int k = 0; k < n_tok; ++k) {
        float f[16];
        r0.get(f);
        r1.get(f + 8);
        E *const y = out;
        // the next token
        in += it;
        out += ot;
        if (++tt == (unsigned)a.T) {
            tt = 0;
            in += ib - (int64_t)a.T * it;
            out += ob - (int64_t)a.T * ot;
        }
        if (on && k + 1 < n_tok) {
            r0.load(in + e0);
            r1.load(in + e1);
        }
        float sum = 0.f, sum1 = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum = fmaf(f[i], f[i], sum);
            sum1 = fmaf(f[i + 8], f[i + 8], sum1);
        }
        sum += sum1;
#pragma unroll
        for (int o = LPV / 2; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
        if (!on) continue;
        if (w) {
            const float r = rsqrtf(sum * inv_d + a.eps);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 g = s_w[is_k][(i >> 2) * LPV + part];
                f[i] = f[i] * r * g.x;
                f[i + 1] = f[i + 1] * r * g.y;
                f[i + 2] = f[i + 2] * r * g.z;
                f[i + 3] = f[i + 3] * r * g.w;
            }
        }
        if (rot) {
            const float4 *cs = reinterpret_cast<const float4 *>(s_cs + k * half) + part;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float4 c = cs[i / 2 * rot_parts];       // pairs i and i + 1
                constexpr int V = PAIRS ? 1 : 8, U = PAIRS ? 2 : 1;
                const float p = f[i * U], q = f[i * U + V], r = f[(i + 1) * U], t = f[(i + 1) * U + V];
                f[i * U] = p * c.x - q * c.y;
                f[i * U + V] = q * c.x + p * c.y;
                f[(i + 1) * U] = r * c.z - t * c.w;
                f[(i + 1) * U + V] = t * c.z + r * c.w;
            }
        }
        Raw8<E>::store(y + e0, f);
        Raw8<E>::store(y + e1, f + 8);
    }
}

template <typename E>
__global__ void __launch_bounds__(NR_ANY_WARPS * 32) k_norm_rope_any(NormRopeArgs a) {
    __shared__ float2 s_cs[NR_MAX_D / 2];
    __shared__ float s_x[NR_ANY_WARPS][NR_MAX_D];
    pdl_wait();
    const int64_t token = blockIdx.x;
    const int64_t bb = token / a.T, tt = token % a.T;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int half = a.R / 2;
    for (int i = threadIdx.x; i < half; i += blockDim.x) s_cs[i] = angle_cs(a.pos[token], a.inv_freq[i]);
    __syncthreads();
    const int total = a.heads[0] + a.heads[1];
    for (int hh = warp; hh < total; hh += NR_ANY_WARPS) {
        const int s = hh >= a.heads[0];
        const int h = s ? hh - a.heads[0] : hh;
        const E *x = reinterpret_cast<const E *>(a.in[s]) + bb * a.ib[s] + tt * a.it[s] + h * a.ih[s];
        E *y = reinterpret_cast<E *>(a.out[s]) + bb * a.ob[s] + tt * a.ot[s] + h * a.oh[s];
        float sum = 0.f;
        for (int d = lane; d < a.D; d += 32) {
            const float v = to_f32<E>(x[d]);
            s_x[warp][d] = v;
            sum += v * v;
        }
        const void *w = a.w[s];
        if (w) {
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
            const float f = rsqrtf(sum / (float)a.D + a.eps);
            for (int d = lane; d < a.D; d += 32)
                s_x[warp][d] *= f * (a.w_f32 ? reinterpret_cast<const float *>(w)[d]
                                             : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(w)[d]));
        }
        __syncwarp();
        for (int d = lane; d < a.D; d += 32) {
            float v = s_x[warp][d];
            if (d < a.R) {
                const int i = a.interleaved ? d >> 1 : (d < half ? d : d - half);
                const bool second = a.interleaved ? (d & 1) : d >= half;
                const int step = a.interleaved ? 1 : half;
                const float o = s_x[warp][second ? d - step : d + step];
                const float2 cs = s_cs[i];
                v = second ? v * cs.x + o * cs.y : v * cs.x - o * cs.y;
            }
            y[d] = from_f32<E>(v);
        }
        __syncwarp();
    }
}

template <typename E, int LPV>
static cudaError_t launch_norm_rope_lpv(const NormRopeArgs &a, unsigned tokens, cudaStream_t stream) {
    // heads: all in one CTA if they fit, in equal shares otherwise; a few tokens spread theirs over the SMs
    const int total = a.heads[0] + a.heads[1], most = (tokens < 148 ? 128 : NR_THREADS) / LPV;
    const int shares = (total + most - 1) / most, heads = (total + shares - 1) / shares;
    const int threads = (heads * LPV + 31) / 32 * 32;
    // tokens of a CTA (their angles fit shared memory): the fewest rounds of resident CTAs (64 registers a
    // thread), each as long as its tokens and a start that is worth about two
    const int64_t slots = 148 * (int64_t)(1024 / threads);
    int span = 1;
    int64_t best = INT64_MAX;
    for (int n = 1; n <= 16 && n * (a.R / 2) <= NR_MAX_ANGLES; ++n) {
        const int64_t ctas = (int64_t)((tokens + n - 1) / n) * shares, cost = (ctas + slots - 1) / slots * (n + 2);
        if (cost < best) {
            best = cost;
            span = n;
        }
    }
    const dim3 g((tokens + span - 1) / span, shares), b(threads);
    return a.interleaved ? launch_pdl(k_norm_rope<E, LPV, true>, g, b, 0, stream, a, tokens, span)
                         : launch_pdl(k_norm_rope<E, LPV, false>, g, b, 0, stream, a, tokens, span);
}

template <typename E>
static cudaError_t launch_norm_rope(const NormRopeArgs &a, unsigned tokens, bool wide, cudaStream_t stream) {
    if (!wide)
        return launch_pdl(k_norm_rope_any<E>, dim3(tokens), dim3(NR_ANY_WARPS * 32), 0, stream, a);
    int lpv = 1;
    while (lpv * 16 < a.D) lpv *= 2;
    switch (lpv) {
        case 1: return launch_norm_rope_lpv<E, 1>(a, tokens, stream);
        case 2: return launch_norm_rope_lpv<E, 2>(a, tokens, stream);
        case 4: return launch_norm_rope_lpv<E, 4>(a, tokens, stream);
        case 8: return launch_norm_rope_lpv<E, 8>(a, tokens, stream);
        case 16: return launch_norm_rope_lpv<E, 16>(a, tokens, stream);
        default: return launch_norm_rope_lpv<E, 32>(a, tokens, stream);
    }
}

}  // namespace hqmq

extern "C" int hqmq_launch_norm_rope(const hqmq_head_view *q, const hqmq_head_view *q_out,
                                     const hqmq_head_view *k, const hqmq_head_view *k_out, int dtype,
                                     int B, int T, int D, const void *qw, const void *kw, int w_dtype,
                                     float eps, const int32_t *pos, const double *inv_freq, int R,
                                     int interleaved, cudaStream_t stream) {
    using namespace hqmq;
    NormRopeArgs a = {};
    const hqmq_head_view *in[2] = {q, k}, *out[2] = {q_out, k_out};
    const void *w[2] = {qw, kw};
    const int64_t esz = dtype == HQMQ_BF16 ? 2 : 4;
    bool wide = R % 16 == 0 && (D - R) % 16 == 0;
    const auto aligned16 = [&](const hqmq_head_view *v) {
        return reinterpret_cast<uintptr_t>(v->data) % 16 == 0 && v->stride_b * esz % 16 == 0 &&
               v->stride_t * esz % 16 == 0 && v->stride_h * esz % 16 == 0;
    };
    for (int s = 0; s < 2; ++s) {
        if (!in[s]) continue;
        a.in[s] = in[s]->data;
        a.out[s] = out[s]->data;
        a.ib[s] = in[s]->stride_b; a.it[s] = in[s]->stride_t; a.ih[s] = in[s]->stride_h;
        a.ob[s] = out[s]->stride_b; a.ot[s] = out[s]->stride_t; a.oh[s] = out[s]->stride_h;
        a.heads[s] = in[s]->heads;
        a.w[s] = w[s];
        wide = wide && aligned16(in[s]) && aligned16(out[s]);
    }
    a.w_f32 = w_dtype == HQMQ_F32;
    a.T = T;
    a.D = D;
    a.R = R;
    a.interleaved = interleaved;
    a.eps = eps;
    a.pos = pos;
    a.inv_freq = inv_freq;
    const unsigned tokens = (unsigned)((int64_t)B * T);
    const cudaError_t e = dtype == HQMQ_BF16 ? launch_norm_rope<__nv_bfloat16>(a, tokens, wide, stream)
                                             : launch_norm_rope<float>(a, tokens, wide, stream);
    return e == cudaSuccess ? HQMQ_OK : HQMQ_ERR_CUDA;
}
