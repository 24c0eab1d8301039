// norm_rope.cu -- RMS norm of query and key head vectors with the position
// rotation, in one pass (include/hqmq.h, hqmq_qk_norm_rope).
//
// One CTA takes one token: the R / 2 angles are computed once, in fp64, and
// serve all of its heads; then a warp takes one head vector at a time.
#include "hqmq_device.cuh"

namespace hqmq {

constexpr int NR_WARPS = 8;
constexpr int NR_MAX_D = 512;

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

template <typename E>
__global__ void __launch_bounds__(NR_WARPS * 32) k_norm_rope(NormRopeArgs a) {
    __shared__ float2 s_cs[NR_MAX_D / 2];
    __shared__ float s_x[NR_WARPS][NR_MAX_D];
    pdl_wait();
    const int64_t token = blockIdx.x;
    const int64_t bb = token / a.T, tt = token % a.T;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int half = a.R / 2;
    for (int i = threadIdx.x; i < half; i += blockDim.x) s_cs[i] = angle_cs(a.pos[token], a.inv_freq[i]);
    __syncthreads();
    const int total = a.heads[0] + a.heads[1];
    for (int hh = warp; hh < total; hh += NR_WARPS) {
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
            const float f = 1.0f / sqrtf(sum / (float)a.D + a.eps);
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
    for (int s = 0; s < 2; ++s) {
        if (!in[s]) continue;
        a.in[s] = in[s]->data;
        a.out[s] = out[s]->data;
        a.ib[s] = in[s]->stride_b; a.it[s] = in[s]->stride_t; a.ih[s] = in[s]->stride_h;
        a.ob[s] = out[s]->stride_b; a.ot[s] = out[s]->stride_t; a.oh[s] = out[s]->stride_h;
        a.heads[s] = in[s]->heads;
        a.w[s] = w[s];
    }
    a.w_f32 = w_dtype == HQMQ_F32;
    a.T = T;
    a.D = D;
    a.R = R;
    a.interleaved = interleaved;
    a.eps = eps;
    a.pos = pos;
    a.inv_freq = inv_freq;
    const unsigned n = (unsigned)((int64_t)B * T);
    const cudaError_t e = dtype == HQMQ_BF16
        ? launch_pdl(k_norm_rope<__nv_bfloat16>, dim3(n), dim3(NR_WARPS * 32), 0, stream, a)
        : launch_pdl(k_norm_rope<float>, dim3(n), dim3(NR_WARPS * 32), 0, stream, a);
    return e == cudaSuccess ? HQMQ_OK : HQMQ_ERR_CUDA;
}
