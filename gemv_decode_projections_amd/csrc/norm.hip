// The norms around a block (include/block.h, blk_norm_run), one pass:
//     t = x                                    or  x * rsqrt(mean x^2 + eps) * w_post
//     y = residual + alpha * gate * t          (written in the residual's type)
//     out = y * rsqrt(mean y^2 + eps) * w_pre
// Memory bound: a workgroup owns a row, keeps it in registers in FP32 through
// both norms, and reads and writes each element once; y enters the second
// norm before it is rounded. Measured at width 8192: one row 4.2 us a call (the
// launch and two reductions), 1000 rows with an FP32 residual 25.5 us for 115
// MB, 4.5 TB/s.
#include <algorithm>

#include "block_common.h"

namespace gdp {
namespace {

struct NormArgs {
    const char *x, *residual, *gate, *w_post, *w_pre;
    char *y, *out;
    int64_t x_stride, residual_stride, gate_stride, y_stride, out_stride;   // bytes
    int width;
    float alpha, eps;
};

constexpr int kNormWaves = 16;

// V consecutive elements from p, as FP32; V is 8 or 1.
template <class T, int V>
__device__ __forceinline__ void load(const char *p, float (&v)[V])
{
    if constexpr (V == 1) {
        v[0] = T::lo(*reinterpret_cast<const uint16_t *>(p));
    } else {
        const u32x4 u = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = T::lo(u[i]);
            v[2 * i + 1] = T::hi(u[i]);
        }
    }
}
template <class T, int V>
__device__ __forceinline__ void store(char *p, const float (&v)[V])
{
    if constexpr (V == 1) {
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)T::pack(v[0], v[0]);
    } else {
        *reinterpret_cast<u32x4 *>(p) = u32x4{T::pack(v[0], v[1]), T::pack(v[2], v[3]), T::pack(v[4], v[5]),
                                              T::pack(v[6], v[7])};
    }
}
template <int V>
__device__ __forceinline__ void load32(const char *p, float (&v)[V])
{
    if constexpr (V == 1) {
        v[0] = *reinterpret_cast<const float *>(p);
    } else {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
}
template <int V>
__device__ __forceinline__ void store32(char *p, const float (&v)[V])
{
    if constexpr (V == 1) {
        *reinterpret_cast<float *>(p) = v[0];
    } else {
        *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4 *>(p + 16) = f32x4{v[4], v[5], v[6], v[7]};
    }
}

// Sum over the workgroup, the same in every thread and every run.
__device__ __forceinline__ float block_sum(float v, float *s)
{
    v += __shfl_xor(v, 1);
    v += __shfl_xor(v, 2);
    v += __shfl_xor(v, 4);
    v += __shfl_xor(v, 8);
    v = sum_quads(v);
    const int waves = blockDim.x / kWave;
    if (waves == 1)
        return v;
    if (threadIdx.x % kWave == 0)
        s[threadIdx.x / kWave] = v;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < waves; ++w)
        t += s[w];
    return t;
}

// V elements per access, U accesses per thread: piece i of a thread starts at
// element (i * blockDim + thread) * V.
template <class T, bool R32, int V, int U>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a)
{
    __shared__ float s_sum[2][kNormWaves];
    const int64_t row = blockIdx.x;
    constexpr int RB = R32 ? 4 : 2;
    float x[U][V], r[U][V];
    int at[U];
    bool in[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        at[i] = (i * blockDim.x + threadIdx.x) * V;
        in[i] = at[i] < a.width;
        if (!in[i])
            continue;
        if (a.x)
            load<T, V>(a.x + row * a.x_stride + (int64_t)at[i] * 2, x[i]);
        const char *p = a.residual + row * a.residual_stride + (int64_t)at[i] * RB;
        if constexpr (R32)
            load32<V>(p, r[i]);
        else
            load<T, V>(p, r[i]);
    }
    const float inv_width = 1.0f / (float)a.width;
    if (a.x) {
        float f = a.alpha;
        if (a.w_post) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (in[i])
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        ss += x[i][e] * x[i][e];
            f = rsqrtf(block_sum(ss, s_sum[0]) * inv_width + a.eps);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (!in[i])
                continue;
            if (a.w_post) {
                float w[V];
                load<T, V>(a.w_post + (int64_t)at[i] * 2, w);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    x[i][e] = x[i][e] * f * w[e] * a.alpha;
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    x[i][e] *= f;
            }
            if (a.gate) {
                float g[V];
                load<T, V>(a.gate + row * a.gate_stride + (int64_t)at[i] * 2, g);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    x[i][e] *= g[e];
            }
#pragma unroll
            for (int e = 0; e < V; ++e)
                r[i][e] += x[i][e];
            if (a.y) {
                char *p = a.y + row * a.y_stride + (int64_t)at[i] * RB;
                if constexpr (R32)
                    store32<V>(p, r[i]);
                else
                    store<T, V>(p, r[i]);
            }
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (in[i])
#pragma unroll
            for (int e = 0; e < V; ++e)
                ss += r[i][e] * r[i][e];
    const float f = rsqrtf(block_sum(ss, s_sum[1]) * inv_width + a.eps);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (!in[i])
            continue;
        float w[V];
        load<T, V>(a.w_pre + (int64_t)at[i] * 2, w);
#pragma unroll
        for (int e = 0; e < V; ++e)
            w[e] = r[i][e] * f * w[e];
        store<T, V>(a.out + row * a.out_stride + (int64_t)at[i] * 2, w);
    }
}

using NormKernel = void (*)(NormArgs);

template <class T, bool R32>
NormKernel pick(bool vec, int u)
{
    if (vec)
        return u <= 1 ? norm_kernel<T, R32, 8, 1> : u <= 2 ? norm_kernel<T, R32, 8, 2> : norm_kernel<T, R32, 8, 4>;
    return u <= 8 ? norm_kernel<T, R32, 1, 8> : norm_kernel<T, R32, 1, 32>;
}

constexpr int kNormMaxWidth = 32768;

}  // namespace
}  // namespace gdp

using namespace gdp;

extern "C" int blk_norm_run(const blk_norm_args *n, int m, void *stream)
{
    if (!n)
        return PROJ_ERR_NULL;
    if (m < 0 || n->width < 1 || n->width > kNormMaxWidth || (n->dtype != BLK_BF16 && n->dtype != BLK_F16) ||
        (n->residual_dtype != n->dtype && n->residual_dtype != BLK_F32))
        return PROJ_ERR_ARG;
    const int64_t strides[] = {stride_of(n->x_stride, m), stride_of(n->residual_stride, m), stride_of(n->gate_stride, m),
                               stride_of(n->residual_out_stride, m), stride_of(n->out_stride, m)};
    for (int64_t s : strides)
        if (s < 0 || s >= ((int64_t)1 << 40))
            return PROJ_ERR_ARG;
    if (!rows_apart<1>(n->width, {n->out_stride}, {m}) ||
        (n->residual_out && !rows_apart<1>(n->width, {n->residual_out_stride}, {m})))
        return PROJ_ERR_ARG;
    if (m == 0)
        return PROJ_OK;
    if (!n->residual || !n->weight_pre || !n->out || (n->x && !n->residual_out) ||
        (!n->x && (n->weight_post || n->gate || n->residual_out)))
        return PROJ_ERR_NULL;
    const bool r32 = n->residual_dtype == BLK_F32;
    // Eight elements per access where every row allows it, single ones elsewhere.
    bool vec = n->width % 8 == 0;
    for (int64_t s : strides)
        vec = vec && s % 8 == 0;
    for (const void *p : {n->x, n->residual, n->gate, n->weight_post, n->weight_pre, (const void *)n->residual_out,
                          (const void *)n->out}) {
        if (!aligned_to(p, 2))
            return PROJ_ERR_ALIGN;
        vec = vec && aligned_to(p, 16);
    }
    if (r32 && (!aligned_to(n->residual, 4) || !aligned_to(n->residual_out, 4)))
        return PROJ_ERR_ALIGN;
    NormArgs a{};
    const int rb = r32 ? 4 : 2;
    a.x = static_cast<const char *>(n->x);
    a.residual = static_cast<const char *>(n->residual);
    a.gate = static_cast<const char *>(n->gate);
    a.w_post = static_cast<const char *>(n->weight_post);
    a.w_pre = static_cast<const char *>(n->weight_pre);
    a.y = static_cast<char *>(n->residual_out);
    a.out = static_cast<char *>(n->out);
    a.x_stride = strides[0] * 2;
    a.residual_stride = strides[1] * rb;
    a.gate_stride = strides[2] * 2;
    a.y_stride = strides[3] * rb;
    a.out_stride = strides[4] * 2;
    a.width = n->width;
    a.alpha = n->alpha;
    a.eps = n->eps;
    const int pieces = vec ? n->width / 8 : n->width;
    const int threads = std::min(1024, (pieces + kWave - 1) / kWave * kWave);
    const int u = (pieces + threads - 1) / threads;
    NormKernel fn = n->dtype == BLK_BF16 ? (r32 ? pick<BF16, true>(vec, u) : pick<BF16, false>(vec, u))
                                         : (r32 ? pick<F16, true>(vec, u) : pick<F16, false>(vec, u));
    void *params[1] = {&a};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(fn), dim3((unsigned)m), dim3(threads), params, 0,
                                         static_cast<hipStream_t>(stream));
    return e == hipSuccess ? PROJ_OK : hip_fail(e);
}
