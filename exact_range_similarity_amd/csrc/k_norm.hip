// Layer norm of rows and its gradient.
#include "encoder_internal.h"

namespace ersj {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// Sum over the workgroup, in every thread.
__device__ __forceinline__ float block_sum(float v, float *red)
{
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.f;
    for (int k = 0; k < kWaves; ++k) t += red[k];
    return t;
}

template <typename T, typename P>
__global__ __launch_bounds__(kThreads) void k_norm(NormArgs a)
{
    __shared__ float red[kWaves];
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.ld_x;
        T *y = (T *)a.y + r * a.ld_y;
        float s = 0.f;
        for (int c = threadIdx.x; c < a.dim; c += kThreads) s += (float)x[c];
        const float mean = block_sum(s, red) / (float)a.dim;
        s = 0.f;
        for (int c = threadIdx.x; c < a.dim; c += kThreads) {
            const float d = (float)x[c] - mean;
            s += d * d;
        }
        const float rstd = 1.f / sqrtf(block_sum(s, red) / (float)a.dim + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        for (int c = threadIdx.x; c < a.dim; c += kThreads) {
            float v = ((float)x[c] - mean) * rstd;
            if (a.weight) v *= (float)((const P *)a.weight)[c];
            if (a.bias) v += (float)((const P *)a.bias)[c];
            y[c] = (T)v;
        }
    }
}

template <typename T, typename P>
__global__ __launch_bounds__(kThreads) void k_norm_grad_x(NormGradArgs a)
{
    __shared__ float red[kWaves];
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.ld_x;
        const T *gy = (const T *)a.gy + r * a.ld_gy;
        T *gx = (T *)a.gx + r * a.ld_gx;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < a.dim; c += kThreads) {
            const float g = (float)gy[c] * (a.weight ? (float)((const P *)a.weight)[c] : 1.f);
            s1 += g;
            s2 += g * (((float)x[c] - mean) * rstd);
        }
        s1 = block_sum(s1, red) / (float)a.dim;
        s2 = block_sum(s2, red) / (float)a.dim;
        for (int c = threadIdx.x; c < a.dim; c += kThreads) {
            const float g = (float)gy[c] * (a.weight ? (float)((const P *)a.weight)[c] : 1.f);
            const float xh = ((float)x[c] - mean) * rstd;
            gx[c] = (T)(rstd * (g - s1 - xh * s2));
        }
    }
}

constexpr int kParts = 256;

int parts_of(int64_t n) { return n < kParts ? (n < 1 ? 1 : (int)n) : kParts; }

// Part p of the sums over rows p, p + parts, ...: part [p][2][dim].
template <typename T>
__global__ __launch_bounds__(kThreads) void k_norm_grad_part(NormGradArgs a, float *part)
{
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.dim) return;
    float sw = 0.f, sb = 0.f;
    for (int64_t r = blockIdx.y; r < a.n; r += gridDim.y) {
        const float dy = (float)((const T *)a.gy)[r * a.ld_gy + c];
        const float xh = ((float)((const T *)a.x)[r * a.ld_x + c] - a.mean[r]) * a.rstd[r];
        sw += dy * xh;
        sb += dy;
    }
    part[(int64_t)blockIdx.y * 2 * a.dim + c] = sw;
    part[((int64_t)blockIdx.y * 2 + 1) * a.dim + c] = sb;
}

template <typename P>
__global__ __launch_bounds__(kThreads) void k_norm_grad_join(const float *part, int parts, int dim, P *gw, P *gb)
{
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= dim) return;
    float sw = 0.f, sb = 0.f;
    for (int p = 0; p < parts; ++p) {
        sw += part[(int64_t)p * 2 * dim + c];
        sb += part[((int64_t)p * 2 + 1) * dim + c];
    }
    if (gw) gw[c] = (P)sw;
    if (gb) gb[c] = (P)sb;
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs &a, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    const dim3 grid((unsigned)(a.n < 65536 ? a.n : 65536)), block(kThreads);
    ERSJ_ELEM_SWITCH(a.type, T, ERSJ_ELEM_SWITCH(a.param_type, P, k_norm<T, P><<<grid, block, 0, s>>>(a)))
    return hipGetLastError();
}

uint64_t layer_norm_grad_work(int64_t n, int dim) { return (uint64_t)parts_of(n) * 2 * 4 * (uint64_t)dim; }

hipError_t launch_layer_norm_grad(const NormGradArgs &a, hipStream_t s)
{
    if (a.gw || a.gb) {
        const int parts = parts_of(a.n);
        const dim3 grid((a.dim + kThreads - 1) / kThreads, parts), block(kThreads);
        ERSJ_ELEM_SWITCH(a.type, T, k_norm_grad_part<T><<<grid, block, 0, s>>>(a, (float *)a.work))
        ERSJ_ELEM_SWITCH(a.param_type, P, k_norm_grad_join<P><<<dim3(grid.x), block, 0, s>>>(
                                              (const float *)a.work, parts, a.dim, (P *)a.gw, (P *)a.gb))
    }
    if (a.gx && a.n) {
        const dim3 grid((unsigned)(a.n < 65536 ? a.n : 65536)), block(kThreads);
        ERSJ_ELEM_SWITCH(a.type, T, ERSJ_ELEM_SWITCH(a.param_type, P,
            k_norm_grad_x<T, P><<<grid, block, 0, s>>>(a)))
    }
    return hipGetLastError();
}

}  // namespace ersj
