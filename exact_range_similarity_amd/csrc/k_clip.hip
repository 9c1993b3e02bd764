// Clipping of a set of gradients by their global norm: one kernel sums the
// squares in binary64, one partial sum per workgroup; the next adds the
// partial sums and scales.
#include "encoder_internal.h"

namespace ersj {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

__device__ __forceinline__ double block_sum(double v, double *red)
{
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.;
    for (int k = 0; k < kWaves; ++k) t += red[k];
    return t;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, uint32_t n)
{
    double s = 0.;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        const double v = (double)(float)p[i];
        s += v * v;
    }
    return s;
}

__global__ __launch_bounds__(kThreads) void k_grad_squares(const GradChunk *chunks, uint32_t n, double *part)
{
    __shared__ double red[kWaves];
    double s = 0.;
    for (uint32_t k = blockIdx.x; k < n; k += gridDim.x) {
        const GradChunk c = chunks[k];
        ERSJ_ELEM_SWITCH(c.type, T, s += chunk_squares((const T *)c.in, c.count))
    }
    s = block_sum(s, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *in, T *out, uint32_t n, float f)
{
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) out[i] = (T)(f * (float)in[i]);
}

__global__ __launch_bounds__(kThreads) void k_grad_scale(const GradChunk *chunks, uint32_t n, const double *part,
                                                         int parts, float max_norm, float *norm_out)
{
    __shared__ double red[kWaves];
    double s = 0.;
    for (int k = threadIdx.x; k < parts; k += kThreads) s += part[k];
    const double norm = sqrt(block_sum(s, red));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    const double bound = norm + 1e-6;
    const float f = (double)max_norm >= bound ? 1.f : (float)((double)max_norm / bound);
    for (uint32_t k = blockIdx.x; k < n; k += gridDim.x) {
        const GradChunk c = chunks[k];
        if (f == 1.f && c.in == c.out) continue;
        ERSJ_ELEM_SWITCH(c.type, T, chunk_scale((const T *)c.in, (T *)c.out, c.count, f))
    }
}

}  // namespace

hipError_t launch_grads_clip(const GradChunk *chunks, uint32_t n_chunks, float max_norm, float *norm, void *work,
                             hipStream_t s)
{
    const int parts = n_chunks < (uint32_t)kGradParts ? (int)n_chunks : kGradParts;
    if (parts) k_grad_squares<<<dim3(parts), dim3(kThreads), 0, s>>>(chunks, n_chunks, (double *)work);
    k_grad_scale<<<dim3(parts ? parts : 1), dim3(kThreads), 0, s>>>(chunks, n_chunks, (const double *)work, parts,
                                                                  max_norm, norm);
    return hipGetLastError();
}

}  // namespace ersj
