// Clipping of a set of gradients by their global norm: one kernel sums the
// squares in binary64 (an f32 gradient's square may leave the range of 32 bits),
// one partial sum per workgroup; the next adds the partial sums, each workgroup
// for itself, and scales.  Bound by memory, and the gradients are read twice:
// the factor depends on all of them.  268M f32 elements: 202 + 389 us for 1.07 +
// 2.14 GB, 5.4 TB/s, as fast as a copy; 21M bf16 elements: 9.5 + 16 us.
#include "encoder_internal.h"

namespace ersj {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kVecs = (int)(kGradChunkBytes / 16) / kThreads;  // 16-byte vectors of a thread in a whole chunk

__device__ __forceinline__ double block_sum(double v, double *red)
{
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.;
    for (int k = 0; k < kWaves; ++k) t += red[k];
    return t;
}

// A chunk's vectors: thread t takes vectors t, t + kThreads, ...; the elements
// after the last whole vector go to the first threads one by one.
template <typename T>
struct Chunk {
    typedef Slot<T, 16 / sizeof(T)> V;
    static constexpr int kLen = 16 / sizeof(T);
    typename V::vec v[kVecs];

    __device__ __forceinline__ void load(const T *p, uint32_t n)
    {
        const uint32_t vecs = n / kLen;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const uint32_t i = threadIdx.x + k * kThreads;
            if (i < vecs) v[k] = V::load(p + i * kLen);
        }
    }
};

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, uint32_t n)
{
    constexpr int kLen = 16 / sizeof(T);
    Chunk<T> c;
    c.load(p, n);
    const uint32_t vecs = n / kLen;
    double s[2] = {0., 0.};
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        if (threadIdx.x + k * kThreads < vecs) {
#pragma unroll
            for (int j = 0; j < kLen; ++j) {
                const double x = (double)(float)c.v[k][j];
                s[j & 1] += x * x;
            }
        }
    }
    const uint32_t i = vecs * kLen + threadIdx.x;
    if (i < n) {
        const double x = (double)(float)p[i];
        s[0] += x * x;
    }
    return s[0] + s[1];
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
    constexpr int kLen = 16 / sizeof(T);
    typedef Slot<T, kLen> V;
    typedef float fvec __attribute__((ext_vector_type(kLen)));
    Chunk<T> c;
    c.load(in, n);
    const uint32_t vecs = n / kLen;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const uint32_t i = threadIdx.x + k * kThreads;
        if (i < vecs)
            V::store(out + i * kLen,
                     __builtin_convertvector(__builtin_convertvector(c.v[k], fvec) * f, typename V::vec));
    }
    const uint32_t i = vecs * kLen + threadIdx.x;
    if (i < n) out[i] = (T)(f * (float)in[i]);
}

__global__ __launch_bounds__(kThreads) void k_grad_scale(const GradChunk *chunks, uint32_t n, const double *part,
                                                         int parts, float max_norm, float *norm_out)
{
    __shared__ double red[kWaves];
    double s = 0.;
#pragma unroll
    for (int k = 0; k < kGradParts / kThreads; ++k) {
        const int i = threadIdx.x + k * kThreads;
        s += i < parts ? part[i] : 0.;
    }
    const double norm = sqrt(block_sum(s, red));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    const double bound = norm + 1e-6;
    const float f = (double)max_norm >= bound ? 1.f : (float)((double)max_norm / bound);
    // from the end: what the other kernel read last is the likeliest to be in a cache
    for (uint32_t k = blockIdx.x; k < n; k += gridDim.x) {
        const GradChunk c = chunks[n - 1 - k];
        if (f == 1.f && c.in == c.out) continue;
        ERSJ_ELEM_SWITCH(c.type, T, chunk_scale((const T *)c.in, (T *)c.out, c.count, f))
    }
}

// The chunks of up to kGradTensors tensors, one to a thread.
__global__ __launch_bounds__(kThreads) void k_grad_table(GradTensors t, GradChunk *chunks)
{
    const uint32_t c = t.t[0].first + blockIdx.x * kThreads + threadIdx.x;
    if (c >= t.end) return;
    int lo = 0, hi = t.count - 1;  // the last tensor whose first chunk is not after c
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.t[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    const GradTensor g = t.t[lo];
    const int64_t es = elem_size(g.type), step = kGradChunkBytes / es, lead = first_chunk(g.in, g.type);
    const uint32_t k = c - g.first;
    const int64_t at = k ? lead + (int64_t)(k - 1) * step : 0, len = k ? step : lead;
    GradChunk out;
    out.in = (const char *)g.in + at * es;
    out.out = (char *)g.out + at * es;
    out.count = (uint32_t)(g.size - at < len ? g.size - at : len);
    out.type = g.type;
    chunks[c] = out;
}

}  // namespace

hipError_t launch_grads_table(const GradTensors &t, GradChunk *chunks, hipStream_t s)
{
    const uint32_t n = t.end - t.t[0].first;
    k_grad_table<<<dim3((n + kThreads - 1) / kThreads), dim3(kThreads), 0, s>>>(t, chunks);
    return hipGetLastError();
}

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
