// Internal declarations of the encoder operators (include/ersj_encoder.h):
// element types, vector access and kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace ersj {

// Error message and device memory of the library (ersj_api.cpp): set_error
// keeps the message for ersj_last_error and returns the code; a block is
// returned with the size it was asked for.
int set_error(int code, const char *msg);
hipError_t device_block_get(int dev, size_t bytes, void **out);
void device_block_put(int dev, void *p, size_t bytes);

enum ElemType { kF32 = 0, kF16 = 1, kBF16 = 2 };

typedef _Float16 f16_t;
typedef __bf16 bf16_t;

// LEN elements at any element-aligned address: gfx950's global loads and stores
// take unaligned addresses, so rows of odd length or spacing use the same
// full-width accesses as aligned ones (300,000 rows of 385 bf16 against 384: layer
// norm 101 and 89 us, its gradient 148 and 139).
template <typename E, int LEN>
struct Slot {
    typedef E vec __attribute__((ext_vector_type(LEN)));
    struct __attribute__((packed, aligned(sizeof(E)))) slot {
        vec v;
    };
    static __device__ __forceinline__ vec load(const E *p) { return ((const slot *)p)->v; }
    static __device__ __forceinline__ void store(E *p, vec v) { ((slot *)p)->v = v; }
};

// The following statements with T as the element type.
#define ERSJ_ELEM_SWITCH(type, T, ...)                         \
    switch (type) {                                            \
    case ersj::kF32: { typedef float T; __VA_ARGS__; } break;  \
    case ersj::kF16: { typedef ersj::f16_t T; __VA_ARGS__; } break; \
    default: { typedef ersj::bf16_t T; __VA_ARGS__; } break;   \
    }

__host__ __device__ inline int elem_size(int type) { return type == kF32 ? 4 : 2; }

struct EmbedArgs {
    const void *table;
    int table_type;
    int64_t rows, ld_table;
    int dim;
    const void *ids;
    int id_type;
    int64_t n;
    float scale;
    int64_t padding_id;
    void *out;
    int out_type;
    int64_t ld_out;
};
hipError_t launch_embed(const EmbedArgs &a, hipStream_t s);

struct EmbedGradArgs {
    const void *grad;
    int grad_type;
    int64_t ld_grad;
    const void *ids;
    int id_type;
    int64_t n;
    float scale;
    int64_t padding_id;
    void *out;
    int out_type;
    int64_t rows;
    int dim;
    int64_t ld_out;
    int accumulate;
    void *work;
};
uint64_t embed_grad_work(int64_t n, int64_t rows, int dim);
hipError_t launch_embed_grad(const EmbedGradArgs &a, hipStream_t s);

struct NormArgs {
    const void *x;
    int type;
    int64_t n;
    int dim;
    int64_t ld_x;
    const void *weight, *bias;
    int param_type;
    float eps;
    void *y;
    int64_t ld_y;
    float *mean, *rstd;
};
hipError_t launch_layer_norm(const NormArgs &a, hipStream_t s);

struct NormGradArgs {
    const void *gy;
    int64_t ld_gy;
    const void *x;
    int64_t ld_x;
    int type;
    int64_t n;
    int dim;
    const float *mean, *rstd;
    const void *weight;
    int param_type;
    void *gx;
    int64_t ld_gx;
    void *gw, *gb;
    void *work;
};
uint64_t layer_norm_grad_work(int64_t n, int dim);
hipError_t launch_layer_norm_grad(const NormGradArgs &a, hipStream_t s);

// A chunk of one gradient tensor.
struct GradChunk {
    const void *in;
    void *out;
    uint32_t count;  // elements
    int32_t type;
};
constexpr uint32_t kGradChunkBytes = 32768;

// Elements of a tensor's first chunk: those after it begin at whole cache
// lines, wherever the tensor lies in a larger buffer (300 odd-sized bf16 views
// of 100M elements: 126 us, 130 with chunks that begin as the tensors do).
__host__ __device__ inline int64_t first_chunk(const void *p, int type)
{
    return (int64_t)(kGradChunkBytes - ((uintptr_t)p & 127)) / elem_size(type);
}

// Tensors with elements, handed to the kernel that writes their chunks as its
// arguments: nothing on the host is read after the launch.
struct GradTensor {
    const void *in;
    void *out;
    int64_t size;
    int32_t type;
    uint32_t first;  // index of its first chunk
};
constexpr int kGradTensors = 96;  // 3 KB of the 4 KB of a kernel's arguments
struct GradTensors {
    GradTensor t[kGradTensors];
    int count;
    uint32_t end;  // chunks up to the last tensor's
};
hipError_t launch_grads_table(const GradTensors &t, GradChunk *chunks, hipStream_t s);
constexpr int kGradParts = 2048;  // partial sums, one per workgroup of the norm kernel
hipError_t launch_grads_clip(const GradChunk *chunks, uint32_t n_chunks, float max_norm, float *norm, void *work,
                             hipStream_t s);

}  // namespace ersj
