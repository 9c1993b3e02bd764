// Internal declarations of the feed-forward operators
// (include/ersj_encoder.h): rows held in 8 bits and the gated block.
#pragma once

#include "encoder_internal.h"

namespace ersj {

// ---- rows held in 8 bits ----

constexpr int kPackBlock = 32;  // neighbours along a row that share a scale
constexpr int kPackNone = 255;  // scale of a block that holds a NaN or an infinity

__host__ __device__ inline int pack_blocks(int dim) { return (dim + kPackBlock - 1) / kPackBlock; }

// Scale byte e + 127 for a block whose largest magnitude has these bits.
__device__ __forceinline__ int pack_scale(uint32_t most)
{
    if (most >= 0x7f800000u) return kPackNone;
    // 2^(exponent - 6), twice that where the fraction is above 127/64
    const int s = (int)(most >> 23) - 6 + ((most & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return s < 1 ? 1 : s;
}

// 2^e of a scale byte; NaN for a block that has none.
__device__ __forceinline__ float pack_step(int scale)
{
    return scale == kPackNone ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)scale << 23);
}

// The codes of a block's values under its scale.  With the largest scale of a
// type 64 of them are beyond its range, so 63 is the most.
template <typename T, int LEN, typename V>
__device__ __forceinline__ void pack_codes(const V &x, int scale, int8_t (&code)[LEN])
{
    const float inverse = __uint_as_float((uint32_t)(254 - (scale == kPackNone ? 127 : scale)) << 23);
    const float most = scale == (__is_same(T, f16_t) ? 137 : 249) ? 63.f : 127.f;
#pragma unroll
    for (int k = 0; k < LEN; ++k) {
        float v = rintf((float)x[k] * inverse);
        v = v > most ? most : v < -most ? -most : v;
        code[k] = scale == kPackNone ? (int8_t)0 : (int8_t)(int)v;
    }
}

// Codes [n][dim] and scales [n][pack_blocks(dim)], both without gaps.
struct PackArgs {
    const void *x;
    int type;
    int64_t n;
    int dim;
    int64_t ld_x;
    int8_t *codes;
    uint8_t *scales;
};
bool pack_fits(int64_t n, int dim);  // a launch's limit
hipError_t launch_pack(const PackArgs &a, hipStream_t s);

struct UnpackArgs {
    const int8_t *codes;
    const uint8_t *scales;
    int64_t n;
    int dim;
    void *x;
    int type;
    int64_t ld_x;
    int width;  // columns written, zeros behind dim (at most dim rounded up to 32)
};
hipError_t launch_unpack(const UnpackArgs &a, hipStream_t s);

// ---- gated block ----

struct GatedArgs {
    const void *x;
    int type;
    int64_t n;
    int dim;
    int64_t ld_x;
    const void *gate;
    int64_t ld_gate;
    const void *up;
    int64_t ld_up;
    int hidden;
    int act;
    void *h;
    int64_t ld_h;
    void *work;
};
uint64_t gated_work(const GatedArgs &a);
hipError_t launch_gated(const GatedArgs &a, hipStream_t s);

struct GatedGradArgs {
    const void *gh;
    int64_t ld_gh;
    const void *x;          // or, where NULL, the rows held in 8 bits:
    const int8_t *codes;
    const uint8_t *scales;
    int type;
    int64_t n;
    int dim;
    int64_t ld_x;
    const void *gate;
    int64_t ld_gate;
    const void *up;
    int64_t ld_up;
    int hidden;
    int act;
    void *gx;
    int64_t ld_gx;
    void *ggate, *gup;
    int64_t ld_ggate, ld_gup;
    void *work;
};
uint64_t gated_grad_work(const GatedGradArgs &a);
hipError_t launch_gated_grad(const GatedGradArgs &a, hipStream_t s);

}  // namespace ersj
