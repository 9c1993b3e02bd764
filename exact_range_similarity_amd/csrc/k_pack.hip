// Rows held in 8 bits: 32 neighbours of a row share a power of two 2^e, the
// least of which 127 reach the largest of them, and each is held as the whole
// number of them nearest to it.  A power of two makes every step exact (scaling,
// the value that a code stands for, also as a 16-bit number), so nothing but
// the one rounding to a whole number is lost: at most half of 2^e, less than
// 1/127 of the largest (but for the ends of the scales: with a type's largest,
// 64 steps are held as 63, up to a whole 2^e off, 1/64 of the largest; with the
// least, 2^-126, runs whose largest is below 63.5 steps are off by half a step).
// Both kernels are bound by memory: 1M x 384 bf16, 1.16 GB each way, 217 to 250
// us to codes and 220 to 234 us back, 4.7 to 5.3 TB/s where a large copy has
// 5.2.  Hence items of 16 values, which make the codes' accesses 16 bytes wide,
// and four of them on their way in every thread.
#include "feedforward_internal.h"

namespace ersj {

namespace {

constexpr int kThreads = 256;
constexpr int kItem = 16;   // values of a lane: two lanes to a block
constexpr int kTurns = 4;   // items of a thread

// The place of item i of a workgroup's stretch: a workgroup works on consecutive
// items, rows of `per` items each, from one 64-bit division for its first.
struct Place {
    int64_t row;
    int item;
    __device__ __forceinline__ Place(int64_t row0, uint32_t item0, uint32_t i, uint32_t per)
    {
        const uint32_t at = item0 + i;
        row = row0 + at / per;
        item = (int)(at % per);
    }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void k_pack(PackArgs a)
{
    typedef Slot<T, kItem> X;
    typedef Slot<int8_t, kItem> C;
    const int blocks = pack_blocks(a.dim);
    const uint32_t per = 2 * blocks;
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kTurns), row0 = first / per;
    const uint32_t item0 = (uint32_t)(first - row0 * per);
    typename X::vec x[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const Place p(row0, item0, t * kThreads + threadIdx.x, per);
        const int c = p.item * kItem;
        if (p.row >= a.n) x[t] = (typename X::vec)(T)0.f;
        else {
            const T *from = (const T *)a.x + p.row * a.ld_x;
            if (c + kItem <= a.dim) x[t] = X::load(from + c);
            else
                for (int k = 0; k < kItem; ++k) x[t][k] = c + k < a.dim ? from[c + k] : (T)0.f;
        }
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const Place p(row0, item0, t * kThreads + threadIdx.x, per);
        uint32_t most = 0;  // as bits, which are ordered like the magnitudes, NaN above infinity
#pragma unroll
        for (int k = 0; k < kItem; ++k) {
            const uint32_t b = __float_as_uint((float)x[t][k]) & 0x7fffffffu;
            most = b > most ? b : most;
        }
        const uint32_t other = __builtin_amdgcn_update_dpp(0, most, 0xb1, 0xf, 0xf, true);  // lane ^ 1
        most = other > most ? other : most;
        const int scale = pack_scale(most);
        int8_t code[kItem];
        pack_codes<T, kItem>(x[t], scale, code);
        if (p.row >= a.n) continue;
        const int c = p.item * kItem;
        int8_t *to = a.codes + p.row * a.dim + c;
        if (c + kItem <= a.dim) {
            typename C::vec v;
#pragma unroll
            for (int k = 0; k < kItem; ++k) v[k] = code[k];
            C::store(to, v);
        } else {
#pragma unroll
            for (int k = 0; k < kItem; ++k)
                if (c + k < a.dim) to[k] = code[k];
        }
        if (!(p.item & 1)) a.scales[p.row * blocks + p.item / 2] = (uint8_t)scale;
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_unpack(UnpackArgs a)
{
    typedef Slot<T, kItem> X;
    typedef Slot<int8_t, kItem> C;
    const int blocks = pack_blocks(a.dim);
    const uint32_t per = 2 * blocks;
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kTurns), row0 = first / per;
    const uint32_t item0 = (uint32_t)(first - row0 * per);
    typename C::vec code[kTurns];
    int scale[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const Place p(row0, item0, t * kThreads + threadIdx.x, per);
        const int c = p.item * kItem;
        code[t] = (typename C::vec)(int8_t)0;
        scale[t] = 1;
        if (p.row >= a.n) continue;
        const int8_t *from = a.codes + p.row * a.dim + c;
        if (c + kItem <= a.dim) code[t] = C::load(from);
        else
            for (int k = 0; k < kItem; ++k) code[t][k] = c + k < a.dim ? from[k] : (int8_t)0;
        scale[t] = a.scales[p.row * blocks + p.item / 2];
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const Place p(row0, item0, t * kThreads + threadIdx.x, per);
        const int c = p.item * kItem;
        if (p.row >= a.n) continue;
        const float step = pack_step(scale[t]);
        typename X::vec x;
#pragma unroll
        for (int k = 0; k < kItem; ++k) x[k] = (T)((float)code[t][k] * step);
        T *to = (T *)a.x + p.row * a.ld_x + c;
        if (c + kItem <= a.dim) X::store(to, x);
        else {
#pragma unroll
            for (int k = 0; k < kItem; ++k)
                if (c + k < a.width) to[k] = c + k < a.dim ? x[k] : (T)0.f;
        }
    }
}

unsigned blocks_of(int64_t n, int dim)
{
    return (unsigned)((n * 2 * pack_blocks(dim) + kThreads * kTurns - 1) / (kThreads * kTurns));
}

}  // namespace

bool pack_fits(int64_t n, int dim) { return n * 2 * pack_blocks(dim) < ((int64_t)1 << 32) * kTurns - (1 << 20); }

hipError_t launch_pack(const PackArgs &a, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    ERSJ_ELEM_SWITCH(a.type, T, k_pack<T><<<blocks_of(a.n, a.dim), kThreads, 0, s>>>(a));
    return hipGetLastError();
}

hipError_t launch_unpack(const UnpackArgs &a, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    ERSJ_ELEM_SWITCH(a.type, T, k_unpack<T><<<blocks_of(a.n, a.dim), kThreads, 0, s>>>(a));
    return hipGetLastError();
}

}  // namespace ersj
