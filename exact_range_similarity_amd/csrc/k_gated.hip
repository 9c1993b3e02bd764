// The gated feed-forward block and its gradient.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u            (one kernel: both projections and the product)
//   du = dh act(g), dg = dh u act'(g)               (one kernel: the projections again)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x  (a product each, the first over both pairs)
//
// All of it is one tiled matrix product with different ends.  A workgroup owns
// tiles of BM x BM results in turn; the two operands' slabs of 64 along k are
// copied to LDS by loads that write it directly, up to two (small tiles: four)
// slabs ahead and into the next tile, and feed 16x16x32 matrix instructions
// (32x32x16 ones, which move more sums through the registers, took 1440 us where
// these take 1283, forward of 8192 x 4096 x 11008 bf16).  An operand whose rows run
// along k is read from LDS 16 bytes a lane; one whose rows run across k (the
// weights for dx, all operands of dW) is staged as it lies in memory and
// transposed by the LDS read itself, so no transposed copy of anything is made.
// For the projections the rows of the weights' slab alternate 32 of Wg and 32 of
// Wu, so a lane holds g and u of the same place.  The matrix instruction's first
// operand is the one along the results' rows in memory: a lane then holds four
// neighbours of a row.
//
// 8192 x 4096 x 11008 bf16: forward 1.13 ms (1.31 PFLOP/s), gradient 3.6 ms (1.22),
// bound by the matrix units at the clock that the power allows (2.0 GHz, 58% of
// their cycles busy, as in the library's product of this size, 1.25 PFLOP/s).
// 65,536 x 384 x 1024: forward 145 us, where a tile's end (activation, 134 MB of
// results) and the fetch of its six slabs weigh as much as its products.  Few rows
// are bound by the weights: 1 x 4096 x 11008, 180 MB, 33 us, 5.4 TB/s.
//
// 32-bit tensors are split into three bf16 parts, x = x1 + x2 + x3, each the
// rounded rest of those before (8 bits each: nothing is left of 24), and the six
// products of parts whose order is 2^-16 and above are summed, smallest first:
// the same kernel with six times the slabs, 215 TFLOP/s for 4096 x 4096 x 4096
// where the library's 32-bit product has 148.  What is dropped (x2 y3, x3 y2, x3
// y3) is at most 2^-23 of each product.
#include "feedforward_internal.h"

namespace ersj {

namespace {

typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f16_t f16x8 __attribute__((ext_vector_type(8)));
typedef bf16_t bf16x8 __attribute__((ext_vector_type(8)));

// Which planes are multiplied in turn, four bits each, smallest products first:
// one plane, three of both operands, three of one of them, two of one.
constexpr uint32_t kPlanes2 = 0x01, kPlanes6P = 0x010201, kPlanes6Q = 0x001021, kPlanes3 = 0x012;

constexpr int kSlab = 64, kSteps = kSlab / 32;

enum { kStore, kGate, kGateGrad };

// Division of numbers below 2^31 by a number known on the host.
struct Divide {
    uint32_t by, factor, shift;
    void set(uint32_t d)
    {
        by = d;
        uint32_t bits = 0;
        while (((uint64_t)1 << bits) < d) ++bits;
        // 2^p / d rounded up, p = 31 + bits: exact quotients below 2^31
        factor = d == 1 ? 0 : (uint32_t)((((uint64_t)1 << (31 + bits)) + d - 1) / d);
        shift = d == 1 ? 0 : bits - 1;
    }
    __device__ __forceinline__ int operator()(int n) const
    {
        return by == 1 ? n : (int)(__umulhi((uint32_t)n, factor) >> shift);
    }
};

struct ProductArgs {
    // P: along the results' rows (n), Q: across them (m); planes of 16-bit values
    const uint16_t *p[2], *q[2];
    int64_t p_plane, q_plane, ld_p, ld_q;
    // of one product.  Of an operand along k whole pieces of 8 values are read: behind
    // k its rows go on to the next multiple of 8, with zeros or values that meet zeros
    int k;
    int products;         // of planes
    uint32_t p_planes, q_planes;
    int sources;          // pairs (p[i], q[i]) summed, 1 or 2
    int m, n;
    int n_room;           // columns that may be read of P across k (a multiple of 8)
    int m_room;           // the same of Q
    int mt, nt, parts, outs;
    int slabs, all, len;  // slabs of a product, of all sources and products, of a part
    Divide by_slabs, by_out, by_tiles, by_column, by_rest;
    void *out[2];
    int64_t ld_out[2];
    float *part;          // [parts][outs][m][n] where parts > 1
    // kGateGrad
    const void *gh;
    int64_t ld_gh;
    uint16_t *dg, *du;
    int64_t d_plane, ld_d;
    int d_planes;         // of dg and du; 16 bits: 1 or 2, 1 in tiles of 256
    int n_pad;            // columns of dg and du that are written, zeros behind n
    int act;
    // f16: parts of k_bounds, and where the factor of dg and du and its inverse go
    const float *bounds;
    int bound_parts;
    float *factor;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// An offset that lies outside of every buffer here, also with what is added to
// it (both below 2^31): a load from outside gives zeros.
constexpr uint32_t kOutside = 0x80000000u;

// 16 bytes from each lane's place in a buffer to LDS, lane by lane from `lds`.
__device__ __forceinline__ void dma16(uint32_t lds, u32x4 buffer, uint32_t off)
{
    // s_nop: the wait state that a write of m0 needs before it is used.  m0 is a
    // reserved register: the compiler keeps nothing in it from one instruction to
    // another and takes it in no list of clobbered ones (none of this file's code
    // uses it but these lines).
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(off), "s"(buffer)
                 : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ void barrier()
{
    asm volatile("s_barrier" ::: "memory");
}

template <typename T>
__device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c)
{
    if constexpr (sizeof(T) == 2 && __is_same(T, f16_t))
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <typename T>
__device__ __forceinline__ uint16_t bits16(float v)
{
    return __builtin_bit_cast(uint16_t, (T)v);
}

// One bf16 part of a 32-bit value: its rounding to nearest, or its upper bits
// where that would overflow; what is not finite becomes NaN, so that no
// infinity meets another value's zero parts.
__device__ __forceinline__ uint16_t part_of(float &v)
{
    const uint32_t b = __float_as_uint(v);
    if ((b & 0x7f800000u) == 0x7f800000u) {
        v = 0.f;
        return 0x7fc0;
    }
    uint16_t r = bits16<bf16_t>(v);
    if ((r & 0x7f80) == 0x7f80) r = (uint16_t)(b >> 16);
    v -= __uint_as_float((uint32_t)r << 16);
    return r;
}

// One operand of a tile: its loads to LDS and its fragments.  ROWS values
// across k.  Along k (ACROSS false) a row of LDS holds kSlab values of k, its
// 16-byte pieces exchanged by the row so that 16 neighbouring rows cover all
// banks; across k it holds the tile's ROWS values at one k, its pieces exchanged
// in pairs by bits 0, 1 and 3 of k.  Either way a wave's reads fall on all banks.
// PAIR: rows of the slab are 32 of one matrix and 32 of another in turn.
//
// A slab is a buffer that begins with its first value, and a lane's loads lie a
// fixed distance apart.  What is outside the matrix is outside the buffer: rows
// behind the last of an operand along k and values of k of one across it by the
// buffer's length, values of k of one along it by the lane's offset.  (Columns
// of one across k that lie behind the tile's edge are the next row's first: they
// only meet results that are not written.)
template <int ROWS, bool ACROSS, bool PAIR>
struct Side {
    static constexpr int kBytes = ROWS * kSlab * 2;
    static constexpr int kLoads = kBytes / 4096;                   // of each of four waves
    static constexpr int kPieces = ACROSS ? ROWS / 8 : kSlab / 8;  // of a row of LDS
    static constexpr int kLoadRows = 64 / kPieces;                 // rows of LDS that a wave's load fills
    uint32_t off[2];  // of even and odd loads
    int piece;

    static __device__ __forceinline__ int exchange(int row)
    {
        if (!ACROSS) return (row >> 1) & 7;
        return ROWS == 64 ? (row & 2) | (row & 8) >> 1 : (row & 3) << 1 | (row & 8);
    }

    __device__ __forceinline__ void init(int wave, int64_t ld)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
            // a wave's first load, but exchanged like its second
            const int row = wave * kLoadRows + lane / kPieces;
            piece = (lane % kPieces) ^ exchange(row + odd * 4 * kLoadRows);
            off[odd] = (uint32_t)(row * (int)ld + piece * 8) * 2;
        }
    }

    // Bytes from one load of a lane to the next but `PAIR`'s, which come in twos.
    static __device__ __forceinline__ uint32_t distance(int j, int64_t ld)
    {
        return (uint32_t)((PAIR ? j >> 1 : j) * 4 * kLoadRows * (int)ld) * 2;
    }

    // The buffer of a slab at `base`: `room` rows (along k) or columns (across
    // it) from the tile's first on and `left` values of k exist.
    static __device__ __forceinline__ u32x4 buffer(const uint16_t *base, int64_t ld, int room, int left)
    {
        const uint64_t b = (uint64_t)base;
        return (u32x4){(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, length(ld, room, left), 0x00020000u};
    }
    static __device__ __forceinline__ uint32_t length(int64_t ld, int room, int left)
    {
        if (!ACROSS) return (uint32_t)((room < ROWS ? room : ROWS) * (int)ld) * 2;
        return (uint32_t)(((left < kSlab + 1 ? left : kSlab + 1) - 1) * (int)ld + room) * 2;
    }
    // To the next slab; `left`: of that.
    static __device__ __forceinline__ void move(u32x4 &b, int64_t ld, int room, int left)
    {
        const uint64_t to = ((uint64_t)b[1] << 32 | b[0]) + kSlab * 2 * (ACROSS ? (uint32_t)ld : 1u);
        b[0] = (uint32_t)to;
        b[1] = (uint32_t)(to >> 32);
        if (ACROSS) b[2] = length(ld, room, left);
    }

    // A lane's offset in load j of a slab.
    __device__ __forceinline__ uint32_t offset(int j, int64_t ld, int left) const
    {
        return (ACROSS || piece * 8 < left ? off[j & 1] : kOutside) + distance(j, ld);
    }

    // Values of 8 consecutive k for 16 consecutive rows from `row` (a multiple
    // of 16), for the matrix instruction of the slab's values 32 kk to 32 kk + 31.
    static __device__ __forceinline__ s16x8 fragment(const char *lds, int row, int kk)
    {
        const int lane = threadIdx.x & 63;
        if constexpr (ACROSS) {
            const int k = kk * 32 + (lane >> 4) * 8 + ((lane & 15) >> 2), col = row + (lane & 3) * 4;
            // four values of k on have the same exchange
            const int at = k * (ROWS * 2) + (((col >> 3) ^ exchange(k)) << 4) + (col & 7) * 2;
            typedef __attribute__((address_space(3))) s16x4 *ptr;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds_char *)(lds + at));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds_char *)(lds + at + 4 * ROWS * 2));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const int r = row + (lane & 15);
            const int c = (kk * 4 + (lane >> 4)) ^ exchange(r);
            return *(const s16x8 *)(lds + r * (kSlab * 2) + c * 16);
        }
    }
};

// exp(v); FAST: the hardware's exponential, off by about |v| 2^-24 of the result,
// for results of 16 bits.
template <bool FAST>
__device__ __forceinline__ float exp_of(float v)
{
    return FAST ? __expf(v) : expf(v);
}

template <bool FAST>
__device__ __forceinline__ float inverse(float v)
{
    return FAST ? __builtin_amdgcn_rcpf(v) : 1.f / v;
}

// The normal distribution Phi(g) and its density phi(g), by the upper tail of
// z = |g|, which keeps the bits of a small Phi.  FAST: the tail is exp(-z^2/2) R(z),
// R as a polynomial in t = 1 / (1 + 0.32 z), fitted to 1.4e-6 of the tail, which
// shares the density's exponential (65,536 x 384 x 1024 bf16: forward 146 us, 181
// with erff).  Otherwise it is erfcf's, and what the rounding of z^2 leaves over
// enters the exponential: off by some g^2 2^-24 of the tail, and not of 1.
template <bool FAST>
__device__ __forceinline__ float normal(float g, float &density)
{
    if constexpr (!FAST) {
        const float z = fminf(fabsf(g), 64.f), square = z * z;
        density = 0.39894228040143268f * expf(-0.5f * square) * (1.f - 0.5f * __builtin_fmaf(z, z, -square));
        const float tail = 0.5f * erfcf(z * 0.70710678118654752f);
        return g < 0.f ? tail : 1.f - tail;
    }
    const float e = exp_of<FAST>(-0.5f * g * g);
    density = 0.39894228040143268f * e;
    const float z = fabsf(g), t = __builtin_amdgcn_rcpf(1.f + 0.32f * z);
    float r = 0.0323464572429657f;
    r = r * t + -0.11485423147678375f;
    r = r * t + 0.09560500830411911f;
    r = r * t + 0.022990422323346138f;
    r = r * t + 0.09457922726869583f;
    r = r * t + 0.11398735642433167f;
    r = r * t + 0.12768389284610748f;
    r = r * t + 0.12766137719154358f;
    const float q = e * r * t;
    return g < 0.f ? q : 1.f - q;
}

// act(g) and its derivative.
template <bool FAST>
__device__ __forceinline__ float act_of(int act, float g)
{
    if (act == 1) {
        float density;
        return g * normal<FAST>(g, density);
    }
    const float k = 0.79788456080286536f;
    return g * inverse<FAST>(1.f + exp_of<FAST>(act == 0 ? -g : -2.f * k * (g + 0.044715f * g * g * g)));
}

template <bool FAST>
__device__ __forceinline__ float slope_of(int act, float g, float &value)
{
    if (act == 1) {
        float density;
        const float c = normal<FAST>(g, density);
        value = g * c;
        return c + g * density;
    }
    const float k = 0.79788456080286536f;
    const float s = inverse<FAST>(1.f + exp_of<FAST>(act == 0 ? -g : -2.f * k * (g + 0.044715f * g * g * g)));
    value = g * s;
    if (act == 0) return s * (1.f + g * (1.f - s));
    // (beyond 64 s is 0 or 1, and g^2 may be infinite)
    return s + value * (1.f - s) * 2.f * k * (1.f + 3 * 0.044715f * fminf(g * g, 4096.f));
}

// The power of two by which f16 dg and du are multiplied.  As they are, a sum
// over many rows would lose the terms below 6e-5 (1e-6 in grad_h: 4% of dW), and
// one above 65,504 would be infinite.  |u| and |act(g)| are at most |x| |w| and
// |act'| at most 1.13: 2^(14 - e) with 2^e the exponent of R W, R the largest of
// max|grad_h| |x| over the rows and W of the weights' |w|, keeps all of them below
// 1.13 * 2^15.  The bound is some sqrt(dim) above their size, which leaves twenty
// binades of normal numbers below it.
__device__ __forceinline__ float factor_of(float rows, float weights)
{
    const float bound = rows * weights;  // 2^-72 to 2^64, or 0
    return bound > 0.f ? __uint_as_float((uint32_t)(127 + 14 + 127 - (int)(__float_as_uint(bound) >> 23)) << 23) : 1.f;
}

__device__ __forceinline__ float wave_most(float v)
{
#pragma unroll
    for (int to = 32; to; to >>= 1) v = fmaxf(v, __shfl_xor(v, to));
    return v;
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int to = 32; to; to >>= 1) v += __shfl_xor(v, to);
    return v;
}

constexpr int kBoundParts = 1024;  // most workgroups of k_bounds

// R (blockIdx.y 0) and W (1) of factor_of over the rows of a workgroup's waves.
// Rows whose bound is not finite are left out: what comes of them is not finite
// whatever the factor.  20,000 x 384 x 1024: 57 MB, 13 us of the gradient's 159; one
// token x 4096 x 11008, where the weights are read once more for it: 37 us of 148.
struct BoundArgs {
    const f16_t *gh;
    int64_t ld_gh;
    // as the products read them: whole pieces of 16 bytes, zeros behind dim
    const f16_t *x, *gate, *up;
    int64_t ld_x, ld_w;
    int64_t n;
    int pad, hidden;  // pad: columns of x and of the weights
    float *part;      // [2][gridDim.x]
};
__global__ __launch_bounds__(256) void k_bounds(BoundArgs a)
{
    typedef Slot<f16_t, 8> S8;
    __shared__ float of_wave[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool weights = blockIdx.y;
    const int64_t count = weights ? 2 * (int64_t)a.hidden : a.n;
    float most = 0.f;
    for (int64_t r = (int64_t)blockIdx.x * 4 + wave; r < count; r += (int64_t)gridDim.x * 4) {
        const f16_t *row = !weights ? a.x + r * a.ld_x : r < a.hidden ? a.gate + r * a.ld_w : a.up + (r - a.hidden) * a.ld_w;
        float square = 0.f;
        for (int c = lane * 8; c < a.pad; c += 512) {
            const auto v = *(const typename S8::vec *)(row + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) square += (float)v[e] * (float)v[e];
        }
        float bound = sqrtf(wave_sum(square));
        if (!weights) {
            uint32_t top = 0;
            const f16_t *gh = a.gh + r * a.ld_gh;
            auto with = [&](f16_t v) {
                const uint32_t b = bits16<f16_t>(v) & 0x7fffu;
                top = b < 0x7c00u && b > top ? b : top;
            };
            for (int c = lane * 8; c < a.hidden; c += 512) {
                if (c + 8 <= a.hidden) {
                    const auto v = S8::load(gh + c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) with(v[e]);
                } else {
                    for (int e = c; e < a.hidden; ++e) with(gh[e]);
                }
            }
            bound *= wave_most((float)__builtin_bit_cast(f16_t, (uint16_t)top));
        }
        if (bound < __builtin_inff()) most = fmaxf(most, bound);
    }
    if (lane == 0) of_wave[wave] = most;
    __syncthreads();
    if (threadIdx.x == 0)
        a.part[blockIdx.y * gridDim.x + blockIdx.x] = fmaxf(fmaxf(of_wave[0], of_wave[1]), fmaxf(of_wave[2], of_wave[3]));
}

// What a workgroup works on next: a tile of one of the outputs, over a part of k.
struct Unit {
    int64_t m0;
    int n0, part, which, first, last;  // slabs [first, last) of all sources and products
};

// T: the 16-bit type multiplied; O: the tensors' type.
template <typename T, typename O, int BM, int kStages, bool PA, bool QA, int END>
__global__ __launch_bounds__(256, BM == 256 || kStages * BM > 256 ? 1 : 2) void k_product(ProductArgs a)
{
    constexpr int BN = BM, WAVES = 4;
    // waves two by two; in the smallest tile one above the other, so that each has g and u of its places
    constexpr int WM = BM == 64 ? 16 : BM / 2, WN = BM == 64 ? 64 : BN / 2, MB = WM / 16, NB = WN / 16;
    constexpr bool kPair = END != kStore;  // P's rows alternate between the two weights
    constexpr int CN = kPair ? BN / 2 : BN;
    constexpr bool FAST = sizeof(O) == 2;
    constexpr bool kFactor = __is_same(O, f16_t) && END != kGate;  // dg and du come multiplied by a factor
    typedef Side<BN, PA, kPair> P;
    typedef Side<BM, QA, false> Q;
    constexpr int STAGE = P::kBytes + Q::kBytes;
    constexpr int kTurn = sizeof(O) == 2 ? WM * 64 : 0;  // a wave's room to turn 32 columns of its results
    __shared__ __align__(1024) char lds[kStages * STAGE + WAVES * kTurn];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char *)lds;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;

    // Workgroups go to the eight dies in turn.  A die works through a stretch of
    // the units of its own, whose tiles lie in columns of eight rows of tiles,
    // so that what its workgroups read at a time stays in its cache.
    const int total = a.by_out.by * a.outs;
    const int die = blockIdx.x & 7, stride = (int)gridDim.x >> 3;
    const int share = total >> 3, rest = total & 7;
    const int end = (die + 1) * share + (die < rest ? die + 1 : rest);
    int unit = die * share + (die < rest ? die : rest) + (int)(blockIdx.x >> 3);
    if (unit >= end) return;
    auto decode = [&](int id) {
        Unit u;
        u.which = a.by_out(id);
        id -= u.which * a.by_out.by;
        u.part = a.by_tiles(id);
        id -= u.part * a.by_tiles.by;
        const int group = a.by_column(id);
        id -= group * a.by_column.by;
        const bool whole = group * 8 + 8 <= a.mt;
        const int tn = whole ? id >> 3 : a.by_rest(id);
        u.n0 = tn * CN;
        u.m0 = (int64_t)(group * 8 + id - tn * (whole ? 8 : (int)a.by_rest.by)) * BM;
        u.first = u.part * a.len;
        u.last = u.first + a.len < a.all ? u.first + a.len : a.all;
        return u;
    };

    // of dg and du, or its inverse for what is summed of them
    float factor = 1.f;
    if constexpr (kFactor && END == kGateGrad) {
        float most[2] = {0.f, 0.f};
        for (int i = lane * 4; i < a.bound_parts; i += 256)
#pragma unroll
            for (int of = 0; of < 2; ++of) {
                const f32x4 v = *(const f32x4 *)(a.bounds + of * a.bound_parts + i);
                most[of] = fmaxf(most[of], fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
            }
        factor = factor_of(wave_most(most[0]), wave_most(most[1]));
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            a.factor[0] = factor;
            a.factor[1] = 1.f / factor;
        }
    } else if constexpr (kFactor) {
        factor = a.factor[1];
    }
    if constexpr (kFactor) factor = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(factor)));

    // The loads run up to two slabs ahead of the products, across units: where
    // the next slab lies, how much of k it has, and how many more slabs follow it
    // side by side.  Most turns only move on.
    P p;
    Q q;
    p.init(wave, a.ld_p);
    q.init(wave, a.ld_q);
    Unit lu = decode(unit);
    int lunit = unit, pos = lu.first, left = 0, run = 0, p_room = 0, q_room = 0;
    u32x4 pb0 = (u32x4)0u, pb1 = (u32x4)0u, qb = (u32x4)0u;
    auto next_slab = [&]() {
        if (--run > 0) {
            left -= kSlab;
            P::move(pb0, a.ld_p, p_room, left);
            if constexpr (kPair) P::move(pb1, a.ld_p, p_room, left);
            Q::move(qb, a.ld_q, q_room, left);
            return;
        }
        if (pos == lu.last) {
            lunit += stride;
            if (lunit >= end) {  // there is none: what is loaded now is not read
                lunit = end;
                pb0[2] = pb1[2] = qb[2] = 0;
                return;
            }
            lu = decode(lunit);
            pos = lu.first;
        }
        const int seg = a.by_slabs(pos), at = pos - seg * a.slabs, k0 = at * kSlab;
        const int src = seg >= a.products, prod = seg - src * a.products;
        const int64_t po = ((a.p_planes >> (4 * prod)) & 15) * a.p_plane +
                           (PA ? (int64_t)k0 * a.ld_p + lu.n0 : (int64_t)lu.n0 * a.ld_p + k0);
        const int64_t qo = ((a.q_planes >> (4 * prod)) & 15) * a.q_plane +
                           (QA ? (int64_t)k0 * a.ld_q + lu.m0 : lu.m0 * a.ld_q + k0);
        left = a.k - k0;
        p_room = (PA ? a.n_room : a.n) - lu.n0;
        q_room = (int)((QA ? a.m_room : a.m) - lu.m0);
        pb0 = P::buffer(a.p[kPair ? 0 : src] + po, a.ld_p, p_room, left);
        if constexpr (kPair) pb1 = P::buffer(a.p[1] + po, a.ld_p, p_room, left);
        qb = Q::buffer(a.q[a.outs == 2 ? lu.which : src] + qo, a.ld_q, q_room, left);
        run = a.slabs - at < lu.last - pos ? a.slabs - at : lu.last - pos;
        pos += run;
    };
    constexpr int kLoads = P::kLoads + Q::kLoads;
    auto load = [&](int l, uint32_t at) {  // load l of the slab
        const uint32_t to = at + wave * 1024 + l * 4096;
        if (l < P::kLoads) dma16(to, kPair && (l & 1) ? pb1 : pb0, p.offset(l, a.ld_p, left));
        else dma16(to, qb, q.offset(l - P::kLoads, a.ld_q, left));
    };

    const int wn = BM == 64 ? 0 : (wave & 1) * WN, wm = (BM == 64 ? wave : wave >> 1) * WM;
    // kStages slabs are in LDS or on their way.  A slab's steps each multiply
    // what the step before read from LDS and read what the next one multiplies;
    // the last step begins with the slab's only barrier, behind which the next
    // slab is whole and this one's place is free for the slab kStages later.
    // (Four slabs of 32 in the same room are no faster, 1240 and 1309 us for dx of
    // 8192 x 4096 x 11008, and slower in tiles of 128, where barriers come often.)
    s16x8 fp[2][NB], fq[2][MB];
    // fragment r of a step, in the order in which the products need them
    auto read = [&](int set, int r, const char *at, int kk) {
        if (r == 0 || r > MB) fp[set][r ? r - MB : 0] = P::fragment(at, wn + (r ? r - MB : 0) * 16, kk);
        else fq[set][r - 1] = Q::fragment(at + P::kBytes, wm + (r - 1) * 16, kk);
    };
    constexpr int kCells = NB * MB, kReads = NB + MB;
    // reads done before product c: all in the first half of a step
    auto next_read = [](int c) constexpr { return c * 2 < kCells ? c * 2 * kReads / kCells : kReads; };
    for (int b = 0; b < kStages; ++b) {
        next_slab();
#pragma unroll
        for (int l = 0; l < kLoads; ++l) load(l, lds0 + b * STAGE);
    }
    wait_loads<(kStages - 1) * kLoads>();
    barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(0, r, lds, 0);

    typedef Slot<T, 4> S4;
    typedef Slot<T, 8> S8;
    auto grad_row = [&](int64_t m, int c) {  // eight values of grad_h, zeros outside
        typename S8::vec v = (typename S8::vec)(T)0.f;
        if (m < a.m) {
            const T *from = (const T *)a.gh + m * a.ld_gh + c;
            if (c + 8 <= a.n) v = S8::load(from);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = c + e < a.n ? from[e] : (T)0.f;
        }
        return v;
    };
    // loads of grad_h ahead of a unit's products, and a lower bound on what a
    // tile inside the block issues after the loads of its last slabs: its results'
    // stores and the next unit's loads of grad_h (at most what the counter holds)
    constexpr int kAhead = END == kGateGrad && sizeof(O) == 2 && BM < 256 ? WM / 16 : 0;
    constexpr int kStores = sizeof(O) == 4 ? (END == kStore ? kCells : END == kGate ? kCells / 2 : 0)
                            : END == kGate ? NB / 4 * (WM / 16) : NB / 2 * (WM / 16);
    // (not in the large tile, whose long sums hide that wait: forward of 8192 x
    // 4096 x 11008 1220 us, 1240 with it, for the registers that it takes)
    constexpr int kSince = BM == 256 ? 0 : kStores + kAhead < 40 ? kStores + kAhead : 40;
    bool before = false;  // the unit before lay inside the block

    char *turn = lds + kStages * STAGE + wave * kTurn;
    int buf = 0;
    for (; unit < end; unit += stride) {
        const Unit u = decode(unit);
        f32x4 acc[NB][MB];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j) acc[i][j] = (f32x4)0.f;
        const int64_t mw = u.m0 + wm;
        const int nw = u.n0 + (kPair ? wn / 2 : wn);
        // grad_h comes while the products are formed, a row's 32 columns over four
        // lanes; the large tile has no registers for it, and less need
        const bool inner = u.m0 + BM <= a.m && u.n0 + CN <= a.n;
        typename S8::vec dh[kAhead ? kAhead : 1];
        if constexpr (kAhead > 0) {
#pragma unroll
            for (int r = 0; r < kAhead; ++r) dh[r] = grad_row(mw + r * 16 + (lane >> 2), nw + (lane & 3) * 8);
        }
        // What was issued after the first slab's loads, in order, need not be waited for with them.
        const bool calm = inner && before;
        before = inner;
        // one workgroup's products go before the end of the other that shares the unit
        // (65,536 x 384 x 1024 bf16: forward 167 us, 161 with it, on one card)
        if constexpr (BM == 128) __builtin_amdgcn_s_setprio(1);
        for (int t = u.first; t < u.last; ++t) {
            const char *at = lds + buf * STAGE;
            const uint32_t free = lds0 + buf * STAGE;
            buf = (buf + 1) % kStages;
            const char *other = lds + buf * STAGE;
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) {
                if (kk == kSteps - 1) {
                    next_slab();
                    // this wave's loads of the next slab, and its reads of this one
                    if (kSince > 0 && calm && t == u.first)
                        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kStages - 2) * kLoads + kSince) : "memory");
                    else
                        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kStages - 2) * kLoads) : "memory");
                    barrier();
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int c = 0; c < kCells; ++c) {
                    const int i = c / MB, j = c % MB;
                    acc[i][j] = mma<T>(fp[kk & 1][i], fq[kk & 1][j], acc[i][j]);
                    if (kk == kSteps - 1) {
#pragma unroll
                        for (int l = c * kLoads / kCells; l < (c + 1) * kLoads / kCells; ++l) load(l, free);
                    }
#pragma unroll
                    for (int r = next_read(c); r < next_read(c + 1); ++r)
                        read((kk + 1) & 1, r, kk == kSteps - 1 ? other : at, (kk + 1) % kSteps);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }

        if constexpr (BM == 128) __builtin_amdgcn_s_setprio(0);

        // A lane's place: row j * 16 + lane % 16 of the wave's and, in register e
        // of block i, column i * 16 + 4 (el / 16) + e.
        // (The lane is hidden from the compiler, which would keep all addresses of
        // the end in registers during the products.)
        int el = lane;
        asm volatile("" : "+v"(el));
        const int ln = (el >> 4) * 4, lm = el & 15;
        // Rows of 32 columns of 16 bits, turned through LDS so that a lane moves
        // 16 bytes and four lanes a row; pieces of 16 bytes are exchanged by the
        // row, so that all banks take part.
        auto place = [&](int row, int piece) { return turn + row * 64 + ((piece ^ ((row >> 2) & 3)) << 4); };
        auto mine = [&](int j, int half) {  // this lane's four of a block's half of 16 columns
            return (typename S4::vec *)(place(j * 16 + lm, half * 2 + (el >> 5)) + ((el >> 4) & 1) * 8);
        };
        auto put = [&](int j, int half, f32x4 v) { *mine(j, half) = __builtin_convertvector(v, typename S4::vec); };
        // What a lane writes there another reads, within a wave and in vectors of
        // another length: nothing is moved across these places.
        auto turned = []() { asm volatile("" ::: "memory"); };
        auto store = [&](T *out, int64_t ld, int col, int64_t width) {  // the wave's rows, columns from col on
            turned();
#pragma unroll
            for (int r = 0; r < WM / 16; ++r) {
                const int row = r * 16 + (el >> 2), c = col + (el & 3) * 8;
                const typename S8::vec v = *(const typename S8::vec *)place(row, el & 3);
                if (mw + row >= a.m) continue;
                T *to = out + (mw + row) * ld + c;
                if (c + 8 <= width) S8::store(to, v);
                else
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e < width) to[e] = v[e];
            }
            turned();
        };
        // 32 bits: a lane's four neighbours as they are, at offsets in a buffer that
        // ends with the tile's last row (few registers for addresses, unlike pointers)
        const bool whole = u.n0 + CN <= a.n;
        __amdgpu_buffer_rsrc_t out32;
        uint32_t at32 = 0, step32 = 0;
        auto open32 = [&](float *out, int64_t ld) {
            const int rows = a.m - u.m0 < BM ? (int)(a.m - u.m0) : BM;
            out32 = __builtin_amdgcn_make_buffer_rsrc(out + u.m0 * ld + u.n0, 0, rows * (int)ld * 4, 0x00020000);
            step32 = (uint32_t)(int)ld * 64;  // 16 rows
            at32 = (uint32_t)((wm + lm) * (int)ld + (nw - u.n0) + ln) * 4;
        };
        auto store32 = [&](int j, int col, f32x4 v) {
            const uint32_t off = at32 + j * step32 + col * 4;
            const auto words = __builtin_bit_cast(u32x4, v);
            if (whole) __builtin_amdgcn_raw_buffer_store_b128(words, out32, off, 0, 0);
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    __builtin_amdgcn_raw_buffer_store_b32(words[e], out32,
                                                          nw + ln + col + e < a.n ? off + 4 * e : kOutside, 0, 0);
        };
        // 32 bits: a sum leaves its accumulation register where it is stored, and not before
        auto take = [](f32x4 v) {
            if constexpr (sizeof(O) == 4) asm volatile("" : "+v"(v));
            return v;
        };
        if constexpr (END == kStore) {
            if (a.parts > 1 || sizeof(O) == 4) {
                if (a.parts > 1) open32(a.part + ((int64_t)u.part * a.outs + u.which) * a.m * a.n, a.n);
                else open32((float *)a.out[u.which], a.ld_out[u.which]);
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int j = 0; j < MB; ++j) {
                        store32(j, i * 16, kFactor ? acc[i][j] * factor : take(acc[i][j]));
                        __builtin_amdgcn_sched_barrier(0);
                    }
            } else if constexpr (sizeof(O) == 2) {
#pragma unroll
                for (int i = 0; i < NB; i += 2) {
#pragma unroll
                    for (int j = 0; j < MB; ++j) {
                        put(j, 0, kFactor ? acc[i][j] * factor : acc[i][j]);
                        put(j, 1, kFactor ? acc[i + 1][j] * factor : acc[i + 1][j]);
                    }
                    store((T *)a.out[u.which], a.ld_out[u.which], nw + i * 16, a.n);
                }
            }
        } else {
            // blocks i and i + 1 hold g, the two after them u
            if constexpr (END == kGate && sizeof(O) == 4) open32((float *)a.out[0], a.ld_out[0]);
#pragma unroll
            for (int i = 0; i < NB; i += 4) {
                const int col = nw + i * 8;
                if constexpr (END == kGateGrad && sizeof(O) == 2) {
                    // grad_h to the lanes that hold g and u
#pragma unroll
                    for (int r = 0; r < WM / 16; ++r)
                        *(typename S8::vec *)place(r * 16 + (el >> 2), el & 3) =
                            kAhead ? dh[kAhead ? r : 0] : grad_row(mw + r * 16 + (el >> 2), col + (el & 3) * 8);
                    turned();
                }
#pragma unroll
                for (int j = 0; j < MB; ++j) {
                    __builtin_amdgcn_sched_barrier(0);  // one block at a time, for the registers' sake
                    const int64_t m = mw + j * 16 + lm;
                    if constexpr (END == kGate) {
                        f32x4 h[2];
                        auto both = [&](int act) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                h[e / 4][e % 4] = act_of<FAST>(act, acc[i + e / 4][j][e % 4]) * acc[i + 2 + e / 4][j][e % 4];
                        };
                        switch (a.act) {
                        case 0: both(0); break;
                        case 1: both(1); break;
                        default: both(2);
                        }
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if constexpr (sizeof(O) == 2) put(j, half, h[half]);
                            else store32(j, i * 8 + half * 16, h[half]);
                        }
                    } else {
                        // g and u give way to dg and du
                        f32x4 d[2];
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if constexpr (sizeof(O) == 2) {
                                d[half] = __builtin_convertvector(*mine(j, half), f32x4);
                                if constexpr (kFactor) d[half] *= factor;
                            } else {
                                const int n = col + half * 16 + ln;
                                const float *gh = (const float *)a.gh + m * a.ld_gh;
                                if (m < a.m && n + 3 < a.n) d[half] = Slot<float, 4>::load(gh + n);
                                else
#pragma unroll
                                    for (int e = 0; e < 4; ++e) d[half][e] = m < a.m && n + e < a.n ? gh[n + e] : 0.f;
                            }
                        }
                        auto both = [&](int act) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float value;
                                const float s = slope_of<FAST>(act, acc[i + e / 4][j][e % 4], value), dh = d[e / 4][e % 4];
                                acc[i + e / 4][j][e % 4] = dh * acc[i + 2 + e / 4][j][e % 4] * s;
                                acc[i + 2 + e / 4][j][e % 4] = dh * value;
                            }
                        };
                        switch (a.act) {
                        case 0: both(0); break;
                        case 1: both(1); break;
                        default: both(2);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (sizeof(O) == 2) {
                    if constexpr (END == kGateGrad) {
                        turned();
                        // zeros behind the block's columns come from the zeros in the place of grad_h
#pragma unroll
                        for (int of = 0; of < 2; ++of) {
                            T *to = (T *)(of ? a.du : a.dg);
                            for (int plane = 0;; ++plane) {
#pragma unroll
                                for (int j = 0; j < MB; ++j) {
                                    put(j, 0, acc[i + 2 * of][j]);
                                    put(j, 1, acc[i + 2 * of + 1][j]);
                                }
                                store(to, a.ld_d, col, a.n_pad);
                                if (BM == 256 || plane + 1 == a.d_planes) break;
                                to += a.d_plane;
#pragma unroll
                                for (int c = 0; c < 2 * MB; ++c) {
                                    f32x4 &v = acc[i + 2 * of + c / MB][c % MB];
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const float h = (float)(T)v[e];
                                        v[e] = fabsf(h) < __builtin_inff() ? v[e] - h : 0.f;
                                    }
                                }
                            }
                        }
                    } else {
                        store((T *)a.out[0], a.ld_out[0], col, a.n);
                    }
                } else if constexpr (END == kGateGrad) {
#pragma unroll
                    for (int of = 0; of < 4; ++of)
#pragma unroll
                        for (int j = 0; j < MB; ++j) {
                            const int64_t m = mw + j * 16 + lm;
                            const int n = col + (of & 1) * 16 + ln;
                            f32x4 v = acc[i + of][j];
                            if (m >= a.m || n >= a.n_pad) continue;
                            uint16_t *to = (of & 2 ? a.du : a.dg) + m * a.ld_d + n;
#pragma unroll
                            for (int k = 0; k < 3; ++k) {
                                s16x4 x;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float f = v[e];
                                    x[e] = (short)part_of(f);
                                    v[e] = f;
                                }
                                *(s16x4 *)(to + k * a.d_plane) = x;
                            }
                        }
                }
            }
        }
    }
    wait_loads<0>();  // no load is on its way to LDS when the workgroup ends
}

// Zeros, for the gradients of weights that no row meets.
template <typename O>
__global__ __launch_bounds__(256) void k_zero(O *out, int64_t ld, int m, int n)
{
    for (int64_t r = blockIdx.x; r < m; r += gridDim.x)
        for (int c = threadIdx.x; c < n; c += 256) out[r * ld + c] = (O)0.f;
}

// Sums of the parts of a product, in order, eight of them on their way at a
// time.  (Only products of few tiles have parts: m n is at most 2^24.)
struct Parts {
    const float *part;
    int parts, m, n, all;  // all: of one or two results [m][n]
    Divide by_n;
    void *out[2];
    int64_t ld[2];
};
struct Joins {
    Parts p[2];
};
template <typename O>
__global__ __launch_bounds__(256) void k_product_join(Joins joins)
{
    const Parts a = joins.p[blockIdx.y];
    const int i = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= a.all) return;
    f32x4 v = (f32x4)0.f;
    if (i + 4 <= a.all) {
        for (int p = 0; p < a.parts; p += 8) {
            f32x4 x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                x[u] = Slot<float, 4>::load(a.part + (int64_t)(p + u < a.parts ? p + u : a.parts - 1) * a.all + i);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (p + u < a.parts) v += x[u];
        }
    } else {
        for (int p = 0; p < a.parts; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < a.all) v[e] += a.part[(int64_t)p * a.all + i + e];
    }
    int row = a.by_n(i), col = i - row * a.n;
    auto at = [&](int r) { return row < a.m ? (O *)a.out[0] + r * a.ld[0] : (O *)a.out[1] + (r - a.m) * a.ld[1]; };
    if (col + 4 <= a.n) {
        Slot<O, 4>::store(at(row) + col, __builtin_convertvector(v, typename Slot<O, 4>::vec));
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e, ++col) {
        if (i + e >= a.all) return;
        while (col >= a.n) {
            col -= a.n;
            ++row;
        }
        at(row)[col] = (O)v[e];
    }
}

// Matrices [n][dim] as the products read them: 16-bit values with rows of `pad`
// (a multiple of 8) and zeros behind the row's end; three planes for 32 bits.
struct Lay {
    const void *src;
    int64_t ld, n;
    int dim, pad;
    uint16_t *out;
};
struct Lays {
    Lay m[3];
};
template <typename S>
__global__ __launch_bounds__(256) void k_lay(Lays l)
{
    constexpr int kLen = 16 / sizeof(S);  // a thread's values
    typedef Slot<S, kLen> V;
    const Lay a = l.m[blockIdx.y];
    const uint32_t per = a.pad / kLen;
    const int64_t all = a.n * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i >> 32 ? i / per : (int64_t)((uint32_t)i / per);
        const int c = (int)(i - r * per) * kLen;
        const S *src = (const S *)a.src + r * a.ld + c;
        typename V::vec v;
        if (c + kLen <= a.dim) v = V::load(src);
        else
#pragma unroll
            for (int e = 0; e < kLen; ++e) v[e] = c + e < a.dim ? src[e] : (S)0.f;
        uint16_t *to = a.out + r * a.pad + c;
        if constexpr (sizeof(S) == 2) {
            *(typename V::vec *)to = v;
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                s16x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float f = v[e];
                    x[e] = (short)part_of(f);
                    v[e] = f;
                }
                *(s16x4 *)(to + k * a.n * a.pad) = x;
            }
        }
    }
}

unsigned blocks_for(int64_t threads)
{
    const int64_t b = (threads + 255) / 256;
    return (unsigned)(b < 1 ? 1 : b > 65536 ? 65536 : b);
}

int pad8(int v) { return (v + 7) & ~7; }

// A matrix as an operand: in place, or laid out in the working memory.
struct Operand {
    const uint16_t *p = nullptr;
    int64_t ld = 0, plane = 0;
    bool laid = false;
};

struct Room {
    char *base;
    uint64_t used = 0;
    void *take(uint64_t bytes)
    {
        void *at = (void *)((uintptr_t)base + used);
        used += (bytes + 255) & ~(uint64_t)255;
        return at;
    }
};

// In place where the loads can take it: 16-bit values, rows that begin at 16
// bytes and hold whole pieces of 16 bytes, spaced so that a tile's offsets stay
// below 2^31 bytes.  Otherwise laid out in `planes` of 16-bit values, with zeros
// behind dim to the next multiple of 8.
Operand operand(Room &room, const void *p, int type, int64_t n, int dim, int64_t ld, int planes)
{
    Operand o;
    if (p && type != kF32 && dim % 8 == 0 && ld % 8 == 0 && ((uintptr_t)p & 15) == 0 && ld < (1 << 22)) {
        o.p = (const uint16_t *)p;
        o.ld = ld;
        return o;
    }
    const int pad = pad8(dim);
    o.laid = true;
    o.ld = pad;
    o.plane = n * pad;
    o.p = (const uint16_t *)room.take((uint64_t)o.plane * 2 * planes);
    return o;
}

// Lays out those of the matrices that are not read in place.
struct Layer {
    Lays l;
    int count = 0;
    int64_t most = 0;
    void add(const Operand &o, const void *src, int64_t n, int dim, int64_t ld)
    {
        if (!o.laid || !src) return;
        l.m[count++] = Lay{src, ld, n, dim, (int)o.ld, const_cast<uint16_t *>(o.p)};
        if (n * o.ld > most) most = n * o.ld;
    }
    hipError_t run(int type, hipStream_t s) const
    {
        if (!count) return hipSuccess;
        const dim3 blocks(blocks_for(most / (type == kF32 ? 4 : 8)), count);
        if (type == kF32) k_lay<float><<<blocks, 256, 0, s>>>(l);
        else k_lay<f16_t><<<blocks, 256, 0, s>>>(l);
        return hipGetLastError();
    }
};

// Tiles of a product, by their edge and the slabs that are in LDS or on their way.
enum Tile { kTile64, kTile128, kTile128Deep, kTile256 };
constexpr int edge_of(Tile t) { return t == kTile64 ? 64 : t == kTile256 ? 256 : 128; }

template <typename T, typename O, bool PA, bool QA, int END>
hipError_t run_product(ProductArgs &a, Tile tile, hipStream_t s)
{
    // that end's code for 32 bits is too long for the large tile; only projections take the deep one
    constexpr bool kLarge = !(END == kGateGrad && sizeof(O) == 4), kDeep = END != kStore;
    if (tile == kTile256 && !kLarge) tile = kTile128;
    const int bm = edge_of(tile), bn = bm / (END == kStore ? 1 : 2);
    a.mt = (a.m + bm - 1) / bm;
    a.nt = (a.n + bn - 1) / bn;
    a.slabs = (a.k + kSlab - 1) / kSlab;
    a.all = a.slabs * a.products * a.sources;
    a.len = (a.all + a.parts - 1) / a.parts;
    a.parts = (a.all + a.len - 1) / a.len;  // none is empty
    const int64_t count = (int64_t)a.mt * a.nt * a.parts * a.outs;
    if (count >= (int64_t)1 << 31) return hipErrorInvalidConfiguration;
    a.by_slabs.set(a.slabs);
    a.by_out.set(a.mt * a.nt * a.parts);
    a.by_tiles.set(a.mt * a.nt);
    a.by_column.set(8 * a.nt);
    a.by_rest.set(a.mt % 8 ? a.mt % 8 : 8);
    // as many workgroups as run at once, a multiple of the dies
    const int64_t most = tile == kTile256 || tile == kTile128Deep ? 256 : 512;
    const unsigned blocks = (unsigned)(count < most ? (count + 7) & ~(int64_t)7 : most);
    switch (tile) {
    case kTile64: k_product<T, O, 64, 4, PA, QA, END><<<blocks, 256, 0, s>>>(a); break;
    case kTile128: k_product<T, O, 128, 2, PA, QA, END><<<blocks, 256, 0, s>>>(a); break;
    case kTile128Deep:
        if constexpr (kDeep) k_product<T, O, 128, 4, PA, QA, END><<<blocks, 256, 0, s>>>(a);
        break;
    default:
        if constexpr (kLarge) k_product<T, O, 256, 2, PA, QA, END><<<blocks, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <bool PA, bool QA, int END>
hipError_t product(ProductArgs &a, int type, Tile tile, hipStream_t s)
{
    if (type == kF32) return run_product<bf16_t, float, PA, QA, END>(a, tile, s);
    if (type == kF16) return run_product<f16_t, f16_t, PA, QA, END>(a, tile, s);
    return run_product<bf16_t, bf16_t, PA, QA, END>(a, tile, s);
}

int64_t tiles_of(int64_t m, int64_t n, Tile t) { return ((m + edge_of(t) - 1) / edge_of(t)) * ((n + edge_of(t) - 1) / edge_of(t)); }

// Whether m x n results of `slabs` slabs each are formed in tiles of 256 x 256:
// where every compute unit gets one and the sum is long enough.  They read less,
// but two workgroups of 128 x 128 overlap one's end with the other's products, and
// wide tiles may lie half outside (dx of 65,536 x 384 x 1024, 384 columns: 121 us with
// 128, 132 with 256).  Forward of 16,384 x 64 slabs x 4096 bf16, in us with 128 and 256:
// 6 slabs 124, 142; 12 210, 214; 16 271, 260; 24 389, 352; 32 507, 443; 64 977, 823.
// dx of 16,384 x 4096 x (32 a slab): 24 slabs 424, 428; 32 506, 477; 64 1011, 910.
bool large_tiles(int64_t m, int64_t n, int64_t slabs)
{
    const int64_t large = tiles_of(m, n, kTile256);
    return slabs >= 24 && large >= 256 && large * 20 <= tiles_of(m, n, kTile128) * 6;
}

// Otherwise, for the projections, whose sums cannot be cut: 64 x 64 where all such
// tiles run at once, 512 of them, else 128 x 128, with four slabs on their way
// where there is one for a compute unit (and two slabs where there are more and
// two share a unit).  In us, tiles of 64, of 128 with four slabs and with two:
//   1 x 4096 x 11008 bf16, 344 of 64:      33.5  35.2  43.0   (180 MB: 5.4 TB/s)
//   64 x 4096 x 11008, 344:                35.6  35.9  51.1
//   128 x 4096 x 11008, 688:               45.4  36.9  53.5
//   200 x 4096 x 4096, 512:                30.2  35.6  43.8
//   200 x 2048 x 5632, 704:                24.4  21.0  24.9
//   600 x 768 x 3000, 940:                 15.6  12.3  11.4
//   1000 x 1000 x 1000 f32, 512:           65.2  67.8  86.7
//   1100 x 1000 x 1000 f32, 576:           88.8  70.3  89.0
//   1999 x 385 x 1001 f32, 1024:           57.5  42.6  47.0
//   64 x 4096 x 11008 f32, 344:             424   405   529   (the other way)
//   3000 x 768 x 1024 f32, 384 of 128:    115.6  98.2  78.2
Tile projection_tile(int64_t m, int64_t n, int64_t slabs)
{
    if (large_tiles(m, n, slabs)) return kTile256;
    if (tiles_of(m, n, kTile128) > 256) return kTile128;
    return tiles_of(m, n, kTile64) <= 512 ? kTile64 : kTile128Deep;
}

// Other sums are cut into parts; small products do better in small tiles, by
// tiles of 128 times slabs (the gradient with dx alone, in us in tiles of 64 and of
// 128; 768: 1000 x 384 x 1024 bf16, 22.6 and 24.5; 4096: 500 x 1024 x 4096 bf16,
// 40.3 and 40.4; 4608: 1000 x 384 x 1024 f32, 67.4 and 63.5; 6048: 8000 x 384 x 1024
// bf16, 53.5 and 48.9; 9216: 2000 x 384 x 1024 f32, 94.4 and 75.6).
Tile sum_tile(int64_t m, int64_t n, int64_t slabs)
{
    if (large_tiles(m, n, slabs)) return kTile256;
    const int64_t tiles = tiles_of(m, n, kTile128);
    return tiles <= 256 && tiles * slabs <= 5000 ? kTile64 : kTile128;
}

// Into how many parts a sum is cut so that the device is filled, each of four
// slabs at least.
int parts_of(int64_t m, int64_t n, int64_t slabs, Tile t)
{
    if (t == kTile256) return 1;
    const int64_t tiles = tiles_of(m, n, t);
    if (t == kTile128 && tiles > 64 && tiles <= 1024) {
        // the parts that come out even: turns of 512 workgroups by what each takes
        // (900 ns a slab, three for the end), and joining (8 bytes a value and part).
        // Both weights' gradient of 16,384 x 1280 x 3328 bf16, 520 tiles: 727 us in
        // one part, 680 in three; of 65,536 x 768 x 2048, 192 tiles: 1051 us in the
        // two that run at once, 1021 in five.
        int best = 1;
        int64_t least = 0;
        for (int p = 1; p <= 8 && (p == 1 || p <= slabs / 4); ++p) {
            const int64_t turns = (tiles * p + 511) / 512, ns = turns * ((slabs + p - 1) / p + 3) * 900;
            const int64_t all = p == 1 ? ns : ns + p * m * n / 625 + 4000;
            if (p > 1 && all * 20 > least * 19) continue;  // for less than a 20th it does not get more room
            best = p;
            least = all;
        }
        return best;
    }
    int64_t parts = 512 / tiles;
    if (parts > slabs / 4) parts = slabs / 4;
    return parts < 1 ? 1 : (int)parts;
}

// The weights as operands, both laid out or both in place with one spacing.
void weights(Room &room, const void *gate, int64_t ld_gate, const void *up, int64_t ld_up, int type, int hidden, int dim,
             Operand &g, Operand &u)
{
    const int planes = type == kF32 ? 3 : 1;
    g = operand(room, gate, type, hidden, dim, ld_gate, planes);
    u = operand(room, up, type, hidden, dim, ld_up, planes);
    if (g.laid && u.laid) return;
    if (g.laid || u.laid || g.ld != u.ld) {
        if (!g.laid) g = operand(room, nullptr, type, hidden, dim, 0, planes);
        if (!u.laid) u = operand(room, nullptr, type, hidden, dim, 0, planes);
    }
}

struct ForwardPlan {
    Operand x, gate, up;
    uint64_t bytes;
};

ForwardPlan plan(const GatedArgs &a)
{
    Room room{(char *)a.work};
    ForwardPlan f;
    f.x = operand(room, a.x, a.type, a.n, a.dim, a.ld_x, a.type == kF32 ? 3 : 1);
    weights(room, a.gate, a.ld_gate, a.up, a.ld_up, a.type, a.hidden, a.dim, f.gate, f.up);
    f.bytes = room.used;
    return f;
}

struct GradPlan {
    Operand x, gate, up;
    uint16_t *dg, *du;
    int64_t d_plane;
    int n_pad, outs, d_planes;
    float *bounds, *factor;  // f16
    int bound_parts;
    float *x_part, *w_part;
    int x_parts, w_parts;
    Tile h_tile, x_tile, w_tile;
    uint64_t bytes;
};

GradPlan plan(const GatedGradArgs &a)
{
    Room room{(char *)a.work};
    GradPlan f{};
    // what a code stands for is a bf16 number (in f16 rows an f16 one): one plane
    f.x = operand(room, a.x, a.type, a.n, a.dim, a.ld_x, a.type == kF32 && a.x ? 3 : 1);
    weights(room, a.gate, a.ld_gate, a.up, a.ld_up, a.type, a.hidden, a.dim, f.gate, f.up);
    // dg and du as 16-bit values are a rounding more than the results' own, 1.4 times
    // its error; in small products, which other things bound, they have a second
    // plane for what the first leaves over.  One plane and two, in us, bf16: 9 x 384 x
    // 1024 28 and 28, 300 x 384 x 1024 28 and 30, 16 x 2048 x 4096 37 and 45 (the most
    // that it costs here); beyond, 2000 x 384 x 1024 43 and 60, 1 x 4096 x 11008, where the
    // weights are read twice for it, 109 and 143.  The projections' large tile writes one.
    const int64_t weight = (int64_t)a.dim * a.hidden, slabs_h = (pad8(a.dim) + kSlab - 1) / kSlab;
    f.h_tile = projection_tile(a.n, 2 * (int64_t)a.hidden, slabs_h * (a.type != kF32 ? 1 : a.x ? 6 : 3));
    const bool two = f.h_tile != kTile256 && a.n * weight <= (int64_t)1 << 27 && weight <= 1 << 23;
    f.d_planes = a.type == kF32 ? 3 : two ? 2 : 1;
    const int planes = f.d_planes;
    f.n_pad = pad8(a.hidden);
    f.d_plane = a.n * f.n_pad;
    f.dg = (uint16_t *)room.take((uint64_t)f.d_plane * 2 * planes);
    f.du = (uint16_t *)room.take((uint64_t)f.d_plane * 2 * planes);
    if (a.type == kF16) {
        // workgroups of k_bounds, four rows or more each, that the projections read 256 at a time
        const int64_t most = a.n > 2 * (int64_t)a.hidden ? a.n : 2 * (int64_t)a.hidden;
        f.bound_parts = most > 4 * (kBoundParts - 256) ? kBoundParts : (int)((most + 1023) / 1024) * 256;
        f.bounds = (float *)room.take(2 * sizeof(float) * f.bound_parts);
        f.factor = (float *)room.take(2 * sizeof(float));
    }
    f.outs = (a.ggate != nullptr) + (a.gup != nullptr);
    const int64_t m = (int64_t)f.outs * a.hidden, slabs_x = (f.n_pad + kSlab - 1) / kSlab, slabs_w = (a.n + kSlab - 1) / kSlab;
    const int64_t all_x = slabs_x * 2 * (planes == 3 ? 6 : planes), all_w = slabs_w * (planes < 3 ? planes : a.x ? 6 : 3);
    f.x_tile = sum_tile(a.n, a.dim, all_x);
    f.w_tile = sum_tile(m, a.dim, all_w);
    f.x_parts = a.gx && a.n ? parts_of(a.n, a.dim, all_x, f.x_tile) : 1;
    f.w_parts = f.outs && a.n ? parts_of(m, a.dim, all_w, f.w_tile) : 1;
    f.x_part = (float *)room.take(f.x_parts > 1 ? (uint64_t)f.x_parts * a.n * a.dim * 4 : 0);
    f.w_part = (float *)room.take(f.w_parts > 1 ? (uint64_t)f.w_parts * m * a.dim * 4 : 0);
    f.bytes = room.used;
    return f;
}

// The parts of one product or two, added in one launch.
struct Joiner {
    Joins j;
    int count = 0, most = 0;
    void add(const ProductArgs &p)
    {
        if (p.parts == 1) return;
        Parts &a = j.p[count++];
        a.part = p.part;
        a.parts = p.parts;
        a.m = p.m;
        a.n = p.n;
        a.all = p.m * p.n * p.outs;
        a.by_n.set(p.n);
        for (int i = 0; i < 2; ++i) {
            a.out[i] = p.out[i];
            a.ld[i] = p.ld_out[i];
        }
        if (a.all > most) most = a.all;
    }
    hipError_t run(int type, hipStream_t s) const
    {
        if (!count) return hipSuccess;
        const dim3 blocks(blocks_for((most + 3) / 4), count);
        ERSJ_ELEM_SWITCH(type, O, k_product_join<O><<<blocks, 256, 0, s>>>(j));
        return hipGetLastError();
    }
};

// P = the weights, Q = the rows: both projections.
ProductArgs projections(const Operand &gate, const Operand &up, const Operand &x, int type, bool held, int64_t n,
                        int dim, int hidden, int act)
{
    ProductArgs p{};
    p.p[0] = gate.p;
    p.p[1] = up.p;
    p.q[0] = x.p;
    p.ld_p = gate.ld;
    p.ld_q = x.ld;
    p.p_plane = gate.plane;
    p.q_plane = x.plane;
    p.k = pad8(dim);
    p.products = type != kF32 ? 1 : held ? 3 : 6;
    p.p_planes = type != kF32 ? 0 : held ? kPlanes3 : kPlanes6P;
    p.q_planes = type != kF32 || held ? 0 : kPlanes6Q;
    p.sources = p.parts = p.outs = 1;
    p.m = (int)n;
    p.n = hidden;
    p.act = act;
    return p;
}

#define TRY_HIP(expr)                        \
    do {                                     \
        const hipError_t e__ = (expr);       \
        if (e__ != hipSuccess) return e__;   \
    } while (0)

}  // namespace

uint64_t gated_work(const GatedArgs &a) { return a.n ? plan(a).bytes : 0; }

hipError_t launch_gated(const GatedArgs &a, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    const ForwardPlan f = plan(a);
    Layer layer;
    layer.add(f.x, a.x, a.n, a.dim, a.ld_x);
    layer.add(f.gate, a.gate, a.hidden, a.dim, a.ld_gate);
    layer.add(f.up, a.up, a.hidden, a.dim, a.ld_up);
    TRY_HIP(layer.run(a.type, s));
    ProductArgs p = projections(f.gate, f.up, f.x, a.type, false, a.n, a.dim, a.hidden, a.act);
    p.out[0] = a.h;
    p.ld_out[0] = a.ld_h;
    return product<false, false, kGate>(p, a.type, projection_tile(a.n, 2 * (int64_t)a.hidden, (int64_t)p.products * ((p.k + kSlab - 1) / kSlab)), s);
}

uint64_t gated_grad_work(const GatedGradArgs &a) { return plan(a).bytes; }

hipError_t launch_gated_grad(const GatedGradArgs &a, hipStream_t s)
{
    const GradPlan f = plan(a);
    if (!f.outs && (!a.gx || a.n == 0)) return hipSuccess;
    if (a.n) {
        Layer layer;
        layer.add(f.x, a.x, a.n, a.dim, a.ld_x);
        layer.add(f.gate, a.gate, a.hidden, a.dim, a.ld_gate);
        layer.add(f.up, a.up, a.hidden, a.dim, a.ld_up);
        TRY_HIP(layer.run(a.type, s));
        if (!a.x) {
            const UnpackArgs u{a.codes, a.scales, a.n, a.dim, const_cast<uint16_t *>(f.x.p),
                               a.type == kF16 ? kF16 : kBF16, f.x.ld, (int)f.x.ld};
            TRY_HIP(launch_unpack(u, s));
        }
        if (a.type == kF16) {
            const BoundArgs b{(const f16_t *)a.gh, a.ld_gh, (const f16_t *)f.x.p, (const f16_t *)f.gate.p,
                              (const f16_t *)f.up.p, f.x.ld, f.gate.ld, a.n, pad8(a.dim), a.hidden, f.bounds};
            k_bounds<<<dim3(f.bound_parts, 2), 256, 0, s>>>(b);
            TRY_HIP(hipGetLastError());
        }
        ProductArgs p = projections(f.gate, f.up, f.x, a.type, !a.x, a.n, a.dim, a.hidden, a.act);
        p.bounds = f.bounds;
        p.bound_parts = f.bound_parts;
        p.factor = f.factor;
        p.gh = a.gh;
        p.ld_gh = a.ld_gh;
        p.dg = f.dg;
        p.du = f.du;
        p.d_plane = f.d_plane;
        p.ld_d = f.n_pad;
        p.d_planes = f.d_planes;
        p.n_pad = f.n_pad;
        TRY_HIP((product<false, false, kGateGrad>(p, a.type, f.h_tile, s)));
    }
    Joiner joiner;
    if (a.gx && a.n) {
        ProductArgs x{};
        x.p[0] = f.gate.p;
        x.p[1] = f.up.p;
        x.q[0] = f.dg;
        x.q[1] = f.du;
        x.ld_p = f.gate.ld;
        x.ld_q = f.n_pad;
        x.p_plane = f.gate.plane;
        x.q_plane = f.d_plane;
        x.k = a.hidden;  // dg and du have zeros behind it, to n_pad; the weights' rows end with it
        x.products = a.type == kF32 ? 6 : f.d_planes;
        x.p_planes = a.type == kF32 ? kPlanes6P : 0;
        x.q_planes = a.type == kF32 ? kPlanes6Q : f.d_planes == 2 ? kPlanes2 : 0;
        x.sources = 2;
        x.outs = 1;
        x.parts = f.x_parts;
        x.part = f.x_part;
        x.factor = f.factor;
        x.m = (int)a.n;
        x.n = a.dim;
        x.n_room = pad8(a.dim);
        x.out[0] = a.gx;
        x.ld_out[0] = a.ld_gx;
        TRY_HIP((product<true, false, kStore>(x, a.type, f.x_tile, s)));
        joiner.add(x);
    }
    if (f.outs && a.n == 0) {
        for (int i = 0; i < 2; ++i) {
            void *out = i ? a.gup : a.ggate;
            const int64_t ld = i ? a.ld_gup : a.ld_ggate;
            if (out) ERSJ_ELEM_SWITCH(a.type, O, k_zero<O><<<blocks_for(a.hidden * 256), 256, 0, s>>>((O *)out, ld, a.hidden, a.dim));
        }
        return hipGetLastError();
    }
    if (f.outs) {
        ProductArgs w{};
        w.p[0] = f.x.p;
        w.q[0] = a.ggate ? f.dg : f.du;
        w.q[1] = f.du;
        w.ld_p = f.x.ld;
        w.ld_q = f.n_pad;
        w.p_plane = f.x.plane;
        w.q_plane = f.d_plane;
        w.k = (int)a.n;
        w.products = a.type != kF32 ? f.d_planes : a.x ? 6 : 3;
        w.p_planes = a.type != kF32 || !a.x ? 0 : kPlanes6P;
        w.q_planes = a.type != kF32 ? (f.d_planes == 2 ? kPlanes2 : 0) : a.x ? kPlanes6Q : kPlanes3;
        w.sources = 1;
        w.outs = f.outs;
        w.parts = f.w_parts;
        w.part = f.w_part;
        w.factor = f.factor;
        w.m = a.hidden;
        w.n = a.dim;
        w.n_room = pad8(a.dim);
        w.m_room = f.n_pad;
        w.out[0] = a.ggate ? a.ggate : a.gup;
        w.out[1] = a.gup;
        w.ld_out[0] = a.ggate ? a.ld_ggate : a.ld_gup;
        w.ld_out[1] = a.ld_gup;
        TRY_HIP((product<true, true, kStore>(w, a.type, f.w_tile, s)));
        joiner.add(w);
    }
    return joiner.run(a.type, s);
}

}  // namespace ersj
