// The gated feed-forward block and its gradient.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u            (one kernel: both projections and the product)
//   du = dh act(g), dg = dh u act'(g)               (one kernel: the projections again)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x  (a product each, the first over both pairs)
//
// All of it is one tiled matrix product with different ends.  A workgroup owns
// BM x BN results; the two operands' slabs of 64 along k are copied to LDS by
// loads that write it directly, one slab ahead, and feed 32x32x16 matrix
// instructions.  An operand whose rows run along k is read from LDS 16 bytes a
// lane; one whose rows run across k (the weights for dx, all operands of dW)
// is staged as it lies in memory and transposed by the LDS read itself, so no
// transposed copy of anything is made.  For the projections the rows of the
// weights' slab alternate 32 of Wg and 32 of Wu, so a lane holds g and u of the
// same place.  The matrix instruction's first operand is the one along the
// results' rows in memory: a lane then holds four neighbours of a row.
//
// 32-bit tensors are split into three bf16 parts, x = x1 + x2 + x3, each the
// rounded rest of those before, and the six products whose order is above 2^-27
// of the whole are summed, smallest first: the same kernel with six times the
// slabs.  What is dropped is at most 3 * 2^-27 of each product.
#include "feedforward_internal.h"

namespace ersj {

namespace {

typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef f16_t f16x8 __attribute__((ext_vector_type(8)));
typedef bf16_t bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kSlab = 64;

// Which planes are multiplied in turn, four bits each, smallest products first:
// one plane, three of both operands, three of one of them.
constexpr uint32_t kPlanes6P = 0x010201, kPlanes6Q = 0x001021, kPlanes3 = 0x012;

enum { kStore, kGate, kGateGrad };

struct ProductArgs {
    // P: along the results' rows (n), Q: across them (m); planes of 16-bit values
    const uint16_t *p[2], *q[2];
    int64_t p_plane, q_plane, ld_p, ld_q;
    int k;                // of one product, a multiple of 8 where an operand lies along it
    int products;         // of planes
    uint32_t p_planes, q_planes;
    int sources;          // pairs (p[i], q[i]) summed
    int m, n;
    int n_room;           // columns that may be read of P across k (a multiple of 8)
    int m_room;           // the same of Q
    int mt, nt, parts, outs;
    void *out[2];
    int64_t ld_out[2];
    float *part;          // [parts][outs][m][n] where parts > 1
    // kGateGrad
    const void *gh;
    int64_t ld_gh;
    uint16_t *dg, *du;
    int64_t d_plane, ld_d;
    int n_pad;            // columns of dg and du that are written, zeros behind n
    int act;
};

// 16 bytes from `base` + `off` of each lane to LDS, lane by lane from `lds`.
__device__ __forceinline__ void dma16(uint32_t lds, uint32_t off, const void *base)
{
    // the wait state that a write of m0 needs before it is used
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "memory");
}

// What is loaded in the place of values behind the end of k.
__device__ const uint32_t kZeros[4] = {0, 0, 0, 0};

__device__ __forceinline__ void dma16_from(uint32_t lds, const void *from)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(from) : "memory");
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
__device__ __forceinline__ f32x16 mma(s16x8 a, s16x8 b, f32x16 c)
{
    if constexpr (sizeof(T) == 2 && __is_same(T, f16_t))
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
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
// across k.  Along k (ACROSS false) a row of LDS holds 64 values of k, its
// 16-byte pieces exchanged by bits 1 to 3 of the row; across k it holds the
// tile's ROWS values at one k, its pieces exchanged in groups of four by the
// low bits of k.  Either way a wave's reads fall on all banks.
template <int ROWS, int WAVES, bool ACROSS>
struct Side {
    static constexpr int kBytes = ROWS * kSlab * 2;
    static constexpr int kLoads = kBytes / (WAVES * 64 * 16);
    static constexpr int kPieces = ACROSS ? ROWS / 8 : kSlab / 8;  // of a row of LDS
    static constexpr int kLoadRows = 64 / kPieces;                 // rows of LDS that a wave's load fills
    uint32_t off[kLoads];
    int piece;  // along k: the lane's piece

    // `room`: rows (along k) or columns (across k) from the tile's first that may be read
    __device__ __forceinline__ void init(int wave, int64_t ld, int room)
    {
        const int lane = threadIdx.x & 63, r = lane / kPieces;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int row = (j * WAVES + wave) * kLoadRows + r;
            if constexpr (ACROSS) {
                int c = (lane % kPieces) ^ ((row & 3) << 2);
                c = c * 8 < room ? c : 0;
                off[j] = (uint32_t)(row * (int)ld + c * 8) * 2;
            } else {
                piece = (lane % kPieces) ^ ((row >> 1) & 7);
                off[j] = (uint32_t)((row < room ? row : room - 1) * (int)ld + piece * 8) * 2;
            }
        }
    }

    // Load j of a slab at `base`; `left`: values of k from the slab's first on (more than 0).
    __device__ __forceinline__ void load(int j, int wave, uint32_t lds, int left, const uint16_t *base) const
    {
        const uint32_t to = lds + (j * WAVES + wave) * 1024;
        if (left >= kSlab) {
            dma16(to, off[j], base);
            return;
        }
        const int k = ACROSS ? (j * WAVES + wave) * kLoadRows + (int)(threadIdx.x & 63) / kPieces : piece * 8;
        dma16_from(to, k < left ? (const char *)base + off[j] : (const char *)kZeros);
    }

    // Values of 8 consecutive k for 32 consecutive rows from `row` (a multiple
    // of 32), for the matrix instruction of the slab's values 16 kk to 16 kk + 15.
    static __device__ __forceinline__ s16x8 fragment(const char *lds, int row, int kk)
    {
        const int lane = threadIdx.x & 63;
        if constexpr (ACROSS) {
            const int k = kk * 16 + (lane >> 5) * 8 + ((lane & 15) >> 2);
            const int col = row + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
            const int at = k * (ROWS * 2) + (((col >> 3) ^ ((k & 3) << 2)) << 4) + (col & 7) * 2;
            typedef __attribute__((address_space(3))) s16x4 *ptr;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds_char *)(lds + at));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds_char *)(lds + at + 4 * ROWS * 2));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const int r = row + (lane & 31);
            const int c = (kk * 2 + (lane >> 5)) ^ ((r >> 1) & 7);
            return *(const s16x8 *)(lds + r * 128 + c * 16);
        }
    }
};

// act(g) and its derivative.
template <bool FAST>
__device__ __forceinline__ float exp_of(float v)
{
    return FAST ? __expf(v) : expf(v);
}

template <bool FAST>
__device__ __forceinline__ float act_of(int act, float g)
{
    if (act == 0) return g / (1.f + exp_of<FAST>(-g));
    if (act == 1) return 0.5f * g * (1.f + erff(g * 0.70710678118654752f));
    const float k = 0.79788456080286536f;
    return g / (1.f + exp_of<FAST>(-2.f * k * (g + 0.044715f * g * g * g)));
}

template <bool FAST>
__device__ __forceinline__ float slope_of(int act, float g, float &value)
{
    if (act == 0) {
        const float s = 1.f / (1.f + exp_of<FAST>(-g));
        value = g * s;
        return s * (1.f + g * (1.f - s));
    }
    if (act == 1) {
        const float c = 0.5f * (1.f + erff(g * 0.70710678118654752f));
        value = g * c;
        return c + g * 0.39894228040143268f * exp_of<FAST>(-0.5f * g * g);
    }
    const float k = 0.79788456080286536f;
    const float s = 1.f / (1.f + exp_of<FAST>(-2.f * k * (g + 0.044715f * g * g * g)));
    value = g * s;
    return s + g * s * (1.f - s) * 2.f * k * (1.f + 3 * 0.044715f * g * g);
}

// T: the 16-bit type multiplied; O: the tensors' type.
template <typename T, typename O, int BM, int BN, int WM, int WN, bool PA, bool QA, int END>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, (BM / WM) * (BN / WN) * 64 == 256 && BM == 256 ? 1 : 2) void k_product(ProductArgs a)
{
    constexpr int WAVES = (BM / WM) * (BN / WN), MB = WM / 32, NB = WN / 32;
    constexpr bool kPair = END != kStore;  // P's rows alternate between the two weights
    constexpr int CN = kPair ? BN / 2 : BN;
    constexpr bool FAST = sizeof(O) == 2;
    typedef Side<BN, WAVES, PA> P;
    typedef Side<BM, WAVES, QA> Q;
    constexpr int STAGE = P::kBytes + Q::kBytes;
    __shared__ __align__(1024) char lds[2 * STAGE];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char *)lds;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;

    // Workgroups go to the eight dies in turn: each die gets a stretch of the
    // tiles, which lie in columns of eight rows of tiles, for its own cache.
    const int tiles = a.mt * a.nt;
    const int total = tiles * a.parts * a.outs;
    int id = blockIdx.x;
    {
        const int q = total >> 3, r = total & 7, die = id & 7;
        id = die * q + (die < r ? die : r) + (id >> 3);
    }
    const int which = id / (tiles * a.parts);
    id -= which * tiles * a.parts;
    const int part = id / tiles;
    id -= part * tiles;
    const int group = id / (8 * a.nt), rows = a.mt - group * 8 < 8 ? a.mt - group * 8 : 8;
    id -= group * 8 * a.nt;
    const int tm = group * 8 + id % rows, tn = id / rows;
    const int64_t m0 = (int64_t)tm * BM;
    const int n0 = tn * CN;

    P p;
    Q q;
    p.init(wave, a.ld_p, PA ? a.n_room - n0 : a.n - n0);
    if constexpr (kPair) {
        // row r of the slab is row n0 + (r / 64) * 32 + r % 32 of Wg (r / 32 even) or Wu
        const int r = lane / P::kPieces;
#pragma unroll
        for (int j = 0; j < P::kLoads; ++j) {
            const int row = (j * WAVES + wave) * P::kLoadRows + r;
            const int of = (row >> 6) * 32 + (row & 31);
            p.off[j] = (uint32_t)((of < a.n - n0 ? of : a.n - n0 - 1) * (int)a.ld_p + p.piece * 8) * 2;
        }
    }
    q.init(wave, a.ld_q, QA ? a.m_room - (int)m0 : (a.m - m0 < BM ? (int)(a.m - m0) : BM));

    const int slabs = (a.k + kSlab - 1) / kSlab, all = slabs * a.products * a.sources;
    const int first = (int)((int64_t)all * part / a.parts), last = (int)((int64_t)all * (part + 1) / a.parts);

    // The slab to load next: its operands and how much of k is left.
    int seg = slabs ? first / slabs : 0, k0 = (first - seg * slabs) * kSlab, left = 0;
    const uint16_t *pb0 = nullptr, *pb1 = nullptr, *qb = nullptr;
    auto next_slab = [&]() {
        const int src = seg / a.products, prod = seg - src * a.products;
        const int64_t po = ((a.p_planes >> (4 * prod)) & 15) * a.p_plane + (PA ? (int64_t)k0 * a.ld_p + n0 : (int64_t)n0 * a.ld_p + k0);
        pb0 = a.p[kPair ? 0 : src] + po;
        pb1 = a.p[1] + po;
        qb = a.q[a.outs == 2 ? which : src] + ((a.q_planes >> (4 * prod)) & 15) * a.q_plane +
             (QA ? (int64_t)k0 * a.ld_q + m0 : m0 * a.ld_q + k0);
        left = a.k - k0;
        k0 += kSlab;
        if (k0 >= a.k) {
            k0 = 0;
            ++seg;
        }
    };
    constexpr int kLoads = P::kLoads + Q::kLoads;
    auto load = [&](int l, uint32_t at) {  // load l of the slab
        if (l < P::kLoads)
            p.load(l, wave, at, left, kPair && (((l * WAVES + wave) * P::kLoadRows) & 32) ? pb1 : pb0);
        else
            q.load(l - P::kLoads, wave, at + P::kBytes, left, qb);
    };

    f32x16 acc[NB][MB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = (f32x16)0.f;

    const int wn = (wave % (BN / WN)) * WN, wm = (wave / (BN / WN)) * WM;
    // Two slabs are in LDS or on their way.  A slab's four steps each multiply
    // what the step before read from LDS and read what the next one multiplies;
    // the last step begins with the slab's only barrier, behind which the next
    // slab is whole and this one's place is free for the slab after it.
    s16x8 fp[2][NB], fq[2][MB];
    auto read = [&](int set, int r, const char *at, int kk) {  // fragment r of a step
        if (r < NB) fp[set][r] = P::fragment(at, wn + r * 32, kk);
        else fq[set][r - NB] = Q::fragment(at + P::kBytes, wm + (r - NB) * 32, kk);
    };
    constexpr int kCells = NB * MB, kReads = NB + MB;
    const int count = last - first;
    for (int b = 0; b < 2; ++b)
        if (b < count) {
            next_slab();
#pragma unroll
            for (int l = 0; l < kLoads; ++l) load(l, lds0 + b * STAGE);
        }
    if (count) {
        if (count > 1) wait_loads<kLoads>();
        else wait_loads<0>();
        barrier();
#pragma unroll
        for (int r = 0; r < kReads; ++r) read(0, r, lds, 0);
    }
    for (int t = 0; t < count; ++t) {
        const char *at = lds + (t & 1) * STAGE, *other = lds + (1 - (t & 1)) * STAGE;
        const uint32_t free = lds0 + (t & 1) * STAGE;
        const bool more = t + 2 < count;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            if (kk == 3) {
                // this wave's loads of the next slab, and its reads of this one
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                barrier();
                if (more) next_slab();
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < kCells; ++c) {
                const int i = c / MB, j = c % MB;
                acc[i][j] = mma<T>(fp[kk & 1][i], fq[kk & 1][j], acc[i][j]);
                if (kk == 3 && more) {
#pragma unroll
                    for (int l = c * kLoads / kCells; l < (c + 1) * kLoads / kCells; ++l) load(l, free);
                }
#pragma unroll
                for (int r = c * kReads / kCells; r < (c + 1) * kReads / kCells; ++r)
                    read((kk + 1) & 1, r, kk == 3 ? other : at, (kk + 1) & 3);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }

    // a lane's place: row m of the results and, in register 4 g + e of block i, column 8 g + e
    const int ln = (lane >> 5) * 4;
#pragma unroll
    for (int j = 0; j < MB; ++j) {
        const int64_t m = m0 + wm + j * 32 + (lane & 31);
        if constexpr (END == kStore) {
            if (m >= a.m) continue;
            float *part_out = a.parts > 1 ? a.part + (((int64_t)part * a.outs + which) * a.m + m) * a.n : nullptr;
            O *out = (O *)a.out[which] + m * a.ld_out[which];
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int n = n0 + wn + i * 32 + g * 8 + ln;
                    f32x4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * g + e];
                    if (a.parts > 1) {
                        if (n + 3 < a.n) Slot<float, 4>::store(part_out + n, v);
                        else
                            for (int e = 0; e < 4; ++e)
                                if (n + e < a.n) part_out[n + e] = v[e];
                    } else {
                        if (n + 3 < a.n) Slot<O, 4>::store(out + n, __builtin_convertvector(v, typename Slot<O, 4>::vec));
                        else
                            for (int e = 0; e < 4; ++e)
                                if (n + e < a.n) out[n + e] = (O)v[e];
                    }
                }
        } else {
#pragma unroll
            for (int i = 0; i < NB; i += 2)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int n = n0 + (wn + i * 32) / 2 + g * 8 + ln;
                    if constexpr (END == kGate) {
                        if (m >= a.m) continue;
                        f32x4 v;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = act_of<FAST>(a.act, acc[i][j][4 * g + e]) * acc[i + 1][j][4 * g + e];
                        O *out = (O *)a.out[0] + m * a.ld_out[0];
                        if (n + 3 < a.n) Slot<O, 4>::store(out + n, __builtin_convertvector(v, typename Slot<O, 4>::vec));
                        else
                            for (int e = 0; e < 4; ++e)
                                if (n + e < a.n) out[n + e] = (O)v[e];
                    } else {
                        if (m >= a.m || n >= a.n_pad) continue;
                        const O *gh = (const O *)a.gh + m * a.ld_gh;
                        f32x4 d = (f32x4)0.f;
                        if (n + 3 < a.n) d = __builtin_convertvector(Slot<O, 4>::load(gh + n), f32x4);
                        else
                            for (int e = 0; e < 4; ++e)
                                if (n + e < a.n) d[e] = (float)gh[n + e];
                        f32x4 dg, du;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float value;
                            const float s = slope_of<FAST>(a.act, acc[i][j][4 * g + e], value);
                            const bool in = n + e < a.n;
                            dg[e] = in ? d[e] * acc[i + 1][j][4 * g + e] * s : 0.f;
                            du[e] = in ? d[e] * value : 0.f;
                        }
                        const int64_t at = m * a.ld_d + n;
                        if constexpr (sizeof(O) == 2) {
                            *(typename Slot<T, 4>::vec *)(a.dg + at) = __builtin_convertvector(dg, typename Slot<T, 4>::vec);
                            *(typename Slot<T, 4>::vec *)(a.du + at) = __builtin_convertvector(du, typename Slot<T, 4>::vec);
                        } else {
#pragma unroll
                            for (int k = 0; k < 3; ++k) {
                                s16x4 x, y;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float v = dg[e], w = du[e];
                                    x[e] = (short)part_of(v);
                                    y[e] = (short)part_of(w);
                                    dg[e] = v;
                                    du[e] = w;
                                }
                                *(s16x4 *)(a.dg + k * a.d_plane + at) = x;
                                *(s16x4 *)(a.du + k * a.d_plane + at) = y;
                            }
                        }
                    }
                }
        }
    }
}

// Sums of the parts of a product, in order.
template <typename O>
__global__ __launch_bounds__(256) void k_product_join(const float *part, int parts, int outs, int m, int n, O *out0,
                                                      O *out1, int64_t ld0, int64_t ld1)
{
    const int64_t size = (int64_t)m * n, all = size * outs;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < all; i += (int64_t)gridDim.x * 1024) {
        const int len = all - i < 4 ? (int)(all - i) : 4;
        f32x4 v = (f32x4)0.f;
        for (int p = 0; p < parts; ++p) {
            const float *at = part + p * all + i;
            if (len == 4) v += Slot<float, 4>::load(at);
            else
                for (int e = 0; e < len; ++e) v[e] += at[e];
        }
        for (int e = 0; e < len; ++e) {
            const int64_t w = i + e >= size, r = i + e - w * size, row = r / n;
            (w ? out1 : out0)[row * (w ? ld1 : ld0) + r - row * n] = (O)v[e];
        }
    }
}

// A matrix [n][dim] as the products read it: 16-bit values with rows of `pad`
// (a multiple of 8) and zeros behind the row's end; three planes for 32 bits.
template <typename S>
__global__ __launch_bounds__(256) void k_lay(const S *src, int64_t ld, int64_t n, int dim, int pad, uint16_t *out)
{
    const int per = pad / 8;
    const int64_t all = n * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per;
        const int c = (int)(i - r * per) * 8;
        typename Slot<S, 8>::vec v;
        if (c + 8 <= dim) v = Slot<S, 8>::load(src + r * ld + c);
        else
            for (int e = 0; e < 8; ++e) v[e] = c + e < dim ? src[r * ld + c + e] : (S)0.f;
        uint16_t *to = out + r * pad + c;
        if constexpr (sizeof(S) == 2) {
            *(typename Slot<S, 8>::vec *)to = v;
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                s16x8 x;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float f = v[e];
                    x[e] = (short)part_of(f);
                    v[e] = f;
                }
                *(s16x8 *)(to + k * n * pad) = x;
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
        char *at = base + used;
        used += (bytes + 255) & ~(uint64_t)255;
        return at;
    }
};

// In place where the loads can take it: 16-bit values, rows that begin at 16
// bytes and hold whole pieces of 16 bytes, spaced so that a tile's offsets fit 32 bits.
Operand operand(Room &room, const void *p, int type, int64_t n, int dim, int64_t ld)
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
    o.p = (const uint16_t *)room.take((uint64_t)o.plane * 2 * (type == kF32 ? 3 : 1));
    return o;
}

hipError_t lay(const Operand &o, const void *src, int type, int64_t n, int dim, int64_t ld, hipStream_t s)
{
    if (!o.laid || n == 0) return hipSuccess;
    const unsigned blocks = blocks_for(n * (o.ld / 8));
    uint16_t *out = const_cast<uint16_t *>(o.p);
    if (type == kF32) k_lay<float><<<blocks, 256, 0, s>>>((const float *)src, ld, n, dim, (int)o.ld, out);
    else k_lay<f16_t><<<blocks, 256, 0, s>>>((const f16_t *)src, ld, n, dim, (int)o.ld, out);
    return hipGetLastError();
}

template <typename T, typename O, bool PA, bool QA, int END>
hipError_t run_product(ProductArgs &a, bool large, hipStream_t s)
{
    const int bm = large ? 256 : 128, bn = (large ? 256 : 128) / (END == kStore ? 1 : 2);
    a.mt = (a.m + bm - 1) / bm;
    a.nt = (a.n + bn - 1) / bn;
    const int64_t count = (int64_t)a.mt * a.nt * a.parts * a.outs;
    if (count * 256 >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
    const unsigned blocks = (unsigned)count;
    if (large) k_product<T, O, 256, 256, 128, 128, PA, QA, END><<<blocks, 256, 0, s>>>(a);
    else k_product<T, O, 128, 128, 64, 64, PA, QA, END><<<blocks, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <bool PA, bool QA, int END>
hipError_t product(ProductArgs &a, int type, bool large, hipStream_t s)
{
    if (type == kF32) return run_product<bf16_t, float, PA, QA, END>(a, large, s);
    if (type == kF16) return run_product<f16_t, f16_t, PA, QA, END>(a, large, s);
    return run_product<bf16_t, bf16_t, PA, QA, END>(a, large, s);
}

// Whether the tiles of 256 x 256 give every compute unit one.
bool large_tiles(int64_t m, int64_t n) { return ((m + 255) / 256) * ((n + 255) / 256) >= 256; }

// Into how many parts the sum over k is cut so that the device is filled.
int parts_of(int64_t m, int64_t n, int64_t slabs)
{
    const int64_t tiles = ((m + 127) / 128) * ((n + 127) / 128);
    int64_t parts = 512 / tiles;
    if (parts > slabs / 4) parts = slabs / 4;
    return parts < 1 ? 1 : (int)parts;
}

// The weights as operands, both laid out or both in place with one spacing.
void weights(Room &room, const void *gate, int64_t ld_gate, const void *up, int64_t ld_up, int type, int hidden, int dim,
             Operand &g, Operand &u)
{
    g = operand(room, gate, type, hidden, dim, ld_gate);
    u = operand(room, up, type, hidden, dim, ld_up);
    if (g.laid && u.laid) return;
    if (g.laid || u.laid || g.ld != u.ld) {
        if (!g.laid) g = operand(room, nullptr, type, hidden, dim, 0);
        if (!u.laid) u = operand(room, nullptr, type, hidden, dim, 0);
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
    f.x = operand(room, a.x, a.type, a.n, a.dim, a.ld_x);
    weights(room, a.gate, a.ld_gate, a.up, a.ld_up, a.type, a.hidden, a.dim, f.gate, f.up);
    f.bytes = room.used;
    return f;
}

struct GradPlan {
    Operand x, gate, up;
    uint16_t *dg, *du;
    int64_t d_plane;
    int n_pad, outs;
    float *part;
    int x_parts, w_parts;
    bool x_large, w_large;
    uint64_t bytes;
};

GradPlan plan(const GatedGradArgs &a)
{
    Room room{(char *)a.work};
    GradPlan f;
    f.x = operand(room, a.x, a.type, a.n, a.dim, a.ld_x);
    weights(room, a.gate, a.ld_gate, a.up, a.ld_up, a.type, a.hidden, a.dim, f.gate, f.up);
    const int planes = a.type == kF32 ? 3 : 1;
    f.n_pad = pad8(a.hidden);
    f.d_plane = a.n * f.n_pad;
    f.dg = (uint16_t *)room.take((uint64_t)f.d_plane * 2 * planes);
    f.du = (uint16_t *)room.take((uint64_t)f.d_plane * 2 * planes);
    f.outs = (a.ggate != nullptr) + (a.gup != nullptr);
    const int64_t m = (int64_t)f.outs * a.hidden, slabs_x = (f.n_pad + 63) / 64, slabs_w = (a.n + 63) / 64;
    f.x_large = large_tiles(a.n, a.dim);
    f.w_large = large_tiles(m, a.dim);
    f.x_parts = a.gx && a.n && !f.x_large ? parts_of(a.n, a.dim, slabs_x * 2 * (planes == 3 ? 6 : 1)) : 1;
    f.w_parts = f.outs && !f.w_large ? parts_of(m, a.dim, slabs_w * (planes == 1 ? 1 : a.x ? 6 : 3)) : 1;
    uint64_t part = 0;
    if (f.x_parts > 1) part = (uint64_t)f.x_parts * a.n * a.dim * 4;
    if (f.w_parts > 1) {
        const uint64_t b = (uint64_t)f.w_parts * m * a.dim * 4;
        if (b > part) part = b;
    }
    f.part = (float *)room.take(part);
    f.bytes = room.used;
    return f;
}

hipError_t join(const ProductArgs &p, int type, hipStream_t s)
{
    if (p.parts == 1) return hipSuccess;
    const int64_t all = (int64_t)p.m * p.n * p.outs;
    const unsigned blocks = blocks_for((all + 3) / 4);
    ERSJ_ELEM_SWITCH(type, O,
        k_product_join<O><<<blocks, 256, 0, s>>>(p.part, p.parts, p.outs, p.m, p.n, (O *)p.out[0], (O *)p.out[1],
                                                 p.ld_out[0], p.ld_out[1]));
    return hipGetLastError();
}

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
    TRY_HIP(lay(f.x, a.x, a.type, a.n, a.dim, a.ld_x, s));
    TRY_HIP(lay(f.gate, a.gate, a.type, a.hidden, a.dim, a.ld_gate, s));
    TRY_HIP(lay(f.up, a.up, a.type, a.hidden, a.dim, a.ld_up, s));
    ProductArgs p = projections(f.gate, f.up, f.x, a.type, false, a.n, a.dim, a.hidden, a.act);
    p.out[0] = a.h;
    p.ld_out[0] = a.ld_h;
    return product<false, false, kGate>(p, a.type, large_tiles(a.n, 2 * (int64_t)a.hidden), s);
}

uint64_t gated_grad_work(const GatedGradArgs &a) { return plan(a).bytes; }

hipError_t launch_gated_grad(const GatedGradArgs &a, hipStream_t s)
{
    const GradPlan f = plan(a);
    if (!f.outs && (!a.gx || a.n == 0)) return hipSuccess;
    if (a.n) {
        if (a.x) TRY_HIP(lay(f.x, a.x, a.type, a.n, a.dim, a.ld_x, s));
        else {
            // what a code stands for is a bf16 number: 32-bit rows have one plane
            const UnpackArgs u{a.codes, a.scales, a.n, a.dim, const_cast<uint16_t *>(f.x.p),
                               a.type == kF16 ? kF16 : kBF16, f.x.ld, (int)f.x.ld};
            TRY_HIP(launch_unpack(u, s));
        }
        TRY_HIP(lay(f.gate, a.gate, a.type, a.hidden, a.dim, a.ld_gate, s));
        TRY_HIP(lay(f.up, a.up, a.type, a.hidden, a.dim, a.ld_up, s));
        ProductArgs p = projections(f.gate, f.up, f.x, a.type, !a.x, a.n, a.dim, a.hidden, a.act);
        p.gh = a.gh;
        p.ld_gh = a.ld_gh;
        p.dg = f.dg;
        p.du = f.du;
        p.d_plane = f.d_plane;
        p.ld_d = f.n_pad;
        p.n_pad = f.n_pad;
        TRY_HIP((product<false, false, kGateGrad>(p, a.type, large_tiles(a.n, 2 * (int64_t)a.hidden), s)));
    }
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
        x.k = a.hidden;
        x.products = a.type == kF32 ? 6 : 1;
        x.p_planes = a.type == kF32 ? kPlanes6P : 0;
        x.q_planes = a.type == kF32 ? kPlanes6Q : 0;
        x.sources = 2;
        x.outs = 1;
        x.parts = f.x_parts;
        x.part = f.part;
        x.m = (int)a.n;
        x.n = a.dim;
        x.n_room = pad8(a.dim);
        x.out[0] = a.gx;
        x.ld_out[0] = a.ld_gx;
        TRY_HIP((product<true, false, kStore>(x, a.type, f.x_large, s)));
        TRY_HIP(join(x, a.type, s));
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
        w.products = a.type != kF32 ? 1 : a.x ? 6 : 3;
        w.p_planes = a.type != kF32 || !a.x ? 0 : kPlanes6P;
        w.q_planes = a.type != kF32 ? 0 : a.x ? kPlanes6Q : kPlanes3;
        w.sources = 1;
        w.outs = f.outs;
        w.parts = f.w_parts;
        w.part = f.part;
        w.m = a.hidden;
        w.n = a.dim;
        w.n_room = pad8(a.dim);
        w.m_room = f.n_pad;
        w.out[0] = a.ggate ? a.ggate : a.gup;
        w.out[1] = a.gup;
        w.ld_out[0] = a.ggate ? a.ld_ggate : a.ld_gup;
        w.ld_out[1] = a.ld_gup;
        TRY_HIP((product<true, true, kStore>(w, a.type, f.w_large, s)));
        TRY_HIP(join(w, a.type, s));
    }
    return hipSuccess;
}

}  // namespace ersj
