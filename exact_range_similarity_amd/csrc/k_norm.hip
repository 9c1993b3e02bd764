// Layer norm of rows and its gradient.
//
// Both are bound by memory: a row is read once, stays in registers through
// its reductions, and its result is written once.  A row belongs to a team of
// L lanes (a part of a wave up to 64, a whole workgroup above), each holding
// NV vectors of 16 bytes; a team works through rows that lie a whole grid
// apart and loads the next one while it reduces the current one.  The variance
// is the mean square of the differences from the mean, which costs a second
// reduction over registers and nothing in memory, and loses nothing where the
// mean is large.  1M x 384 bf16: 287 us for 1.54 GB, 5.4 TB/s; gradient over
// 32,768 x 4096 bf16: 158 us for 0.81 GB, 5.1 TB/s, and over 20,000 x 384 f16 12.6
// + 3.7 us for 46 MB, where starting, the last turns and the sums' join count.
#include "feedforward_internal.h"

namespace ersj {

namespace {

constexpr int kThreads = 256;

// Threads of a workgroup whose teams have `lanes` lanes: a team above a wave
// is a workgroup of its own.
constexpr int block_of(int lanes) { return lanes > 64 ? lanes : kThreads; }

template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// Sum over the L lanes of a team (L a power of two up to 64), in every lane.
template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
    if constexpr (L >= 2) v += dpp<0xb1>(v);   // lane ^ 1
    if constexpr (L >= 4) v += dpp<0x4e>(v);   // lane ^ 2
    if constexpr (L >= 8) v += dpp<0x141>(v);  // the other half of 8, mirrored
    if constexpr (L >= 16) v += dpp<0x140>(v); // the other half of 16, mirrored
    if constexpr (L >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if constexpr (L >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    return v;
}

// Sum over the teams of a wave, lane by lane (over the lanes that differ by a
// multiple of L), in every lane.
template <int L>
__device__ __forceinline__ float teams_sum(float v)
{
    if constexpr (L <= 8) v += dpp<0x128>(v);  // rotations within 16 lanes, by 8, 4, 2, 1
    if constexpr (L <= 4) v += dpp<0x124>(v);
    if constexpr (L <= 2) v += dpp<0x122>(v);
    if constexpr (L <= 1) v += dpp<0x121>(v);
    if constexpr (L <= 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if constexpr (L <= 32) {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    return v;
}

// Sums of K values over a team of L lanes.  A team of a workgroup goes through
// `red`, one slot of which is free of readers when the next sum writes it
// (two slots used in turn, one barrier a sum).
template <int L, int K>
__device__ __forceinline__ void team_sum(float (&v)[K], float (*red)[L > 64 ? L / 64 : 1][K], int &slot)
{
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lanes_sum<(L > 64 ? 64 : L)>(v[k]);
    if constexpr (L > 64) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) red[slot][threadIdx.x >> 6][k] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = 0.f;
#pragma unroll
        for (int j = 0; j < L / 64; ++j) {
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += red[slot][j][k];
        }
        slot ^= 1;
    }
}

// A lane's columns: vector k covers LEN columns from col[k].  Vectors of all
// but the last turn are whole; the last vector of a row whose length is not a
// multiple of LEN begins earlier, so that it ends with the row, and its first
// `skip` columns are its neighbour's (skip = LEN: nothing of it is the
// lane's own).  Skipped columns hold right values but enter no sum.
template <int LEN, int L, int NV>
struct Columns {
    int col[NV];
    int skip;
    __device__ __forceinline__ Columns(int dim)
    {
        const int lane = threadIdx.x & (L - 1);
#pragma unroll
        for (int k = 0; k < NV; ++k) col[k] = (k * L + lane) * LEN;
        const int c = col[NV - 1];
        col[NV - 1] = c + LEN <= dim ? c : dim - LEN;
        skip = c - col[NV - 1] < LEN ? c - col[NV - 1] : LEN;
    }
};

// The largest magnitude, as bits, over the lanes of a team that share a block
// of rows held in 8 bits, in each of them.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_most(uint32_t v)
{
    auto with = [&](uint32_t o) { v = o > v ? o : v; };
    if constexpr (LANES >= 2) with(__builtin_amdgcn_update_dpp(0, v, 0xb1, 0xf, 0xf, true));
    if constexpr (LANES >= 4) with(__builtin_amdgcn_update_dpp(0, v, 0x4e, 0xf, 0xf, true));
    if constexpr (LANES >= 8) with(__builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true));
    return v;
}

// Holds a lane's columns of a row in 8 bits.  A block's lanes lie side by side
// in one vector of the team, since teams of fewer lanes have no second one.
template <typename T, int LEN, int L, int NV, typename V>
__device__ __forceinline__ void hold_row(const NormArgs &a, const Columns<LEN, L, NV> &at, const V (&v)[NV], int64_t r)
{
    constexpr int kLanes = kPackBlock / LEN < L ? kPackBlock / LEN : L;
    static_assert(L >= kPackBlock / LEN || NV == 1, "a block within a vector");
    static_assert(kLanes <= 8, "lanes of a block");
    const int blocks = pack_blocks(a.dim), lane = threadIdx.x & (L - 1);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < LEN; ++j) {
            const uint32_t b = k < NV - 1 || j >= at.skip ? __float_as_uint(v[k][j]) & 0x7fffffffu : 0;
            most = b > most ? b : most;
        }
        most = lanes_most<kLanes>(most);
        const int scale = pack_scale(most);
        int8_t code[LEN];
        pack_codes<T, LEN>(v[k], scale, code);
        const int c = (k * L + lane) * LEN;
        if (r >= a.n || c >= a.dim) continue;
        int8_t *to = a.codes + r * a.dim + at.col[k];
        if (k < NV - 1 || at.skip == 0) {
            typename Slot<int8_t, LEN>::vec w;
#pragma unroll
            for (int j = 0; j < LEN; ++j) w[j] = code[j];
            Slot<int8_t, LEN>::store(to, w);
        } else {
#pragma unroll
            for (int j = 0; j < LEN; ++j)
                if (j >= at.skip) to[j] = code[j];
        }
        if (c % kPackBlock == 0) a.scales[r * blocks + c / kPackBlock] = (uint8_t)scale;
    }
}

// HOLD: the rows are held in 8 bits as well, one reading of the rows less than
// a pass of its own (1M x 384 bf16, 1.93 GB: 366 us, 5.3 TB/s, where the norm
// takes 286 and the pass 250).
template <typename T, typename P, int LEN, int L, int NV, bool HOLD>
__global__ __launch_bounds__(block_of(L)) void k_norm(NormArgs a)
{
    constexpr int kTeams = block_of(L) / L;
    constexpr bool kKeep = L <= 256;  // weight and bias stay in registers
    typedef float fvec __attribute__((ext_vector_type(LEN)));
    typedef Slot<T, LEN> X;
    typedef Slot<P, LEN> W;
    __shared__ float red[2][L > 64 ? L / 64 : 1][1];
    int slot = 0;
    const Columns<LEN, L, NV> at(a.dim);
    const P *pw = (const P *)a.weight, *pb = (const P *)a.bias;
    fvec w[NV], b[NV];
    if constexpr (kKeep) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            w[k] = pw ? __builtin_convertvector(W::load(pw + at.col[k]), fvec) : (fvec)1.f;
            b[k] = pb ? __builtin_convertvector(W::load(pb + at.col[k]), fvec) : (fvec)0.f;
        }
    }
    const float dim = (float)a.dim;  // divided by, not multiplied with its inverse: an exact sum gives an exact mean
    const int64_t step = (int64_t)gridDim.x * kTeams;
    int64_t r = (int64_t)blockIdx.x * kTeams + threadIdx.x / L;
    typename X::vec next[NV];
    {
        const T *x = (const T *)a.x + (r < a.n ? r : a.n - 1) * a.ld_x;
#pragma unroll
        for (int k = 0; k < NV; ++k) next[k] = X::load(x + at.col[k]);
    }
    // every lane of a wave, and every wave of a workgroup's team, takes the same turns
    const int64_t turns = (a.n + step - 1) / step;
    for (int64_t turn = 0; turn < turns; ++turn, r += step) {
        fvec v[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) v[k] = __builtin_convertvector(next[k], fvec);
        if (turn + 1 < turns) {
            const int64_t q = r + step < a.n ? r + step : a.n - 1;
            const T *x = (const T *)a.x + q * a.ld_x;
#pragma unroll
            for (int k = 0; k < NV; ++k) next[k] = X::load(x + at.col[k]);
        }
        if constexpr (HOLD) hold_row<T>(a, at, v, r);
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int j = 0; j < LEN; ++j) s[0] += k < NV - 1 || j >= at.skip ? v[k][j] : 0.f;
        }
        team_sum<L, 1>(s, red, slot);
        const float mean = s[0] / dim;
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            v[k] -= mean;
#pragma unroll
            for (int j = 0; j < LEN; ++j) s[0] += k < NV - 1 || j >= at.skip ? v[k][j] * v[k][j] : 0.f;
        }
        team_sum<L, 1>(s, red, slot);
        const float rstd = 1.f / sqrtf(s[0] / dim + a.eps);
        if (r < a.n) {
            if ((threadIdx.x & (L - 1)) == 0) {
                if (a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
            T *y = (T *)a.y + r * a.ld_y;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (k == NV - 1 && at.skip == LEN) continue;
                v[k] *= rstd;
                if constexpr (kKeep) v[k] = v[k] * w[k] + b[k];
                else {
                    if (pw) v[k] *= __builtin_convertvector(W::load(pw + at.col[k]), fvec);
                    if (pb) v[k] += __builtin_convertvector(W::load(pb + at.col[k]), fvec);
                }
                X::store(y + at.col[k], __builtin_convertvector(v[k], typename X::vec));
            }
        }
    }
}

// Rows longer than the registers of a workgroup: read again for each step, an
// element a load.  4096 x 40,000 f32: 614 us, 246 for one reading and the writing
// at the rate of a copy; 4096 x 65,536 bf16 860 and 202.
template <typename T, typename P>
__global__ __launch_bounds__(1024) void k_norm_long(NormArgs a)
{
    __shared__ float red[2][16][1];
    int slot = 0;
    const P *pw = (const P *)a.weight, *pb = (const P *)a.bias;
    const float dim = (float)a.dim;
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.ld_x;
        T *y = (T *)a.y + r * a.ld_y;
        float s[1] = {0.f};
        for (int c = threadIdx.x; c < a.dim; c += 1024) s[0] += (float)x[c];
        team_sum<1024, 1>(s, red, slot);
        const float mean = s[0] / dim;
        s[0] = 0.f;
        for (int c = threadIdx.x; c < a.dim; c += 1024) {
            const float d = (float)x[c] - mean;
            s[0] += d * d;
        }
        team_sum<1024, 1>(s, red, slot);
        const float rstd = 1.f / sqrtf(s[0] / dim + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        for (int c = threadIdx.x; c < a.dim; c += 1024) {
            float v = ((float)x[c] - mean) * rstd;
            if (pw) v *= (float)pw[c];
            if (pb) v += (float)pb[c];
            y[c] = (T)v;
        }
    }
}

// A lane's columns of a row of x, as loaded: the values themselves, or the codes
// of rows held in 8 bits and their scales.  Only the last vector, which may
// begin before its place, can lie in two blocks.
template <typename T, int LEN, int NV, bool HELD>
struct RowOfX {
    typename Slot<T, LEN>::vec v[NV];
    template <typename C>
    __device__ __forceinline__ void load(const NormGradArgs &a, const C &at, int64_t q)
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) v[k] = Slot<T, LEN>::load((const T *)a.x + q * a.ld_x + at.col[k]);
    }
    template <typename V, typename C>
    __device__ __forceinline__ V get(const C &, int k) const
    {
        return __builtin_convertvector(v[k], V);
    }
};

template <typename T, int LEN, int NV>
struct RowOfX<T, LEN, NV, true> {
    typename Slot<int8_t, LEN>::vec code[NV];
    uint8_t scale[NV], end;
    template <typename C>
    __device__ __forceinline__ void load(const NormGradArgs &a, const C &at, int64_t q)
    {
        const int8_t *codes = a.codes + q * a.dim;
        const uint8_t *scales = a.scales + q * pack_blocks(a.dim);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            code[k] = Slot<int8_t, LEN>::load(codes + at.col[k]);
            scale[k] = scales[at.col[k] / kPackBlock];
        }
        end = scales[(at.col[NV - 1] + LEN - 1) / kPackBlock];
    }
    template <typename V, typename C>
    __device__ __forceinline__ V get(const C &at, int k) const
    {
        V v = __builtin_convertvector(code[k], V);
        const float step = pack_step(scale[k]);
        if (k < NV - 1) return v * step;
        const float last = pack_step(end);
        const int own = kPackBlock - at.col[k] % kPackBlock;
#pragma unroll
        for (int j = 0; j < LEN; ++j) v[j] *= j < own ? step : last;
        return v;
    }
};

// The gradient.  dw and db are sums over rows: each team keeps its own in
// registers, a workgroup's teams are added in a fixed order at the end, and
// k_norm_grad_join adds the workgroups' sums, part [workgroup][2][dim].
// HELD: x comes from rows held in 8 bits (1M x 384 bf16, 1.94 GB: 356 us, and
// 451 from the rows themselves, 2.3 GB).
template <typename T, typename P, int LEN, int L, int NV, bool HELD>
__global__ __launch_bounds__(block_of(L)) void k_norm_grad(NormGradArgs a, float *part)
{
    constexpr int kBlock = block_of(L);
    constexpr int kTeams = kBlock / L;
    constexpr bool kKeep = L <= 256;
    typedef float fvec __attribute__((ext_vector_type(LEN)));
    typedef Slot<T, LEN> X;
    typedef Slot<P, LEN> W;
    __shared__ float red[2][L > 64 ? L / 64 : 1][2];
    __shared__ __align__(16) float sums[L > 64 ? 1 : kBlock / 64][L > 64 ? 1 : 2 * L * NV * LEN];
    int slot = 0;
    const Columns<LEN, L, NV> at(a.dim);
    const P *pw = (const P *)a.weight;
    fvec w[NV], dw[NV], db[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if constexpr (kKeep) w[k] = pw ? __builtin_convertvector(W::load(pw + at.col[k]), fvec) : (fvec)1.f;
        dw[k] = (fvec)0.f;
        db[k] = (fvec)0.f;
    }
    const float inv = 1.f / (float)a.dim;
    const int64_t step = (int64_t)gridDim.x * kTeams;
    int64_t r = (int64_t)blockIdx.x * kTeams + threadIdx.x / L;
    RowOfX<T, LEN, NV, HELD> nx;
    typename X::vec ng[NV];
    float nmean = 0.f, nrstd = 0.f;
    const int64_t turns = (a.n + step - 1) / step;
    if (turns) {
        const int64_t q = r < a.n ? r : a.n - 1;
        nx.load(a, at, q);
#pragma unroll
        for (int k = 0; k < NV; ++k) ng[k] = X::load((const T *)a.gy + q * a.ld_gy + at.col[k]);
        nmean = a.mean[q];
        nrstd = a.rstd[q];
    }
    for (int64_t turn = 0; turn < turns; ++turn, r += step) {
        fvec xh[NV], g[NV];
        const float rstd = nrstd;
        const bool mine = r < a.n;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            xh[k] = (nx.template get<fvec>(at, k) - nmean) * rstd;
            g[k] = __builtin_convertvector(ng[k], fvec);
            if (mine) {
                dw[k] += g[k] * xh[k];
                db[k] += g[k];
            }
        }
        if (turn + 1 < turns) {
            const int64_t q = r + step < a.n ? r + step : a.n - 1;
            nx.load(a, at, q);
#pragma unroll
            for (int k = 0; k < NV; ++k) ng[k] = X::load((const T *)a.gy + q * a.ld_gy + at.col[k]);
            nmean = a.mean[q];
            nrstd = a.rstd[q];
        }
        if (!a.gx) continue;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if constexpr (kKeep) g[k] *= w[k];
            else if (pw) g[k] *= __builtin_convertvector(W::load(pw + at.col[k]), fvec);
#pragma unroll
            for (int j = 0; j < LEN; ++j) {
                const bool in = k < NV - 1 || j >= at.skip;
                s[0] += in ? g[k][j] : 0.f;
                s[1] += in ? g[k][j] * xh[k][j] : 0.f;
            }
        }
        team_sum<L, 2>(s, red, slot);
        const float m1 = s[0] * inv, m2 = s[1] * inv;
        if (mine) {
            T *gx = (T *)a.gx + r * a.ld_gx;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (k == NV - 1 && at.skip == LEN) continue;
                X::store(gx + at.col[k],
                         __builtin_convertvector((g[k] - m1 - xh[k] * m2) * rstd, typename X::vec));
            }
        }
    }
    if (!a.gw && !a.gb) return;
    // the only workgroup writes the results, one of several its part
    P *gw = part ? nullptr : (P *)a.gw, *gb = part ? nullptr : (P *)a.gb;
    float *out = part + (uint64_t)blockIdx.x * 2 * a.dim;
    typedef Slot<float, LEN> S;
    // a lane's own columns of vector k to p[column] (p in LDS or not)
    auto put = [&](float *p, int k, fvec v) {
        if (k < NV - 1 || at.skip == 0) S::store(p + at.col[k], v);
        else {
#pragma unroll
            for (int j = 0; j < LEN; ++j)
                if (j >= at.skip) p[at.col[k] + j] = v[j];
        }
    };
    if constexpr (L > 64) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (part) {
                put(out, k, dw[k]);
                put(out + a.dim, k, db[k]);
                continue;
            }
#pragma unroll
            for (int j = 0; j < LEN; ++j) {
                if (k == NV - 1 && j < at.skip) continue;
                if (gw) gw[at.col[k] + j] = (P)dw[k][j];
                if (gb) gb[at.col[k] + j] = (P)db[k][j];
            }
        }
    } else {
        // the teams of a wave by lane exchanges, then the waves in order
        float *own = sums[threadIdx.x >> 6];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int j = 0; j < LEN; ++j) {
                dw[k][j] = teams_sum<L>(dw[k][j]);
                db[k][j] = teams_sum<L>(db[k][j]);
            }
            if ((threadIdx.x & 63) < L) {
                put(own, k, dw[k]);
                put(own + L * NV * LEN, k, db[k]);
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.dim; c += kBlock) {
            const int i = c < a.dim ? c : c - a.dim + L * NV * LEN;
            float s = sums[0][i];
#pragma unroll
            for (int t = 1; t < kBlock / 64; ++t) s += sums[t][i];
            if (part) out[c] = s;
            else if (c < a.dim) {
                if (gw) gw[c] = (P)s;
            } else if (gb)
                gb[c - a.dim] = (P)s;
        }
    }
}

// The gradient of such rows: twice over them for grad_x here, once for the sums
// over rows in k_norm_grad_long_part.  4096 x 40,000 f32: 1515 us, 369 for one
// reading and the writing at the rate of a copy.
template <typename T, typename P>
__global__ __launch_bounds__(1024) void k_norm_grad_long(NormGradArgs a)
{
    __shared__ float red[2][16][2];
    int slot = 0;
    const P *pw = (const P *)a.weight;
    const float inv = 1.f / (float)a.dim;
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.ld_x, *gy = (const T *)a.gy + r * a.ld_gy;
        T *gx = (T *)a.gx + r * a.ld_gx;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x; c < a.dim; c += 1024) {
            const float g = (float)gy[c] * (pw ? (float)pw[c] : 1.f);
            s[0] += g;
            s[1] += g * (((float)x[c] - mean) * rstd);
        }
        team_sum<1024, 2>(s, red, slot);
        const float m1 = s[0] * inv, m2 = s[1] * inv;
        for (int c = threadIdx.x; c < a.dim; c += 1024) {
            const float g = (float)gy[c] * (pw ? (float)pw[c] : 1.f);
            const float xh = ((float)x[c] - mean) * rstd;
            gx[c] = (T)((g - m1 - xh * m2) * rstd);
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_norm_grad_long_part(NormGradArgs a, float *part)
{
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.dim) return;
    float sw = 0.f, sb = 0.f;
    for (int64_t r = blockIdx.y; r < a.n; r += gridDim.y) {
        const float dy = (float)((const T *)a.gy)[r * a.ld_gy + c];
        sw += dy * (((float)((const T *)a.x)[r * a.ld_x + c] - a.mean[r]) * a.rstd[r]);
        sb += dy;
    }
    part[(int64_t)blockIdx.y * 2 * a.dim + c] = sw;
    part[((int64_t)blockIdx.y * 2 + 1) * a.dim + c] = sb;
}

// Sums of the parts: 16 columns of [2][dim] a workgroup, 64 threads to a
// column, their sums added in order.
template <typename P>
__global__ __launch_bounds__(1024) void k_norm_grad_join(const float *part, int parts, int dim, P *gw, P *gb)
{
    __shared__ float sums[64][17];
    const int c = blockIdx.x * 16 + (threadIdx.x & 15), g = threadIdx.x >> 4;
    float s = 0.f;
    if (c < 2 * dim) {
        for (int p = g; p < parts; p += 64 * 8) {
            float x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int q = p + 64 * u < parts ? p + 64 * u : parts - 1;
                x[u] = part[(int64_t)q * 2 * dim + c];
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (p + 64 * u < parts) s += x[u];
        }
    }
    sums[g][threadIdx.x & 15] = s;
    __syncthreads();
    if (threadIdx.x < 16 && c < 2 * dim) {
        s = sums[0][threadIdx.x];
        for (int k = 1; k < 64; ++k) s += sums[k][threadIdx.x];
        if (c < dim) {
            if (gw) gw[c] = (P)s;
        } else if (gb)
            gb[c - dim] = (P)s;
    }
}

// Lanes of a team and vectors of a lane for rows of `dim` elements.  Within a
// wave: the smallest team of at least eight lanes (128 consecutive bytes a
// load) whose lanes need no more than four vectors (1M rows of 384 bf16: 16
// lanes 295 us, 32 lanes 301, 64 lanes 331).  Teams of a workgroup: up to three
// vectors, since a fourth costs more occupancy than half-empty lanes cost
// (gradient over 32,768 x 4096 bf16: 256 lanes of two vectors 155 us, 128 of
// four 167), but four where the lanes would double for it at 256 (10,000 x
// 8192 bf16: 110 us, 512 lanes of two 121) and at the longest.  lanes = 0: the
// row is too long.
struct Shape {
    int len, lanes, nv;
};

// `most` lanes fit the registers: 1024 for the norm, 512 for its gradient,
// which holds about twice as much (1024 lanes leave 128 registers each).
Shape shape_of(int type, int dim, int most)
{
    Shape s;
    s.len = 16 / elem_size(type);
    if (dim < s.len) s.len = 1;
    const int vecs = (dim + s.len - 1) / s.len;
    s.lanes = 1;
    while (s.lanes < 8 && s.lanes < vecs) s.lanes *= 2;
    while (s.lanes < 64 && s.lanes * 4 < vecs) s.lanes *= 2;
    if (s.lanes * 4 < vecs) {
        s.lanes = vecs <= 128 * 3 ? 128 : vecs <= 256 * 4 ? 256 : 512;
        if (s.lanes < most && vecs > 512 * 3) s.lanes = 1024;
        if (s.lanes * 4 < vecs) s.lanes = 0;
    }
    s.nv = s.lanes ? (vecs + s.lanes - 1) / s.lanes : 0;
    return s;
}

// Workgroups of the norm: one turn each for up to kNormFull workgroups of 256
// threads, then up to eight turns (four of the large workgroups), which pay
// for the weights' loads; more workgroups than fit the device start as others
// end, so that no few are left for a round of their own (30,000 x 4097 f32: 203
// us, 272 with a fixed 1024 workgroups of 29 turns).
constexpr int kNormFull = 2048;

unsigned norm_blocks(int64_t n, const Shape &s)
{
    const int block = s.lanes ? block_of(s.lanes) : 1024;
    const int64_t teams = s.lanes ? block / s.lanes : 1, need = (n + teams - 1) / teams;
    int64_t turns = need / (kNormFull * 256 / block);
    const int64_t top = block > 256 ? 4 : 8;
    turns = turns < 1 ? 1 : turns > top ? top : turns;
    return (unsigned)((need + turns - 1) / turns);
}

// Workgroups of the gradient.  One where its teams get up to four rows each:
// it needs no join.  Else no more than the registers let run at once (512 of
// 256 threads; 512 of 512 where a lane holds little), with one, two or four rows
// to a team as the sums that they leave, 8 bytes a column and workgroup, grow
// beside the rows (turns 1, 2, 4: 1000 x 384 bf16 7.5, 8.2, 9.9 us; 2000 x 1024
// f32 12.2, 10.2, 10.8; 1000 x 8192 bf16 28.5, 27.9, 22.4).
unsigned grad_blocks(int64_t n, int dim, const Shape &s)
{
    const int block = s.lanes ? block_of(s.lanes) : 1024;
    const int64_t teams = s.lanes ? block / s.lanes : 1, need = (n + teams - 1) / teams;
    if (need <= 4) return 1;
    const int64_t columns = need * dim;
    const int64_t turns = columns <= 1 << 17 ? 1 : columns <= 1 << 21 ? 2 : 4;
    const int64_t most = (s.lanes == 512 && s.len * s.nv <= 12 ? 1024 : 512) * 256 / block;
    const int64_t blocks = (need + turns - 1) / turns;
    return (unsigned)(blocks < most ? blocks : most);
}

template <typename T, typename P, template <typename, typename, int, int, int> class F, typename... A>
hipError_t by_shape(const Shape &s, A... args)
{
    constexpr int LEN = 16 / sizeof(T);
#define CASE(L, NV)          \
    case L * 8 + NV:         \
        F<T, P, LEN, L, NV>::run(args...); \
        return hipGetLastError();
    if (s.len == 1) {
        switch (s.lanes) {
        case 1: F<T, P, 1, 1, 1>::run(args...); return hipGetLastError();
        case 2: F<T, P, 1, 2, 1>::run(args...); return hipGetLastError();
        case 4: F<T, P, 1, 4, 1>::run(args...); return hipGetLastError();
        default: F<T, P, 1, 8, 1>::run(args...); return hipGetLastError();
        }
    }
    switch (s.lanes * 8 + s.nv) {
        CASE(1, 1) CASE(2, 1) CASE(4, 1)
        CASE(8, 1) CASE(8, 2) CASE(8, 3) CASE(8, 4)
        CASE(16, 3) CASE(16, 4) CASE(32, 3) CASE(32, 4) CASE(64, 3) CASE(64, 4)
        CASE(128, 3) CASE(256, 2) CASE(256, 3) CASE(256, 4) CASE(512, 3)
    }
    if constexpr (F<T, P, LEN, 1024, 4>::kLong) {
        switch (s.lanes * 8 + s.nv) { CASE(1024, 2) CASE(1024, 3) CASE(1024, 4) }
    } else {
        switch (s.lanes * 8 + s.nv) { CASE(512, 4) }
    }
#undef CASE
    return hipErrorInvalidConfiguration;  // a shape without a kernel
}

template <bool HOLD>
struct Norm {
    template <typename T, typename P, int LEN, int L, int NV>
    struct Run {
        static constexpr bool kLong = true;  // 1024 lanes as well
        static void run(const NormArgs *a, unsigned blocks, hipStream_t s)
        {
            k_norm<T, P, LEN, L, NV, HOLD><<<dim3(blocks), dim3(block_of(L)), 0, s>>>(*a);
        }
    };
};

template <bool HELD>
struct Grad {
    template <typename T, typename P, int LEN, int L, int NV>
    struct Run {
        static constexpr bool kLong = false;
        static void run(const NormGradArgs *a, float *part, unsigned blocks, hipStream_t s)
        {
            k_norm_grad<T, P, LEN, L, NV, HELD><<<dim3(blocks), dim3(block_of(L)), 0, s>>>(*a, part);
        }
    };
};

// Calls ... with T and P for the admissible pairs: P is T or float.
#define ERSJ_NORM_SWITCH(type, param, T, P, ...)                                                          \
    do {                                                                                                  \
        if ((type) == kF32) { typedef float T; typedef float P; __VA_ARGS__; }                            \
        else if ((type) == kF16 && (param) == kF32) { typedef f16_t T; typedef float P; __VA_ARGS__; }    \
        else if ((type) == kF16) { typedef f16_t T; typedef f16_t P; __VA_ARGS__; }                       \
        else if ((param) == kF32) { typedef bf16_t T; typedef float P; __VA_ARGS__; }                     \
        else { typedef bf16_t T; typedef bf16_t P; __VA_ARGS__; }                                         \
    } while (0)

}  // namespace

hipError_t launch_layer_norm(const NormArgs &a, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    const Shape sh = shape_of(a.type, a.dim, 1024);
    const unsigned blocks = norm_blocks(a.n, sh);
    ERSJ_NORM_SWITCH(a.type, a.param_type, T, P,
        if (sh.lanes && a.codes) return by_shape<T, P, Norm<true>::template Run>(sh, &a, blocks, s);
        if (sh.lanes) return by_shape<T, P, Norm<false>::template Run>(sh, &a, blocks, s);
        k_norm_long<T, P><<<dim3(blocks), dim3(1024), 0, s>>>(a));
    return hipGetLastError();
}

bool norm_holds(int type, int dim) { return shape_of(type, dim, 1024).lanes != 0; }

bool norm_grad_of_held(int type, int dim) { return shape_of(type, dim, 512).lanes != 0; }

uint64_t layer_norm_grad_work(int64_t n, int dim)
{
    // a shape depends on the type: the larger of the two
    uint64_t most = 0;
    for (int type : {(int)kF32, (int)kBF16}) {
        const Shape sh = shape_of(type, dim, 512);
        const unsigned blocks = grad_blocks(n, dim, sh);
        const uint64_t b = blocks == 1 && sh.lanes ? 0 : (uint64_t)blocks * 2 * 4 * (uint64_t)dim;
        if (b > most) most = b;
    }
    return most;
}

hipError_t launch_layer_norm_grad(const NormGradArgs &a, hipStream_t s)
{
    const Shape sh = shape_of(a.type, a.dim, 512);
    const unsigned blocks = grad_blocks(a.n, a.dim, sh);
    const bool params = a.gw || a.gb;
    if (!params && (!a.gx || a.n == 0)) return hipSuccess;
    float *part = params && (blocks > 1 || !sh.lanes) ? (float *)a.work : nullptr;
    ERSJ_NORM_SWITCH(a.type, a.param_type, T, P,
        if (sh.lanes) {
            const hipError_t e = a.x || !a.n ? by_shape<T, P, Grad<false>::template Run>(sh, &a, part, blocks, s)
                                             : by_shape<T, P, Grad<true>::template Run>(sh, &a, part, blocks, s);
            if (e != hipSuccess) return e;
        } else {
            // the sums before the gradient of x, which may replace an input
            if (part)
                k_norm_grad_long_part<T><<<dim3((a.dim + kThreads - 1) / kThreads, blocks), dim3(kThreads), 0, s>>>(a, part);
            if (a.gx && a.n) k_norm_grad_long<T, P><<<dim3(blocks), dim3(1024), 0, s>>>(a);
        }
        if (part)
            k_norm_grad_join<P><<<dim3((2 * a.dim + 15) / 16), dim3(1024), 0, s>>>(part, (int)blocks, a.dim, (P *)a.gw,
                                                                                  (P *)a.gb));
    return hipGetLastError();
}

}  // namespace ersj
