// Token embedding and the gradient of its table.
#include "encoder_internal.h"

namespace ersj {

namespace {

constexpr int kThreads = 256;

template <typename I>
__device__ __forceinline__ int64_t id_at(const void *ids, int64_t t)
{
    return (int64_t)((const I *)ids)[t];
}

template <typename T, typename O, typename I>
__global__ __launch_bounds__(kThreads) void k_embed(EmbedArgs a)
{
    for (int64_t t = blockIdx.x; t < a.n; t += gridDim.x) {
        const int64_t id = id_at<I>(a.ids, t);
        O *out = (O *)a.out + t * a.ld_out;
        const bool pad = id >= 0 && id == a.padding_id, bad = id < 0 || id >= a.rows;
        const T *row = (const T *)a.table + (bad ? 0 : id) * a.ld_table;
        for (int c = threadIdx.x; c < a.dim; c += kThreads) {
            float v = pad ? 0.f : __builtin_nanf("");
            if (!pad && !bad) v = a.scale * (float)row[c];
            out[c] = (O)v;
        }
    }
}

// ---- sort of the tokens by id -------------------------------------------
//
// Stable least-significant-digit radix sort of (key, t), key = id or `rows`
// for tokens that add nothing.  A workgroup counts the digits of its kSortRun
// consecutive entries; the scatter kernel derives its own offsets from the
// table of all counts.

constexpr int kSortRun = 4096;
constexpr int kSortItems = kSortRun / kThreads;
constexpr int kMaxDigitBits = 9;
constexpr int kWaves = kThreads / 64;

struct SortPlan {
    int passes, bits;
    int64_t runs;
};

SortPlan sort_plan(int64_t n, int64_t rows)
{
    int kb = 0;
    while (((int64_t)1 << kb) <= rows) ++kb;  // keys 0 .. rows
    SortPlan p;
    p.passes = (kb + kMaxDigitBits - 1) / kMaxDigitBits;
    p.bits = (kb + p.passes - 1) / p.passes;
    p.runs = (n + kSortRun - 1) / kSortRun;
    return p;
}

struct SortSource {
    const void *ids;
    const uint32_t *keys, *pos;  // null on the first pass
    int64_t padding_id, rows;
    uint32_t n;
};

template <typename I>
__device__ __forceinline__ uint32_t sort_key(const SortSource &s, uint32_t i)
{
    if (s.keys) return s.keys[i];
    const int64_t id = id_at<I>(s.ids, i);
    return id < 0 || id >= s.rows || id == s.padding_id ? (uint32_t)s.rows : (uint32_t)id;
}

template <typename I>
__global__ __launch_bounds__(kThreads) void k_sort_count(SortSource s, int shift, int bits, uint32_t *counts)
{
    __shared__ uint32_t cnt[1 << kMaxDigitBits];
    const int nd = 1 << bits;
    for (int k = threadIdx.x; k < nd; k += kThreads) cnt[k] = 0;
    __syncthreads();
    const uint32_t i0 = blockIdx.x * kSortRun;
    for (uint32_t i = i0 + threadIdx.x; i < i0 + kSortRun && i < s.n; i += kThreads)
        atomicAdd(&cnt[(sort_key<I>(s, i) >> shift) & (nd - 1)], 1u);
    __syncthreads();
    for (int k = threadIdx.x; k < nd; k += kThreads) counts[(size_t)blockIdx.x * nd + k] = cnt[k];
}

template <typename I>
__global__ __launch_bounds__(kThreads) void k_sort_scatter(SortSource s, int shift, int bits, uint32_t *counts,
                                                           uint32_t *keys_out, uint32_t *pos_out)
{
    __shared__ uint32_t base[1 << kMaxDigitBits];
    __shared__ uint32_t cnt[kWaves][1 << kMaxDigitBits];
    __shared__ uint32_t wsum[kWaves];
    const int nd = 1 << bits, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    for (int k = tid; k < kWaves * nd; k += kThreads) cnt[k / nd][k % nd] = 0;

    // offsets: all smaller digits, then the same digit in earlier runs
    uint32_t carry = 0;
    for (int k0 = 0; k0 < nd; k0 += kThreads) {
        const int k = k0 + tid;
        uint32_t total = 0, before = 0;
        if (k < nd) {
            for (uint32_t g = 0; g < gridDim.x; ++g) {
                const uint32_t c = counts[(size_t)g * nd + k];
                total += c;
                if (g < blockIdx.x) before += c;
            }
        }
        uint32_t inc = total;
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t v = __shfl_up(inc, o, 64);
            if (lane >= o) inc += v;
        }
        if (lane == 63) wsum[w] = inc;
        __syncthreads();
        uint32_t below = carry;
        for (int j = 0; j < kWaves; ++j) {
            if (j < w) below += wsum[j];
            carry += wsum[j];
        }
        if (k < nd) base[k] = below + inc - total + before;
        __syncthreads();
    }

    // ranks within the wave's stretch of the run, in order
    uint32_t key[kSortItems], rank[kSortItems];
    const uint32_t i0 = blockIdx.x * kSortRun + w * (kSortRun / kWaves) + lane;
#pragma unroll
    for (int r = 0; r < kSortItems; ++r) {
        const uint32_t i = i0 + r * 64;
        const bool ok = i < s.n;
        key[r] = ok ? sort_key<I>(s, i) : 0;
        const uint32_t dg = (key[r] >> shift) & (nd - 1);
        uint64_t same = __ballot(ok);
        for (int b = 0; b < bits; ++b) {
            const uint64_t m = __ballot((dg >> b) & 1);
            same &= (dg >> b) & 1 ? m : ~m;
        }
        uint32_t old = 0;
        const int leader = ok ? __ffsll((unsigned long long)same) - 1 : lane;
        if (ok && lane == leader) old = atomicAdd(&cnt[w][dg], (uint32_t)__popcll(same));
        old = __shfl(old, leader, 64);
        rank[r] = old + __popcll(same & (((uint64_t)1 << lane) - 1));
    }
    __syncthreads();
    for (int k = tid; k < nd; k += kThreads) {
        uint32_t at = base[k];
        for (int j = 0; j < kWaves; ++j) {
            const uint32_t c = cnt[j][k];
            cnt[j][k] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortItems; ++r) {
        const uint32_t i = i0 + r * 64;
        if (i < s.n) {
            const uint32_t at = cnt[w][(key[r] >> shift) & (nd - 1)] + rank[r];
            keys_out[at] = key[r];
            pos_out[at] = s.pos ? s.pos[i] : i;
        }
    }
}

// ---- sums over the sorted tokens ------------------------------------------
//
// The output is the merge of two sequences: the sorted tokens, each an
// addition, and the table's rows, each finished (written) after its last
// token.  Token i is at place i + key[i] of the merge (i tokens and key[i]
// rows come before it), so a wave finds its share, `share` consecutive
// places, by a search over i for that strictly rising sum.  Shares cost the
// same whatever the distribution of the ids: a frequent token spans several
// waves, and a stretch of unused rows is spread over several as well.
//
// A share that begins inside a row leaves up to kSnap - 1 tokens that remain
// of it, and the row's end, to the wave before.  Only a longer rest is cut:
// its waves write their sums to `part` (the share's first row if that was
// begun before, its last row if that is not finished), and k_embed_grad_join
// adds them up in order.

constexpr int kSnap = 32;
constexpr int kShareMin = 32;
constexpr int kMaxShares = 8192;  // waves of the sum kernel: 8 per SIMD
enum { kFirstCut = 1, kLastCut = 2, kInside = 4 };

struct SumPlan {
    int cols;        // columns of one wave: 64 lanes of 16 bytes of the 16-bit types
    int col_blocks;
    int64_t shares, share;
};

SumPlan sum_plan(int64_t n, int64_t rows, int dim)
{
    SumPlan p;
    p.cols = 512;
    p.col_blocks = (dim + p.cols - 1) / p.cols;
    const int64_t total = n + rows;
    const int64_t most = p.col_blocks < kMaxShares / 64 ? kMaxShares / p.col_blocks : 64;
    p.share = (total + most - 1) / most;  // shares <= kMaxShares
    if (p.share < kShareMin) p.share = kShareMin;
    p.shares = (total + p.share - 1) / p.share;
    return p;
}

struct Cut {
    uint32_t i;   // tokens before
    uint32_t v;   // rows finished before
    bool inside;  // row v was begun before and is long
};

// The cut at place `at`, by the 32 lanes of each half of the wave for its own
// `at`: a 32-way search, then a look at the rest of the row that it falls in.
__device__ __forceinline__ Cut find_cut(const uint32_t *keys, uint32_t n, uint32_t rows, int64_t at)
{
    const int lane = threadIdx.x & 31;
    const int half = (threadIdx.x & 32);
    // least i with i + keys[i] >= at, in [lo, hi]
    int64_t lo = at > rows ? at - rows : 0, hi = at < n ? at : n;
    while (__ballot(lo < hi)) {
        const int64_t step = (hi - lo + 31) >> 5;
        const int64_t i = lo + (int64_t)lane * step;
        bool less = false;
        if (lo < hi && i < hi) less = i + (int64_t)keys[i] < at;
        const uint32_t m = (uint32_t)(__ballot(less) >> half);
        if (lo < hi) {
            // `less` holds for the first c probes: the answer lies after
            // probe c - 1 and not after probe c
            const int c = __popc(m);
            const int64_t top = lo + (int64_t)c * step;
            if (c > 0) lo = lo + (int64_t)(c - 1) * step + 1;
            if (c < 32 && top < hi) hi = top;
        }
    }
    Cut r;
    r.i = (uint32_t)lo;
    r.v = (uint32_t)(at - lo);
    r.inside = false;
    const bool begun = r.i > 0 && r.v < rows && keys[r.i - 1] == r.v;
    const uint32_t j = r.i + lane;
    const bool same = begun && j < n && keys[j] == r.v;
    const uint32_t m = (uint32_t)(__ballot(same) >> half);
    if (begun) {
        if (m == 0xffffffffu) r.inside = true;
        else {
            r.i += __popc(m);
            r.v += 1;
        }
    }
    return r;
}

// Columns of a lane: NV vectors of LEN elements.  A vector that would pass
// the row's end begins LEN before it instead; the columns it shares with its
// neighbour hold the same sums.
template <typename T, typename O, int LEN, int NV>
__global__ __launch_bounds__(kThreads) void k_embed_grad_sum(EmbedGradArgs a, const uint32_t *keys,
                                                             const uint32_t *pos, int64_t share, uint32_t shares,
                                                             float *part, uint8_t *flags)
{
    typedef T tvec __attribute__((ext_vector_type(LEN)));
    typedef O ovec __attribute__((ext_vector_type(LEN)));
    typedef float fvec __attribute__((ext_vector_type(LEN)));
    struct __attribute__((packed, aligned(sizeof(T)))) tslot { tvec v; };
    struct __attribute__((packed, aligned(sizeof(O)))) oslot { ovec v; };
    struct __attribute__((packed, aligned(4))) fslot { fvec v; };
    constexpr int kAhead = 8 / NV;  // rows in flight

    const int lane = threadIdx.x & 63;
    const uint32_t w = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6));
    if (w >= shares) return;
    const uint32_t n = (uint32_t)a.n, rows = (uint32_t)a.rows;
    const int64_t total = (int64_t)n + rows;

    int64_t at = (int64_t)(w + (lane >> 5)) * share;
    if (at > total) at = total;
    const Cut cut = find_cut(keys, n, rows, at);
    uint32_t i = __builtin_amdgcn_readlane(cut.i, 0), v = __builtin_amdgcn_readlane(cut.v, 0);
    const uint32_t i1 = __builtin_amdgcn_readlane(cut.i, 32);
    uint32_t v1 = __builtin_amdgcn_readlane(cut.v, 32);
    const bool begun = __builtin_amdgcn_readlane((int)cut.inside, 0);
    const bool open = __builtin_amdgcn_readlane((int)cut.inside, 32);
    if (v1 > rows) v1 = rows;

    // even blocks of whole vectors: the last has several, so a vector that is
    // shifted back from the row's end stays inside its wave's own columns
    const int vecs = (a.dim + LEN - 1) / LEN;
    const int c0 = (int)((int64_t)blockIdx.y * vecs / gridDim.y) * LEN;
    const int block_cols = (int)((int64_t)(blockIdx.y + 1) * vecs / gridDim.y) * LEN - c0;
    int cols[NV];
    bool on[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        int c = (k * 64 + lane) * LEN;
        on[k] = c < block_cols;
        c += c0;
        cols[k] = c + LEN > a.dim ? a.dim - LEN : c;
    }

    fvec acc[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) acc[k] = (fvec)0.f;
    bool any = false;         // acc holds tokens of row v
    bool first = begun;       // row v was begun before this share
    uint32_t flag = 0;

    auto finish = [&]() {
        if (first) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (on[k]) ((fslot *)(part + (uint64_t)w * 2 * a.dim + cols[k]))->v = acc[k];
            flag |= kFirstCut;
        } else if (any || !a.accumulate) {
            O *out = (O *)a.out + (int64_t)v * a.ld_out;
#pragma unroll
            for (int k = 0; k < NV; ++k) acc[k] *= a.scale;
            if (a.accumulate) {  // all read before any is written: shifted vectors overlap
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (on[k]) acc[k] += __builtin_convertvector(((const oslot *)(out + cols[k]))->v, fvec);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (on[k]) ((oslot *)(out + cols[k]))->v = __builtin_convertvector(acc[k], ovec);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) acc[k] = (fvec)0.f;
        any = first = false;
        ++v;
    };

    while (i < i1) {
        // up to 64 tokens' keys and places, one to a lane
        const uint32_t m = i1 - i < 64 ? i1 - i : 64;
        const uint32_t kk = keys[i + (lane < (int)m ? lane : 0)];
        const uint32_t pp = pos[i + (lane < (int)m ? lane : 0)];
        if (__builtin_amdgcn_readlane(kk, 0) >= rows) { i = i1; break; }
        for (uint32_t t = 0; t < m; t += kAhead) {
            tvec x[kAhead][NV];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const uint32_t tu = t + u < m ? t + u : m - 1;
                // tokens that add nothing (key `rows`) are not read
                const uint32_t p = __builtin_amdgcn_readlane(kk, tu) < rows ? __builtin_amdgcn_readlane(pp, tu)
                                                                              : __builtin_amdgcn_readlane(pp, 0);
                const T *row = (const T *)a.grad + (int64_t)p * a.ld_grad;
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (on[k]) x[u][k] = ((const tslot *)(row + cols[k]))->v;
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (t + u < m) {
                    const uint32_t key = __builtin_amdgcn_readlane(kk, t + u);
                    if (key < rows) {
                        while (v < key) finish();
#pragma unroll
                        for (int k = 0; k < NV; ++k)
                            if (on[k]) acc[k] += __builtin_convertvector(x[u][k], fvec);
                        any = true;
                    }
                }
            }
        }
        i += m;
    }
    while (v < v1) finish();
    if (open) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on[k]) ((fslot *)(part + ((uint64_t)w * 2 + 1) * a.dim + cols[k]))->v = acc[k];
        flag |= kLastCut | (first ? kInside : 0);
    }
    if (lane == 0 && blockIdx.y == 0) flags[w] = (uint8_t)flag;
}

// Rows cut over several shares.  A workgroup goes through its share of the
// flags; for each row that ends there it finds the share where the row was
// begun, and its waves add equal stretches of the parts between, which are
// then added in order.
constexpr int kJoinThreads = 512;
constexpr int kJoinBlocks = 512;
static_assert(kMaxShares / kJoinBlocks <= 64, "a join block's flags fit one wave");

template <typename O>
__global__ __launch_bounds__(kJoinThreads) void k_embed_grad_join(EmbedGradArgs a, const uint32_t *keys,
                                                                  int64_t share, uint32_t shares, const float *part,
                                                                  const uint8_t *flags)
{
    constexpr int kJoinWaves = kJoinThreads / 64;
    __shared__ float sums[kJoinWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t per = (shares + gridDim.x - 1) / gridDim.x;
    const uint32_t w0 = blockIdx.x * per, w1 = w0 + per < shares ? w0 + per : shares;
    // a block has at most kMaxShares / kJoinBlocks shares, one to a lane
    const uint32_t mine = w0 + lane < w1 ? flags[w0 + lane] : 0;
    for (uint64_t todo = __ballot((mine & kFirstCut) != 0); todo; todo &= todo - 1) {  // the same for all waves
        const uint32_t w = w0 + (__ffsll((unsigned long long)todo) - 1);
        // the share where the row was begun: the first before w that is not all inside it
        uint32_t b = w;
        for (bool more = true; more;) {
            const int64_t q = (int64_t)b - 1 - lane;
            const uint64_t m = __ballot(q < 0 || !(flags[q] & kInside));
            if (m) {
                b = b - 1 - (__ffsll((unsigned long long)m) - 1);
                more = false;
            } else
                b -= 64;
        }
        const int64_t at = (int64_t)w * share;
        const Cut cut = find_cut(keys, (uint32_t)a.n, (uint32_t)a.rows, at);
        const uint32_t v = __builtin_amdgcn_readfirstlane(cut.v);
        const uint32_t count = w - b + 1;  // parts: the last rows of b .. w - 1, the first row of w
        const uint32_t each = (count + kJoinWaves - 1) / kJoinWaves;
        const uint32_t p0 = wave * each, p1 = p0 + each < count ? p0 + each : count;
        for (int c0 = 0; c0 < a.dim; c0 += 64) {
            const int c = c0 + lane;
            float s = 0.f;
            if (c < a.dim) {
#pragma unroll 8
                for (uint32_t p = p0; p < p1; ++p)
                    s += part[((uint64_t)(b + p) * 2 + (b + p < w ? 1 : 0)) * a.dim + c];
            }
            __syncthreads();
            sums[wave][lane] = s;
            __syncthreads();
            if (wave == 0 && c < a.dim) {
                s = 0.f;
                for (int k = 0; k < kJoinWaves; ++k) s += sums[k][lane];
                s *= a.scale;
                O *out = (O *)a.out + (int64_t)v * a.ld_out + c;
                if (a.accumulate) s += (float)*out;
                *out = (O)s;
            }
        }
    }
}

uint64_t up256(uint64_t b) { return (b + 255) & ~(uint64_t)255; }

}  // namespace

hipError_t launch_embed(const EmbedArgs &a, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    const dim3 grid((unsigned)(a.n < 65536 ? a.n : 65536)), block(kThreads);
    ERSJ_ELEM_SWITCH(a.table_type, T, ERSJ_ELEM_SWITCH(a.out_type, O,
        if (a.id_type) k_embed<T, O, int64_t><<<grid, block, 0, s>>>(a);
        else k_embed<T, O, int32_t><<<grid, block, 0, s>>>(a)))
    return hipGetLastError();
}

uint64_t embed_grad_work(int64_t n, int64_t rows, int dim)
{
    const SortPlan p = sort_plan(n, rows);
    const SumPlan q = sum_plan(n, rows, dim);
    return 4 * up256(4 * (uint64_t)n) + up256(((uint64_t)4 << p.bits) * (uint64_t)p.runs) +
           up256((uint64_t)q.shares) + (uint64_t)q.shares * 2 * 4 * (uint64_t)dim;
}

hipError_t launch_embed_grad(const EmbedGradArgs &a, hipStream_t s)
{
    const SortPlan p = sort_plan(a.n, a.rows);
    char *at = (char *)a.work;
    uint32_t *buf[4];
    for (int k = 0; k < 4; ++k, at += up256(4 * (uint64_t)a.n)) buf[k] = (uint32_t *)at;
    uint32_t *counts = (uint32_t *)at;
    at += up256(((uint64_t)4 << p.bits) * (uint64_t)p.runs);
    SortSource src{a.ids, nullptr, nullptr, a.padding_id, a.rows, (uint32_t)a.n};
    int side = 0;
    for (int k = 0; k < p.passes && a.n; ++k, side ^= 1) {
        const dim3 grid((unsigned)p.runs), block(kThreads);
        uint32_t *ko = buf[2 * side], *po = buf[2 * side + 1];
        if (a.id_type) {
            k_sort_count<int64_t><<<grid, block, 0, s>>>(src, k * p.bits, p.bits, counts);
            k_sort_scatter<int64_t><<<grid, block, 0, s>>>(src, k * p.bits, p.bits, counts, ko, po);
        } else {
            k_sort_count<int32_t><<<grid, block, 0, s>>>(src, k * p.bits, p.bits, counts);
            k_sort_scatter<int32_t><<<grid, block, 0, s>>>(src, k * p.bits, p.bits, counts, ko, po);
        }
        src.keys = ko;
        src.pos = po;
    }
    const SumPlan q = sum_plan(a.n, a.rows, a.dim);
    uint8_t *flags = (uint8_t *)at;
    float *part = (float *)(at + up256((uint64_t)q.shares));
    const int len = a.grad_type == kF32 ? 4 : 8;
    const dim3 grid((unsigned)((q.shares + kWaves - 1) / kWaves), q.col_blocks), block(kThreads);
#define SUM(T, O)                                                                                                  \
    do {                                                                                                           \
        if (a.dim < len)                                                                                           \
            k_embed_grad_sum<T, O, 1, 1><<<grid, block, 0, s>>>(a, src.keys, src.pos, q.share, (uint32_t)q.shares, \
                                                                part, flags);                                      \
        else                                                                                                       \
            k_embed_grad_sum<T, O, 16 / sizeof(T), sizeof(T) / 2><<<grid, block, 0, s>>>(                          \
                a, src.keys, src.pos, q.share, (uint32_t)q.shares, part, flags);                                   \
    } while (0)
    switch (a.grad_type * 4 + a.out_type) {
    case kF32 * 4 + kF32: SUM(float, float); break;
    case kF16 * 4 + kF32: SUM(f16_t, float); break;
    case kBF16 * 4 + kF32: SUM(bf16_t, float); break;
    case kF16 * 4 + kF16: SUM(f16_t, f16_t); break;
    default: SUM(bf16_t, bf16_t); break;
    }
#undef SUM
    if (a.n > kSnap)
        ERSJ_ELEM_SWITCH(a.out_type, O, k_embed_grad_join<O><<<dim3(kJoinBlocks), dim3(kJoinThreads), 0, s>>>(
                                            a, src.keys, q.share, (uint32_t)q.shares, part, flags))
    return hipGetLastError();
}

}  // namespace ersj
