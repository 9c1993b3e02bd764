// Token embedding and the gradient of its table.
#include "encoder_internal.h"
#include "embed_few_plan.h"

namespace ersj {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

template <typename I>
__device__ __forceinline__ int64_t id_at(const void *ids, int64_t t)
{
    return (int64_t)((const I *)ids)[t];
}

// out[t] = scale * table[ids[t]].  Bound by memory: rows of the table in, rows
// of the output out (65,536 tokens x 384, f32 table of 32,768 rows to bf16:
// 14.7 us for 70 MB, 4.8 TB/s; a copy of 512 MiB reaches 5.3).  A token
// belongs to a team of L lanes, each with NV vectors of LEN elements (16
// bytes of the output); a team takes tokens that lie a whole grid apart and
// has the next token's row and the id after that on the way.  A vector that
// would pass the row's end begins earlier, so that it ends with the row, and
// writes its neighbour's values a second time.
template <typename T, typename O, typename I, int LEN, int L, int NV>
__global__ __launch_bounds__(kThreads) void k_embed(EmbedArgs a)
{
    typedef Slot<T, LEN> In;
    typedef Slot<O, LEN> Out;
    typedef float fvec __attribute__((ext_vector_type(LEN)));
    const int lane = threadIdx.x & (L - 1);
    const int c0 = blockIdx.y * (L * NV * LEN);
    int col[NV];
    bool on[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = c0 + (k * L + lane) * LEN;
        on[k] = c < a.dim;
        col[k] = c + LEN <= a.dim ? c : a.dim - LEN;
    }
    const int64_t step = (int64_t)gridDim.x * (kThreads / L);
    int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    if (t >= a.n) return;
    auto id_of = [&](int64_t at) { return id_at<I>(a.ids, at < a.n ? at : a.n - 1); };
    auto load = [&](int64_t id, typename In::vec (&x)[NV]) {
        // the first row in the place of one that is not used
        const bool use = id >= 0 && id < a.rows && id != a.padding_id;
        const T *row = (const T *)a.table + (use ? id : 0) * a.ld_table;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on[k]) x[k] = In::load(row + col[k]);
    };
    int64_t id = id_of(t), next_id = id_of(t + step);
    typename In::vec x[NV], y[NV];
    load(id, x);
    while (true) {
        const int64_t after = id_of(t + 2 * step);
        const bool more = t + step < a.n;
        if (more) load(next_id, y);
        const bool pad = id >= 0 && id == a.padding_id, bad = id < 0 || id >= a.rows;
        O *out = (O *)a.out + t * a.ld_out;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            fvec v = __builtin_convertvector(x[k], fvec) * a.scale;
            if (pad || bad) v = (fvec)(pad ? 0.f : __builtin_nanf(""));
            if (on[k]) Out::store(out + col[k], __builtin_convertvector(v, typename Out::vec));
            x[k] = y[k];
        }
        if (!more) break;
        t += step;
        id = next_id;
        next_id = after;
    }
}

// ---- sort of the tokens by id -------------------------------------------
//
// Stable least-significant-digit radix sort of (key, t), key = id or `rows`
// for tokens that add nothing.  A workgroup takes a run of consecutive
// entries: one kernel counts the runs' digits, the next ranks a run's entries
// and moves them, to offsets that it derives from the counts of all runs.
// With many runs a scan kernel lies between.  (Adding each moved entry to the
// next pass's counts instead of counting anew costs more: device-wide atomics,
// 44 us for a million entries against 5 us for the kernel.)  Tokens that fit
// one workgroup are sorted by it in one kernel, through LDS.  Bound by the
// latency of its steps: count and scatter take 3.0 and 6.4 us a pass for 65,536
// tokens, and 5.4 and 11.4 us with 4.9 us of scan for a million.

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxDigitBits = 10;  // a digit's count to each thread
constexpr int kMaxDigits = 1 << kMaxDigitBits;
static_assert(kMaxDigits <= kSortThreads, "one thread to a digit");
// More runs than this are scanned by a kernel of their own: up to it a thread
// reads the counts of a digit in 64 runs or less in one or two batches of loads.
constexpr int kScanRuns = 64;
constexpr int kLocalMax = kSortThreads * 4;  // entries of the one-workgroup sort

struct SortPlan {
    int passes, bits;
    int items;  // per thread
    int64_t runs;
};

SortPlan sort_plan(int64_t n, int64_t rows)
{
    int kb = 0;
    while (((int64_t)1 << kb) <= rows) ++kb;  // keys 0 .. rows
    SortPlan p;
    p.passes = (kb + kMaxDigitBits - 1) / kMaxDigitBits;
    p.bits = (kb + p.passes - 1) / p.passes;
    // short runs while their counts need no scan: more workgroups, fewer steps
    // each (65,536 tokens, scatter: one entry a thread 6.3 us, two 6.6, four 8.5;
    // above 131,072 four with the scan 11.4 us for a million, eight 15.9)
    const int64_t unit = (int64_t)kScanRuns * kSortThreads;
    p.items = n <= unit ? 1 : n <= 2 * unit ? 2 : 4;
    const int64_t run = (int64_t)p.items * kSortThreads;
    p.runs = (n + run - 1) / run;
    return p;
}

struct SortSource {
    const void *ids;
    const uint2 *entries;  // (key, t); null on the first pass
    int64_t padding_id, rows;
    uint32_t n;
};

template <typename I>
__device__ __forceinline__ uint2 sort_entry(const SortSource &s, uint32_t i)
{
    if (s.entries) return s.entries[i];
    const int64_t id = id_at<I>(s.ids, i);
    return make_uint2(id < 0 || id >= s.rows || id == s.padding_id ? (uint32_t)s.rows : (uint32_t)id, i);
}

template <typename I, int ITEMS>
__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortSource s, int shift, int bits, uint32_t *counts)
{
    __shared__ uint32_t cnt[kMaxDigits];
    const int nd = 1 << bits;
    uint32_t key[ITEMS];
    const uint64_t i0 = (uint64_t)blockIdx.x * (kSortThreads * ITEMS) + threadIdx.x;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
        const uint64_t i = i0 + r * kSortThreads;
        key[r] = sort_entry<I>(s, i < s.n ? (uint32_t)i : s.n - 1).x;
    }
    if ((int)threadIdx.x < nd) cnt[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
        if (i0 + r * kSortThreads < s.n) atomicAdd(&cnt[(key[r] >> shift) & (nd - 1)], 1u);
    __syncthreads();
    if ((int)threadIdx.x < nd) counts[(size_t)blockIdx.x * nd + threadIdx.x] = cnt[threadIdx.x];
}

// Each digit's counts over the runs become their exclusive prefix; the total
// goes to row `runs`.  One wave per digit, four loads of 64 runs at a time.
__global__ __launch_bounds__(kThreads) void k_sort_scan(uint32_t *counts, uint32_t runs, int bits)
{
    const int lane = threadIdx.x & 63;
    const uint32_t nd = 1u << bits, k = blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (k >= nd) return;
    uint32_t carry = 0;
    for (uint32_t g0 = 0; g0 < runs; g0 += 256) {
        uint32_t c[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t g = g0 + 64 * u + lane;
            c[u] = g < runs ? counts[(size_t)g * nd + k] : 0;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t g = g0 + 64 * u + lane;
            uint32_t inc = c[u];
            for (int o = 1; o < 64; o <<= 1) {
                const uint32_t v = __shfl_up(inc, o, 64);
                if (lane >= o) inc += v;
            }
            if (g < runs) counts[(size_t)g * nd + k] = carry + inc - c[u];
            carry += __shfl(inc, 63, 64);
        }
    }
    if (lane == 0) counts[(size_t)runs * nd + k] = carry;
}

// Exclusive prefix over the first kMaxDigits threads' values, in those threads.
__device__ __forceinline__ uint32_t digit_prefix(uint32_t v, uint32_t *wsum)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint32_t inc = v;
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t u = __shfl_up(inc, o, 64);
        if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 63 && w < kMaxDigits / 64) wsum[w] = inc;
    __syncthreads();
    for (int j = 0; j < kMaxDigits / 64; ++j)
        if (j < w) inc += wsum[j];
    return inc - v;
}

// Rank of each of the thread's ITEMS entries among the wave's entries with
// the same digit, in order (entry r of a lane comes before entry r + 1 of any
// lane); cnt, the wave's own counters, ends as its digit counts.
template <int ITEMS>
__device__ __forceinline__ void wave_ranks(const uint32_t (&dg)[ITEMS], const bool (&ok)[ITEMS], int bits,
                                           uint32_t *cnt, uint32_t (&rank)[ITEMS])
{
    const int lane = threadIdx.x & 63;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
        uint64_t same = __ballot(ok[r]);
        for (int b = 0; b < bits; ++b) {
            const uint64_t m = __ballot((dg[r] >> b) & 1);
            same &= (dg[r] >> b) & 1 ? m : ~m;
        }
        // the lanes of a digit read its counter together; the first then writes it
        const uint32_t old = ok[r] ? ((volatile uint32_t *)cnt)[dg[r]] : 0;
        if (ok[r] && (same & below) == 0) ((volatile uint32_t *)cnt)[dg[r]] = old + (uint32_t)__popcll(same);
        __builtin_amdgcn_wave_barrier();
        rank[r] = old + (uint32_t)__popcll(same & below);
    }
}

template <typename I, int ITEMS>
__global__ __launch_bounds__(kSortThreads) void k_sort_scatter(SortSource s, int shift, int bits,
                                                               const uint32_t *counts, bool scanned, uint2 *out)
{
    __shared__ uint32_t cnt[kSortWaves][kMaxDigits];
    __shared__ uint32_t halves[2][kSortThreads];
    __shared__ uint32_t wsum[kMaxDigits / 64];
    const uint32_t nd = 1u << bits, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    constexpr uint32_t run = kSortThreads * ITEMS;

    // a wave's entries are consecutive
    uint2 e[ITEMS];
    uint32_t dg[ITEMS], rank[ITEMS];
    bool ok[ITEMS];
    const uint64_t i0 = (uint64_t)blockIdx.x * run + w * (64 * ITEMS) + lane;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
        const uint64_t i = i0 + r * 64;
        ok[r] = i < s.n;
        e[r] = sort_entry<I>(s, ok[r] ? (uint32_t)i : s.n - 1);
    }
    // offsets: all smaller digits, then the same digit in earlier runs
    uint32_t total = 0, before = 0;
    if (scanned) {
        if (tid < nd) {
            before = counts[(size_t)blockIdx.x * nd + tid];
            total = counts[(size_t)gridDim.x * nd + tid];
        }
    } else {
        // kSortThreads / nd threads share a digit's runs
        const uint32_t k = tid & (nd - 1), part = tid >> bits, parts = kSortThreads >> bits;
        for (uint32_t g = part; g < gridDim.x; g += parts * 8) {
            uint32_t c[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint32_t q = g + u * parts;
                c[u] = q < gridDim.x ? counts[(size_t)q * nd + k] : 0;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                total += c[u];
                before += g + u * parts < blockIdx.x ? c[u] : 0;
            }
        }
        halves[0][tid] = total;
        halves[1][tid] = before;
    }
    for (uint32_t k = tid; k < kSortWaves * nd; k += kSortThreads) cnt[k >> bits][k & (nd - 1)] = 0;
    if (!scanned) {
        __syncthreads();
        if (tid < nd) {
            const uint32_t parts = kSortThreads >> bits;
            for (uint32_t j = 1; j < parts; ++j) {
                total += halves[0][j * nd + tid];
                before += halves[1][j * nd + tid];
            }
        } else
            total = 0;
    }
    uint32_t base = digit_prefix(total, wsum) + before;  // its barriers also publish the cleared counters

#pragma unroll
    for (int r = 0; r < ITEMS; ++r) dg[r] = (e[r].x >> shift) & (nd - 1);
    wave_ranks<ITEMS>(dg, ok, bits, cnt[w], rank);
    __syncthreads();
    if (tid < nd) {
        uint32_t c[kSortWaves];
#pragma unroll
        for (int j = 0; j < kSortWaves; ++j) c[j] = cnt[j][tid];
#pragma unroll
        for (int j = 0; j < kSortWaves; ++j) {
            cnt[j][tid] = base;
            base += c[j];
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
        if (ok[r]) out[cnt[w][dg[r]] + rank[r]] = e[r];
}

// The whole sort of up to kSortThreads * ITEMS tokens by one workgroup.
template <typename I, int ITEMS>
__global__ __launch_bounds__(kSortThreads) void k_sort_local(SortSource s, int passes, int bits, uint2 *out)
{
    __shared__ uint32_t cnt[kSortWaves][kMaxDigits];
    __shared__ uint2 sorted[kSortThreads * ITEMS];
    __shared__ uint32_t wsum[kMaxDigits / 64];
    const uint32_t nd = 1u << bits, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    uint2 e[ITEMS];
    uint32_t dg[ITEMS], rank[ITEMS];
    bool ok[ITEMS];
    const uint32_t i0 = w * 64 * ITEMS + lane;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
        const uint32_t i = i0 + r * 64;
        ok[r] = i < s.n;
        e[r] = sort_entry<I>(s, ok[r] ? i : s.n - 1);
    }
    for (int p = 0; p < passes; ++p) {
        for (uint32_t k = tid; k < kSortWaves * nd; k += kSortThreads) cnt[k >> bits][k & (nd - 1)] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ITEMS; ++r) dg[r] = (e[r].x >> (p * bits)) & (nd - 1);
        wave_ranks<ITEMS>(dg, ok, bits, cnt[w], rank);
        __syncthreads();
        uint32_t c[kSortWaves], total = 0;
        if (tid < nd) {
#pragma unroll
            for (int j = 0; j < kSortWaves; ++j) {
                c[j] = cnt[j][tid];
                total += c[j];
            }
        }
        uint32_t base = digit_prefix(total, wsum);
        if (tid < nd) {
#pragma unroll
            for (int j = 0; j < kSortWaves; ++j) {
                cnt[j][tid] = base;
                base += c[j];
            }
        }
        __syncthreads();
        const bool last = p == passes - 1;
#pragma unroll
        for (int r = 0; r < ITEMS; ++r) {
            if (!ok[r]) continue;
            const uint32_t to = cnt[w][dg[r]] + rank[r];
            if (last) out[to] = e[r];
            else sorted[to] = e[r];
        }
        if (last) break;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ITEMS; ++r)
            if (ok[r]) e[r] = sorted[i0 + r * 64];
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

// A wave handles its share in sequence, about 0.1 us a token, so a share and
// what it takes over from the next are short where there are few (65,536 tokens
// and 32,768 rows of 384 bf16: 15 us with these; 20 us with shares of 32 and
// rests of up to 31 tokens).
constexpr int kSnap = 8;
constexpr int kShareMin = 16;
// Waves of the sum kernel, 5 to a SIMD of the 6 that its registers allow.  A
// million tokens and 250,001 rows of 385: sum and join 268 + 15 us, with 8192
// 268 + 18, with 16,384 257 + 31.
constexpr int kMaxShares = 5120;
constexpr int kSumCols = 512;  // columns of a wave: 64 lanes of 16 bytes of the 16-bit types
enum { kFirstCut = 1, kInside = 2 };

// What a share leaves to the join: whether it ends a row begun before it
// (row), and whether it lies inside one row.
struct Note {
    uint32_t row, flags;
};

struct SumPlan {
    int col_blocks;
    int64_t shares, share;
};

SumPlan sum_plan(int64_t n, int64_t rows, int dim)
{
    SumPlan p;
    p.col_blocks = (dim + kSumCols - 1) / kSumCols;
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
__device__ __forceinline__ Cut find_cut(const uint2 *entries, uint32_t n, uint32_t rows, int64_t at)
{
    const int lane = threadIdx.x & 31;
    const int half = (threadIdx.x & 32);
    // least i with i + key[i] >= at, in [lo, hi]
    int64_t lo = at > rows ? at - rows : 0, hi = at < n ? at : n;
    while (__ballot(lo < hi)) {
        const int64_t step = (hi - lo + 31) >> 5;
        const int64_t i = lo + (int64_t)lane * step;
        bool less = false;
        if (lo < hi && i < hi) less = i + (int64_t)entries[i].x < at;
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
    const uint32_t j = r.i + lane;
    const uint32_t prev = entries[r.i ? r.i - 1 : 0].x, here = entries[j < n ? j : n - 1].x;
    const bool begun = r.i > 0 && r.v < rows && prev == r.v;
    const bool same = begun && j < n && here == r.v;
    const uint32_t m = (uint32_t)(__ballot(same) >> half);
    if (begun) {
        if (__popc(m) >= kSnap) r.inside = true;
        else {
            r.i += __popc(m);
            r.v += 1;
        }
    }
    return r;
}

// out[v] = scale * sum of grad[t] over the tokens of v.  Bound by memory for
// wide rows: 15.3 us for 66 MB at 65,536 x 384 bf16 (4.3 TB/s, two sets of row
// loads in flight and five waves a SIMD cover the latency), 270 us for 1.08 GB at
// 1M x 385 bf16 to f32 (4.0 TB/s; rows of 770 bytes touch a sixth more in whole
// cache lines).  Columns of a lane: NV vectors of LEN elements.  A vector that
// would pass the row's end ends with it instead; the columns it shares with its
// neighbour hold the same sums.
template <typename T, typename O, int LEN, int NV>
__global__ __launch_bounds__(kThreads) void k_embed_grad_sum(EmbedGradArgs a, const uint2 *entries,
                                                             int64_t share, uint32_t shares,
                                                             float *part, Note *notes)
{
    typedef Slot<T, LEN> In;
    typedef Slot<O, LEN> Out;
    typedef float fvec __attribute__((ext_vector_type(LEN)));
    // tokens of one set of loads, of which two are in flight: more of narrow rows
    // (1M x 32 bf16, 32,768 rows: the whole call 86 us with eight, 92 with four)
    constexpr int kAhead = LEN <= 2 ? 8 : 4 / NV;

    const int lane = threadIdx.x & 63;
    const uint32_t w = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6));
    if (w >= shares) return;
    const uint32_t n = (uint32_t)a.n, rows = (uint32_t)a.rows;
    const int64_t total = (int64_t)n + rows;

    int64_t at = (int64_t)(w + (lane >> 5)) * share;
    if (at > total) at = total;
    const Cut cut = find_cut(entries, n, rows, at);
    uint32_t i = __builtin_amdgcn_readlane(cut.i, 0), v = __builtin_amdgcn_readlane(cut.v, 0);
    const uint32_t v0 = v;
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
    uint32_t cols[NV];
    bool on[NV];  // lanes beyond the columns load and add the last vector, and write nothing
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * 64 + lane) * LEN;
        on[k] = c < block_cols;
        const int last = c0 + block_cols < a.dim ? c0 + block_cols - LEN : a.dim - LEN;
        cols[k] = (uint32_t)(c0 + c < last ? c0 + c : last);
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
                if (on[k]) Slot<float, LEN>::store(part + (uint64_t)w * 2 * a.dim + cols[k], acc[k]);
            flag |= kFirstCut;
        } else if (any || !a.accumulate) {
            O *out = (O *)a.out + (int64_t)v * a.ld_out;
            const float scale = any ? a.scale : 1.f;  // zeros stay zeros under a scale of infinity or NaN
#pragma unroll
            for (int k = 0; k < NV; ++k) acc[k] *= scale;
            if (a.accumulate) {  // all read before any is written: shifted vectors overlap
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (on[k]) acc[k] += __builtin_convertvector(Out::load(out + cols[k]), fvec);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (on[k]) Out::store(out + cols[k], __builtin_convertvector(acc[k], typename Out::vec));
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) acc[k] = (fvec)0.f;
        any = first = false;
        ++v;
    };

    while (i < i1) {
        // up to 64 tokens, one to a lane: key and place of the row of grad in bytes
        uint32_t m = i1 - i < 64 ? i1 - i : 64;
        const uint32_t mine = i + (lane < (int)m ? lane : 0);
        const uint2 e = entries[mine];
        const uint32_t kk = e.x;
        const uint64_t place = (uint64_t)e.y * (uint64_t)a.ld_grad * sizeof(T);
        const uint32_t place_lo = (uint32_t)place, place_hi = (uint32_t)(place >> 32);
        // tokens that add nothing come last
        const uint32_t real = (uint32_t)__popcll(__ballot(lane < (int)m && kk < rows));
        i = real < m ? i1 : i + m;
        m = real;
        if (m == 0) break;
        auto load = [&](uint32_t t, typename In::vec (&x)[kAhead][NV]) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const uint32_t tu = t + u < m ? t + u : m - 1;
                const char *row = (const char *)a.grad + (((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)place_hi, tu) << 32) |
                                                          (uint32_t)__builtin_amdgcn_readlane((int)place_lo, tu));
#pragma unroll
                for (int k = 0; k < NV; ++k) x[u][k] = In::load((const T *)(row + cols[k] * (uint32_t)sizeof(T)));
            }
        };
        auto add = [&](uint32_t t, const typename In::vec (&x)[kAhead][NV]) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (t + u >= m) continue;
                const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)kk, t + u);
                while (v != key) finish();
#pragma unroll
                for (int k = 0; k < NV; ++k) acc[k] += __builtin_convertvector(x[u][k], fvec);
                any = true;
            }
        };
        typename In::vec x[kAhead][NV], y[kAhead][NV];
        load(0, x);
        for (uint32_t t = 0; t < m; t += 2 * kAhead) {
            if (t + kAhead < m) load(t + kAhead, y);
            add(t, x);
            if (t + 2 * kAhead < m) load(t + 2 * kAhead, x);
            add(t + kAhead, y);
        }
    }
    while (v < v1) finish();
    if (open) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on[k]) Slot<float, LEN>::store(part + ((uint64_t)w * 2 + 1) * a.dim + cols[k], acc[k]);
        flag |= first ? kInside : 0;
    }
    if (lane == 0 && blockIdx.y == 0) notes[w] = Note{v0, flag};
}

// Rows cut over several shares: the last rows of shares b .. w - 1 and the
// first row of share w are parts of one row of the table.  A wave looks at one
// share w; where a row that was begun before ends there, it finds b and adds
// the parts in order.  More than kJoinAlone parts are added by the whole
// workgroup: its waves form groups that cover a block of columns, each group
// adds an equal stretch of the parts, and the groups' sums are added in order.
// Bound by the latency of the chain notes, parts, result: 5.9 us at 65,536 x
// 384, 15 us at 1M x 385.
constexpr int kJoinThreads = 512;
constexpr int kJoinWaves = kJoinThreads / 64;
constexpr uint32_t kJoinAlone = 16;

template <typename O>
__global__ __launch_bounds__(kJoinThreads) void k_embed_grad_join(EmbedGradArgs a, uint32_t shares,
                                                                  const float *part, const Note *notes)
{
    typedef Slot<float, 4>::vec fvec;
    __shared__ fvec sums[kJoinWaves][64];
    __shared__ uint32_t first[kJoinWaves], row[kJoinWaves], count[kJoinWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t w = blockIdx.x * kJoinWaves + wave;

    // sum of parts p0 .. p1 - 1 of the row begun in share b and ended in share e, four columns from c;
    // the loads of eight parts are in flight together, the last ones repeated where there are fewer
    auto sum = [&](uint32_t b, uint32_t e, uint32_t p0, uint32_t p1, int c) {
        fvec s = (fvec)0.f;
        if (c + 4 <= a.dim) {
            for (uint32_t p = p0; p < p1; p += 8) {
                fvec x[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const uint32_t q = b + (p + u < p1 ? p + u : p1 - 1);
                    x[u] = Slot<float, 4>::load(part + ((uint64_t)q * 2 + (q < e ? 1 : 0)) * a.dim + c);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (p + u < p1) s += x[u];
            }
        } else {
            for (uint32_t p = p0; p < p1; ++p) {
                const float *x = part + ((uint64_t)(b + p) * 2 + (b + p < e ? 1 : 0)) * a.dim + c;
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (c + k < a.dim) s[k] += x[k];
            }
        }
        return s;
    };
    auto write = [&](uint32_t v, fvec s, int c) {
        O *out = (O *)a.out + (int64_t)v * a.ld_out + c;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (c + k < a.dim) {
                float t = s[k] * a.scale;
                if (a.accumulate) t += (float)out[k];
                out[k] = (O)t;
            }
        }
    };

    uint32_t parts = 0, b = w;
    const Note note = w < shares ? notes[w] : Note{0, 0};
    // whether each of the 256 shares before b lies inside one row; for w without
    // waiting for its own note
    uint32_t inside[4];
    auto look = [&]() {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t q = (int64_t)b - 1 - 64 * k - lane;
            inside[k] = notes[q < 0 || b > shares ? 0 : q].flags & (q < 0 ? 0 : kInside);
        }
    };
    look();
    if (note.flags & kFirstCut) {
        // b: the first share before w that is not all inside the row
        for (bool more = true; more;) {
            uint64_t m[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[k] = __ballot(!inside[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (!more) continue;
                if (m[k]) {
                    b = b - 1 - (__ffsll((unsigned long long)m[k]) - 1);
                    more = false;
                } else
                    b -= 64;
            }
            if (more) look();
        }
        parts = w - b + 1;
        if (parts <= kJoinAlone)
            for (int c = lane * 4; c < a.dim; c += 256) write(note.row, sum(b, w, 0, parts, c), c);
    }
    if (lane == 0) {
        first[wave] = b;
        row[wave] = note.row;
        count[wave] = parts > kJoinAlone ? parts : 0;
    }
    __syncthreads();
    const int blocks = (a.dim + 255) / 256;  // blocks of columns, one per wave of a group
    const int across = blocks < kJoinWaves ? blocks : kJoinWaves;
    const int groups = kJoinWaves / across, group = wave / across, block = wave - group * across;
    for (int j = 0; j < kJoinWaves; ++j) {
        const uint32_t n = count[j];
        if (n == 0) continue;
        const uint32_t e = blockIdx.x * kJoinWaves + j, each = (n + groups - 1) / groups;
        const uint32_t p0 = group * each < n ? group * each : n, p1 = p0 + each < n ? p0 + each : n;
        for (int c0 = 0; c0 < blocks; c0 += across) {
            const int c = (c0 + block) * 256 + lane * 4;
            __syncthreads();
            if (group < groups && c < a.dim) sums[wave][lane] = sum(first[j], e, p0, p1, c);
            __syncthreads();
            if (group == 0 && c < a.dim) {
                fvec s = sums[wave][lane];
                for (int k = 1; k < groups; ++k) s += sums[k * across + wave][lane];
                write(row[j], s, c);
            }
        }
    }
}

// ---- few tokens -----------------------------------------------------------
//
// Up to kFewMax tokens need no sort: a workgroup owns `own` rows of the table,
// picks the tokens of its rows out of all ids, in order, into LDS, and its
// waves order them by row with ballots.  Rows of up to kFewAlone tokens are
// summed by a wave each; the tokens of a longer one are split evenly over the
// waves, whose sums are added in order.  One launch and no working memory in
// place of three kernels.  GPU time against the sort's three kernels, ids by a
// Zipf law: 16 tokens and 5000 rows of 64 f32 5.8 against 13.9 us, 512 tokens
// 7.3 against 17.1, 1024 tokens and 32,768 rows of 384 bf16 14.7 against 22.1,
// 250,000 rows of 64 32 against 32; 1024 tokens of one id and 32,768 rows 26
// against 22, and the gap widens with more tokens: hence the limit.  Of a tall
// table it writes mostly zeros, a row an instruction: 512 tokens and 250,000 rows
// of 64 f32 21 us a call, 12 at the rate of a copy.
constexpr uint32_t kFewAlone = 32;

template <typename T, typename O, typename I, int LEN, int NV>
__global__ __launch_bounds__(kFewThreads) void k_embed_grad_few(EmbedGradArgs a, int own, int64_t base)
{
    typedef Slot<T, LEN> In;
    typedef Slot<O, LEN> Out;
    typedef float fvec __attribute__((ext_vector_type(LEN)));
    constexpr int kPer = kFewMax / kFewThreads;
    constexpr int kAhead = 16 / NV;
    __shared__ uint16_t token[kFewMax], order[kFewMax];
    __shared__ uint8_t rel[kFewMax];
    __shared__ uint32_t found[kPer * kFewWaves], count[kFewRows], first[kFewRows];
    __shared__ fvec sums[kFewWaves][NV][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    const uint32_t n = (uint32_t)a.n;
    const int64_t v0 = base + (int64_t)blockIdx.x * own, v1 = v0 + own < a.rows ? v0 + own : a.rows;
    const int rows = (int)(v1 - v0);

    // the tokens of these rows, in order
    int64_t id[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const uint32_t i = k * kFewThreads + threadIdx.x;
        id[k] = i < n ? id_at<I>(a.ids, i) : -1;
    }
    uint64_t in[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const bool mine = id[k] >= v0 && id[k] < v1 && id[k] != a.padding_id;
        in[k] = __ballot(mine);
        if (lane == 0) found[k * kFewWaves + wave] = (uint32_t)__popcll(in[k]);
    }
    __syncthreads();
    uint32_t total = 0, at[kPer];
#pragma unroll
    for (int j = 0; j < kPer * kFewWaves; ++j) {
        if ((j & (kFewWaves - 1)) == wave) at[j / kFewWaves] = total;
        total += found[j];
    }
    total = __builtin_amdgcn_readfirstlane(total);

    // columns of the lanes, as in k_embed_grad_sum
    const int vecs = (a.dim + LEN - 1) / LEN;
    const int c0 = (int)((int64_t)blockIdx.y * vecs / gridDim.y) * LEN;
    const int block_cols = (int)((int64_t)(blockIdx.y + 1) * vecs / gridDim.y) * LEN - c0;
    uint32_t cols[NV];
    bool on[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * 64 + lane) * LEN;
        on[k] = c < block_cols;
        const int last = c0 + block_cols < a.dim ? c0 + block_cols - LEN : a.dim - LEN;
        cols[k] = (uint32_t)(c0 + c < last ? c0 + c : last);
    }
    auto write = [&](int r, bool any, fvec (&acc)[NV]) {
        O *out = (O *)a.out + (v0 + r) * a.ld_out;
        const float scale = any ? a.scale : 1.f;  // zeros stay zeros under a scale of infinity or NaN
#pragma unroll
        for (int k = 0; k < NV; ++k) acc[k] *= scale;
        if (a.accumulate) {  // all read before any is written: shifted vectors overlap
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (on[k]) acc[k] += __builtin_convertvector(Out::load(out + cols[k]), fvec);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on[k]) Out::store(out + cols[k], __builtin_convertvector(acc[k], typename Out::vec));
    };
    fvec acc[NV];
    if (total == 0) {
        if (a.accumulate) return;
        for (int r = wave; r < rows; r += kFewWaves) {
#pragma unroll
            for (int k = 0; k < NV; ++k) acc[k] = (fvec)0.f;
            write(r, false, acc);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (in[k] >> lane & 1) {
            const uint32_t to = at[k] + (uint32_t)__popcll(in[k] & below);
            token[to] = (uint16_t)(k * kFewThreads + threadIdx.x);
            rel[to] = (uint8_t)(id[k] - v0);
        }
    }
    __syncthreads();

    // each row's tokens side by side, in order: counts, their prefix, places
    constexpr int kChunks = kFewMax / 64;
    const int chunks = (int)(total + 63) / 64;
    uint32_t to[kChunks];  // row of each of the lane's tokens, 64 j + lane
#pragma unroll
    for (int j = 0; j < kChunks; ++j) to[j] = j * 64 + lane < (int)total ? rel[j * 64 + lane] : kFewRows;
    for (int r = wave; r < rows; r += kFewWaves) {
        uint32_t c = 0;
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
            if (j < chunks) c += (uint32_t)__popcll(__ballot(to[j] == (uint32_t)r));
        if (lane == 0) count[r] = c;
    }
    __syncthreads();
    if (wave == 0) {
        const uint32_t c = lane < rows ? count[lane] : 0;
        uint32_t inc = c;
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t u = __shfl_up(inc, o, 64);
            if (lane >= o) inc += u;
        }
        if (lane < rows) first[lane] = inc - c;
    }
    __syncthreads();
    for (int r = wave; r < rows; r += kFewWaves) {
        uint32_t p = first[r];
        if (count[r] == 0) continue;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            if (j >= chunks) continue;
            const uint64_t m = __ballot(to[j] == (uint32_t)r);
            if (to[j] == (uint32_t)r) order[p + (uint32_t)__popcll(m & below)] = token[j * 64 + lane];
            p += (uint32_t)__popcll(m);
        }
    }
    __syncthreads();

    auto sum = [&](uint32_t p0, uint32_t p1, fvec (&acc)[NV]) {
#pragma unroll
        for (int k = 0; k < NV; ++k) acc[k] = (fvec)0.f;
        for (uint32_t p = p0; p < p1; p += kAhead) {
            typename In::vec x[kAhead][NV];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const uint32_t t = __builtin_amdgcn_readfirstlane(order[p + u < p1 ? p + u : p1 - 1]);
                const T *row = (const T *)a.grad + (int64_t)t * a.ld_grad;
#pragma unroll
                for (int k = 0; k < NV; ++k) x[u][k] = In::load(row + cols[k]);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (p + u >= p1) continue;
#pragma unroll
                for (int k = 0; k < NV; ++k) acc[k] += __builtin_convertvector(x[u][k], fvec);
            }
        }
    };
    for (int r = wave; r < rows; r += kFewWaves) {
        const uint32_t c = __builtin_amdgcn_readfirstlane(count[r]), p = __builtin_amdgcn_readfirstlane(first[r]);
        if (c > kFewAlone || (c == 0 && a.accumulate)) continue;
        sum(p, p + c, acc);
        write(r, c > 0, acc);
    }
    if (total <= kFewAlone) return;
    for (int r = 0; r < rows; ++r) {  // the same for all waves
        const uint32_t c = __builtin_amdgcn_readfirstlane(count[r]), p = __builtin_amdgcn_readfirstlane(first[r]);
        if (c <= kFewAlone) continue;
        sum(p + c * wave / kFewWaves, p + c * (wave + 1) / kFewWaves, acc);
#pragma unroll
        for (int k = 0; k < NV; ++k) sums[wave][k][lane] = acc[k];
        __syncthreads();
        if (wave == (r & (kFewWaves - 1))) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                acc[k] = sums[0][k][lane];
                for (int j = 1; j < kFewWaves; ++j) acc[k] += sums[j][k][lane];
            }
            write(r, true, acc);
        }
        __syncthreads();
    }
}

uint64_t up256(uint64_t b) { return (b + 255) & ~(uint64_t)255; }

}  // namespace

constexpr int kEmbedBlocks = 2048;  // 8 workgroups to each CU

template <typename T, typename O, typename I>
static void run_embed(const EmbedArgs &a, hipStream_t s)
{
    // the smallest team of at least eight lanes (fewer where the row has fewer
    // vectors) that covers the row with up to four vectors a lane; longer rows
    // are split over the grid's second axis
    constexpr int kLen = 16 / sizeof(O);
    const int len = a.dim < kLen ? 1 : kLen;
    const int vecs = (a.dim + len - 1) / len;
    int lanes = 1;
    while (lanes < 8 && lanes < vecs) lanes *= 2;
    while (lanes < 64 && lanes * 4 < vecs) lanes *= 2;
    const int nv = (vecs + lanes - 1) / lanes;
    const int64_t need = (a.n + kThreads / lanes - 1) / (kThreads / lanes);
    const dim3 grid((unsigned)(need < kEmbedBlocks ? need : kEmbedBlocks), nv > 4 ? (unsigned)((nv + 3) / 4) : 1u);
    const dim3 block(kThreads);
#define CASE(L, NV)                                                     \
    case L * 8 + NV:                                                    \
        k_embed<T, O, I, kLen, L, NV><<<grid, block, 0, s>>>(a);        \
        break;
    if (len == 1) {
        switch (lanes) {
        case 1: k_embed<T, O, I, 1, 1, 1><<<grid, block, 0, s>>>(a); return;
        case 2: k_embed<T, O, I, 1, 2, 1><<<grid, block, 0, s>>>(a); return;
        case 4: k_embed<T, O, I, 1, 4, 1><<<grid, block, 0, s>>>(a); return;
        default: k_embed<T, O, I, 1, 8, 1><<<grid, block, 0, s>>>(a); return;
        }
    }
    switch (lanes * 8 + (nv < 4 ? nv : 4)) {
        CASE(1, 1) CASE(2, 1) CASE(4, 1) CASE(8, 1) CASE(8, 2) CASE(8, 3) CASE(8, 4) CASE(16, 3) CASE(16, 4) CASE(32, 3) CASE(32, 4) CASE(64, 3)
        CASE(64, 4)
    }
#undef CASE
}

hipError_t launch_embed(const EmbedArgs &a, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
#define RUN(T, O)                                      \
    do {                                               \
        if (a.id_type) run_embed<T, O, int64_t>(a, s); \
        else run_embed<T, O, int32_t>(a, s);           \
    } while (0)
    switch (a.table_type * 4 + a.out_type) {
    case kF32 * 4 + kF32: RUN(float, float); break;
    case kF32 * 4 + kF16: RUN(float, f16_t); break;
    case kF32 * 4 + kBF16: RUN(float, bf16_t); break;
    case kF16 * 4 + kF16: RUN(f16_t, f16_t); break;
    default: RUN(bf16_t, bf16_t); break;
    }
#undef RUN
    return hipGetLastError();
}

static uint64_t count_bytes(const SortPlan &p) { return up256(((uint64_t)4 << p.bits) * (uint64_t)(p.runs + 1)); }

uint64_t embed_grad_work(int64_t n, int64_t rows, int dim)
{
    const SortPlan p = sort_plan(n, rows);
    if (n <= kFewMax) return 0;
    const SumPlan q = sum_plan(n, rows, dim);
    return 2 * up256(8 * (uint64_t)n) + count_bytes(p) + up256(q.shares * sizeof(Note)) +
           (uint64_t)q.shares * 2 * 4 * (uint64_t)dim;
}

template <typename I, int ITEMS>
static void launch_sort_pass(const SortPlan &p, const SortSource &src, int shift, uint32_t *counts, uint2 *out,
                             hipStream_t s)
{
    const dim3 grid((unsigned)p.runs), block(kSortThreads);
    const bool scan = p.runs > kScanRuns;
    k_sort_count<I, ITEMS><<<grid, block, 0, s>>>(src, shift, p.bits, counts);
    if (scan)
        k_sort_scan<<<dim3(((1u << p.bits) + kWaves - 1) / kWaves), dim3(kThreads), 0, s>>>(counts, (uint32_t)p.runs,
                                                                                           p.bits);
    k_sort_scatter<I, ITEMS><<<grid, block, 0, s>>>(src, shift, p.bits, counts, scan, out);
}

template <typename I>
static void launch_sort(const SortPlan &p, SortSource &src, uint2 *const (&buf)[2], uint32_t *counts, hipStream_t s)
{
    if (src.n <= (uint32_t)kLocalMax) {
        k_sort_local<I, kLocalMax / kSortThreads><<<dim3(1), dim3(kSortThreads), 0, s>>>(src, p.passes, p.bits, buf[0]);
        src.entries = buf[0];
        return;
    }
    for (int k = 0; k < p.passes; ++k) {
        uint2 *out = buf[k & 1];
        if (p.items == 1) launch_sort_pass<I, 1>(p, src, k * p.bits, counts, out, s);
        else if (p.items == 2) launch_sort_pass<I, 2>(p, src, k * p.bits, counts, out, s);
        else launch_sort_pass<I, 4>(p, src, k * p.bits, counts, out, s);
        src.entries = out;
    }
}

template <typename T, typename O, int LEN, int NV>
static void launch_few(const EmbedGradArgs &a, int col_blocks, hipStream_t s)
{
    const FewPlan p = few_plan(a.rows);
    for (int64_t v = 0; v < a.rows; v += p.step) {
        const dim3 grid(few_groups(p, a.rows, v), col_blocks), block(kFewThreads);
        if (a.id_type) k_embed_grad_few<T, O, int64_t, LEN, NV><<<grid, block, 0, s>>>(a, p.own, v);
        else k_embed_grad_few<T, O, int32_t, LEN, NV><<<grid, block, 0, s>>>(a, p.own, v);
    }
}

template <typename T, typename O, int LEN, int NV>
static void launch_sum_of(const EmbedGradArgs &a, const uint2 *entries, const SumPlan &q, float *part, Note *notes,
                          hipStream_t s)
{
    if (a.n <= kFewMax) {
        launch_few<T, O, LEN, NV>(a, q.col_blocks, s);
        return;
    }
    const dim3 grid((unsigned)((q.shares + kWaves - 1) / kWaves), q.col_blocks), block(kThreads);
    k_embed_grad_sum<T, O, LEN, NV><<<grid, block, 0, s>>>(a, entries, q.share, (uint32_t)q.shares, part, notes);
    k_embed_grad_join<O><<<dim3((unsigned)((q.shares + kJoinWaves - 1) / kJoinWaves)), dim3(kJoinThreads), 0, s>>>(
        a, (uint32_t)q.shares, part, notes);
}

// Narrow rows are spread over all lanes: a token costs the wave as many
// additions as a lane has columns.
template <typename T, typename O>
static void launch_sum(const EmbedGradArgs &a, const uint2 *entries, const SumPlan &q, float *part, Note *notes,
                       hipStream_t s)
{
    if (a.dim <= 64) launch_sum_of<T, O, 1, 1>(a, entries, q, part, notes, s);
    else if (a.dim <= 128) launch_sum_of<T, O, 2, 1>(a, entries, q, part, notes, s);
    else if (a.dim <= 256) launch_sum_of<T, O, 4, 1>(a, entries, q, part, notes, s);
    else if constexpr (sizeof(T) == 4) launch_sum_of<T, O, 4, 2>(a, entries, q, part, notes, s);
    else launch_sum_of<T, O, 8, 1>(a, entries, q, part, notes, s);
}

hipError_t launch_embed_grad(const EmbedGradArgs &a, hipStream_t s)
{
    const SortPlan p = sort_plan(a.n, a.rows);
    char *at = (char *)a.work;
    uint2 *buf[2];
    for (int k = 0; k < 2; ++k, at += up256(8 * (uint64_t)a.n)) buf[k] = (uint2 *)at;
    uint32_t *counts = (uint32_t *)at;
    at += count_bytes(p);
    SortSource src{a.ids, nullptr, a.padding_id, a.rows, (uint32_t)a.n};
    if (a.n > kFewMax) {
        if (a.id_type) launch_sort<int64_t>(p, src, buf, counts, s);
        else launch_sort<int32_t>(p, src, buf, counts, s);
    }
    const SumPlan q = sum_plan(a.n, a.rows, a.dim);
    Note *notes = (Note *)at;
    float *part = (float *)(at + up256(q.shares * sizeof(Note)));
    switch (a.grad_type * 4 + a.out_type) {
    case kF32 * 4 + kF32: launch_sum<float, float>(a, src.entries, q, part, notes, s); break;
    case kF16 * 4 + kF32: launch_sum<f16_t, float>(a, src.entries, q, part, notes, s); break;
    case kBF16 * 4 + kF32: launch_sum<bf16_t, float>(a, src.entries, q, part, notes, s); break;
    case kF16 * 4 + kF16: launch_sum<f16_t, f16_t>(a, src.entries, q, part, notes, s); break;
    default: launch_sum<bf16_t, bf16_t>(a, src.entries, q, part, notes, s); break;
    }
    return hipGetLastError();
}

}  // namespace ersj
