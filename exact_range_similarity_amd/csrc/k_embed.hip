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

__device__ __forceinline__ uint32_t lower_bound(const uint32_t *keys, uint32_t n, uint32_t v)
{
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
        const uint32_t mid = lo + ((hi - lo) >> 1);
        if (keys[mid] < v) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// One wave per row of the table.
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void k_embed_grad_rows(EmbedGradArgs a, const uint32_t *keys,
                                                              const uint32_t *pos)
{
    const int lane = threadIdx.x & 63;
    const int64_t v = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (v >= a.rows) return;
    const uint32_t b = lower_bound(keys, (uint32_t)a.n, (uint32_t)v);
    const uint32_t e = lower_bound(keys, (uint32_t)a.n, (uint32_t)v + 1);
    if (a.accumulate && b == e) return;
    O *out = (O *)a.out + v * a.ld_out;
    for (int c = lane; c < a.dim; c += 64) {
        float sum = 0.f;
        for (uint32_t i = b; i < e; ++i) sum += (float)((const T *)a.grad)[(int64_t)pos[i] * a.ld_grad + c];
        float r = sum * a.scale;
        if (a.accumulate) r += (float)out[c];
        out[c] = (O)r;
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

uint64_t embed_grad_work(int64_t n, int64_t rows, int)
{
    const SortPlan p = sort_plan(n, rows);
    return 4 * up256(4 * (uint64_t)n) + up256(((uint64_t)4 << p.bits) * (uint64_t)p.runs);
}

hipError_t launch_embed_grad(const EmbedGradArgs &a, hipStream_t s)
{
    const SortPlan p = sort_plan(a.n, a.rows);
    char *at = (char *)a.work;
    uint32_t *buf[4];
    for (int k = 0; k < 4; ++k, at += up256(4 * (uint64_t)a.n)) buf[k] = (uint32_t *)at;
    uint32_t *counts = (uint32_t *)at;
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
    const dim3 grid((unsigned)((a.rows + kWaves - 1) / kWaves)), block(kThreads);
    ERSJ_ELEM_SWITCH(a.grad_type, T, ERSJ_ELEM_SWITCH(a.out_type, O,
        k_embed_grad_rows<T, O><<<grid, block, 0, s>>>(a, src.keys, src.pos)))
    return hipGetLastError();
}

}  // namespace ersj
