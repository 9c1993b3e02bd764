// C ABI of the encoder operators (see include/ersj_encoder.h): argument
// validation, and the chunks of a set of gradients.
#include "ersj_encoder.h"
#include "encoder_internal.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <vector>

using namespace ersj;

static_assert(ERSJ_F32 == kF32 && ERSJ_F16 == kF16 && ERSJ_BF16 == kBF16, "element types");
static_assert(kGradParts * sizeof(double) == ERSJ_GRADS_WORK, "working memory of ersj_grads_clip");

struct ersj_grads {
    int device = 0;
    GradChunk *chunks = nullptr;  // device
    uint32_t n_chunks = 0;
    size_t bytes = 0;
};

namespace {

int refuse(const char *fmt, ...)
{
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return set_error(ERSJ_ERR_INVALID_ARG, buf);
}

int done(hipError_t e, const char *what)
{
    if (e == hipSuccess) return ERSJ_OK;
    (void)hipGetLastError();
    char buf[256];
    snprintf(buf, sizeof buf, "%s: %s", what, hipGetErrorString(e));
    return set_error(e == hipErrorOutOfMemory ? ERSJ_ERR_OOM : ERSJ_ERR_HIP, buf);
}

bool is_type(int32_t t) { return t == ERSJ_F32 || t == ERSJ_F16 || t == ERSJ_BF16; }

bool aligned(const void *p, size_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;

int check_rows(int64_t n, int32_t dim)
{
    if (n < 0 || n > kMaxRows) return refuse("n = %lld: must be in [0, 2^31)", (long long)n);
    if (dim < 1 || dim > ERSJ_ENCODER_MAX_DIM)
        return refuse("dim = %d: must be in [1, %d]", dim, ERSJ_ENCODER_MAX_DIM);
    return ERSJ_OK;
}

int check_tensor(const void *p, int32_t type, int64_t ld, int32_t dim, bool used, const char *what)
{
    if (!is_type(type)) return refuse("%s: unknown element type %d", what, type);
    if (ld < dim) return refuse("%s: row spacing %lld is below dim = %d", what, (long long)ld, dim);
    if (ld > (int64_t)1 << 40) return refuse("%s: row spacing %lld is out of range", what, (long long)ld);
    if (used && !p) return refuse("%s is NULL", what);
    if (!aligned(p, elem_size(type))) return refuse("%s is not aligned to its element size", what);
    return ERSJ_OK;
}

int check_ids(const void *ids, int32_t type, int64_t n, int64_t rows)
{
    if (type != ERSJ_I32 && type != ERSJ_I64) return refuse("ids: unknown id type %d", type);
    if (n > 0 && !ids) return refuse("ids is NULL");
    if (!aligned(ids, type == ERSJ_I64 ? 8 : 4)) return refuse("ids is not aligned to its element size");
    if (rows < 1 || rows >= kMaxRows) return refuse("rows = %lld: must be in [1, 2^31 - 1)", (long long)rows);
    return ERSJ_OK;
}

int check_work(const void *work, uint64_t have, uint64_t need, size_t align)
{
    if (have < need)
        return refuse("working memory of %llu bytes, %llu are needed", (unsigned long long)have,
                      (unsigned long long)need);
    if (need && !work) return refuse("d_work is NULL");
    if (!aligned(work, align)) return refuse("d_work is not aligned to %zu bytes", align);
    return ERSJ_OK;
}

#define TRY(expr)                       \
    do {                                \
        int r__ = (expr);               \
        if (r__ != ERSJ_OK) return r__; \
    } while (0)

int check_clip(float max_norm, const float *d_norm, const void *d_work, uint64_t have, uint64_t need)
{
    if (!(max_norm >= 0.f)) return refuse("max_norm = %g: must not be negative", (double)max_norm);
    if (!aligned(d_norm, 4)) return refuse("d_norm is not aligned to 4 bytes");
    return check_work(d_work, have, need, 8);
}

// Whether memory that is written for one tensor is read or written for another
// as well, or for the same one at another place.
bool shared_memory(int32_t count, const void *const *d_grad, void *const *d_out, const int64_t *size,
                   const int32_t *type)
{
    struct Range {
        uintptr_t first, end;
        bool operator<(const Range &r) const { return first < r.first; }
    };
    auto range = [&](const void *p, int32_t i) {
        return Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)size[i] * elem_size(type[i])};
    };
    std::vector<Range> written;
    written.reserve(count);
    for (int32_t i = 0; i < count; ++i)
        if (size[i]) written.push_back(range(d_out ? d_out[i] : d_grad[i], i));
    if (!std::is_sorted(written.begin(), written.end())) std::sort(written.begin(), written.end());
    for (size_t k = 1; k < written.size(); ++k)
        if (written[k].first < written[k - 1].end) return true;
    for (int32_t i = 0; d_out && i < count; ++i) {
        if (!size[i] || d_out[i] == d_grad[i]) continue;
        const Range in = range(d_grad[i], i);
        // the last range that begins before the input's end
        auto at = std::lower_bound(written.begin(), written.end(), Range{in.end, 0});
        if (at != written.begin() && (at - 1)->end > in.first) return true;
    }
    return false;
}

int check_shared_memory(int32_t count, const void *const *d_grad, void *const *d_out, const int64_t *size,
                        const int32_t *type)
{
    try {
        if (shared_memory(count, d_grad, d_out, size, type))
            return refuse("tensors share memory that is written");
    } catch (const std::exception &) {
        return set_error(ERSJ_ERR_OOM, "host memory for the check of a set of gradients");
    }
    return ERSJ_OK;
}

// Checks the tensors of a set; *total: how many chunks they have.
int check_grads(int32_t count, const void *const *d_grad, void *const *d_out, const int64_t *size,
                const int32_t *type, uint32_t *total)
{
    if (count < 1 || count > 65536) return refuse("count = %d: must be in [1, 65536]", count);
    if (!d_grad || !size || !type) return refuse("d_grad, size or type is NULL");
    uint64_t chunks = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (!is_type(type[i])) return refuse("tensor %d: unknown element type %d", i, type[i]);
        if (size[i] < 0 || size[i] > (int64_t)1 << 40)
            return refuse("tensor %d: size %lld is out of range", i, (long long)size[i]);
        if (size[i] == 0) continue;
        if (!d_grad[i] || (d_out && !d_out[i])) return refuse("tensor %d is NULL", i);
        if (!aligned(d_grad[i], elem_size(type[i])) || (d_out && !aligned(d_out[i], elem_size(type[i]))))
            return refuse("tensor %d is not aligned to its element size", i);
        const int64_t first = first_chunk(d_grad[i], type[i]), step = kGradChunkBytes / elem_size(type[i]);
        chunks += 1 + (size[i] > first ? (uint64_t)((size[i] - first + step - 1) / step) : 0);
    }
    // half a terabyte, more than the memory of any one device
    if (chunks > ((uint64_t)1 << 24)) return refuse("the tensors hold too many elements");
    *total = (uint32_t)chunks;
    return ERSJ_OK;
}

// Enqueues the kernels that write the chunks of tensors that check_grads passed.
hipError_t write_chunks(int32_t count, const void *const *d_grad, void *const *d_out, const int64_t *size,
                        const int32_t *type, GradChunk *chunks, hipStream_t stream)
{
    GradTensors t;
    t.count = 0;
    t.end = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (size[i]) {
            const int64_t first = first_chunk(d_grad[i], type[i]), step = kGradChunkBytes / elem_size(type[i]);
            t.t[t.count++] = GradTensor{d_grad[i], d_out ? d_out[i] : const_cast<void *>(d_grad[i]), size[i], type[i],
                                        t.end};
            t.end += 1 + (size[i] > first ? (uint32_t)((size[i] - first + step - 1) / step) : 0);
        }
        if (t.count == kGradTensors || (i == count - 1 && t.count)) {
            const hipError_t e = launch_grads_table(t, chunks, stream);
            if (e != hipSuccess) return e;
            t.count = 0;
        }
    }
    return hipSuccess;
}

}  // namespace

extern "C" {

int ersj_embed(const void *d_table, int32_t table_type, int64_t rows, int32_t dim, int64_t ld_table,
               const void *d_ids, int32_t id_type, int64_t n, float scale, int64_t padding_id, void *d_out,
               int32_t out_type, int64_t ld_out, void *stream)
{
    TRY(check_rows(n, dim));
    TRY(check_tensor(d_table, table_type, ld_table, dim, true, "table"));
    TRY(check_ids(d_ids, id_type, n, rows));
    TRY(check_tensor(d_out, out_type, ld_out, dim, n > 0, "out"));
    if (table_type != ERSJ_F32 && out_type != table_type)
        return refuse("out: a table of 16 bits gives rows of its own type");
    if (padding_id < -1) return refuse("padding_id = %lld: must be an id or -1", (long long)padding_id);
    const EmbedArgs a{d_table, table_type, rows, ld_table, dim, d_ids, id_type, n, scale, padding_id, d_out, out_type,
                      ld_out};
    return done(launch_embed(a, (hipStream_t)stream), "embed kernel");
}

uint64_t ersj_embed_grad_work(int64_t n, int64_t rows, int32_t dim)
{
    if (n < 0 || n > kMaxRows || rows < 1 || rows >= kMaxRows || dim < 1 || dim > ERSJ_ENCODER_MAX_DIM) return 0;
    return embed_grad_work(n, rows, dim);
}

int ersj_embed_grad(const void *d_grad, int32_t grad_type, int64_t ld_grad, const void *d_ids, int32_t id_type,
                    int64_t n, float scale, int64_t padding_id, void *d_out, int32_t out_type, int64_t rows,
                    int32_t dim, int64_t ld_out, int32_t accumulate, void *d_work, uint64_t d_work_bytes,
                    void *stream)
{
    TRY(check_rows(n, dim));
    TRY(check_tensor(d_grad, grad_type, ld_grad, dim, n > 0, "grad"));
    TRY(check_ids(d_ids, id_type, n, rows));
    TRY(check_tensor(d_out, out_type, ld_out, dim, true, "out"));
    if (out_type != ERSJ_F32 && out_type != grad_type)
        return refuse("out: must have the type of grad or 32 bits");
    if (padding_id < -1) return refuse("padding_id = %lld: must be an id or -1", (long long)padding_id);
    TRY(check_work(d_work, d_work_bytes, embed_grad_work(n, rows, dim), 256));
    const EmbedGradArgs a{d_grad, grad_type, ld_grad, d_ids, id_type, n, scale, padding_id, d_out, out_type, rows,
                          dim, ld_out, accumulate, d_work};
    return done(launch_embed_grad(a, (hipStream_t)stream), "embed gradient kernels");
}

int ersj_layer_norm(const void *d_x, int32_t type, int64_t n, int32_t dim, int64_t ld_x, const void *d_weight,
                    const void *d_bias, int32_t param_type, float eps, void *d_y, int64_t ld_y, float *d_mean,
                    float *d_rstd, void *stream)
{
    TRY(check_rows(n, dim));
    TRY(check_tensor(d_x, type, ld_x, dim, n > 0, "x"));
    TRY(check_tensor(d_y, type, ld_y, dim, n > 0, "y"));
    TRY(check_tensor(d_weight, param_type, dim, dim, false, "weight"));
    TRY(check_tensor(d_bias, param_type, dim, dim, false, "bias"));
    if (param_type != ERSJ_F32 && param_type != type)
        return refuse("weight and bias must have the type of x or 32 bits");
    if (!(eps >= 0.f) || std::isinf(eps)) return refuse("eps = %g: must be finite and not negative", (double)eps);
    if (d_y == d_x && ld_y != ld_x) return refuse("y: in place, its row spacing must be that of x");
    if (!aligned(d_mean, 4) || !aligned(d_rstd, 4)) return refuse("mean and rstd must be aligned to 4 bytes");
    const NormArgs a{d_x, type, n, dim, ld_x, d_weight, d_bias, param_type, eps, d_y, ld_y, d_mean, d_rstd};
    return done(launch_layer_norm(a, (hipStream_t)stream), "layer norm kernel");
}

uint64_t ersj_layer_norm_grad_work(int64_t n, int32_t dim)
{
    if (n < 0 || n > kMaxRows || dim < 1 || dim > ERSJ_ENCODER_MAX_DIM) return 0;
    return layer_norm_grad_work(n, dim);
}

int ersj_layer_norm_grad(const void *d_grad_y, int64_t ld_grad_y, const void *d_x, int64_t ld_x, int32_t type,
                         int64_t n, int32_t dim, const float *d_mean, const float *d_rstd, const void *d_weight,
                         int32_t param_type, void *d_grad_x, int64_t ld_grad_x, void *d_grad_weight,
                         void *d_grad_bias, void *d_work, uint64_t d_work_bytes, void *stream)
{
    TRY(check_rows(n, dim));
    TRY(check_tensor(d_grad_y, type, ld_grad_y, dim, n > 0, "grad_y"));
    TRY(check_tensor(d_x, type, ld_x, dim, n > 0, "x"));
    TRY(check_tensor(d_grad_x, type, ld_grad_x, dim, false, "grad_x"));
    TRY(check_tensor(d_weight, param_type, dim, dim, false, "weight"));
    TRY(check_tensor(d_grad_weight, param_type, dim, dim, false, "grad_weight"));
    TRY(check_tensor(d_grad_bias, param_type, dim, dim, false, "grad_bias"));
    if (param_type != ERSJ_F32 && param_type != type)
        return refuse("weight and its gradients must have the type of x or 32 bits");
    if (n > 0 && (!d_mean || !d_rstd)) return refuse("mean or rstd is NULL");
    if (!aligned(d_mean, 4) || !aligned(d_rstd, 4)) return refuse("mean and rstd must be aligned to 4 bytes");
    if ((d_grad_x == d_grad_y && ld_grad_x != ld_grad_y && d_grad_x) ||
        (d_grad_x == d_x && ld_grad_x != ld_x && d_grad_x))
        return refuse("grad_x: in place, its row spacing must be that of the tensor it replaces");
    if (d_grad_weight || d_grad_bias) TRY(check_work(d_work, d_work_bytes, layer_norm_grad_work(n, dim), 256));
    const NormGradArgs a{d_grad_y, ld_grad_y, d_x, ld_x, type, n, dim, d_mean, d_rstd, d_weight, param_type,
                         d_grad_x, ld_grad_x, d_grad_weight, d_grad_bias, d_work};
    return done(launch_layer_norm_grad(a, (hipStream_t)stream), "layer norm gradient kernels");
}

int ersj_grads_create(int32_t count, const void *const *d_grad, void *const *d_out, const int64_t *size,
                      const int32_t *type, void *stream, ersj_grads **out)
{
    if (!out) return refuse("out is NULL");
    *out = nullptr;
    uint32_t total = 0;
    TRY(check_grads(count, d_grad, d_out, size, type, &total));
    try {
        ersj_grads *h = new ersj_grads;
        h->n_chunks = total;
        h->bytes = total * sizeof(GradChunk);
        int r = ERSJ_OK;
        if (total) {
            r = done(hipGetDevice(&h->device), "hipGetDevice");
            if (r == ERSJ_OK) r = check_shared_memory(count, d_grad, d_out, size, type);
            if (r == ERSJ_OK) {
                void *p = nullptr;
                r = done(device_block_get(h->device, h->bytes, &p), "table of a set of gradients");
                h->chunks = (GradChunk *)p;
            }
            if (r == ERSJ_OK)
                r = done(write_chunks(count, d_grad, d_out, size, type, h->chunks, (hipStream_t)stream),
                         "table of a set of gradients");
            if (r == ERSJ_OK) r = done(hipStreamSynchronize((hipStream_t)stream), "table of a set of gradients");
        }
        if (r != ERSJ_OK) {
            ersj_grads_free(h);
            return r;
        }
        *out = h;
        return ERSJ_OK;
    } catch (const std::exception &) {
        return set_error(ERSJ_ERR_OOM, "host memory for a set of gradients");
    }
}

int ersj_grads_clip(const ersj_grads *h, float max_norm, float *d_norm, void *d_work, uint64_t d_work_bytes,
                    void *stream)
{
    if (!h) return refuse("handle is NULL");
    TRY(check_clip(max_norm, d_norm, d_work, d_work_bytes, ERSJ_GRADS_WORK));
    return done(launch_grads_clip(h->chunks, h->n_chunks, max_norm, d_norm, d_work, (hipStream_t)stream),
                "gradient clipping kernels");
}

uint64_t ersj_clip_tensors_work(int32_t count, const int64_t *size, const int32_t *type)
{
    if (count < 1 || count > 65536 || !size || !type) return 0;
    uint64_t chunks = 0;  // the most that the tensors have at any alignment
    for (int32_t i = 0; i < count; ++i) {
        if (!is_type(type[i]) || size[i] < 0 || size[i] > (int64_t)1 << 40) return 0;
        if (size[i]) chunks += 2 + (uint64_t)size[i] * elem_size(type[i]) / kGradChunkBytes;
    }
    return ERSJ_GRADS_WORK + chunks * sizeof(GradChunk);
}

int ersj_clip_tensors(int32_t count, const void *const *d_grad, void *const *d_out, const int64_t *size,
                      const int32_t *type, float max_norm, float *d_norm, void *d_work, uint64_t d_work_bytes,
                      void *stream)
{
    uint32_t total = 0;
    TRY(check_grads(count, d_grad, d_out, size, type, &total));
    TRY(check_clip(max_norm, d_norm, d_work, d_work_bytes, ersj_clip_tensors_work(count, size, type)));
    TRY(check_shared_memory(count, d_grad, d_out, size, type));
    GradChunk *chunks = (GradChunk *)((char *)d_work + ERSJ_GRADS_WORK);
    TRY(done(write_chunks(count, d_grad, d_out, size, type, chunks, (hipStream_t)stream), "table of gradients"));
    return done(launch_grads_clip(chunks, total, max_norm, d_norm, d_work, (hipStream_t)stream),
                "gradient clipping kernels");
}

void ersj_grads_free(ersj_grads *h)
{
    if (!h) return;
    if (h->chunks) {
        try {
            device_block_put(h->device, h->chunks, h->bytes);
        } catch (...) {  // no host memory for the pool's entry
            (void)hipFree(h->chunks);
        }
    }
    delete h;
}

}  // extern "C"
