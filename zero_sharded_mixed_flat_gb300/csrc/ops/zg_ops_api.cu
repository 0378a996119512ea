// zg_ops_api.cu -- the C ABI of the training operators (include/zg.h):
// argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <new>
#include <vector>

#include "zg.h"
#include "zg_launch.h"
#include "zg_ops.h"

struct zg_scan {
    int device;
    int64_t batch, tokens, channels;
    int64_t record_bytes;
    char *d_mem;  // ctl (8 bytes), status and gave_up (4 bytes each), and from kHead on the records
    long long wait_limit;
};

struct zg_grads {
    int device;
    int64_t parts;
    zg::GradPart *d_parts;
};

namespace {

int fail(int code, const char *fmt, ...)
{
    char msg[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return zg::report_error(code, msg);
}

int finish(cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return ZG_OK;
    return fail(ZG_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

// A call's body. The pointer checks and the launch helpers keep what they know in
// containers, whose allocations may throw: nothing of that crosses the C ABI.
template <class Body>
int guarded(Body body)
{
    try {
        return body();
    } catch (...) {
        return fail(ZG_ERR_NO_MEMORY, "host allocation failed");
    }
}

int element_size(int dtype) { return dtype == ZG_DTYPE_BF16 ? 2 : 4; }

int check_dtype(int dtype, const char *what)
{
    if (dtype == ZG_DTYPE_BF16 || dtype == ZG_DTYPE_F32) return ZG_OK;
    return fail(ZG_ERR_INVALID_ARG, "%s must be ZG_DTYPE_BF16 or ZG_DTYPE_F32 (got %d)", what, dtype);
}

// Device memory aligned to `align` bytes; NULL only where `optional`.
int check_ptr(const void *p, int align, bool optional, const char *what)
{
    if (!p) return optional ? ZG_OK : fail(ZG_ERR_INVALID_ARG, "%s is NULL", what);
    if (reinterpret_cast<uintptr_t>(p) % align) return fail(ZG_ERR_MISALIGNED, "%s is not %d-byte aligned", what, align);
    return zg::check_memory(p, false, what);
}

// ------------------------------------------------------------------ scan

constexpr int64_t kFar = int64_t(1) << 60;  // strides and extents stay below this
constexpr int64_t kHead = 256;
constexpr long long kScanWaitLimit = 4000000;

zg::ScanWork work_of(const zg_scan *s)
{
    return zg::ScanWork{reinterpret_cast<unsigned long long *>(s->d_mem), reinterpret_cast<int *>(s->d_mem + 8),
                        reinterpret_cast<uint32_t *>(s->d_mem + 12), s->d_mem + kHead, s->wait_limit};
}

// `out`: no two elements may share memory.
int check_view(const zg_view *v, const zg_scan_shape *s, bool out, const char *what)
{
    if (!v) return fail(ZG_ERR_INVALID_ARG, "%s is NULL", what);
    const int64_t b = v->batch_stride, t = v->token_stride;
    if (b < 0 || t < 0) return fail(ZG_ERR_INVALID_ARG, "%s has a negative stride", what);
    if (double(b) * double(s->batch) + double(t) * double(s->tokens) + double(s->channels) >= double(kFar))
        return fail(ZG_ERR_INVALID_ARG, "%s has strides out of range", what);
    if (out) {
        // the tighter of the two strides steps over one row of channels, the
        // other over all that the tighter one spans
        const bool apart_t = s->tokens == 1 || t >= s->channels;
        const bool apart_b = s->batch == 1 || b >= s->channels;
        const bool nested = s->tokens == 1 || s->batch == 1 || b >= (s->tokens - 1) * t + s->channels ||
                            t >= (s->batch - 1) * b + s->channels;
        if (!apart_t || !apart_b || !nested) return fail(ZG_ERR_INVALID_ARG, "%s has elements that overlap", what);
    }
    return check_ptr(v->ptr, element_size(s->dtype), false, what);
}

int check_shape(const zg_scan *scan, const zg_scan_shape *s)
{
    if (!scan) return fail(ZG_ERR_INVALID_ARG, "scan handle is NULL");
    if (!s) return fail(ZG_ERR_INVALID_ARG, "shape is NULL");
    if (int rc = check_dtype(s->dtype, "dtype")) return rc;
    if (s->batch < 1 || s->tokens < 1 || s->channels < 1)
        return fail(ZG_ERR_INVALID_ARG, "batch, tokens and channels must be at least 1");
    if (s->batch > scan->batch || s->tokens > scan->tokens || s->channels > scan->channels)
        return fail(ZG_ERR_INVALID_ARG, "shape %lld x %lld x %lld is larger than the handle's %lld x %lld x %lld",
                    (long long)s->batch, (long long)s->tokens, (long long)s->channels, (long long)scan->batch,
                    (long long)scan->tokens, (long long)scan->channels);
    if (s->seq_start) {
        if (s->batch != 1) return fail(ZG_ERR_INVALID_ARG, "packed sequences need batch = 1 (got %lld)", (long long)s->batch);
        if (s->n_seq < 1 || s->n_seq >= (int64_t(1) << 31))
            return fail(ZG_ERR_INVALID_ARG, "n_seq must be in [1, 2^31) (got %lld)", (long long)s->n_seq);
        if (int rc = check_ptr(s->seq_start, 8, false, "seq_start")) return rc;
    }
    if (zg::scan_record_bytes(s->batch, s->tokens, s->channels) > scan->record_bytes)
        return fail(ZG_ERR_INVALID_ARG, "the shape needs more workspace than the handle has");
    int dev = 0;
    if (int rc = finish(cudaGetDevice(&dev), "zg_gated_scan")) return rc;
    if (dev != scan->device)
        return fail(ZG_ERR_INVALID_ARG, "the handle belongs to device %d, but the current device is %d", scan->device, dev);
    return ZG_OK;
}

zg::ScanView view(const zg_view *v) { return zg::ScanView{v->ptr, v->batch_stride, v->token_stride}; }

zg::ScanArgs scan_args(const zg_scan_shape *s)
{
    zg::ScanArgs a{};
    a.batch = s->batch;
    a.tokens = s->tokens;
    a.channels = s->channels;
    a.seq_start = s->seq_start;
    a.n_seq = s->seq_start ? s->n_seq : s->batch;
    a.dtype = s->dtype;
    a.clear_rest = s->clear_rest != 0;
    return a;
}

// ------------------------------------------------------------------ rows of logits

int check_rows(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride, int k)
{
    if (int rc = check_dtype(dtype, "dtype")) return rc;
    if (rows < 0) return fail(ZG_ERR_INVALID_ARG, "rows must not be negative (got %lld)", (long long)rows);
    if (vocab < 1 || vocab > (int64_t(1) << 30))
        return fail(ZG_ERR_INVALID_ARG, "vocab must be in [1, 2^30] (got %lld)", (long long)vocab);
    if (stride < vocab || stride >= kFar)
        return fail(ZG_ERR_INVALID_ARG, "row_stride %lld is not at least vocab %lld", (long long)stride, (long long)vocab);
    if (double(rows) * double(stride) >= double(kFar)) return fail(ZG_ERR_INVALID_ARG, "rows x row_stride is out of range");
    if (k < 1 || k > ZG_TOPK_MAX) return fail(ZG_ERR_INVALID_ARG, "k must be in [1, %d] (got %d)", ZG_TOPK_MAX, k);
    if (rows == 0) return ZG_OK;
    return check_ptr(logits, element_size(dtype), false, "logits");
}

int check_distill(const zg_distill_args *d, float scale, zg::DistillArgs &a)
{
    if (!d) return fail(ZG_ERR_INVALID_ARG, "args is NULL");
    if (int rc = check_rows(d->logits, d->dtype, d->rows, d->vocab, d->row_stride, d->k)) return rc;
    if (int rc = check_dtype(d->t_dtype, "t_dtype")) return rc;
    // the kernels scale by log2(e) / T
    if (!(d->temperature > 0.0f) || !isfinite(d->temperature) || !isfinite(1.0f / d->temperature * 1.44269504f))
        return fail(ZG_ERR_INVALID_ARG, "temperature must be finite and > 0, and log2(e) over it finite (got %g)",
                    double(d->temperature));
    if (!isfinite(scale)) return fail(ZG_ERR_INVALID_ARG, "scale must be finite");
    if (d->rows) {
        if (int rc = check_ptr(d->t_logits, element_size(d->t_dtype), false, "t_logits")) return rc;
        if (int rc = check_ptr(d->t_index, 4, false, "t_index")) return rc;
    }
    a = zg::DistillArgs{};
    a.logits = d->logits;
    a.rows = d->rows;
    a.row_stride = d->row_stride;
    a.vocab = int(d->vocab);
    a.dtype = d->dtype;
    a.t_logits = d->t_logits;
    a.t_index = d->t_index;
    a.t_dtype = d->t_dtype;
    a.k = d->k;
    a.temperature = d->temperature;
    a.scale = scale;
    return ZG_OK;
}

int check_dlogits(const zg_distill_args *d, const float *dloss, void *dlogits, int64_t stride, zg::DistillArgs &a)
{
    if (stride < d->vocab || stride >= kFar || double(d->rows) * double(stride) >= double(kFar))
        return fail(ZG_ERR_INVALID_ARG, "drow_stride %lld is not at least vocab %lld, or out of range", (long long)stride,
                    (long long)d->vocab);
    if (d->rows) {
        if (dlogits == d->logits && stride != d->row_stride)
            return fail(ZG_ERR_INVALID_ARG, "a gradient in the logits' own memory needs their row_stride");
        if (int rc = check_ptr(dloss, 4, true, "dloss")) return rc;
        if (int rc = check_ptr(dlogits, element_size(d->dtype), false, "dlogits")) return rc;
    }
    a.dloss = dloss;
    a.dlogits = dlogits;
    a.drow_stride = stride;
    return ZG_OK;
}

// ------------------------------------------------------------------ tokens, blocks, policies, gradients

// Rows of `width` elements, `stride` apart.
int check_stride(int64_t rows, int64_t width, int64_t stride, const char *what)
{
    if (stride < width || stride >= kFar || double(rows) * double(stride) >= double(kFar))
        return fail(ZG_ERR_INVALID_ARG, "%s %lld is not at least the row's %lld, or out of range", what, (long long)stride,
                    (long long)width);
    return ZG_OK;
}

int check_tokens(const void *tokens, int token_bytes, int64_t n)
{
    if (token_bytes != 4 && token_bytes != 8) return fail(ZG_ERR_INVALID_ARG, "token_bytes must be 4 or 8 (got %d)", token_bytes);
    return n ? check_ptr(tokens, token_bytes, false, "tokens") : ZG_OK;
}

int check_work(const void *work, int64_t have, int64_t need)
{
    if (have < need) return fail(ZG_ERR_INVALID_ARG, "work has %lld bytes, needs %lld", (long long)have, (long long)need);
    return need ? check_ptr(work, 16, false, "work") : ZG_OK;
}

int check_embed(int64_t n, int64_t vocab, int64_t width, float scale)
{
    constexpr int64_t kMost = (int64_t(1) << 31) - 1;
    if (n < 0 || n > kMost) return fail(ZG_ERR_INVALID_ARG, "n must be in [0, 2^31) (got %lld)", (long long)n);
    if (vocab < 1 || vocab > kMost) return fail(ZG_ERR_INVALID_ARG, "vocab must be in [1, 2^31) (got %lld)", (long long)vocab);
    if (width < 1 || width > ZG_EMBED_MAX_WIDTH)
        return fail(ZG_ERR_INVALID_ARG, "width must be in [1, %d] (got %lld)", ZG_EMBED_MAX_WIDTH, (long long)width);
    if (!isfinite(scale)) return fail(ZG_ERR_INVALID_ARG, "scale must be finite");
    return ZG_OK;
}

// One of a block's tensors of rows, of which `there` says whether it takes part.
int check_block_rows(const zg_block *b, const void *p, int64_t stride, bool there, const char *what, zg::RowsView &v)
{
    v = zg::RowsView{nullptr, 0};
    if (!b->rows) return ZG_OK;
    if (!there) return p ? fail(ZG_ERR_INVALID_ARG, "%s must be NULL here", what) : ZG_OK;
    if (!p) return fail(ZG_ERR_INVALID_ARG, "%s is NULL", what);
    if (int rc = check_stride(b->rows, b->width, stride, what)) return rc;
    if (int rc = check_ptr(p, element_size(b->dtype), false, what)) return rc;
    v = zg::RowsView{const_cast<void *>(p), stride};
    return ZG_OK;
}

int check_block_shape(int64_t rows, int64_t width, int64_t groups)
{
    if (rows < 0 || rows >= kFar) return fail(ZG_ERR_INVALID_ARG, "rows is out of range (got %lld)", (long long)rows);
    if (width < 1 || width > ZG_BLOCK_MAX_WIDTH)
        return fail(ZG_ERR_INVALID_ARG, "width must be in [1, %d] (got %lld)", ZG_BLOCK_MAX_WIDTH, (long long)width);
    if (groups < 1 || rows % groups || (rows && groups > rows))
        return fail(ZG_ERR_INVALID_ARG, "groups must divide rows (got %lld and %lld)", (long long)groups, (long long)rows);
    return ZG_OK;
}

int check_block(const zg_block *b, zg::BlockArgs &a)
{
    if (!b) return fail(ZG_ERR_INVALID_ARG, "block is NULL");
    if (int rc = check_dtype(b->dtype, "dtype")) return rc;
    if (int rc = check_block_shape(b->rows, b->width, b->groups)) return rc;
    if (!isfinite(b->res_scale)) return fail(ZG_ERR_INVALID_ARG, "res_scale must be finite");
    if (!(b->eps >= 0.0f) || !isfinite(b->eps)) return fail(ZG_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (b->rows && !b->o && (b->w_post || b->gate))
        return fail(ZG_ERR_INVALID_ARG, "w_post and gate must be NULL where o is");
    a = zg::BlockArgs{};
    a.rows = b->rows;
    a.width = int(b->width);
    a.groups = b->gate ? b->groups : 1;
    a.dtype = b->dtype;
    a.res_scale = b->res_scale;
    a.eps = b->eps;
    const int size = element_size(b->dtype);
    if (int rc = check_block_rows(b, b->x, b->x_stride, true, "x", a.x)) return rc;
    if (int rc = check_block_rows(b, b->o, b->o_stride, b->o != nullptr, "o", a.o)) return rc;
    if (int rc = check_ptr(b->w_post, size, true, "w_post")) return rc;
    if (int rc = check_ptr(b->gate, size, true, "gate")) return rc;
    if (int rc = check_ptr(b->w_pre, size, true, "w_pre")) return rc;
    a.w_post = b->w_post;
    a.gate = b->gate;
    a.w_pre = b->w_pre;
    return ZG_OK;
}

// A weight's gradient, there exactly where the weight is.
int check_weight(const void *w, const void *dw, int dtype, const char *what)
{
    if (!w) return dw ? fail(ZG_ERR_INVALID_ARG, "%s must be NULL here", what) : ZG_OK;
    return check_ptr(dw, element_size(dtype), false, what);
}

int check_temperature(float t)
{
    // the kernels scale by log2(e) / T
    if (t > 0.0f && isfinite(t) && isfinite(1.0f / t * 1.44269504f)) return ZG_OK;
    return fail(ZG_ERR_INVALID_ARG, "temperature must be finite and > 0, and log2(e) over it finite (got %g)", double(t));
}

int check_policy(const zg_policy_args *p, float scale, zg::PolicyArgs &a)
{
    if (!p) return fail(ZG_ERR_INVALID_ARG, "args is NULL");
    if (int rc = check_rows(p->logits, p->dtype, p->rows, p->vocab, p->row_stride, 1)) return rc;
    if (int rc = check_tokens(p->tokens, p->token_bytes, p->rows)) return rc;
    if (int rc = check_temperature(p->temperature)) return rc;
    if (!(p->clip_low >= 0.0f && p->clip_low <= 1.0f))
        return fail(ZG_ERR_INVALID_ARG, "clip_low must be in [0, 1] (got %g)", double(p->clip_low));
    if (!(p->clip_high >= 0.0f) || !isfinite(p->clip_high))
        return fail(ZG_ERR_INVALID_ARG, "clip_high must be finite and >= 0 (got %g)", double(p->clip_high));
    if (!isfinite(p->kl)) return fail(ZG_ERR_INVALID_ARG, "kl must be finite");
    if (!isfinite(scale)) return fail(ZG_ERR_INVALID_ARG, "scale must be finite");
    if (p->rows) {
        if (int rc = check_ptr(p->old_logp, 4, false, "old_logp")) return rc;
        if (int rc = check_ptr(p->advantage, 4, false, "advantage")) return rc;
        if (int rc = check_ptr(p->ref_logp, 4, true, "ref_logp")) return rc;
    }
    a = zg::PolicyArgs{};
    a.logits = p->logits;
    a.rows = p->rows;
    a.row_stride = p->row_stride;
    a.vocab = int(p->vocab);
    a.dtype = p->dtype;
    a.token_bytes = p->token_bytes;
    a.tokens = p->tokens;
    a.old_logp = p->old_logp;
    a.advantage = p->advantage;
    a.ref_logp = p->ref_logp;
    a.clip_low = p->clip_low;
    a.clip_high = p->clip_high;
    a.kl = p->kl;
    a.temperature = p->temperature;
    a.scale = scale;
    return ZG_OK;
}

int check_policy_gradient(const zg_policy_args *p, const float *dloss, void *dlogits, int64_t stride, zg::PolicyArgs &a)
{
    if (int rc = check_stride(p->rows, p->vocab, stride, "drow_stride")) return rc;
    if (p->rows) {
        if (dlogits == p->logits && stride != p->row_stride)
            return fail(ZG_ERR_INVALID_ARG, "a gradient in the logits' own memory needs their row_stride");
        if (int rc = check_ptr(dloss, 4, true, "dloss")) return rc;
        if (int rc = check_ptr(dlogits, element_size(p->dtype), false, "dlogits")) return rc;
    }
    a.dloss = dloss;
    a.dlogits = dlogits;
    a.drow_stride = stride;
    return ZG_OK;
}

// No output overlaps another, or a gradient that is not its own.
int check_apart(const zg_grad *list, int64_t count)
{
    struct Span {
        uintptr_t lo, hi;
        int64_t of;
    };
    std::vector<Span> outs;
    for (int64_t i = 0; i < count; ++i) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(list[i].out);
        if (list[i].n) outs.push_back(Span{lo, lo + uintptr_t(list[i].n) * element_size(list[i].out_dtype), i});
    }
    std::sort(outs.begin(), outs.end(), [](const Span &a, const Span &b) { return a.lo < b.lo; });
    for (size_t i = 1; i < outs.size(); ++i)
        if (outs[i].lo < outs[i - 1].hi)
            return fail(ZG_ERR_INVALID_ARG, "the outputs of list[%lld] and list[%lld] overlap", (long long)outs[i - 1].of,
                        (long long)outs[i].of);
    for (int64_t i = 0; i < count; ++i) {
        if (!list[i].n) continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(list[i].grad);
        const uintptr_t hi = lo + uintptr_t(list[i].n) * element_size(list[i].dtype);
        auto it = std::upper_bound(outs.begin(), outs.end(), lo, [](uintptr_t v, const Span &s) { return v < s.hi; });
        for (; it != outs.end() && it->lo < hi; ++it)
            if (it->of != i || list[i].grad != list[i].out)
                return fail(ZG_ERR_INVALID_ARG, "list[%lld] overlaps the output of list[%lld]", (long long)i, (long long)it->of);
    }
    return ZG_OK;
}

int grads_call(const zg_grads *g, float max_norm, float eps, float scale, float *stats, void *work, int64_t work_bytes,
               bool write, cudaStream_t stream)
{
    if (!g) return fail(ZG_ERR_INVALID_ARG, "list is NULL");
    if (!(scale > 0.0f) || !isfinite(scale)) return fail(ZG_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (write && !(max_norm > 0.0f)) return fail(ZG_ERR_INVALID_ARG, "max_norm must be > 0");
    if (write && (!(eps >= 0.0f) || !isfinite(eps))) return fail(ZG_ERR_INVALID_ARG, "eps must be finite and >= 0");
    int dev = 0;
    if (int rc = finish(cudaGetDevice(&dev), "zg_grads")) return rc;
    if (dev != g->device)
        return fail(ZG_ERR_INVALID_ARG, "the list belongs to device %d, but the current device is %d", g->device, dev);
    if (int rc = check_ptr(stats, 4, false, "stats")) return rc;
    if (int rc = check_work(work, work_bytes, zg_grads_workspace(g))) return rc;
    return finish(zg::launch_grads_norm(g->d_parts, g->parts, static_cast<double *>(work), scale, max_norm, eps, stats, write,
                                        stream),
                  "gradient list launch");
}

}  // namespace

extern "C" {

int zg_scan_init(int64_t batch, int64_t tokens, int64_t channels, zg_scan **out)
{
    if (!out) return fail(ZG_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (batch < 1 || tokens < 1 || channels < 1)
        return fail(ZG_ERR_INVALID_ARG, "batch, tokens and channels must be at least 1");
    if (double(batch) * double(tokens) * double(channels) >= double(kFar))
        return fail(ZG_ERR_INVALID_ARG, "batch x tokens x channels is out of range");
    zg_scan *s = new (std::nothrow) zg_scan();
    if (!s) return fail(ZG_ERR_NO_MEMORY, "host allocation of the scan handle failed");
    s->batch = batch;
    s->tokens = tokens;
    s->channels = channels;
    s->wait_limit = kScanWaitLimit;
    s->record_bytes = zg::scan_record_bytes(batch, tokens, channels);
    cudaError_t e = cudaGetDevice(&s->device);
    if (e == cudaSuccess) e = cudaMalloc(&s->d_mem, size_t(kHead + s->record_bytes));
    if (e == cudaSuccess) e = cudaMemset(s->d_mem, 0, size_t(kHead + s->record_bytes));
    // epoch 1: the cleared records belong to no launch
    const unsigned long long ctl = 1ull << 32;
    if (e == cudaSuccess) e = cudaMemcpy(s->d_mem, &ctl, sizeof ctl, cudaMemcpyHostToDevice);
    // Both may return before they are done on the device, and a stream of the caller's
    // that does not wait for the default stream could overtake them.
    if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
    if (e != cudaSuccess) {
        const int rc = e == cudaErrorMemoryAllocation
                           ? fail(ZG_ERR_NO_MEMORY, "zg_scan_init: %lld bytes of workspace: %s",
                                  (long long)(kHead + s->record_bytes), cudaGetErrorString(e))
                           : finish(e, "zg_scan_init workspace");
        cudaGetLastError();
        zg_scan_destroy(s);
        return rc;
    }
    *out = s;
    return ZG_OK;
}

void zg_scan_destroy(zg_scan *s)
{
    if (!s) return;
    if (s->d_mem) cudaFree(s->d_mem);
    delete s;
}

int zg_scan_set_wait_limit(zg_scan *s, int64_t polls)
{
    if (!s) return fail(ZG_ERR_INVALID_ARG, "scan handle is NULL");
    if (polls < 0) return fail(ZG_ERR_INVALID_ARG, "polls must be >= 0");
    s->wait_limit = polls;
    return ZG_OK;
}

int zg_scan_status(zg_scan *s, zg_stream stream, int *status)
{
    if (!s) return fail(ZG_ERR_INVALID_ARG, "scan handle is NULL");
    if (!status) return fail(ZG_ERR_INVALID_ARG, "status is NULL");
    int *d_status = work_of(s).status;
    int found = 0;
    cudaError_t e = cudaMemcpyAsync(&found, d_status, sizeof(int), cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return finish(e, "zg_scan_status");
    *status = found;
    if (*status == ZG_OK) return ZG_OK;
    return finish(cudaMemsetAsync(d_status, 0, sizeof(int), stream), "zg_scan_status reset");
}

int zg_gated_scan(zg_scan *scan, const zg_scan_shape *shape, const zg_view *x, const zg_view *f, const float *h0,
                  const zg_view *y, float *h_last, float *states, zg_stream stream)
{
    return guarded([&]() -> int {
        if (int rc = check_shape(scan, shape)) return rc;
        if (int rc = check_view(x, shape, false, "x")) return rc;
        if (int rc = check_view(f, shape, false, "f")) return rc;
        if (int rc = check_view(y, shape, true, "y")) return rc;
        if (int rc = check_ptr(h0, 4, true, "h0")) return rc;
        if (int rc = check_ptr(h_last, 4, true, "h_last")) return rc;
        if (int rc = check_ptr(states, 4, true, "states")) return rc;
        zg::ScanArgs a = scan_args(shape);
        a.x = view(x);
        a.f = view(f);
        a.y = view(y);
        a.h0 = h0;
        a.h_last = h_last;
        a.states = states;
        return finish(zg::launch_scan(a, work_of(scan), stream), "scan launch");
    });
}

int zg_gated_scan_bwd(zg_scan *scan, const zg_scan_shape *shape, const zg_view *x, const zg_view *f,
                      const zg_view *dy, const float *states, const float *h0, const float *dh_last,
                      const zg_view *dx, const zg_view *df, float *dh0, zg_stream stream)
{
    return guarded([&]() -> int {
        if (int rc = check_shape(scan, shape)) return rc;
        if (int rc = check_view(x, shape, false, "x")) return rc;
        if (int rc = check_view(f, shape, false, "f")) return rc;
        if (int rc = check_view(dy, shape, false, "dy")) return rc;
        if (int rc = check_view(dx, shape, true, "dx")) return rc;
        if (int rc = check_view(df, shape, true, "df")) return rc;
        if (int rc = check_ptr(states, 4, false, "states")) return rc;
        if (int rc = check_ptr(h0, 4, true, "h0")) return rc;
        if (int rc = check_ptr(dh_last, 4, true, "dh_last")) return rc;
        if (int rc = check_ptr(dh0, 4, true, "dh0")) return rc;
        zg::ScanArgs a = scan_args(shape);
        a.x = view(x);
        a.f = view(f);
        a.y = view(dy);
        a.h0 = h0;
        a.states = const_cast<float *>(states);
        a.dx = view(dx);
        a.df = view(df);
        a.dh_last = dh_last;
        a.dh0 = dh0;
        return finish(zg::launch_scan_bwd(a, work_of(scan), stream), "scan backward launch");
    });
}

int zg_topk(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride, int k, void *values,
            int32_t *index, zg_stream stream)
{
    return guarded([&]() -> int {
        if (int rc = check_rows(logits, dtype, rows, vocab, row_stride, k)) return rc;
        if (k > vocab) return fail(ZG_ERR_INVALID_ARG, "k = %d is more than vocab = %lld", k, (long long)vocab);
        if (rows == 0) return ZG_OK;
        if (int rc = check_ptr(values, element_size(dtype), false, "values")) return rc;
        if (int rc = check_ptr(index, 4, false, "index")) return rc;
        return finish(zg::launch_topk(logits, dtype, rows, int(vocab), row_stride, k, values, index, stream), "top-k launch");
    });
}

int zg_distill_loss(const zg_distill_args *args, float *loss, float *lse, zg_stream stream)
{
    return guarded([&]() -> int {
        zg::DistillArgs a;
        if (int rc = check_distill(args, 0.0f, a)) return rc;
        if (a.rows == 0) return ZG_OK;
        if (int rc = check_ptr(loss, 4, false, "loss")) return rc;
        if (int rc = check_ptr(lse, 4, true, "lse")) return rc;
        a.loss = loss;
        a.lse = lse;
        return finish(zg::launch_distill(a, stream), "distillation loss launch");
    });
}

int zg_distill_grad(const zg_distill_args *args, const float *lse, float scale, const float *dloss, void *dlogits,
                    int64_t drow_stride, zg_stream stream)
{
    return guarded([&]() -> int {
        zg::DistillArgs a;
        if (int rc = check_distill(args, scale, a)) return rc;
        if (int rc = check_dlogits(args, dloss, dlogits, drow_stride, a)) return rc;
        if (a.rows == 0) return ZG_OK;
        if (int rc = check_ptr(lse, 4, false, "lse")) return rc;
        a.lse_in = lse;
        return finish(zg::launch_distill(a, stream), "distillation gradient launch");
    });
}

int zg_distill_loss_grad(const zg_distill_args *args, float scale, const float *dloss, float *loss, float *lse,
                         void *dlogits, int64_t drow_stride, zg_stream stream)
{
    return guarded([&]() -> int {
        zg::DistillArgs a;
        if (int rc = check_distill(args, scale, a)) return rc;
        if (int rc = check_dlogits(args, dloss, dlogits, drow_stride, a)) return rc;
        if (a.rows == 0) return ZG_OK;
        if (int rc = check_ptr(loss, 4, false, "loss")) return rc;
        if (int rc = check_ptr(lse, 4, true, "lse")) return rc;
        a.loss = loss;
        a.lse = lse;
        return finish(zg::launch_distill(a, stream), "distillation launch");
    });
}

int zg_embed(const void *table, int dtype, int64_t vocab, int64_t width, int64_t table_stride, const void *tokens,
             int token_bytes, int64_t n, float scale, void *out, int64_t out_stride, zg_stream stream)
{
    return guarded([&]() -> int {
        if (int rc = check_dtype(dtype, "dtype")) return rc;
        if (int rc = check_embed(n, vocab, width, scale)) return rc;
        if (int rc = check_stride(vocab, width, table_stride, "table_stride")) return rc;
        if (int rc = check_stride(n, width, out_stride, "out_stride")) return rc;
        if (int rc = check_tokens(tokens, token_bytes, n)) return rc;
        if (n == 0) return ZG_OK;
        if (int rc = check_ptr(table, element_size(dtype), false, "table")) return rc;
        if (int rc = check_ptr(out, element_size(dtype), false, "out")) return rc;
        zg::EmbedArgs a{};
        a.table = table;
        a.dtype = dtype;
        a.vocab = vocab;
        a.width = width;
        a.table_stride = table_stride;
        a.tokens = tokens;
        a.token_bytes = token_bytes;
        a.n = n;
        a.scale = scale;
        a.out = out;
        a.out_stride = out_stride;
        return finish(zg::launch_embed(a, stream), "embedding launch");
    });
}

int64_t zg_embed_grad_workspace(int64_t n, int64_t vocab, int64_t width)
{
    if (check_embed(n, vocab, width, 1.0f)) return -1;
    return zg::embed_grad_workspace(n, vocab, width);
}

int zg_embed_grad(const void *drows, int dtype, int64_t drow_stride, const void *tokens, int token_bytes, int64_t n,
                  int64_t vocab, int64_t width, float scale, const void *add, int64_t add_stride, void *dtable,
                  int table_dtype, int64_t dtable_stride, void *work, int64_t work_bytes, zg_stream stream)
{
    return guarded([&]() -> int {
        if (int rc = check_dtype(dtype, "dtype")) return rc;
        if (int rc = check_dtype(table_dtype, "table_dtype")) return rc;
        if (int rc = check_embed(n, vocab, width, scale)) return rc;
        if (int rc = check_stride(n, width, drow_stride, "drow_stride")) return rc;
        if (int rc = check_stride(vocab, width, dtable_stride, "dtable_stride")) return rc;
        if (add)
            if (int rc = check_stride(vocab, width, add_stride, "add_stride")) return rc;
        if (add && add == dtable && add_stride != dtable_stride)
            return fail(ZG_ERR_INVALID_ARG, "a gradient in add's own memory needs its stride");
        if (int rc = check_tokens(tokens, token_bytes, n)) return rc;
        if (n)
            if (int rc = check_ptr(drows, element_size(dtype), false, "drows")) return rc;
        if (int rc = check_ptr(add, element_size(table_dtype), true, "add")) return rc;
        if (int rc = check_ptr(dtable, element_size(table_dtype), false, "dtable")) return rc;
        if (int rc = check_work(work, work_bytes, zg::embed_grad_workspace(n, vocab, width))) return rc;
        zg::EmbedArgs a{};
        a.table = add;
        a.dtype = table_dtype;
        a.vocab = vocab;
        a.width = width;
        a.table_stride = add_stride;
        a.tokens = tokens;
        a.token_bytes = token_bytes;
        a.n = n;
        a.scale = scale;
        a.out = dtable;
        a.out_stride = dtable_stride;
        a.drows = drows;
        a.drow_dtype = dtype;
        a.drow_stride = drow_stride;
        a.work = work;
        return finish(zg::launch_embed_grad(a, stream), "embedding gradient launch");
    });
}

int zg_block_norm(const zg_block *block, void *x_new, int64_t x_new_stride, void *n, int64_t n_stride, float *kept,
                  zg_stream stream)
{
    return guarded([&]() -> int {
        zg::BlockArgs a;
        if (int rc = check_block(block, a)) return rc;
        if (int rc = check_block_rows(block, x_new, x_new_stride, x_new || block->o, "x_new", a.x_new)) return rc;
        if (int rc = check_block_rows(block, n, n_stride, block->w_pre != nullptr, "n", a.n)) return rc;
        if (a.rows == 0) return ZG_OK;
        if (!x_new && !n) return fail(ZG_ERR_INVALID_ARG, "neither x_new nor n is asked for");
        if (x_new && ((x_new == block->x && x_new_stride != block->x_stride) || x_new == block->o || x_new == n))
            return fail(ZG_ERR_INVALID_ARG, "x_new must not overlap o or n, and in x's own memory it needs x's stride");
        if (n && ((n == block->o && n_stride != block->o_stride) || n == block->x))
            return fail(ZG_ERR_INVALID_ARG, "n must not overlap x, and in o's own memory it needs o's stride");
        if (int rc = check_ptr(kept, 4, true, "kept")) return rc;
        a.kept = kept;
        return finish(a.dtype == ZG_DTYPE_BF16 ? zg::launch_block_norm_bf16(a, stream) : zg::launch_block_norm_f32(a, stream),
                      "block norm launch");
    });
}

int64_t zg_block_norm_workspace(int64_t rows, int64_t width, int64_t groups)
{
    if (check_block_shape(rows, width, groups)) return -1;
    return rows ? zg::block_norm_workspace(rows, width, groups) : 0;
}

int zg_block_norm_grad(const zg_block *block, const float *kept, const void *dn, int64_t dn_stride,
                       const void *dx_new, int64_t dx_new_stride, void *dx, int64_t dx_stride, void *d_o,
                       int64_t d_o_stride, void *dw_pre, void *dw_post, void *dgate, void *work, int64_t work_bytes,
                       zg_stream stream)
{
    return guarded([&]() -> int {
        zg::BlockArgs a;
        if (int rc = check_block(block, a)) return rc;
        if (int rc = check_block_rows(block, dn, dn_stride, block->w_pre != nullptr, "dn", a.n)) return rc;
        if (int rc = check_block_rows(block, dx_new, dx_new_stride, dx_new != nullptr, "dx_new", a.x_new)) return rc;
        if (int rc = check_block_rows(block, dx, dx_stride, true, "dx", a.dx)) return rc;
        if (int rc = check_block_rows(block, d_o, d_o_stride, block->o != nullptr, "d_o", a.d_o)) return rc;
        if (int rc = check_weight(block->w_pre, dw_pre, block->dtype, "dw_pre")) return rc;
        if (int rc = check_weight(block->w_post, dw_post, block->dtype, "dw_post")) return rc;
        if (int rc = check_weight(block->gate, dgate, block->dtype, "dgate")) return rc;
        const int size = element_size(block->dtype);
        if (a.rows == 0) {  // sums over nothing
            const size_t row = size_t(a.width) * size;
            cudaError_t e = dw_pre ? cudaMemsetAsync(dw_pre, 0, row, stream) : cudaSuccess;
            if (e == cudaSuccess && dw_post) e = cudaMemsetAsync(dw_post, 0, row, stream);
            if (e == cudaSuccess && dgate) e = cudaMemsetAsync(dgate, 0, row * size_t(a.groups), stream);
            return finish(e, "block norm gradient of no rows");
        }
        if (dx == d_o || dx == block->x || dx == block->o || (d_o && (d_o == block->x || d_o == block->o)) ||
            (dx == dx_new && dx_stride != dx_new_stride) || (d_o && d_o == dn && d_o_stride != dn_stride) || dx == dn ||
            (d_o && d_o == dx_new))
            return fail(ZG_ERR_INVALID_ARG, "dx and d_o overlap an input or each other");
        if (int rc = check_ptr(kept, 4, false, "kept")) return rc;
        if (int rc = check_work(work, work_bytes, zg::block_norm_workspace(a.rows, a.width, a.groups))) return rc;
        a.kept = const_cast<float *>(kept);
        a.dw_pre = dw_pre;
        a.dw_post = dw_post;
        a.dgate = dgate;
        a.work = static_cast<float *>(work);
        return finish(a.dtype == ZG_DTYPE_BF16 ? zg::launch_block_norm_grad_bf16(a, stream)
                                               : zg::launch_block_norm_grad_f32(a, stream),
                      "block norm gradient launch");
    });
}

int zg_token_logp(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride, const void *tokens,
                  int token_bytes, float temperature, float *logp, float *lse, zg_stream stream)
{
    return guarded([&]() -> int {
        if (int rc = check_rows(logits, dtype, rows, vocab, row_stride, 1)) return rc;
        if (int rc = check_tokens(tokens, token_bytes, rows)) return rc;
        if (int rc = check_temperature(temperature)) return rc;
        if (rows == 0) return ZG_OK;
        if (int rc = check_ptr(logp, 4, false, "logp")) return rc;
        if (int rc = check_ptr(lse, 4, true, "lse")) return rc;
        zg::PolicyArgs a{};
        a.logits = logits;
        a.rows = rows;
        a.row_stride = row_stride;
        a.vocab = int(vocab);
        a.dtype = dtype;
        a.token_bytes = token_bytes;
        a.tokens = tokens;
        a.temperature = temperature;
        a.logp = logp;
        a.lse = lse;
        return finish(zg::launch_policy(a, stream), "token log-probability launch");
    });
}

int zg_policy_loss(const zg_policy_args *args, float *loss, float *logp, float *kept, zg_stream stream)
{
    return guarded([&]() -> int {
        zg::PolicyArgs a;
        if (int rc = check_policy(args, 0.0f, a)) return rc;
        if (a.rows == 0) return ZG_OK;
        if (int rc = check_ptr(loss, 4, false, "loss")) return rc;
        if (int rc = check_ptr(logp, 4, true, "logp")) return rc;
        if (int rc = check_ptr(kept, 4, true, "kept")) return rc;
        a.loss = loss;
        a.logp = logp;
        a.kept = kept;
        return finish(zg::launch_policy(a, stream), "policy loss launch");
    });
}

int zg_policy_grad(const zg_policy_args *args, const float *kept, float scale, const float *dloss, void *dlogits,
                   int64_t drow_stride, zg_stream stream)
{
    return guarded([&]() -> int {
        zg::PolicyArgs a;
        if (int rc = check_policy(args, scale, a)) return rc;
        if (int rc = check_policy_gradient(args, dloss, dlogits, drow_stride, a)) return rc;
        if (a.rows == 0) return ZG_OK;
        if (int rc = check_ptr(kept, 4, false, "kept")) return rc;
        a.kept_in = kept;
        return finish(zg::launch_policy(a, stream), "policy gradient launch");
    });
}

int zg_policy_loss_grad(const zg_policy_args *args, float scale, const float *dloss, float *loss, float *logp,
                        void *dlogits, int64_t drow_stride, zg_stream stream)
{
    return guarded([&]() -> int {
        zg::PolicyArgs a;
        if (int rc = check_policy(args, scale, a)) return rc;
        if (int rc = check_policy_gradient(args, dloss, dlogits, drow_stride, a)) return rc;
        if (a.rows == 0) return ZG_OK;
        if (int rc = check_ptr(loss, 4, false, "loss")) return rc;
        if (int rc = check_ptr(logp, 4, true, "logp")) return rc;
        a.loss = loss;
        a.logp = logp;
        return finish(zg::launch_policy(a, stream), "policy launch");
    });
}

int zg_grads_init(const zg_grad *list, int64_t count, zg_grads **out)
{
    if (!out) return fail(ZG_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    return guarded([&]() -> int {
        if (count < 0 || (count && !list)) return fail(ZG_ERR_INVALID_ARG, "list is NULL or count negative");
        std::vector<zg::GradPart> parts;
        double total = 0.0;
        for (int64_t i = 0; i < count; ++i) total += double(list[i].n > 0 ? list[i].n : 0);
        int64_t each = zg::kGradPartLeast;
        while (each < zg::kGradPartMost && total > 1024.0 * double(each)) each *= 2;
        for (int64_t i = 0; i < count; ++i) {
            const zg_grad &g = list[i];
            char what[48];
            snprintf(what, sizeof what, "list[%lld]", (long long)i);
            if (int rc = check_dtype(g.dtype, what)) return rc;
            if (int rc = check_dtype(g.out_dtype, what)) return rc;
            if (g.n < 0 || g.n >= (int64_t(1) << 40))
                return fail(ZG_ERR_INVALID_ARG, "%s: n must be in [0, 2^40) (got %lld)", what, (long long)g.n);
            if (g.n == 0) continue;
            if (int rc = check_ptr(g.grad, element_size(g.dtype), false, what)) return rc;
            if (int rc = check_ptr(g.out, element_size(g.out_dtype), false, what)) return rc;
            if (g.grad == g.out && g.dtype != g.out_dtype)
                return fail(ZG_ERR_INVALID_ARG, "%s: a gradient clipped in its own memory keeps its dtype", what);
            for (int64_t at = 0; at < g.n; at += each) {
                zg::GradPart p{};
                p.grad = static_cast<const char *>(g.grad) + at * element_size(g.dtype);
                p.out = static_cast<char *>(g.out) + at * element_size(g.out_dtype);
                p.n = int(g.n - at < each ? g.n - at : each);
                p.dtype = uint8_t(g.dtype);
                p.out_dtype = uint8_t(g.out_dtype);
                parts.push_back(p);
            }
        }
        if (int rc = check_apart(list, count)) return rc;
        if (parts.size() >= (size_t(1) << 31)) return fail(ZG_ERR_INVALID_ARG, "the list has too many elements");
        zg_grads *g = new zg_grads();
        g->parts = int64_t(parts.size());
        const size_t bytes = parts.size() * sizeof(zg::GradPart);
        cudaError_t e = cudaGetDevice(&g->device);
        if (e == cudaSuccess) e = cudaMalloc(&g->d_parts, bytes ? bytes : 16);
        if (e == cudaSuccess && bytes) e = cudaMemcpy(g->d_parts, parts.data(), bytes, cudaMemcpyHostToDevice);
        // The copy may return before it is done on the device, and a stream of the caller's
        // that does not wait for the default stream could overtake it.
        if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
        if (e != cudaSuccess) {
            const int rc = e == cudaErrorMemoryAllocation
                               ? fail(ZG_ERR_NO_MEMORY, "zg_grads_init: %zu bytes: %s", bytes, cudaGetErrorString(e))
                               : finish(e, "zg_grads_init");
            cudaGetLastError();
            zg_grads_destroy(g);
            return rc;
        }
        *out = g;
        return ZG_OK;
    });
}

void zg_grads_destroy(zg_grads *g)
{
    if (!g) return;
    if (g->d_parts) cudaFree(g->d_parts);
    delete g;
}

int64_t zg_grads_workspace(const zg_grads *g) { return g ? (g->parts + 2) / 2 * 16 : -1; }

int zg_grads_norm(const zg_grads *grads, float scale, float *stats, void *work, int64_t work_bytes, zg_stream stream)
{
    return guarded([&]() -> int { return grads_call(grads, 1.0f, 0.0f, scale, stats, work, work_bytes, false, stream); });
}

int zg_grads_clip(const zg_grads *grads, float max_norm, float eps, float scale, float *stats, void *work,
                  int64_t work_bytes, zg_stream stream)
{
    return guarded([&]() -> int { return grads_call(grads, max_norm, eps, scale, stats, work, work_bytes, true, stream); });
}

}  // extern "C"
