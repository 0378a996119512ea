// zg_ops_api.cu -- the C ABI of the training operators (include/zg.h):
// argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

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

}  // extern "C"
