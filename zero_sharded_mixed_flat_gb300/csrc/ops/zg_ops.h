// zg_ops.h -- launchers of the training operators (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "zg.h"

namespace zg {

// One tensor of a scan: element (b, t, c) at ptr[b * sb + t * st + c].
struct ScanView {
    void *ptr;
    int64_t sb, st;
};

struct ScanArgs {
    int64_t batch, tokens, channels;
    const int64_t *seq_start;  // device, or null
    int64_t n_seq;             // sequences: batch when seq_start is null
    int dtype;
    bool clear_rest;           // zeros to the outputs of tokens past the last packed sequence
    ScanView x, f, y;          // y: forward's output; dy in backward
    const float *h0;           // or null
    float *h_last;             // or null
    float *states;             // written by forward (or null), read by backward
    ScanView dx, df;           // backward only, as the next two
    const float *dh_last;      // or null
    float *dh0;                // or null
};

// Device memory of a scan handle: the words that blocks take their places from
// and hand states on through.
struct ScanWork {
    unsigned long long *ctl;
    int *status;
    uint32_t *gave_up;
    void *records;
    long long wait_limit;
};

// Bytes of `records` that a shape needs (none when one chunk holds every row).
int64_t scan_record_bytes(int64_t batch, int64_t tokens, int64_t channels);

cudaError_t launch_scan(const ScanArgs &a, const ScanWork &w, cudaStream_t st);
cudaError_t launch_scan_bwd(const ScanArgs &a, const ScanWork &w, cudaStream_t st);

cudaError_t launch_topk(const void *logits, int dtype, int64_t rows, int vocab, int64_t stride, int k, void *values,
                        int32_t *index, cudaStream_t st);

// Any of loss, lse and dlogits may be null; with lse_in the loss is not
// computed and lse is taken from there.
struct DistillArgs {
    const void *logits;
    int64_t rows, row_stride;
    int vocab, dtype;
    const void *t_logits;
    const int32_t *t_index;
    int t_dtype, k;
    float temperature;
    float *loss, *lse;
    const float *lse_in;
    float scale;
    const float *dloss;
    void *dlogits;
    int64_t drow_stride;
};

cudaError_t launch_distill(const DistillArgs &a, cudaStream_t st);

}  // namespace zg
