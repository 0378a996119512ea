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

struct EmbedArgs {
    const void *table;  // of the lookup, or add of the gradient (or null)
    int dtype;          // of table and out
    int64_t vocab, width, table_stride;
    const void *tokens;
    int token_bytes;
    int64_t n;
    float scale;
    void *out;  // rows, or dtable
    int64_t out_stride;
    const void *drows;  // of the gradient
    int drow_dtype;
    int64_t drow_stride;
    void *work;
};

cudaError_t launch_embed(const EmbedArgs &a, cudaStream_t st);
int64_t embed_grad_workspace(int64_t n, int64_t vocab, int64_t width);
cudaError_t launch_embed_grad(const EmbedArgs &a, cudaStream_t st);

// One tensor of a block's norms: element (r, c) at ptr[r * stride + c].
struct RowsView {
    void *ptr;
    int64_t stride;
};

struct BlockArgs {
    int64_t rows, groups;
    int width, dtype;
    RowsView x, o;  // o.ptr may be null, as the weights
    const void *w_post, *gate, *w_pre;
    float res_scale, eps;
    float *kept;         // 2 x rows: written by forward (or null), read by backward
    RowsView x_new, n;   // forward's outputs (either may be null); dx_new (or null) and dn of backward
    RowsView dx, d_o;    // backward only, as the rest
    void *dw_pre, *dw_post, *dgate;
    float *work;
};

// A translation unit to each dtype.
cudaError_t launch_block_norm_bf16(const BlockArgs &a, cudaStream_t st);
cudaError_t launch_block_norm_f32(const BlockArgs &a, cudaStream_t st);
cudaError_t launch_block_norm_grad_bf16(const BlockArgs &a, cudaStream_t st);
cudaError_t launch_block_norm_grad_f32(const BlockArgs &a, cudaStream_t st);
int64_t block_norm_workspace(int64_t rows, int64_t width, int64_t groups);

// loss alone, gradient alone (from kept), or both; with old_logp null the
// log-probabilities alone.
struct PolicyArgs {
    const void *logits;
    int64_t rows, row_stride;
    int vocab, dtype, token_bytes;
    const void *tokens;
    const float *old_logp, *advantage, *ref_logp;
    float clip_low, clip_high, kl, temperature;
    float *loss, *logp, *lse;  // written where not null
    float *kept;               // rows x 3: written with the loss (or null)
    const float *kept_in;      // the gradient alone starts from these
    float scale;
    const float *dloss;
    void *dlogits;
    int64_t drow_stride;
};

cudaError_t launch_policy(const PolicyArgs &a, cudaStream_t st);

// A share of one tensor of a gradient list.
struct GradPart {
    const void *grad;
    void *out;
    int n;
    uint8_t dtype, out_dtype;
};
// Elements of a part: at most some 1,024 parts to a list of up to 33 M elements, so that small lists have work for all SMs;
// of larger lists the most that a block reads well, in as many parts as that makes (124 M gradients: parts of 8192
// elements 163 us, 16384 126, 32768, some 3,900 parts, 123, 65536 124; 0.6 M: of 8192 14.5 us, 16384 16.5, 32768 19.9).
constexpr int64_t kGradPartLeast = 4096, kGradPartMost = 32768;

cudaError_t launch_grads_norm(const GradPart *parts, int64_t count, double *sums, float scale, float max_norm, float eps,
                              float *stats, bool write, cudaStream_t st);

}  // namespace zg
