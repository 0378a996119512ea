// The log-probabilities of tokens, the clipped policy loss with its KL term, and
// its gradient by the logits.
//
// With z a row of logits, T the temperature and t its token, logp = (z_t - m) / T
// - log S with m the row's maximum and S = sum exp((z - m) / T); the loss and its
// slope by logp are the row's own few values; dz = g ([v = t] - exp((z - m) / T) / S)
// with g = scale dloss slope / T.
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

constexpr int kThreads = 512;
constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest of a set of logits and the sum of 2^((z - top) c) over it.
struct Sum {
    float top, sum;
};
__device__ __forceinline__ Sum join(Sum a, Sum b, float c)
{
    const float top = max_nan(a.top, b.top);
    const float sa = a.top == -INFINITY ? 0.0f : a.sum * exp2_approx((a.top - top) * c);
    const float sb = b.top == -INFINITY ? 0.0f : b.sum * exp2_approx((b.top - top) * c);
    return Sum{top, sa + sb};
}

__device__ __forceinline__ int token_of(const PolicyArgs &a, int64_t r)
{
    const int64_t t = a.token_bytes == 8 ? static_cast<const int64_t *>(a.tokens)[r] : static_cast<const int32_t *>(a.tokens)[r];
    return t >= 0 && t < a.vocab ? int(t) : -1;
}

// The loss of a row and its slope by logp.
__device__ __forceinline__ float2 loss_of(const PolicyArgs &a, int64_t r, float logp)
{
    const float adv = a.advantage[r], ratio = expf(logp - a.old_logp[r]);
    const float high = 1.0f + a.clip_high, low = 1.0f - a.clip_low;
    const float held = fminf(fmaxf(ratio, low), high);
    const bool cut = (adv > 0.0f && ratio > high) || (adv < 0.0f && ratio < low);
    float loss = cut ? -held * adv : -ratio * adv, slope = cut ? 0.0f : -ratio * adv;
    if (a.ref_logp) {
        const float d = a.ref_logp[r] - logp, e = expm1f(d);
        loss = fmaf(a.kl, e - d, loss);
        slope = fmaf(-a.kl, e, slope);
    }
    return make_float2(loss, slope);
}

template <class T, bool LOSS, bool GRAD>
__global__ void __launch_bounds__(kThreads) policy_kernel(PolicyArgs a)
{
    __shared__ Sum part[kThreads / 32];
    __shared__ float g_row;
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    const float c = 1.0f / a.temperature * kLog2e;
    const int token = token_of(a, r);
    const T *const z = static_cast<const T *>(a.logits) + r * a.row_stride;
    T *const dz = GRAD ? static_cast<T *>(a.dlogits) + r * a.drow_stride : nullptr;
    if (token < 0) {
        if (LOSS && tid == 0) {
            if (a.loss) a.loss[r] = 0.0f;
            if (a.logp) a.logp[r] = 0.0f;
            if (a.lse) a.lse[r] = 0.0f;
            if (a.kept) a.kept[2 * r] = a.kept[2 * r + 1] = 0.0f;
        }
        if (GRAD)
            for (int v = tid; v < a.vocab; v += kThreads) store1(dz + v, 0.0f);
        return;
    }
    Sum s{-INFINITY, 0.0f};
    const float zt = load1(z + token);
    if (LOSS) {
        for (int v = tid; v < a.vocab; v += kThreads) {
            const float x = load1(z + v);
            s = join(s, Sum{x, x == -INFINITY ? 0.0f : x - x + 1.0f}, c);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            s = join(s, Sum{__shfl_xor_sync(0xffffffffu, s.top, o), __shfl_xor_sync(0xffffffffu, s.sum, o)}, c);
        if (tid % 32 == 0) part[tid / 32] = s;
        __syncthreads();
        s = part[0];
        for (int i = 1; i < kThreads / 32; ++i) s = join(s, part[i], c);
    } else {
        s = Sum{a.kept_in[2 * r], a.kept_in[2 * r + 1]};
    }
    const float rt = 1.0f / a.temperature, log_sum = logf(s.sum);
    if (tid == 0) {
        const float logp = fmaf(zt - s.top, rt, -log_sum);
        float2 l = make_float2(0.0f, 0.0f);
        if (a.old_logp) l = loss_of(a, r, logp);
        if (LOSS) {
            if (a.loss) a.loss[r] = l.x;
            if (a.logp) a.logp[r] = logp;
            if (a.lse) a.lse[r] = fmaf(s.top, rt, log_sum);
            if (a.kept) {
                a.kept[2 * r] = s.top;
                a.kept[2 * r + 1] = s.sum;
            }
        }
        g_row = a.scale * (a.dloss ? a.dloss[r] : 1.0f) * l.y * rt;
    }
    if (!GRAD) return;
    __syncthreads();
    const float g = g_row, q = -g / s.sum;
    for (int v = tid; v < a.vocab; v += kThreads)
        store1(dz + v, fmaf(exp2_approx((load1(z + v) - s.top) * c), q, v == token ? g : 0.0f));
}

template <class T>
cudaError_t of_type(const PolicyArgs &a, cudaStream_t st)
{
    if (a.rows >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    const unsigned blocks = unsigned(a.rows);
    if (a.kept_in)
        policy_kernel<T, false, true><<<blocks, kThreads, 0, st>>>(a);
    else if (a.dlogits)
        policy_kernel<T, true, true><<<blocks, kThreads, 0, st>>>(a);
    else
        policy_kernel<T, true, false><<<blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_policy(const PolicyArgs &a, cudaStream_t st)
{
    return a.dtype == ZG_DTYPE_BF16 ? of_type<uint16_t>(a, st) : of_type<float>(a, st);
}

}  // namespace zg
