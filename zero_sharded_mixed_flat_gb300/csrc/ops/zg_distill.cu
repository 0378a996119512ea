// The distillation loss from a teacher's top logits, and its gradient.
//
// With z a row of the student's logits, T the temperature and p the softmax of
// the teacher's k entries, loss = T^2 sum_j p_j (log p_j - z_{i_j} / T + lse),
// lse = log sum exp(z / T), and dz = scale dloss T (exp(z / T - lse) - p), where
// p acts on its k indices alone. So a row costs a sum over the vocabulary, k
// gathered values, and for the gradient one exponential per logit again.
//
// Bound by memory: each logit is read once (2 bytes in bf16) and its gradient
// written once. A row is read by one small block with a running maximum and sum;
// for loss and gradient together it is read again, from L2, where the rows in
// flight are kept few enough to stay. (Copies of the row in shared memory, with
// the blocks large enough to hold it, took 92 us for the loss below and 156 for
// both: the blocks' ends left memory idle.) Few rows take a cluster of blocks to
// a row, which exchange their maximum and sum through distributed shared memory.
// A part is whole 16-byte units of the row but for its two ends, so any row,
// however it is aligned, moves in wide loads; a gradient whose rows are aligned
// differently is stored in its own units, each from the two that it lies across.
//
// Measured at 4096 x 50257 in bf16, k = 64: the loss 64 us (6.5 TB/s), the
// gradient 126 (6.5 TB/s), both in one launch 154 (5.3 TB/s of the once-read,
// once-written bytes; what is left is the second read out of L2 and the phases
// of a row). With gradient rows that are not aligned as the logits' are, 2048
// rows: gradient 74, both 90. One row: 5 and 4 us, the latency of the launch and
// of the row's three phases.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "zg_launch.h"
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f;
constexpr int kAhead = 4;  // units that a thread asks for before it uses the first

__device__ __forceinline__ float exp2_approx(float v)
{
    float d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
    return d;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t *>(&a)), "l"(*reinterpret_cast<const uint64_t *>(&b)));
    return *reinterpret_cast<const float2 *>(&d);
}

// A sum of exponentials as sum 2^((v - top) c), with top the largest v seen:
// differences first, so that rows of a type's lowest value neither overflow nor
// count as masked. Nothing but -inf gives top = -inf and sum = 0; a NaN or +inf
// makes the sum NaN.
struct Sum {
    float top, sum;
};
__device__ __forceinline__ Sum none() { return Sum{-INFINITY, 0.0f}; }
__device__ __forceinline__ float rescaled(Sum s, float top, float c)
{
    return s.top == -INFINITY ? 0.0f : s.sum * exp2_approx((s.top - top) * c);
}
__device__ __forceinline__ Sum join(Sum a, Sum b, float c)
{
    const float top = max_nan(a.top, b.top);
    return Sum{top, rescaled(a, top, c) + rescaled(b, top, c)};
}
// Over WIDTH neighbouring lanes, the same in all of them.
template <int WIDTH>
__device__ __forceinline__ Sum across(Sum s, float c)
{
    float top = s.top;
#pragma unroll
    for (int o = WIDTH / 2; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = rescaled(s, top, c);
#pragma unroll
    for (int o = WIDTH / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return Sum{top, sum};
}

// Raises a running sum's top, and adds a unit's logits under it.
__device__ __forceinline__ void raise(Sum &s, float top, float c)
{
    top = max_nan(s.top, top);
    if (top != s.top) {
        s.sum = rescaled(s, top, c);
        s.top = top;
    }
}
// sum 2^((v - top) c) over units, each element one packed multiply-add and an
// exponential: top c is rounded once, and what that takes off every exponent
// is given back to the sum. Where that rounding is no longer small (a top that is
// a mask, or rows far from zero) differences come first.
template <class T, bool FAR>
struct Under {
    float top, c, off;
    float2 sum;
    __device__ __forceinline__ Under(float t, float cc) : top(t), c(cc), off(t * cc), sum(make_float2(0.0f, 0.0f)) {}
    __device__ __forceinline__ void add(const Unit<T> &x)
    {
        float2 v[Unit<T>::kN / 2];
        x.get(v);
#pragma unroll
        for (int i = 0; i < Unit<T>::kN / 2; ++i) {
            const float2 t = FAR ? mul_f32x2(add_f32x2(v[i], make_float2(-top, -top)), make_float2(c, c))
                                 : fma_f32x2(v[i], make_float2(c, c), make_float2(-off, -off));
            sum = add_f32x2(sum, make_float2(exp2_approx(t.x), exp2_approx(t.y)));
        }
    }
    __device__ __forceinline__ float get() const
    {
        const float s = sum.x + sum.y;
        return FAR ? s : s * exp2_approx(-fmaf(top, c, -off));
    }
};
// An exponent from which on differences come first. Below this its rounding is at most
// 2^-17; from 2^31 on what has to be made good would pass the exponent's range and
// give inf * 0.
__device__ __forceinline__ bool is_far(float v) { return !(fabsf(v) < 256.0f); }
// A given lse whose last place would show: half of it is 2^-13 of q from here on.
__device__ __forceinline__ bool is_lost(float lse) { return !(fabsf(lse * kLog2e) < 4096.0f); }

template <int THREADS>
struct Shared {
    Sum student[THREADS / 32], teacher[THREADS / 32];
    float red[THREADS / 32];
    Sum block;  // this block's part, read by the others of its row
    // the teacher's entries: exponential, and index (-1: absent)
    __align__(16) float e[ZG_TOPK_MAX];
    __align__(16) int at[ZG_TOPK_MAX];
};

// Sixteen bytes that begin `at` elements into the first of two units.
template <class T>
__device__ __forceinline__ uint4 across(uint4 p, uint4 q, int at)
{
    const int words = at * int(sizeof(T)) / 4, bits = sizeof(T) == 2 ? 16 * (at & 1) : 0;
    const bool two = words & 2, one = words & 1;
    const uint32_t a0 = two ? p.z : p.x, a1 = two ? p.w : p.y, a2 = two ? q.x : p.z, a3 = two ? q.y : p.w;
    const uint32_t a4 = two ? q.z : q.x, a5 = two ? q.w : q.y;
    const uint32_t b0 = one ? a1 : a0, b1 = one ? a2 : a1, b2 = one ? a3 : a2, b3 = one ? a4 : a3, b4 = one ? a5 : a4;
    if (sizeof(T) == 4) return make_uint4(b0, b1, b2, b3);
    return make_uint4(__funnelshift_r(b0, b1, bits), __funnelshift_r(b1, b2, bits), __funnelshift_r(b2, b3, bits),
                      __funnelshift_r(b3, b4, bits));
}

// Threads to an SM: as many as registers allow without spilling what is asked
// for ahead (the loss of 4096 x 50257 in bf16: 67 us at 1024, 63 at 1280, 67 at
// 1536; the gradient 130, 128, 125; both 154, 164, 167).
template <bool LOSS, bool GRAD>
constexpr int kToSm = !LOSS ? 1536 : GRAD ? 1024 : 1280;

// Without LOSS, lse is given. A row takes `blocks` blocks of `each` units: with
// LOSS a cluster, in which they exchange sums. A row whose given lse is_lost has its
// maximum and sum taken again, all of it by its first block alone: the logits may be
// written over. (What that asks of the registers takes 1 % from the other rows'
// gradient: 126 us for 125 of 4096 x 50257 in bf16.)
template <class T, class E, bool LOSS, bool GRAD, int THREADS>
__global__ void __launch_bounds__(THREADS, (kToSm<LOSS, GRAD> / THREADS)) distill_kernel(DistillArgs a, int blocks, int each)
{
    __shared__ Shared<THREADS> sh;
    constexpr int N = Unit<T>::kN, kWarps = THREADS / 32, kEntries = (ZG_TOPK_MAX + THREADS - 1) / THREADS;
    const int tid = threadIdx.x;
    const unsigned number = blockIdx.x / unsigned(blocks);
    const int64_t r = number;
    const int rank = int(blockIdx.x - number * unsigned(blocks));
    const float given = LOSS ? 0.0f : a.lse_in[r];
    const float rt = 1.0f / a.temperature, c = rt * kLog2e;
    const T *const z = static_cast<const T *>(a.logits) + r * a.row_stride;

    // The teacher's entries, one or two to a thread, and the logits at them
    // before anything is written over those.
    int at[kEntries];
    float te[kEntries], zt[kEntries];
    const bool entries = (tid & ~31) < a.k;  // of this warp
#pragma unroll
    for (int n = 0; n < kEntries; ++n) {
        const int j = tid + n * THREADS;
        const bool in = entries && j < a.k;
        at[n] = in ? a.t_index[r * a.k + j] : -1;
        te[n] = in ? load1(static_cast<const E *>(a.t_logits) + r * a.k + j) : -INFINITY;
    }
#pragma unroll
    for (int n = 0; n < kEntries; ++n) {
        if (at[n] < 0 || at[n] >= a.vocab) at[n] = -1, te[n] = -INFINITY;
        zt[n] = at[n] >= 0 ? load1(z + at[n]) : 0.0f;
    }
    const bool lost = !LOSS && is_lost(given);
    if (lost) {
        if (rank != 0) return;
        each = a.vocab / N + 2;
    }
    const Row<T> row(z, a.vocab, each, rank);
    const Part &part = row.part;
    const T *const base = row.base;
    const uint4 *const from = row.from();
    const int units = row.units;

    Sum s = none();
    if (LOSS) {
        auto take_in = [&](const Unit<T> (&x)[kAhead], int u, bool whole) {
            typename Unit<T>::Top top;
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (whole || u + i * THREADS < units) top.add(x[i]);
            raise(s, top.get(), c);
            if (s.top == -INFINITY) return;  // nothing but masked logits so far
            if (is_far(s.top * c)) {
                Under<T, true> under(s.top, c);
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (whole || u + i * THREADS < units) under.add(x[i]);
                s.sum += under.get();
            } else {
                Under<T, false> under(s.top, c);
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (whole || u + i * THREADS < units) under.add(x[i]);
                s.sum += under.get();
            }
        };
        int u = tid;
        for (; u + (kAhead - 1) * THREADS < units; u += kAhead * THREADS) {
            Unit<T> x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) x[i].w = GRAD ? from[u + i * THREADS] : __ldcs(from + u + i * THREADS);
            take_in(x, u, true);
        }
        if (u < units) {
            Unit<T> x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (u + i * THREADS < units) x[i].w = from[u + i * THREADS];
            take_in(x, u, false);
        }
    }
    if (lost) {  // differences first throughout
#pragma unroll 1
        for (int u = tid; u < units; u += THREADS) {
            Unit<T> x;
            x.w = from[u];
            typename Unit<T>::Top top;
            top.add(x);
            raise(s, top.get(), c);
            Under<T, true> under(s.top, c);
            under.add(x);
            if (s.top != -INFINITY) s.sum += under.get();
        }
    }
    if (LOSS || lost) {
        const int i = row.ragged(tid);
        if (i >= 0) {
            const float v = load1(base + i);
            s = join(s, Sum{v, v == -INFINITY ? 0.0f : v - v + 1.0f}, c);
        }
    }
    // one barrier for both sums, the student's and the teacher's
    {
        Sum t = none();
#pragma unroll
        for (int n = 0; n < kEntries; ++n) {
            const int j = tid + n * THREADS;
            if (entries && j < ZG_TOPK_MAX) sh.at[j] = at[n];
            if (entries) t = join(t, Sum{te[n], te[n] == -INFINITY ? 0.0f : te[n] - te[n] + 1.0f}, c);
        }
        if (entries) t = across<32>(t, c);
        if (LOSS || lost) s = across<32>(s, c);
        if (tid % 32 == 0) {
            sh.teacher[tid / 32] = t;
            sh.student[tid / 32] = s;
        }
    }
    __syncthreads();
    // the lower half of a warp joins the student's, the upper the teacher's
    Sum t = across<kWarps>((tid & 16 ? sh.teacher : sh.student)[tid % kWarps], c);
    s = Sum{__shfl_sync(0xffffffffu, t.top, 0), __shfl_sync(0xffffffffu, t.sum, 0)};
    t = Sum{__shfl_sync(0xffffffffu, t.top, 16), __shfl_sync(0xffffffffu, t.sum, 16)};
    const bool empty = t.top == -INFINITY;
    float lse = 0.0f;
    if (LOSS) {
        if (blocks > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            if (tid == 0) sh.block = s;
            cluster.sync();
            s = none();
            for (int i = 0; i < blocks; ++i) s = join(s, cluster.map_shared_rank(&sh, i)->block, c);
            cluster.barrier_arrive();  // its reads are done; nobody leaves before all are
        }
        const float log_sum = logf(s.sum);
        lse = fmaf(s.top, rt, log_sum);
        if (rank == 0 && !entries && tid % 32 == 0) sh.red[tid / 32] = 0.0f;
        if (rank == 0 && entries) {
            // p = 0 leaves its term out; a NaN stays
            float term = 0.0f;
            const float log_total = logf(t.sum);
#pragma unroll
            for (int n = 0; n < kEntries; ++n) {
                const float d = te[n] - t.top, p = at[n] >= 0 ? exp2_approx(d * c) / t.sum : 0.0f;
                if (p != 0.0f) term += p * ((d * rt - log_total) - ((zt[n] - s.top) * rt - log_sum));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
            if (tid % 32 == 0) sh.red[tid / 32] = term;
        }
        if (rank == 0 && tid == 0 && a.lse) a.lse[r] = empty ? 0.0f : lse;
    } else {
        lse = given;
    }
    if (GRAD) {
#pragma unroll
        for (int n = 0; n < kEntries; ++n) {
            const int j = tid + n * THREADS;
            if (entries && j < ZG_TOPK_MAX) sh.e[j] = at[n] >= 0 ? exp2_approx((te[n] - t.top) * c) : 0.0f;
        }
        const float g = a.scale * a.temperature * (a.dloss ? a.dloss[r] : 1.0f);
        T *const dz = static_cast<T *>(a.dlogits) + r * a.drow_stride - part.head;
        // 2^(v c - low), low = lse log2(e) rounded once and made good in the factor.
        // For rows far from zero lse's own last place would show, and q is
        // 2^((v - top) c) / sum.
        const float low = lse * kLog2e;
        const bool far = LOSS ? is_far(low) : lost;
        const float gg = far ? g / s.sum : g * exp2_approx(-fmaf(lse, kLog2eRest, fmaf(lse, kLog2e, -low)));
        auto gradient1 = [&](float v) {
            return empty ? 0.0f : exp2_approx(far ? (v - s.top) * c : fmaf(v, c, -low)) * gg;
        };
        auto gradient = [&](Unit<T> &x, auto is_far_too) {
            float2 v[N / 2];
            x.get(v);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float2 q = decltype(is_far_too)::value
                                     ? mul_f32x2(add_f32x2(v[i], make_float2(-s.top, -s.top)), make_float2(c, c))
                                     : fma_f32x2(v[i], make_float2(c, c), make_float2(-low, -low));
                v[i] = mul_f32x2(make_float2(exp2_approx(q.x), exp2_approx(q.y)), make_float2(gg, gg));
            }
            x.set(v);
        };
        const int phase = int((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T));
        int i0, i1;  // what is written in whole units
        if (phase == 0) {
            i0 = part.u0 * N;
            i1 = part.u1 * N;
        } else {
            // the output's units lie across the input's: whole ones of the output
            // that lie across whole ones of the part
            i0 = (part.u0 * N + 1 + phase + N - 1) / N * N - phase;
            i1 = max((part.u1 * N - 1 + phase) / N * N - phase, i0);
        }
        auto pass = [&](auto is_far_too) {
            if (phase != 0) {
                // each from the two units that it lies across, the second of which a
                // neighbour reads first; two at a time (one: 80 and 94 us for 72 and 89)
                const uint4 *const in = reinterpret_cast<const uint4 *>(base);
                const int at = (N - phase) % N;
                for (int i = i0 + tid * N; i < i1; i += 2 * THREADS * N) {
                    uint4 p[2], q[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int u = (i + j * THREADS * N) / N;
                        if (i + j * THREADS * N < i1) {
                            p[j] = in[u];
                            q[j] = in[u + 1];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (i + j * THREADS * N >= i1) break;
                        Unit<T> x;
                        x.w = across<T>(p[j], q[j], at);
                        gradient(x, is_far_too);
                        __stcs(reinterpret_cast<uint4 *>(dz + i + j * THREADS * N), x.w);
                    }
                }
                return;
            }
            uint4 *const to = reinterpret_cast<uint4 *>(dz) + part.u0;
            int u = tid;
            for (; u + (kAhead - 1) * THREADS < units; u += kAhead * THREADS) {
                Unit<T> x[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) x[i].w = LOSS ? __ldcs(from + u + i * THREADS) : from[u + i * THREADS];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    gradient(x[i], is_far_too);
                    __stcs(to + u + i * THREADS, x[i].w);
                }
            }
            for (; u < units; u += THREADS) {
                Unit<T> x;
                x.w = from[u];
                gradient(x, is_far_too);
                __stcs(to + u, x.w);
            }
        };
        if (empty)
            for (int i = i0 + tid * N; i < i1; i += THREADS * N)
                __stcs(reinterpret_cast<uint4 *>(dz + i), make_uint4(0u, 0u, 0u, 0u));
        else if (far)
            pass(std::true_type{});
        else
            pass(std::false_type{});
        // the rest, less than two units at either end
        i0 = min(i0, part.last);
        i1 = min(i1, part.last);
        if (part.first + tid < i0) store1(dz + part.first + tid, gradient1(load1(base + part.first + tid)));
        if (i1 + tid < part.last) store1(dz + i1 + tid, gradient1(load1(base + i1 + tid)));
        __syncthreads();
        // The entries of this part; the first of a repeated index answers for all.
#pragma unroll
        for (int n = 0; n < kEntries; ++n) {
            const int j = tid + n * THREADS, i = part.head + at[n];
            if (empty || at[n] < 0 || i < part.first || i >= part.last) continue;
            float sum = 0.0f;
            int first = j;
#pragma unroll 2
            for (int m = 0; m < a.k; m += 4) {
                const int4 other = *reinterpret_cast<const int4 *>(&sh.at[m]);
                const float4 e = *reinterpret_cast<const float4 *>(&sh.e[m]);
                sum += other.x == at[n] ? e.x : 0.0f;
                sum += other.y == at[n] ? e.y : 0.0f;
                sum += other.z == at[n] ? e.z : 0.0f;
                sum += other.w == at[n] ? e.w : 0.0f;
                first = min(first, min(min(other.x == at[n] ? m : j, other.y == at[n] ? m + 1 : j),
                                       min(other.z == at[n] ? m + 2 : j, other.w == at[n] ? m + 3 : j)));
            }
            const bool write = first == j;
            const float p = sum / t.sum;
            if (write)
                store1(dz + i, far ? exp2_approx((zt[n] - s.top) * c) * gg - p * g
                                   : (exp2_approx(fmaf(zt[n], rt, -lse) * kLog2e) - p) * g);
        }
    } else {
        __syncthreads();
    }
    if (LOSS && rank == 0 && tid == 0) {
        float loss = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) loss += sh.red[i];
        a.loss[r] = empty ? 0.0f : a.temperature * a.temperature * loss;
    }
    if (LOSS && blocks > 1) cg::this_cluster().barrier_wait();
}

template <class T, class E, bool LOSS, bool GRAD, int THREADS>
cudaError_t launch(const DistillArgs &a, int64_t blocks, int64_t units, cudaStream_t st)
{
    if (a.rows * blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(a.rows * blocks));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(blocks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = LOSS && blocks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, &distill_kernel<T, E, LOSS, GRAD, THREADS>, a, int(blocks),
                              int((units + blocks - 1) / blocks));
}

template <class T, class E, bool LOSS, bool GRAD>
cudaError_t by_size(const DistillArgs &a, cudaStream_t st)
{
    const int64_t units = (int64_t(a.vocab) * int64_t(sizeof(T)) + 30) / 16;
    if constexpr (!LOSS) {
        // Nothing to exchange: as many small blocks as a row has parts for, of up to
        // 1,728 units (at 1,152, 1,728, 2,304 and 3,456: 4096 x 50257 in bf16 132, 126,
        // 126 and 130 us, in binary32 249, 241, 243 and 248; 1000 rows 37.5, 37.2, 36.3
        // and 44.5; 777 x 131075 67.8, 66.7, 66.0 and 72.2). 1 to 60 rows take 4.2 to
        // 5.0 us with either these or smaller parts.
        const int64_t blocks = (units + 1727) / 1728;
        return launch<T, E, false, true, 128>(a, blocks, units, st);
    } else {
        // The smallest blocks keep most rows in flight, at different places at
        // once, so that the ends of some do not leave memory idle: for the loss
        // of 4096 x 50257 in bf16, 128 threads to a row 70 us, 256 79, 512 98. A
        // row that is read again for its gradient has to be in L2 still, so the
        // rows in flight (1024 threads to an SM) have 64 MB together: 128
        // threads 201 us, 256 159, 512 181; of 777 x 131075, 106, 112 and 91.
        // Rows too few to fill half the GPU take more threads, then more blocks.
        const int64_t held = GRAD ? (int64_t(64) << 20) / (152 * units * 16) : 8;  // rows to an SM
        int threads = held >= 8 ? 128 : held >= 4 ? 256 : 512;
        int64_t blocks = 1;
        while (a.rows * blocks * threads < 152 * 512 && units / blocks > 4 * threads) {
            if (threads < 512)
                threads *= 2;
            else if (blocks < 8)
                blocks *= 2;
            else
                break;
        }
        if (threads == 128) return launch<T, E, true, GRAD, 128>(a, blocks, units, st);
        if (threads == 256) return launch<T, E, true, GRAD, 256>(a, blocks, units, st);
        return launch<T, E, true, GRAD, 512>(a, blocks, units, st);
    }
}

template <class T, class E>
cudaError_t by_pass(const DistillArgs &a, cudaStream_t st)
{
    if (!a.loss) return by_size<T, E, false, true>(a, st);
    return a.dlogits ? by_size<T, E, true, true>(a, st) : by_size<T, E, true, false>(a, st);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs &a, cudaStream_t st)
{
    const bool bf = a.dtype == ZG_DTYPE_BF16, tbf = a.t_dtype == ZG_DTYPE_BF16;
    if (bf) return tbf ? by_pass<uint16_t, uint16_t>(a, st) : by_pass<uint16_t, float>(a, st);
    return tbf ? by_pass<float, uint16_t>(a, st) : by_pass<float, float>(a, st);
}

}  // namespace zg
