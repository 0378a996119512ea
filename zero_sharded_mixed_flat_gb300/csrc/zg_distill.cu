// The distillation loss from a teacher's top logits, and its gradient.
//
// With z a row of the student's logits, T the temperature and p the softmax of
// the teacher's k entries, loss = T^2 sum_j p_j (log p_j - z_{i_j} / T + lse),
// lse = log sum exp(z / T), and dz = scale dloss T (exp(z / T - lse) - p), where
// p acts on its k indices alone. So a row costs a sum over the vocabulary, k
// gathered values, and for the gradient one exponential per logit again.
//
// Bound by memory: each logit is read once (2 bytes in bf16) and its gradient
// written once. The row is shared out over a cluster of blocks, each of which
// copies its part into shared memory, so that the second pass reads nothing
// from memory: the blocks exchange their maximum and sum, no more. A part is
// whole 16-byte units of the row but for its two ends, so any row, however it
// is aligned, moves in wide copies.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "zg_launch.h"
#include "zg_ops.h"

namespace zg {
namespace {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.44269504f;
constexpr int kAhead = 4;  // units that a thread asks for before it uses the first

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = uint16_t(pack_bf16x2(v, 0.0f)); }

__device__ __forceinline__ float exp2_approx(float v)
{
    float d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
    return d;
}
// max that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
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

// A sum of exponentials as sum 2^((z - top) c), c = log2(e) / T, with top the
// largest z seen: differences first, so that rows of a type's lowest value
// neither overflow nor count as masked.
struct Sum {
    float top, sum;
};
__device__ __forceinline__ Sum none() { return Sum{-INFINITY, 0.0f}; }
// An empty part (top = -inf) adds nothing; a NaN or +inf makes the sum NaN.
__device__ __forceinline__ Sum join(Sum a, Sum b, float c)
{
    const float top = max_nan(a.top, b.top);
    const float sa = a.top == -INFINITY ? 0.0f : a.sum * exp2_approx((a.top - top) * c);
    const float sb = b.top == -INFINITY ? 0.0f : b.sum * exp2_approx((b.top - top) * c);
    return Sum{top, sa + sb};
}

// Sixteen bytes of logits: eight bf16 or four binary32.
template <class T>
struct Unit;
template <>
struct Unit<uint16_t> {
    static constexpr int kN = 8;
    uint4 w;
    __device__ __forceinline__ void get(float2 (&v)[4]) const
    {
        v[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
        v[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
        v[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
        v[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
    }
    __device__ __forceinline__ void set(const float2 (&v)[4])
    {
        w = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                       pack_bf16x2(v[3].x, v[3].y));
    }
};
template <>
struct Unit<float> {
    static constexpr int kN = 4;
    uint4 w;
    __device__ __forceinline__ void get(float2 (&v)[2]) const
    {
        v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
        v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    __device__ __forceinline__ void set(const float2 (&v)[2])
    {
        w = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
    }
};

// A unit's logits joined to a thread's running sum.
template <int N>
__device__ __forceinline__ void take_in(const float2 (&v)[N], float c, Sum &s)
{
    float top = s.top;
#pragma unroll
    for (int i = 0; i < N; ++i) top = max_nan(top, max_nan(v[i].x, v[i].y));
    if (top == -INFINITY) return;  // nothing but masked logits so far
    if (top != s.top) {
        s.sum = s.top == -INFINITY ? 0.0f : s.sum * exp2_approx((s.top - top) * c);
        s.top = top;
    }
    float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 t = mul_f32x2(add_f32x2(v[i], make_float2(-top, -top)), make_float2(c, c));
        part = add_f32x2(part, make_float2(exp2_approx(t.x), exp2_approx(t.y)));
    }
    s.sum += part.x + part.y;
}

template <int THREADS>
struct Shared {
    Sum warps[THREADS / 32];
    float red[THREADS / 32];
    Sum block;  // this block's part, read by the others of its row
    // the teacher's entries: weight, index (-1: absent), the student's logit
    float p[ZG_TOPK_MAX], z[ZG_TOPK_MAX];
    __align__(16) int at[ZG_TOPK_MAX];
};

template <int WARPS, class Op>
__device__ __forceinline__ float block_fold(float v, float *red, Op op)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = red[threadIdx.x % WARPS];
#pragma unroll
    for (int o = WARPS / 2; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    return v;
}

// The parts of a row. Elements are counted from the 16-byte boundary at or
// below the row's first: the row is [head, head + vocab), units [lo, hi) are a
// block's, and its elements [first, last).
struct Part {
    int head;
    int64_t lo, hi, first, last;
};
template <class T>
__device__ __forceinline__ Part part_of(const T *row, int vocab, int blocks, int rank)
{
    constexpr int N = Unit<T>::kN;
    Part p;
    p.head = int((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int64_t units = (int64_t(p.head) + vocab + N - 1) / N, each = (units + blocks - 1) / blocks;
    p.lo = rank * each < units ? rank * each : units;
    p.hi = p.lo + each < units ? p.lo + each : units;
    p.first = p.lo * N > p.head ? p.lo * N : p.head;
    p.last = p.hi * N < p.head + int64_t(vocab) ? p.hi * N : p.head + int64_t(vocab);
    return p;
}

__device__ __forceinline__ void copy_async(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sixteen bytes from element i of `base`, which is aligned to its units only,
// by whole words: up to one element before and after them is read too.
__device__ __forceinline__ void read_shifted(const uint16_t *base, int64_t i, Unit<uint16_t> &x)
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(base) + (i >> 1);
    x.w = make_uint4(w[0], w[1], w[2], w[3]);
    if (i & 1) {
        const uint32_t last = w[4];
        x.w = make_uint4(__funnelshift_r(x.w.x, x.w.y, 16), __funnelshift_r(x.w.y, x.w.z, 16),
                         __funnelshift_r(x.w.z, x.w.w, 16), __funnelshift_r(x.w.w, last, 16));
    }
}
__device__ __forceinline__ void read_shifted(const float *base, int64_t i, Unit<float> &x)
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(base) + i;
    x.w = make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kStages = 4;

// KEEP: the part is copied into shared memory, in kStages groups, and both
// passes read it there; else each reads it from memory (L2). Without LOSS, lse
// is given. A row takes `blocks` blocks: a cluster where they exchange sums.
template <class T, class E, bool LOSS, bool GRAD, bool KEEP, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) distill_kernel(DistillArgs a, int blocks)
{
    extern __shared__ __align__(16) unsigned char raw[];
    __shared__ Shared<THREADS> sh;
    constexpr int N = Unit<T>::kN, kWarps = THREADS / 32;
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x / unsigned(blocks);
    const int rank = int(blockIdx.x % unsigned(blocks));
    const T *const z = static_cast<const T *>(a.logits) + r * a.row_stride;
    const float rt = 1.0f / a.temperature, c = rt * kLog2e;
    const Part part = part_of(z, a.vocab, blocks, rank);
    const T *const base = z - part.head;  // only elements [head, head + vocab) are touched
    const int64_t u0 = (part.first + N - 1) / N, u1 = part.last / N;  // whole units; the ends are ragged
    const uint4 *const from = reinterpret_cast<const uint4 *>(base);
    Unit<T> *const kept = reinterpret_cast<Unit<T> *>(raw) - part.lo;
    const int per_stage = int((u1 - u0 + THREADS * kStages - 1) / (THREADS * kStages)) * THREADS;

    if (KEEP) {
#pragma unroll
        for (int g = 0; g < kStages; ++g) {
            for (int64_t u = u0 + g * per_stage + tid; u < u1 && u < u0 + (g + 1) * per_stage; u += THREADS)
                copy_async(&kept[u], from + u);
            commit_copies();
        }
    }

    // The teacher's entries, and the logits at them before anything is written
    // over those: a block needs those of its part for their gradients, the first
    // block all for the loss.
    float tm = -INFINITY;
    for (int j = tid; j < ZG_TOPK_MAX; j += THREADS) {
        int at = -1;
        float t = -INFINITY, zt = 0.0f;
        if (j < a.k) {
            at = a.t_index[r * a.k + j];
            if (at < 0 || at >= a.vocab) at = -1;
            if (at >= 0) {
                t = load1(static_cast<const E *>(a.t_logits) + r * a.k + j) * rt;
                zt = load1(z + at);
            }
        }
        sh.at[j] = at;
        sh.p[j] = t;
        sh.z[j] = zt;
        tm = max_nan(tm, t);
    }
    tm = block_fold<kWarps>(tm, sh.red, [](float x, float y) { return max_nan(x, y); });
    if (tm == -INFINITY) {  // a row without entries: the same in every block of it
        if (KEEP) wait_copies<0>();
        if (LOSS && rank == 0 && tid == 0) {
            a.loss[r] = 0.0f;
            if (a.lse) a.lse[r] = 0.0f;
        }
        if (GRAD) {
            T *const dz = static_cast<T *>(a.dlogits) + r * a.drow_stride - part.head;
            if ((reinterpret_cast<uintptr_t>(dz) & 15u) == 0) {
                for (int64_t u = u0 + tid; u < u1; u += THREADS)
                    __stcs(reinterpret_cast<uint4 *>(dz) + u, make_uint4(0u, 0u, 0u, 0u));
                for (int64_t i = part.first + tid; i < part.last && i < u0 * N; i += THREADS) store1(dz + i, 0.0f);
                for (int64_t i = (u1 > u0 ? u1 : u0) * N + tid; i < part.last; i += THREADS) store1(dz + i, 0.0f);
            } else {
                for (int64_t i = part.first + tid; i < part.last; i += THREADS) store1(dz + i, 0.0f);
            }
        }
        return;
    }
    float mine = 0.0f;
    for (int j = tid; j < a.k; j += THREADS) {
        const float e = sh.at[j] >= 0 ? exp2_approx((sh.p[j] - tm) * kLog2e) : 0.0f;
        mine += e;
        if (!LOSS) sh.p[j] = e;
    }
    const float total = block_fold<kWarps>(mine, sh.red, [](float x, float y) { return x + y; });

    float lse;
    if (LOSS) {
        Sum s = none();
        if (KEEP) {
#pragma unroll
            for (int g = 0; g < kStages; ++g) {
                if (g == 0) wait_copies<3>();
                if (g == 1) wait_copies<2>();
                if (g == 2) wait_copies<1>();
                if (g == 3) wait_copies<0>();
                // a thread reads what it copied itself
                for (int64_t u = u0 + g * per_stage + tid; u < u1 && u < u0 + (g + 1) * per_stage; u += THREADS) {
                    float2 v[N / 2];
                    kept[u].get(v);
                    take_in(v, c, s);
                }
            }
        } else {
            int64_t u = u0 + tid;
            for (; u + (kAhead - 1) * THREADS < u1; u += kAhead * THREADS) {
                Unit<T> x[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) x[i].w = from[u + i * THREADS];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    float2 v[N / 2];
                    x[i].get(v);
                    take_in(v, c, s);
                }
            }
            for (; u < u1; u += THREADS) {
                Unit<T> x;
                x.w = from[u];
                float2 v[N / 2];
                x.get(v);
                take_in(v, c, s);
            }
        }
        {  // the ragged ends
            const int64_t head_end = u0 * N < part.last ? u0 * N : part.last;
            const int64_t tail = u1 * N > head_end ? u1 * N : head_end;
            int64_t i = -1;
            if (part.first + tid < head_end) i = part.first + tid;
            if (tid >= 32 && tail + tid - 32 < part.last) i = tail + tid - 32;
            if (i >= 0) {
                const float v = load1(base + i);
                s = join(s, Sum{v, v == -INFINITY ? 0.0f : v - v + 1.0f}, c);
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            s = join(s, Sum{__shfl_xor_sync(0xffffffffu, s.top, o), __shfl_xor_sync(0xffffffffu, s.sum, o)}, c);
        if (tid % 32 == 0) sh.warps[tid / 32] = s;
        __syncthreads();
        s = sh.warps[tid % kWarps];
#pragma unroll
        for (int o = kWarps / 2; o; o >>= 1)
            s = join(s, Sum{__shfl_xor_sync(0xffffffffu, s.top, o), __shfl_xor_sync(0xffffffffu, s.sum, o)}, c);
        if (blocks > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            if (tid == 0) sh.block = s;
            cluster.sync();
            s = none();
            for (int i = 0; i < blocks; ++i) s = join(s, cluster.map_shared_rank(&sh, i)->block, c);
            cluster.sync();  // nobody leaves while its part may be read
        }
        const float log_sum = logf(s.sum);
        lse = fmaf(s.top, rt, log_sum);
        if (rank == 0) {
            // p_j = 0 leaves its term out; a NaN stays
            float term = 0.0f;
            const float log_total = logf(total);
            for (int j = tid; j < a.k; j += THREADS) {
                const float t = sh.p[j] - tm, p = sh.at[j] >= 0 ? exp2_approx(t * kLog2e) / total : 0.0f;
                if (p != 0.0f) term += p * ((t - log_total) - ((sh.z[j] - s.top) * rt - log_sum));
            }
            const float loss = block_fold<kWarps>(term, sh.red, [](float x, float y) { return x + y; });
            if (tid == 0) {
                a.loss[r] = a.temperature * a.temperature * loss;
                if (a.lse) a.lse[r] = lse;
            }
        }
        if (GRAD) {
            for (int j = tid; j < a.k; j += THREADS) sh.p[j] = sh.at[j] >= 0 ? exp2_approx((sh.p[j] - tm) * kLog2e) : 0.0f;
            __syncthreads();
        }
    } else {
        lse = a.lse_in[r];
    }
    if (!GRAD) return;

    const float g = a.scale * a.temperature * (a.dloss ? a.dloss[r] : 1.0f);
    T *const dz = static_cast<T *>(a.dlogits) + r * a.drow_stride - part.head;
    auto gradient = [&](Unit<T> &x) {
        float2 v[N / 2];
        x.get(v);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 q = mul_f32x2(fma_f32x2(v[i], make_float2(rt, rt), make_float2(-lse, -lse)), make_float2(kLog2e, kLog2e));
            v[i] = mul_f32x2(make_float2(exp2_approx(q.x), exp2_approx(q.y)), make_float2(g, g));
        }
        x.set(v);
    };
    const int phase = int((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T));
    int64_t i0, i1;  // what is written in whole units
    if (phase == 0) {
        uint4 *const to = reinterpret_cast<uint4 *>(dz);
        i0 = u0 * N;
        i1 = (u1 > u0 ? u1 : u0) * N;
        int64_t u = u0 + tid;
        if (!KEEP)
            for (; u + (kAhead - 1) * THREADS < u1; u += kAhead * THREADS) {
                Unit<T> x[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) x[i].w = from[u + i * THREADS];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    gradient(x[i]);
                    __stcs(to + u + i * THREADS, x[i].w);
                }
            }
        for (; u < u1; u += THREADS) {
            Unit<T> x;
            if (KEEP)
                x = kept[u];
            else
                x.w = from[u];
            gradient(x);
            __stcs(to + u, x.w);
        }
    } else {
        // the output's units lie across the input's: whole ones of the output,
        // read a word at a time, with an element to spare at both ends
        i0 = (u0 * N + 1 + phase + N - 1) / N * N - phase;
        i1 = (u1 * N - 1 + phase) / N * N - phase;
        if (i1 < i0) i1 = i0;
        const T *const src = KEEP ? reinterpret_cast<const T *>(kept) : base;
        for (int64_t i = i0 + int64_t(tid) * N; i < i1; i += THREADS * N) {
            Unit<T> x;
            read_shifted(src, i, x);
            gradient(x);
            __stcs(reinterpret_cast<uint4 *>(dz + i), x.w);
        }
    }
    // the rest, at most two units' elements at either end
    if (i0 > part.last) i0 = i1 = part.last;
    for (int64_t i = part.first + tid; i < i0; i += THREADS) store1(dz + i, exp2_approx(fmaf(load1(base + i), rt, -lse) * kLog2e) * g);
    for (int64_t i = i1 + tid; i < part.last; i += THREADS) store1(dz + i, exp2_approx(fmaf(load1(base + i), rt, -lse) * kLog2e) * g);
    __syncthreads();
    // The entries of this part; the first of a repeated index answers for all.
    const float weight = 1.0f / total;
    for (int j = tid; j < a.k; j += THREADS) {
        const int at = sh.at[j];
        const int64_t i = part.head + int64_t(at);
        if (at < 0 || i < part.first || i >= part.last) continue;
        float sum = 0.0f;
        bool write = true;
        for (int n = 0; n < a.k; n += 4) {
            const int4 other = *reinterpret_cast<const int4 *>(&sh.at[n]);
            if (other.x == at) sum += sh.p[n], write = write && n >= j;
            if (other.y == at) sum += sh.p[n + 1], write = write && n + 1 >= j;
            if (other.z == at) sum += sh.p[n + 2], write = write && n + 2 >= j;
            if (other.w == at) sum += sh.p[n + 3], write = write && n + 3 >= j;
        }
        if (write) store1(dz + i, (exp2_approx(fmaf(sh.z[j], rt, -lse) * kLog2e) - sum * weight) * g);
    }
}

template <class T, class E, bool LOSS, bool GRAD, bool KEEP, int THREADS>
cudaError_t launch(const DistillArgs &a, int blocks, size_t smem, cudaStream_t st)
{
    auto *kernel = &distill_kernel<T, E, LOSS, GRAD, KEEP, THREADS>;
    if (smem) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    if (a.rows * blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(a.rows * blocks));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(blocks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = LOSS && blocks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, blocks);
}

#ifndef ZG_DT
#define ZG_DT 0
#endif
#ifndef ZG_DB
#define ZG_DB 0
#endif

template <class T, class E, bool LOSS, bool GRAD>
cudaError_t by_size(const DistillArgs &a, cudaStream_t st)
{
    const int64_t bytes = int64_t(a.vocab) * int64_t(sizeof(T)) + 32;
    constexpr int64_t kEach = 27 * 1024;  // shared memory of 128 threads: eight such blocks to an SM
    int threads = bytes <= kEach ? 128 : bytes <= 2 * kEach ? 256 : 512;
    int blocks = 1;
    while (blocks < 8 && ((bytes + blocks - 1) / blocks > kEach * threads / 128 || (a.rows * blocks < 152 && bytes / blocks > 16384)))
        blocks *= 2;
    if (ZG_DT && threads == 512) threads = ZG_DT;
    if (ZG_DB && blocks == 1 && bytes > 2 * kEach) blocks = ZG_DB;
    const int64_t part = ((bytes + 15) / 16 + blocks - 1) / blocks * 16 + 32;
    if (LOSS && part <= 200 * 1024) {
        if (threads == 128) return launch<T, E, LOSS, GRAD, LOSS, 128>(a, blocks, size_t(part), st);
        if (threads == 256) return launch<T, E, LOSS, GRAD, LOSS, 256>(a, blocks, size_t(part), st);
        return launch<T, E, LOSS, GRAD, LOSS, 512>(a, blocks, size_t(part), st);
    }
    if (threads == 128) return launch<T, E, LOSS, GRAD, false, 128>(a, blocks, 0, st);
    return launch<T, E, LOSS, GRAD, false, 512>(a, blocks, 0, st);
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
