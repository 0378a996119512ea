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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
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

struct Teacher {
    float p[ZG_TOPK_MAX];
    int at[ZG_TOPK_MAX];
};

struct Shared {
    Sum warps[kWarps];
    Sum block;         // this block's part, read by the others
    float red[kWarps];
    Teacher t;
};

__device__ __forceinline__ float block_sum(float v, float *red)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = red[threadIdx.x % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float block_max(float v, float *red)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = red[threadIdx.x % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
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

// KEEP: the part lies in shared memory between the passes; else the second pass
// reads it from memory (L2) again. C: blocks of the cluster.
template <class T, class E, bool LOSS, bool GRAD, bool KEEP>
__global__ void __launch_bounds__(kThreads, 2) distill_kernel(DistillArgs a, int blocks)
{
    extern __shared__ __align__(16) unsigned char raw[];
    __shared__ Shared sh;
    constexpr int N = Unit<T>::kN;
    Unit<T> *const kept = reinterpret_cast<Unit<T> *>(raw);
    const int tid = threadIdx.x, rank = blocks > 1 ? int(cg::this_cluster().block_rank()) : 0;
    const int64_t r = blockIdx.x / blocks;
    const T *const z = static_cast<const T *>(a.logits) + r * a.row_stride;
    const float rt = 1.0f / a.temperature, c = rt * kLog2e;
    const Part part = part_of(z, a.vocab, blocks, rank);
    const T *const base = z - part.head;  // only elements [head, head + vocab) are touched

    // the teacher's entries (k is at most the number of threads)
    float t = -INFINITY;
    int at = -1;
    if (tid < a.k) {
        at = a.t_index[r * a.k + tid];
        if (at < 0 || at >= a.vocab) at = -1;
        if (at >= 0) t = load1(static_cast<const E *>(a.t_logits) + r * a.k + tid) * rt;
    }
    const float tm = block_max(t, sh.red);
    if (tm == -INFINITY) {  // a row without entries: the same in every block of it
        if (LOSS && rank == 0 && tid == 0) {
            a.loss[r] = 0.0f;
            if (a.lse) a.lse[r] = 0.0f;
        }
        if (GRAD) {
            T *const dz = static_cast<T *>(a.dlogits) + r * a.drow_stride - part.head;
            for (int64_t i = part.first + tid; i < part.last; i += kThreads) store1(dz + i, 0.0f);
        }
        return;
    }
    const bool mine = at >= 0 && part.head + int64_t(at) >= part.first && part.head + int64_t(at) < part.last;
    // the entries' logits, before anything is written over them: a block needs
    // those of its part for their gradients, the first block all for the loss
    const float zt = at >= 0 && (mine || (LOSS && rank == 0)) ? load1(z + at) : 0.0f;

    float lse;
    if (LOSS) {
        // first pass: whole units, and the elements of the part's ragged ends
        Sum s = none();
        const int64_t u0 = (part.first + N - 1) / N, u1 = part.last / N;
        const uint4 *const from = reinterpret_cast<const uint4 *>(base);
        int64_t u = u0 + tid;
        for (; u + (kAhead - 1) * kThreads < u1; u += kAhead * kThreads) {
            Unit<T> x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) x[i].w = KEEP ? __ldcs(from + u + i * kThreads) : from[u + i * kThreads];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (KEEP) kept[u + i * kThreads - part.lo] = x[i];
                float2 v[N / 2];
                x[i].get(v);
                take_in(v, c, s);
            }
        }
        for (; u < u1; u += kThreads) {
            Unit<T> x;
            x.w = from[u];
            if (KEEP) kept[u - part.lo] = x;
            float2 v[N / 2];
            x.get(v);
            take_in(v, c, s);
        }
        {
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
        const float e = at >= 0 ? exp2_approx((t - tm) * kLog2e) : 0.0f;
        const float total = block_sum(e, sh.red);
        const float p = e / total;
        if (tid < a.k) {
            sh.t.p[tid] = p;
            sh.t.at[tid] = at;
        }
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
            const float term = at >= 0 && p != 0.0f ? p * (((t - tm) - logf(total)) - ((zt - s.top) * rt - log_sum)) : 0.0f;
            const float loss = block_sum(term, sh.red);
            if (tid == 0) {
                a.loss[r] = a.temperature * a.temperature * loss;
                if (a.lse) a.lse[r] = lse;
            }
        }
    } else {
        lse = a.lse_in[r];
        const float e = at >= 0 ? exp2_approx((t - tm) * kLog2e) : 0.0f;
        const float total = block_sum(e, sh.red);
        if (tid < a.k) {
            sh.t.p[tid] = e / total;
            sh.t.at[tid] = at;
        }
        __syncthreads();
    }
    if (!GRAD) return;

    const float g = a.scale * a.temperature * (a.dloss ? a.dloss[r] : 1.0f);
    // an entry's gradient; the first of a repeated index answers for all of them
    float patch = 0.0f;
    bool write = mine;
    if (mine) {
        float sum = 0.0f;
        for (int j = 0; j < a.k; ++j)
            if (sh.t.at[j] == at) {
                if (j < tid) write = false;
                sum += sh.t.p[j];
            }
        patch = (exp2_approx(fmaf(zt, rt, -lse) * kLog2e) - sum) * g;
    }
    if (!KEEP || !LOSS) __syncthreads();  // the entries' logits are read before they are written over
    // second pass
    T *const dz = static_cast<T *>(a.dlogits) + r * a.drow_stride - part.head;
    const bool wide = (reinterpret_cast<uintptr_t>(dz) & 15u) == 0;
    const int64_t u0 = (part.first + N - 1) / N, u1 = part.last / N;
    const uint4 *const from = reinterpret_cast<const uint4 *>(base);
    auto finish = [&](Unit<T> x, int64_t u) {
        float2 v[N / 2];
        x.get(v);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 q = mul_f32x2(fma_f32x2(v[i], make_float2(rt, rt), make_float2(-lse, -lse)), make_float2(kLog2e, kLog2e));
            v[i] = mul_f32x2(make_float2(exp2_approx(q.x), exp2_approx(q.y)), make_float2(g, g));
        }
        if (wide) {
            x.set(v);
            __stcs(reinterpret_cast<uint4 *>(dz) + u, x.w);
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                store1(dz + u * N + 2 * i, v[i].x);
                store1(dz + u * N + 2 * i + 1, v[i].y);
            }
        }
    };
    int64_t u = u0 + tid;
    if (!(KEEP && LOSS))
        for (; u + (kAhead - 1) * kThreads < u1; u += kAhead * kThreads) {
            Unit<T> x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) x[i].w = from[u + i * kThreads];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) finish(x[i], u + i * kThreads);
        }
    for (; u < u1; u += kThreads) {
        Unit<T> x;
        if (KEEP && LOSS)
            x = kept[u - part.lo];
        else
            x.w = from[u];
        finish(x, u);
    }
    {
        const int64_t head_end = u0 * N < part.last ? u0 * N : part.last;
        const int64_t tail = u1 * N > head_end ? u1 * N : head_end;
        int64_t i = -1;
        if (part.first + tid < head_end) i = part.first + tid;
        if (tid >= 32 && tail + tid - 32 < part.last) i = tail + tid - 32;
        if (i >= 0) store1(dz + i, exp2_approx(fmaf(load1(base + i), rt, -lse) * kLog2e) * g);
    }
    __syncthreads();
    if (write) store1(dz + part.head + at, patch);
}

constexpr size_t kKeepMost = 110 * 1024;  // bytes of a part in shared memory: two blocks to an SM

template <class T, class E, bool LOSS, bool GRAD, bool KEEP>
cudaError_t launch(const DistillArgs &a, int blocks, size_t smem, cudaStream_t st)
{
    auto *kernel = &distill_kernel<T, E, LOSS, GRAD, KEEP>;
    if (smem) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    if (a.rows * blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(a.rows * blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(blocks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, blocks);
}

template <class T, class E>
cudaError_t by_pass(const DistillArgs &a, cudaStream_t st)
{
    const bool loss = a.loss != nullptr, grad = a.dlogits != nullptr;
    const int64_t bytes = int64_t(a.vocab) * int64_t(sizeof(T)) + 32;
    // Blocks to a row: enough that a part fits, and more while the rows leave
    // SMs idle and parts are long.
    int blocks = 1;
    const bool hold = loss && grad;
    while (blocks < 8 && ((hold && (bytes + blocks - 1) / blocks > int64_t(kKeepMost)) ||
                          (a.rows * blocks < 152 && bytes / blocks > 16384)))
        blocks *= 2;
    const int64_t part = ((bytes + 15) / 16 + blocks - 1) / blocks * 16 + 16;
    if (!loss) return launch<T, E, false, true, false>(a, blocks, 0, st);
    if (!grad) return launch<T, E, true, false, false>(a, blocks, 0, st);
    if (part > int64_t(kKeepMost) + 64) return launch<T, E, true, true, false>(a, blocks, 0, st);
    return launch<T, E, true, true, true>(a, blocks, size_t(part), st);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs &a, cudaStream_t st)
{
    const bool bf = a.dtype == ZG_DTYPE_BF16, tbf = a.t_dtype == ZG_DTYPE_BF16;
    if (bf) return tbf ? by_pass<uint16_t, uint16_t>(a, st) : by_pass<uint16_t, float>(a, st);
    return tbf ? by_pass<float, uint16_t>(a, st) : by_pass<float, float>(a, st);
}

}  // namespace zg
