// The log-probabilities of tokens, the clipped policy loss with its KL term, and
// its gradient by the logits.
//
// With z a row of logits, T the temperature and t its token, logp = (z_t - m) / T
// - log S with m the row's maximum and S = sum exp((z - m) / T); the loss and its
// slope by logp are the row's own few values; dz = g ([v = t] - exp((z - m) / T) / S)
// with g = scale dloss slope / T. Differences to the maximum come first throughout, so
// masks of any size and rows far from zero have their values.
//
// Bound by memory: each logit is read once and its gradient written once. The gradient needs the whole
// row's sum, so a team of warps copies its next row into shared memory (cp.async) while it goes over
// the present one, there, twice: a row of 50257 bf16 logits takes an SM's memory with the next one. A
// thread reads the units that it copied, which needs no barrier. Rows larger than that, and few rows, are
// shared out over a cluster of blocks, which exchange their maxima and sums through distributed shared
// memory. The gradient alone, from a kept maximum and sum, is a stream.
#include <cooperative_groups.h>

#include <map>
#include <mutex>
#include <tuple>

#include "zg_async.cuh"
#include "zg_launch.h"
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kAhead = 4;  // units of a thread at a time
constexpr int kMemory = 224 * 1024;  // shared memory of a block
constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t *>(&a)), "l"(*reinterpret_cast<const uint64_t *>(&b)));
    return *reinterpret_cast<const float2 *>(&d);
}

// The largest of a set of logits and the sum of 2^((z - top) c) over it.
struct Sum {
    float top, sum;
};
__device__ __forceinline__ float rescaled(Sum s, float top, float c)
{
    return s.top == -INFINITY ? 0.0f : s.sum * exp2_approx((s.top - top) * c);
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
    const bool cut = (adv > 0.0f && ratio > high) || (adv < 0.0f && ratio < low);
    float loss = -(cut ? (adv > 0.0f ? high : low) : ratio) * adv, slope = cut ? 0.0f : -ratio * adv;
    if (a.ref_logp) {
        const float d = a.ref_logp[r] - logp, e = expm1f(d);
        loss = fmaf(a.kl, e - d, loss);
        slope = fmaf(-a.kl, e, slope);
    }
    return make_float2(loss, slope);
}
// What the gradient multiplies: g of the row's token.
__device__ __forceinline__ float factor_of(const PolicyArgs &a, int64_t r, float slope)
{
    return a.scale * (a.dloss ? a.dloss[r] : 1.0f) * slope * (1.0f / a.temperature);
}

// A unit's gradient in place of its logits: k 2^((z - top) c), k = -g / S.
template <class T>
__device__ __forceinline__ void gradient(Unit<T> &x, float top, float c, float k)
{
    float2 v[Unit<T>::kN / 2];
    x.get(v);
#pragma unroll
    for (int i = 0; i < Unit<T>::kN / 2; ++i) {
        const float2 t = mul_f32x2(add_f32x2(v[i], make_float2(-top, -top)), make_float2(c, c));
        v[i] = mul_f32x2(make_float2(exp2_approx(t.x), exp2_approx(t.y)), make_float2(k, k));
    }
    x.set(v);
}
template <class T>
__device__ __forceinline__ float gradient1(float z, float top, float c, float k, float g, bool token)
{
    return fmaf(exp2_approx((z - top) * c), k, token ? g : 0.0f);
}

// A unit of logits from element e0 on, t the token's element, to its gradient's place.
template <class T>
__device__ __forceinline__ void put_unit(Unit<T> &x, T *dz, int e0, int t, bool zero, float top, float c, float k, float g)
{
    constexpr int N = Unit<T>::kN;
    if (zero) {
        x.w = make_uint4(0u, 0u, 0u, 0u);
    } else if (t >= e0 && t < e0 + N) {
        float2 v[N / 2];
        x.get(v);
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            v[i] = make_float2(gradient1<T>(v[i].x, top, c, k, g, e0 + 2 * i == t),
                               gradient1<T>(v[i].y, top, c, k, g, e0 + 2 * i + 1 == t));
        x.set(v);
    } else {
        gradient(x, top, c, k);
    }
    __stcs(reinterpret_cast<uint4 *>(dz + e0), x.w);
}

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

// Where the units of a part's span lie: from memory, or from a stage in shared memory.
// Unit 0 is the one that holds the part's first element.
template <class T>
struct Span {
    Part part;
    const T *base;   // element 0 of the part's count
    int first_unit, units;
    uint32_t at;     // shared address of unit 0, where staged
    __device__ __forceinline__ Span(const T *row, int vocab, int each, int rank, uint32_t shared) : at(shared)
    {
        constexpr int N = Unit<T>::kN;
        part = part_of(row, vocab, each, rank);
        base = row - part.head;
        first_unit = part.first / N;
        units = part.last > part.first ? (part.last + N - 1) / N - first_unit : 0;
    }
    __device__ __forceinline__ const uint4 *from() const { return reinterpret_cast<const uint4 *>(base) + first_unit; }
    __device__ __forceinline__ uint4 unit(int i, bool staged) const
    {
        uint4 w;
        if (!staged) return from()[i];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at + i * 16));
        return w;
    }
    __device__ __forceinline__ bool whole(int i) const { return first_unit + i >= part.u0 && first_unit + i < part.u1; }
    // Elements of unit i that are the part's: [lo, hi) of its N.
    __device__ __forceinline__ int lo(int i) const { return max(part.first - (first_unit + i) * Unit<T>::kN, 0); }
    __device__ __forceinline__ int hi(int i) const { return min(part.last - (first_unit + i) * Unit<T>::kN, Unit<T>::kN); }
};

struct RowShape {
    int blocks, each;   // of a cluster, which shares a row; units of a block's part
    int stages, slot;   // parts of a team in shared memory, and the bytes of one
};

template <int TEAM>
struct TeamShared {
    Sum warp[2][TEAM / 32];  // of rows in turn, as the next: who is two rows ahead has been through a barrier
    Sum block[2];            // this block's part, read by the others of the cluster
    float top, k, g;  // of the row
    int token;
};

// Each team (or, with several blocks, each cluster) takes rows in turn.
template <class T, int TEAM, bool GRAD>
__global__ void __launch_bounds__(kThreads, 1) row_kernel(PolicyArgs a, RowShape shape)
{
    constexpr int kTeams = kThreads / TEAM, N = Unit<T>::kN;
    __shared__ TeamShared<TEAM> shared[kTeams];
    extern __shared__ __align__(16) char rows[];
    const int id = threadIdx.x / TEAM, tid = threadIdx.x % TEAM, lane = tid % 32;
    TeamShared<TEAM> &sh = shared[id];
    const int rank = shape.blocks > 1 ? int(blockIdx.x % unsigned(shape.blocks)) : 0;
    const int64_t step = shape.blocks > 1 ? gridDim.x / shape.blocks : int64_t(gridDim.x) * kTeams;
    const int64_t begin = shape.blocks > 1 ? blockIdx.x / unsigned(shape.blocks) : int64_t(blockIdx.x) * kTeams + id;
    const bool staged = shape.stages > 0;
    const int stages = staged ? shape.stages : 1;
    const uint32_t mine = uint32_t(__cvta_generic_to_shared(rows)) + id * (shape.slot * shape.stages);
    const float rt = 1.0f / a.temperature, c = rt * kLog2e;
    const T *const logits = static_cast<const T *>(a.logits);
    auto ask = [&](int64_t r, int stage) {
        if (staged && r < a.rows) {
            const Span<T> s(logits + r * a.row_stride, a.vocab, shape.each, rank, mine + stage * shape.slot);
            const uint4 *const from = s.from();
            for (int i = tid; i < s.units; i += TEAM) copy16(s.at + i * 16, from + i);
        }
        commit_copies();
    };
    for (int i = 0; i < stages; ++i) ask(begin + i * step, i);
    int token = begin < a.rows ? token_of(a, begin) : -1;
    int stage = 0, turn = 0;
    for (int64_t r = begin; r < a.rows; r += step) {
        const Span<T> s(logits + r * a.row_stride, a.vocab, shape.each, rank, mine + stage * shape.slot);
        // asked for now, needed when the sum is known
        const float zt = tid == 0 && token >= 0 ? load1(logits + r * a.row_stride + token) : 0.0f;
        const int next_token = r + step < a.rows ? token_of(a, r + step) : -1;
        wait_copies(stages - 1);
        Sum sum{-INFINITY, 0.0f};
        auto take_in = [&](const Unit<T> (&x)[kAhead], int n) {  // the first n
            typename Unit<T>::Top most;
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (i < n) most.add(x[i]);
            const float top = max_nan(sum.top, most.get());
            if (top != sum.top) sum = Sum{top, rescaled(sum, top, c)};
            if (top == -INFINITY) return;  // nothing but masked logits so far
            float2 add = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (i >= n) break;
                float2 v[N / 2];
                x[i].get(v);
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    const float2 t = mul_f32x2(add_f32x2(v[j], make_float2(-top, -top)), make_float2(c, c));
                    add = add_f32x2(add, make_float2(exp2_approx(t.x), exp2_approx(t.y)));
                }
            }
            sum.sum += add.x + add.y;
        };
        // a thread's units in turn; those at the part's ends count what is not theirs as masked
        auto fetch = [&](int i) {
            Unit<T> x;
            x.w = s.unit(i, staged);
            if (!s.whole(i)) {
                const int lo = s.lo(i), hi = s.hi(i);
                float2 v[N / 2];
                x.get(v);
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    if (2 * j < lo || 2 * j >= hi) v[j].x = -INFINITY;
                    if (2 * j + 1 < lo || 2 * j + 1 >= hi) v[j].y = -INFINITY;
                }
                x.set(v);
            }
            return x;
        };
        int i = tid;
        for (; i + (kAhead - 1) * TEAM < s.units; i += kAhead * TEAM) {
            Unit<T> x[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) x[j] = fetch(i + j * TEAM);
            take_in(x, kAhead);
        }
        if (i < s.units) {
            Unit<T> x[kAhead];
            int n = 0;
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (i + j * TEAM < s.units) {
                    x[j] = fetch(i + j * TEAM);
                    n = j + 1;
                }
            take_in(x, n);
        }
        if (!GRAD) ask(r + stages * step, stage);
        sum = across<32>(sum, c);
        if (TEAM > 32) {
            if (lane == 0) sh.warp[turn][tid / 32] = sum;
            team_sync(id, TEAM);
            sum = lane < TEAM / 32 ? sh.warp[turn][lane] : Sum{-INFINITY, 0.0f};
            sum = across<32>(sum, c);
        }
        if (shape.blocks > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            if (tid == 0) sh.block[turn] = sum;
            cluster.sync();
            Sum x = lane < shape.blocks ? cluster.map_shared_rank(&sh, lane)->block[turn] : Sum{-INFINITY, 0.0f};
            sum = across<32>(x, c);
        }
        turn ^= 1;
        if (tid == 0) {
            float loss = 0.0f, logp = 0.0f, lse = 0.0f, g = 0.0f;
            if (token >= 0) {
                const float log_sum = logf(sum.sum);
                logp = fmaf(zt - sum.top, rt, -log_sum);
                lse = fmaf(sum.top, rt, log_sum);
                if (a.old_logp) {
                    const float2 l = loss_of(a, r, logp);
                    loss = l.x;
                    if (GRAD) g = factor_of(a, r, l.y);
                }
            } else {
                sum = Sum{0.0f, 0.0f};
            }
            if (rank == 0) {
                if (a.loss) a.loss[r] = loss;
                if (a.logp) a.logp[r] = logp;
                if (a.lse) a.lse[r] = lse;
                if (a.kept) {
                    a.kept[3 * r] = sum.top;
                    a.kept[3 * r + 1] = sum.sum;
                    a.kept[3 * r + 2] = logp;
                }
            }
            sh.top = sum.top;
            sh.k = -g / sum.sum;
            sh.g = g;
            sh.token = token;
        }
        if (GRAD) {
            team_sync(id, TEAM);
            const float top = sh.top, k = sh.k, g = sh.g;
            const int t = sh.token < 0 ? -1 : sh.token + s.part.head;  // counted as the part's elements
            const bool zero = sh.token < 0 || g == 0.0f;  // nothing to compute: padding, and ratios that are cut off
            T *const dz = static_cast<T *>(a.dlogits) + r * a.drow_stride - s.part.head;
            const int phase = int((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T));
            auto put = [&](Unit<T> &x, int e0) { put_unit(x, dz, e0, t, zero, top, c, k, g); };
            auto put1 = [&](int e) {  // element e of the part's count
                const uint4 w = s.unit(e / N - s.first_unit, staged);
                const uint32_t word = (e % N) * int(sizeof(T)) / 4 == 0 ? w.x : (e % N) * int(sizeof(T)) / 4 == 1 ? w.y
                                      : (e % N) * int(sizeof(T)) / 4 == 2 ? w.z : w.w;
                const float z = sizeof(T) == 4 ? __uint_as_float(word) : e & 1 ? bf16_hi(word) : bf16_lo(word);
                store1(dz + e, zero ? 0.0f : gradient1<T>(z, top, c, k, g, e == t));
            };
            if (phase == 0) {
                uint4 *const to = reinterpret_cast<uint4 *>(dz) + s.first_unit;
#pragma unroll 4
                for (int u = tid; u < s.units; u += TEAM) {
                    if (!s.whole(u)) {
                        for (int e = s.lo(u); e < s.hi(u); ++e) put1((s.first_unit + u) * N + e);
                        continue;
                    }
                    Unit<T> x;
                    x.w = zero ? make_uint4(0u, 0u, 0u, 0u) : s.unit(u, staged);
                    put(x, (s.first_unit + u) * N);
                }
            } else {
                // the output's units lie across the input's: whole ones of the output inside the part, each
                // from the two that it lies across
                const int i0 = (s.part.first + phase + N - 1) / N * N - phase;
                const int i1 = max((s.part.last + phase) / N * N - phase, i0);
                const int at = (N - phase) % N;
#pragma unroll 2
                for (int e0 = i0 + tid * N; e0 < i1; e0 += TEAM * N) {
                    const int u = e0 / N - s.first_unit;
                    Unit<T> x;
                    x.w = zero ? make_uint4(0u, 0u, 0u, 0u)
                               : across<T>(s.unit(u, staged), s.unit(min(u + 1, s.units - 1), staged), at);
                    put(x, e0);
                }
                for (int e = s.part.first + tid; e < min(i0, s.part.last); e += TEAM) put1(e);
                for (int e = max(i1, s.part.first) + tid; e < s.part.last; e += TEAM) put1(e);
                team_sync(id, TEAM);  // the others' units have been read
            }
            ask(r + stages * step, stage);
        }
        token = next_token;
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
    wait_copies(0);
    if (shape.blocks > 1) cg::this_cluster().sync();  // nobody leaves while its sums may be read
}

// The gradient alone: parts of a row, nothing to exchange.
constexpr int kStream = 128;

template <class T>
__global__ void __launch_bounds__(kStream) gradient_kernel(PolicyArgs a, int blocks, int each)
{
    constexpr int N = Unit<T>::kN;
    const unsigned number = blockIdx.x / unsigned(blocks);
    const int64_t r = number;
    const int rank = int(blockIdx.x - number * unsigned(blocks)), tid = threadIdx.x;
    const T *const z = static_cast<const T *>(a.logits) + r * a.row_stride;
    const int token = token_of(a, r);
    const float c = 1.0f / a.temperature * kLog2e;
    // logp is kept too: another block may have written over the token's logit
    const float top = a.kept_in[3 * r], sum = a.kept_in[3 * r + 1], logp = a.kept_in[3 * r + 2];
    const float g = token < 0 ? 0.0f : factor_of(a, r, loss_of(a, r, logp).y);
    const Row<T> row(z, a.vocab, each, rank);
    const Part &part = row.part;
    const int t = token < 0 ? -1 : token + part.head;
    const bool zero = token < 0 || g == 0.0f;
    const float k = -g / sum;
    T *const dz = static_cast<T *>(a.dlogits) + r * a.drow_stride - part.head;
    const int phase = int((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T));
    const uint4 *const in = reinterpret_cast<const uint4 *>(row.base);
    auto put = [&](Unit<T> &x, int e0) { put_unit(x, dz, e0, t, zero, top, c, k, g); };
    int i0, i1;  // what is written in whole units
    if (phase == 0) {
        i0 = part.u0 * N;
        i1 = part.u1 * N;
        int e = i0 + tid * N;
        for (; e + (kAhead - 1) * kStream * N < i1; e += kAhead * kStream * N) {
            Unit<T> x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) x[i].w = in[e / N + i * kStream];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) put(x[i], e + i * kStream * N);
        }
        for (; e < i1; e += kStream * N) {
            Unit<T> x;
            x.w = in[e / N];
            put(x, e);
        }
    } else {
        i0 = (part.u0 * N + 1 + phase + N - 1) / N * N - phase;
        i1 = max((part.u1 * N - 1 + phase) / N * N - phase, i0);
        const int at = (N - phase) % N;
        for (int e = i0 + tid * N; e < i1; e += 2 * kStream * N) {
            const int e2 = e + kStream * N;
            Unit<T> x, y;
            const uint4 p0 = in[e / N], p1 = in[e / N + 1];
            uint4 q0 = p0, q1 = p1;
            if (e2 < i1) q0 = in[e2 / N], q1 = in[e2 / N + 1];
            x.w = across<T>(p0, p1, at);
            put(x, e);
            if (e2 < i1) {
                y.w = across<T>(q0, q1, at);
                put(y, e2);
            }
        }
    }
    i0 = min(i0, part.last);
    i1 = min(i1, part.last);
    for (int e = part.first + tid; e < i0; e += kStream)
        store1(dz + e, zero ? 0.0f : gradient1<T>(load1(row.base + e), top, c, k, g, e == t));
    for (int e = i1 + tid; e < part.last; e += kStream)
        store1(dz + e, zero ? 0.0f : gradient1<T>(load1(row.base + e), top, c, k, g, e == t));
}

// Clusters of `blocks` blocks of a kernel that the device holds at once (its groups of SMs need not be
// multiples of them), asked for once.
cudaError_t resident(const void *kernel, cudaLaunchConfig_t cfg, int *clusters)
{
    static std::mutex mu;
    static std::map<std::tuple<int, const void *, unsigned, size_t>, int> known;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    std::lock_guard<std::mutex> lock(mu);
    auto [it, fresh] = known.try_emplace({dev, kernel, cfg.attrs[0].val.clusterDim.x, cfg.dynamicSmemBytes}, 0);
    if (fresh) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(cfg.dynamicSmemBytes));
        if (e == cudaSuccess && cfg.numAttrs) e = cudaOccupancyMaxActiveClusters(&it->second, kernel, &cfg);
        if (e == cudaSuccess && !cfg.numAttrs) it->second = 152;
        if (e != cudaSuccess || it->second < 1) {
            known.erase(it);
            return e != cudaSuccess ? e : cudaErrorInvalidConfiguration;
        }
    }
    *clusters = it->second;
    return cudaSuccess;
}

template <class T, int TEAM, bool GRAD>
cudaError_t rows_of(const PolicyArgs &a, const RowShape &shape, cudaStream_t st)
{
    constexpr int kTeams = kThreads / TEAM;
    auto *kernel = &row_kernel<T, TEAM, GRAD>;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(unsigned(152 / shape.blocks * shape.blocks));
    cfg.blockDim = dim3(kThreads);
    // always the most that any shape takes: the attribute that allows it is set once
    cfg.dynamicSmemBytes = kMemory;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(shape.blocks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = shape.blocks > 1 ? 1 : 0;
    int clusters = 0;
    if (cudaError_t e = resident(reinterpret_cast<const void *>(kernel), cfg, &clusters)) return e;
    const int64_t want = (a.rows + kTeams - 1) / kTeams;
    cfg.gridDim = dim3(unsigned((clusters < want ? clusters : want) * shape.blocks));
    return cudaLaunchKernelEx(&cfg, kernel, a, shape);
}

template <class T, bool GRAD>
cudaError_t by_size(const PolicyArgs &a, cudaStream_t st)
{
    const int64_t units = (int64_t(a.vocab) * int64_t(sizeof(T)) + 30) / 16;
    RowShape s{};
    s.blocks = 1;
    auto hold = [&](int teams) {
        s.each = int((units + s.blocks - 1) / s.blocks);
        s.slot = (s.each + 1) * 16;  // a part may begin and end inside a unit
        const int64_t fit = kMemory / (int64_t(s.slot) * teams);
        s.stages = int(fit < 4 ? fit : 4);
    };
    if (units <= 192) {
        hold(kThreads / 32);
        return rows_of<T, 32, GRAD>(a, s, st);
    }
    if (units <= 1536) {
        hold(kThreads / 128);
        return rows_of<T, 128, GRAD>(a, s, st);
    }
    hold(1);
    while (s.blocks < 8 && (s.stages < 2 || (a.rows * (s.blocks + 1) <= 152 && s.each > 1024))) {
        ++s.blocks;
        hold(1);
    }
    return rows_of<T, kThreads, GRAD>(a, s, st);
}

template <class T>
cudaError_t of_type(const PolicyArgs &a, cudaStream_t st)
{
    if (!a.kept_in) return a.dlogits ? by_size<T, true>(a, st) : by_size<T, false>(a, st);
    const int64_t units = (int64_t(a.vocab) * int64_t(sizeof(T)) + 30) / 16, blocks = (units + 1727) / 1728;
    if (a.rows * blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    gradient_kernel<T><<<unsigned(a.rows * blocks), kStream, 0, st>>>(a, int(blocks), int((units + blocks - 1) / blocks));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_policy(const PolicyArgs &a, cudaStream_t st)
{
    return a.dtype == ZG_DTYPE_BF16 ? of_type<uint16_t>(a, st) : of_type<float>(a, st);
}

}  // namespace zg
