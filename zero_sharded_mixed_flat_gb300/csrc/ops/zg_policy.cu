// The log-probabilities of tokens, the clipped policy loss with its KL term, and
// its gradient by the logits.
//
// With z a row of logits, T the temperature and t its token, logp = (z_t - m) / T
// - log S with m the row's maximum and S = sum exp((z - m) / T); the loss and its
// slope by logp are the row's own few values; dz = g ([v = t] - exp((z - m) / T) / S)
// with g = scale dloss slope / T.
//
// Bound by memory: each logit is read once and its gradient written once. The loss alone is one pass of small
// blocks with a running maximum and sum. The gradient needs the whole row's sum first, so a block copies
// its row into shared memory (cp.async) and goes over it there twice; a thread reads the units that it
// copied, which needs no barrier, and an SM has several rows, of which some are copied while others
// wait for their sums. Rows larger than that, and few rows, are shared out over a cluster of blocks, which
// exchange their maxima and sums through distributed shared memory. The gradient alone, from a kept
// maximum and sum, is a stream.
//
// Measured at 4096 x 50257 in bf16: the loss alone 72 us (5.7 TB/s), loss and gradient 145 (5.7 TB/s of the once-read,
// once-written bytes), the gradient alone 115 (7.2 TB/s); in binary32 131, 316 and 233 us. 777 x 131075 in bf16, the
// loss alone and the gradient 39 and 60 us. 37 x 50257 in binary32, eight blocks to a row, 7.9 us. With gradient rows
// that are not aligned as the logits' are, both 162 and the gradient 122 us. Both in one launch issue in 51 % of the
// cycles with two rows to an SM; what is left is what the phases of a row wait for.
#include <cooperative_groups.h>

#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

#include "zg_async.cuh"
#include "zg_launch.h"
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

namespace cg = cooperative_groups;

constexpr int kAhead = 4;  // units of a thread at a time
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

// a e^x, where e^x may be beyond binary32 though the product is not: an advantage or a KL factor of
// zero, say, beside a ratio that a rare token makes as large as it likes.
constexpr float kLarge = 80.0f;
__device__ __forceinline__ float times_exp(float x, float a)
{
    if (x <= kLarge) return a * expf(x);
    if (a == 0.0f && x < INFINITY) return a;
    return a * expf(0.5f * x) * expf(0.5f * x);
}

// What a row's loss and slope are made of, beside logp.
struct Values {
    float adv, old, ref, weight;
    __device__ __forceinline__ Values(const PolicyArgs &a, int64_t r, bool there)
    {
        adv = there && a.advantage ? a.advantage[r] : 0.0f;
        old = there && a.old_logp ? a.old_logp[r] : 0.0f;
        ref = there && a.ref_logp ? a.ref_logp[r] : 0.0f;
        weight = there && a.dloss ? a.dloss[r] : 1.0f;
    }
    // The loss and its slope by logp.
    __device__ __forceinline__ float2 loss(const PolicyArgs &a, float logp) const
    {
        const float x = logp - old, ratio = expf(x), high = 1.0f + a.clip_high, low = 1.0f - a.clip_low;
        const bool cut = (adv > 0.0f && ratio > high) || (adv < 0.0f && ratio < low);
        float slope = cut ? 0.0f : -times_exp(x, adv), l = cut ? -(adv > 0.0f ? high : low) * adv : slope;
        if (a.ref_logp) {
            const float d = ref - logp;
            if (d > kLarge) {  // 1 + d is far below the exponential's last place
                const float t = times_exp(d, a.kl);
                l += t;
                slope -= t;
            } else {
                const float e = expm1f(d);
                l = fmaf(a.kl, e - d, l);
                slope = fmaf(-a.kl, e, slope);
            }
        }
        return make_float2(l, slope);
    }
    // The gradient's factor at the token.
    __device__ __forceinline__ float factor(const PolicyArgs &a, float slope) const
    {
        return a.scale * weight * slope * (1.0f / a.temperature);
    }
};

// 2^((z - top) c) for a unit's logits, one packed multiply-add and an exponential each: top c is
// rounded once, and what that takes off every exponent is `rest`, a factor to make good. Where the
// rounding is no longer small (a top that is a mask, or a row far from zero) differences come first.
struct Scale {
    float top, c, off;
    bool far;
    __device__ __forceinline__ Scale(float t, float cc) : top(t), c(cc), off(t * cc), far(!(fabsf(off) < 256.0f)) {}
    __device__ __forceinline__ float rest() const { return far ? 1.0f : exp2_approx(-fmaf(top, c, -off)); }
    template <bool FAR>
    __device__ __forceinline__ float2 of(float2 z) const
    {
        const float2 t = FAR ? mul_f32x2(add_f32x2(z, make_float2(-top, -top)), make_float2(c, c))
                             : fma_f32x2(z, make_float2(c, c), make_float2(-off, -off));
        return make_float2(exp2_approx(t.x), exp2_approx(t.y));
    }
    // The same of one logit, to the last bit: what a row's alignment makes of its units does not show.
    __device__ __forceinline__ float of(float z) const { return exp2_approx(far ? (z - top) * c : fmaf(z, c, -off)); }
};
// A unit's gradient in place of its logits: k 2^((z - top) c).
template <bool FAR, class T>
__device__ __forceinline__ void gradient(Unit<T> &x, const Scale &s, float k)
{
    float2 v[Unit<T>::kN / 2];
    x.get(v);
#pragma unroll
    for (int i = 0; i < Unit<T>::kN / 2; ++i) v[i] = mul_f32x2(s.of<FAR>(v[i]), make_float2(k, k));
    x.set(v);
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

// A block's part of a row: from memory, or from a stage in shared memory, where the whole units come
// first and then the (at most two) units of its ragged ends.
template <class T>
struct Span : Row<T> {
    static constexpr int N = Unit<T>::kN;
    uint32_t at;    // shared address of the first whole unit, where staged
    uint32_t ends;  // and of the ragged ends' units, where no row has a whole one
    __device__ __forceinline__ Span(const T *row, int vocab, int each, int rank, uint32_t shared)
        : Row<T>(row, vocab, each, rank), at(shared), ends(shared + each * 16)
    {
    }
    __device__ __forceinline__ int head_end() const { return min(this->part.u0 * N, this->part.last); }
    __device__ __forceinline__ int tail() const { return max(this->part.u1 * N, head_end()); }
    // The team's copies: each thread's are what it reads itself.
    template <int TEAM>
    __device__ __forceinline__ void copy(int tid) const
    {
        const uint4 *const from = this->from();
#pragma unroll 4
        for (int u = tid; u < this->units; u += TEAM) copy16(at + u * 16, from + u);
        if (tid == 0 && this->part.first < head_end()) copy16(ends, from - 1);
        if (tid == 31 && tail() < this->part.last) copy16(ends + 16, reinterpret_cast<const uint4 *>(this->base) + tail() / N);
    }
    template <bool STAGED>
    __device__ __forceinline__ uint4 unit(int u) const
    {
        if (!STAGED) return this->from()[u];
        uint4 w;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at + u * 16));
        return w;
    }
    // One element of the part's count. Staged, those of the ragged ends are for the threads 0 and 31.
    template <bool STAGED>
    __device__ __forceinline__ float one(int e) const
    {
        if (!STAGED) return load1(this->base + e);
        const int u = e / N - this->part.u0;
        const uint32_t a = (e < head_end() ? ends : e >= tail() ? ends + 16 : at + u * 16) + e % N * int(sizeof(T));
        if constexpr (sizeof(T) == 2) {
            uint16_t w;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(a));
            return __uint_as_float(uint32_t(w) << 16);
        } else {
            float w;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w) : "r"(a));
            return w;
        }
    }
    // The ragged elements, of the thread that has them.
    template <class F>
    __device__ __forceinline__ void ragged(int tid, F f) const
    {
        if (tid == 0)
            for (int e = this->part.first; e < head_end(); ++e) f(e);
        if (tid == 31)
            for (int e = tail(); e < this->part.last; ++e) f(e);
    }
};

struct RowShape {
    int blocks, each;  // of a cluster, which shares a row; units of a block's part
    int stages, slot;  // parts of a team in shared memory, and the bytes of one
};

template <int TEAM>
struct TeamShared {
    Sum warp[2][TEAM / 32];  // of rows in turn, as the next: who is two rows ahead has been through a barrier
    Sum block[2];            // this block's part, read by the others of the cluster
    float top, k, g, zt;     // of the row
    int token;
};

// Each team (or, with several blocks, each cluster) takes rows in turn.
template <class T, int TEAM, int THREADS, bool GRAD, bool STAGED>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) row_kernel(PolicyArgs a, RowShape shape)
{
    constexpr int kTeams = THREADS / TEAM, N = Unit<T>::kN;
    __shared__ TeamShared<TEAM> shared[kTeams];
    extern __shared__ __align__(16) char rows[];
    const int id = threadIdx.x / TEAM, tid = threadIdx.x % TEAM, lane = tid % 32;
    TeamShared<TEAM> &sh = shared[id];
    const int rank = shape.blocks > 1 ? int(blockIdx.x % unsigned(shape.blocks)) : 0;
    const int64_t step = shape.blocks > 1 ? gridDim.x / shape.blocks : int64_t(gridDim.x) * kTeams;
    const int64_t begin = shape.blocks > 1 ? blockIdx.x / unsigned(shape.blocks) : int64_t(blockIdx.x) * kTeams + id;
    const int stages = STAGED ? shape.stages : 1;
    const uint32_t mine = uint32_t(__cvta_generic_to_shared(rows)) + id * (shape.slot * shape.stages);
    const float rt = 1.0f / a.temperature, c = rt * kLog2e;
    const T *const logits = static_cast<const T *>(a.logits);
    auto span = [&](int64_t r, int stage) {
        return Span<T>(logits + r * a.row_stride, a.vocab, shape.each, rank, mine + stage * shape.slot);
    };
    auto ask = [&](int64_t r, int stage) {
        if (!STAGED) return;
        if (r < a.rows) span(r, stage).template copy<TEAM>(tid);
        commit_copies();
    };
    for (int i = 0; i < stages; ++i) ask(begin + i * step, i);
    int token = begin < a.rows ? token_of(a, begin) : -1;
    int stage = 0, turn = 0;
    for (int64_t r = begin; r < a.rows; r += step) {
        const Span<T> s = span(r, stage);
        // asked for now, needed when the sum is known
        const bool has = tid == 0 && token >= 0;
        const float zt = has ? load1(logits + r * a.row_stride + token) : 0.0f;
        const Values values(a, r, has);
        const int next_token = r + step < a.rows ? token_of(a, r + step) : -1;
        Sum sum{-INFINITY, 0.0f};
        auto take_in = [&](const Unit<T> (&x)[kAhead], int n) {  // the first n
            typename Unit<T>::Top most;
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (i < n) most.add(x[i]);
            const float top = max_nan(sum.top, most.get());
            if (top != sum.top) sum = Sum{top, rescaled(sum, top, c)};
            if (top == -INFINITY) return;  // nothing but masked logits so far
            const Scale scale(top, c);
            float2 add = make_float2(0.0f, 0.0f);
            auto all = [&](auto far) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (i >= n) break;
                    float2 v[N / 2];
                    x[i].get(v);
#pragma unroll
                    for (int j = 0; j < N / 2; ++j) add = add_f32x2(add, scale.template of<decltype(far)::value>(v[j]));
                }
            };
            if (scale.far)
                all(std::true_type{});
            else
                all(std::false_type{});
            sum.sum += (add.x + add.y) * scale.rest();
        };
        if (STAGED) wait_copies(stages - 1);
        int u = tid;
        for (; u + (kAhead - 1) * TEAM < s.units; u += kAhead * TEAM) {
            Unit<T> x[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) x[j].w = s.template unit<STAGED>(u + j * TEAM);
            take_in(x, kAhead);
        }
        if (u < s.units) {
            Unit<T> x[kAhead];
            int n = 0;
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (u + j * TEAM < s.units) {
                    x[j].w = s.template unit<STAGED>(u + j * TEAM);
                    n = j + 1;
                }
            take_in(x, n);
        }
        s.ragged(tid, [&](int e) {
            const float z = s.template one<STAGED>(e), top = max_nan(sum.top, z);
            if (top != -INFINITY) sum = Sum{top, rescaled(sum, top, c) + exp2_approx((z - top) * c)};
        });
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
                    const float2 l = values.loss(a, logp);
                    loss = l.x;
                    if (GRAD) g = values.factor(a, l.y);
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
            sh.zt = zt;
            sh.token = token;
        }
        if (GRAD) {
            team_sync(id, TEAM);
            const float g = sh.g;
            const Scale scale(sh.top, c);
            const float kk = sh.k * scale.rest();
            // nothing to compute: padding, and ratios that are cut off
            const bool zero = sh.token < 0 || g == 0.0f;
            T *const dz = static_cast<T *>(a.dlogits) + r * a.drow_stride - s.part.head;
            const int phase = int((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T));
            auto put1 = [&](int e) { store1(dz + e, zero ? 0.0f : scale.of(s.template one<STAGED>(e)) * kk); };
            int owner = 0;  // who writes the token's element
            const int t = sh.token + s.part.head;
            if (phase == 0) {
                uint4 *const to = reinterpret_cast<uint4 *>(dz) + s.part.u0;
                auto pass = [&](auto far) {
                    int u = tid;
                    for (; u + (kAhead - 1) * TEAM < s.units; u += kAhead * TEAM) {
                        Unit<T> x[kAhead];
#pragma unroll
                        for (int j = 0; j < kAhead; ++j) x[j].w = s.template unit<STAGED>(u + j * TEAM);
#pragma unroll
                        for (int j = 0; j < kAhead; ++j) {
                            gradient<decltype(far)::value>(x[j], scale, kk);
                            __stcs(to + u + j * TEAM, x[j].w);
                        }
                    }
                    for (; u < s.units; u += TEAM) {
                        Unit<T> x;
                        x.w = s.template unit<STAGED>(u);
                        gradient<decltype(far)::value>(x, scale, kk);
                        __stcs(to + u, x.w);
                    }
                };
                if (zero)
                    for (int u = tid; u < s.units; u += TEAM) __stcs(to + u, make_uint4(0u, 0u, 0u, 0u));
                else if (scale.far)
                    pass(std::true_type{});
                else
                    pass(std::false_type{});
                s.ragged(tid, put1);
                owner = t < s.head_end() ? 0 : t >= s.tail() ? 31 : (t / N - s.part.u0) % TEAM;
            } else {
                // the output's units lie across the input's: whole ones of the output that lie across whole
                // ones of the part, each from the two that it lies across
                const int i0 = (s.part.u0 * N + 1 + phase + N - 1) / N * N - phase;
                const int i1 = max((s.part.u1 * N - 1 + phase) / N * N - phase, i0);
                const int at = (N - phase) % N;
                auto pass = [&](auto far) {
#pragma unroll 2
                    for (int e = i0 + tid * N; e < i1; e += TEAM * N) {
                        const int u = e / N - s.part.u0;
                        Unit<T> x;
                        x.w = across<T>(s.template unit<STAGED>(u), s.template unit<STAGED>(u + 1), at);
                        gradient<decltype(far)::value>(x, scale, kk);
                        __stcs(reinterpret_cast<uint4 *>(dz + e), x.w);
                    }
                };
                if (zero)
                    for (int e = i0 + tid * N; e < i1; e += TEAM * N)
                        __stcs(reinterpret_cast<uint4 *>(dz + e), make_uint4(0u, 0u, 0u, 0u));
                else if (scale.far)
                    pass(std::true_type{});
                else
                    pass(std::false_type{});
                // the rest: less than two units at either end
                for (int e = s.part.first + tid; e < min(i0, s.part.last); e += TEAM) put1(e);
                for (int e = max(i1, s.part.first) + tid; e < s.part.last; e += TEAM) put1(e);
                team_sync(id, TEAM);  // the others' units have been read, and the token's element is written
            }
            if (tid == owner && !zero && t >= s.part.first && t < s.part.last)
                store1(dz + t, fmaf(scale.of(sh.zt), kk, g));
            if (TEAM == 32) __syncwarp();
            ask(r + stages * step, stage);
        }
        token = next_token;
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
    if (STAGED) wait_copies(0);
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
    const Values values(a, r, token >= 0);
    const float g = token < 0 ? 0.0f : values.factor(a, values.loss(a, logp).y);
    const Row<T> row(z, a.vocab, each, rank);
    const Part &part = row.part;
    const int t = token < 0 ? -1 : token + part.head;
    const bool zero = token < 0 || g == 0.0f;
    const Scale scale(top, c);
    const float kk = -g / sum * scale.rest();
    T *const dz = static_cast<T *>(a.dlogits) + r * a.drow_stride - part.head;
    const int phase = int((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T));
    const uint4 *const in = reinterpret_cast<const uint4 *>(row.base);
    auto value = [&](float z, int e) {
        return zero ? 0.0f : e == t ? fmaf(scale.of(z), kk, g) : scale.of(z) * kk;
    };
    int i0, i1;  // what is written in whole units
    if (phase == 0) {
        i0 = part.u0 * N;
        i1 = part.u1 * N;
    } else {
        i0 = (part.u0 * N + 1 + phase + N - 1) / N * N - phase;
        i1 = max((part.u1 * N - 1 + phase) / N * N - phase, i0);
    }
    // the token's logit, before its unit is written over
    const float zt = t >= i0 && t < i1 ? load1(row.base + t) : 0.0f;
    auto pass = [&](auto far) {
        if (phase == 0) {
            int e = i0 + tid * N;
            for (; e + (kAhead - 1) * kStream * N < i1; e += kAhead * kStream * N) {
                Unit<T> x[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) x[i].w = in[e / N + i * kStream];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    gradient<decltype(far)::value>(x[i], scale, kk);
                    __stcs(reinterpret_cast<uint4 *>(dz + e) + i * kStream, x[i].w);
                }
            }
            for (; e < i1; e += kStream * N) {
                Unit<T> x;
                x.w = in[e / N];
                gradient<decltype(far)::value>(x, scale, kk);
                __stcs(reinterpret_cast<uint4 *>(dz + e), x.w);
            }
            return;
        }
        const int at = (N - phase) % N;
        for (int e = i0 + tid * N; e < i1; e += 2 * kStream * N) {
            const int e2 = e + kStream * N;
            Unit<T> x;
            const uint4 p0 = in[e / N], p1 = in[e / N + 1];
            uint4 q0 = p0, q1 = p1;
            if (e2 < i1) q0 = in[e2 / N], q1 = in[e2 / N + 1];
            x.w = across<T>(p0, p1, at);
            gradient<decltype(far)::value>(x, scale, kk);
            __stcs(reinterpret_cast<uint4 *>(dz + e), x.w);
            if (e2 >= i1) break;
            x.w = across<T>(q0, q1, at);
            gradient<decltype(far)::value>(x, scale, kk);
            __stcs(reinterpret_cast<uint4 *>(dz + e2), x.w);
        }
    };
    if (phase == 0) __syncthreads();  // the token's logit has been read where the gradient takes its place
    if (zero)
        for (int e = i0 + tid * N; e < i1; e += kStream * N) __stcs(reinterpret_cast<uint4 *>(dz + e), make_uint4(0u, 0u, 0u, 0u));
    else if (scale.far)
        pass(std::true_type{});
    else
        pass(std::false_type{});
    if (!zero && t >= i0 && t < i1 && (t - i0) / N % kStream == tid) store1(dz + t, value(zt, t));
    i0 = min(i0, part.last);
    i1 = min(i1, part.last);
    for (int e = part.first + tid; e < i0; e += kStream) store1(dz + e, value(load1(row.base + e), e));
    for (int e = i1 + tid; e < part.last; e += kStream) store1(dz + e, value(load1(row.base + e), e));
}

// Clusters of a kernel that the device holds at once (its groups of SMs need not be multiples of
// them), asked for once; `blocks` where there are none.
cudaError_t resident(const void *kernel, cudaLaunchConfig_t cfg, int blocks, int *clusters)
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
        if (e == cudaSuccess && !cfg.numAttrs) it->second = blocks;
        if (e != cudaSuccess || it->second < 1) {
            known.erase(it);
            return e != cudaSuccess ? e : cudaErrorInvalidConfiguration;
        }
    }
    *clusters = it->second;
    return cudaSuccess;
}

// Shared memory of a block where an SM has `to_sm` of them, and the kernel's own few variables.
constexpr int memory_of(int to_sm) { return 224 * 1024 / to_sm - (to_sm - 1) * 512; }

template <class T, int TEAM, int THREADS, bool GRAD, bool STAGED>
cudaError_t rows_of(const PolicyArgs &a, const RowShape &shape, cudaStream_t st)
{
    constexpr int kTeams = THREADS / TEAM, kToSm = 1024 / THREADS;
    auto *kernel = &row_kernel<T, TEAM, THREADS, GRAD, STAGED>;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(unsigned(152 * kToSm / shape.blocks * shape.blocks));
    cfg.blockDim = dim3(THREADS);
    // always the most that any shape takes: the attribute that allows it is set once
    cfg.dynamicSmemBytes = STAGED ? memory_of(kToSm) : 0;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(shape.blocks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = shape.blocks > 1 ? 1 : 0;
    int clusters = 0;
    if (cudaError_t e = resident(reinterpret_cast<const void *>(kernel), cfg, 152 * kToSm, &clusters)) return e;
    // what is staged takes rows in turn; otherwise a block has one
    const int64_t want = (a.rows + kTeams - 1) / kTeams, most = STAGED || shape.blocks > 1 ? clusters : (int64_t(1) << 31) - 1;
    cfg.gridDim = dim3(unsigned((most < want ? most : want) * shape.blocks));
    return cudaLaunchKernelEx(&cfg, kernel, a, shape);
}

template <class T, bool GRAD>
cudaError_t by_size(const PolicyArgs &a, cudaStream_t st)
{
    const int64_t units = (int64_t(a.vocab) * int64_t(sizeof(T)) + 30) / 16;
    RowShape s{};
    // the parts that a block holds, of rows cut into `blocks`, each team with its own
    auto hold = [&](int blocks, int teams, int to_sm) {
        s.blocks = blocks;
        s.each = int((units + blocks - 1) / blocks);
        s.slot = (s.each + 2) * 16;  // whole units, and one at either end
        const int64_t fit = memory_of(to_sm) / (int64_t(s.slot) * teams);
        s.stages = int(fit < 2 ? fit : 2);
    };
    hold(1, 128 / 32, 8);
    if (units <= 192) return rows_of<T, 32, 128, GRAD, true>(a, s, st);
    if constexpr (!GRAD) {
        // once over the row, straight from memory: small blocks keep most rows in flight; few rows take more
        // threads, then more blocks
        s.blocks = 1;
        while (s.blocks < 8 && a.rows * (s.blocks + 1) <= 304 && units / s.blocks > 1024) ++s.blocks;
        s.each = int((units + s.blocks - 1) / s.blocks);
        s.stages = 0;
        return a.rows >= 608 ? rows_of<T, 128, 128, GRAD, false>(a, s, st) : rows_of<T, 512, 512, GRAD, false>(a, s, st);
    } else {
        hold(1, 1, 8);
        if (units <= 1536) return rows_of<T, 128, 128, GRAD, true>(a, s, st);
        // The smallest blocks that have room for a part, without a cluster where that can be. (4096 x 50257 in bf16:
        // two blocks of 512 threads to an SM 145 us, one of 1024 with two rows in its memory 214, clusters of four
        // blocks of 256 201, of two 158: what a row costs every warp of its own, and the waits for its sum.) Few rows
        // take the most blocks of the smallest size (37 x 50257 in binary32: eight of 256 threads 8.0 us, of 512 11.4).
        for (int to_sm = 4; to_sm; to_sm /= 2)
            for (int blocks = 1; blocks <= (to_sm == 4 && a.rows * 8 > 152 * 4 ? 1 : 8); ++blocks) {
                hold(blocks, 1, to_sm);
                if (s.stages < 1) continue;
                while (s.blocks < 8 && a.rows * (s.blocks + 1) <= 152 * to_sm && s.each > 1024) hold(s.blocks + 1, 1, to_sm);
                if (to_sm == 4) return rows_of<T, 256, 256, GRAD, true>(a, s, st);
                if (to_sm == 2) return rows_of<T, 512, 512, GRAD, true>(a, s, st);
                return rows_of<T, 1024, 1024, GRAD, true>(a, s, st);
            }
        hold(8, 1, 1);
        s.stages = 0;
        return rows_of<T, 1024, 1024, GRAD, false>(a, s, st);
    }
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
