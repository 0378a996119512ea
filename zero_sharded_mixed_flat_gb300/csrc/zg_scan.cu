// The gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t with
// a_t = sigmoid(f_t), forward and backward, in one pass over the data.
//
// The recurrence is a scan over affine maps: a run of tokens takes the state
// h to A h + B, with A the product of its gates, and two runs compose to
// (A2 A1, A2 B1 + B2). Backward is the same scan from the end, of
// r -> a_t (dy_t + r). A block takes a tile of kTile channels by kChunk
// tokens: each warp holds its few tokens of the tile in registers, reduces
// them to one map, the warps' maps are composed through shared memory, and
// the blocks' maps through a workspace in global memory, where a block waits
// for those before it. With the state at its first token known, each warp runs
// the recurrence through its tokens again from the registers and stores.
//
// So x and f are read once and y is written once: 6 bytes per element in
// bf16 (10 in backward, with dy, dx and df) and about 0.3 in the workspace.
//
// The maps of earlier blocks are composed in a fixed order, by a tree of
// kGroup chunks to a group and kGroup groups to a span, whatever the order
// in which blocks run: the same inputs give the same bits. Only the state at
// the end of a span hangs on the span before it, so the chain of waits is one
// step per kGroup^2 chunks.
//
// Sequences that begin inside a chunk cut the scan: a run that holds a
// beginning has a constant map, marked by A = kConst (every real A is >= 0),
// so nothing before it, a NaN included, is multiplied into what follows.
#include <cuda_bf16.h>

#include "zg_launch.h"
#include "zg_ops.h"

namespace zg {
namespace {

constexpr int kTile = 64;  // channels of a block: two to a lane
constexpr int kChunk = ZG_SCAN_CHUNK;
constexpr int kGroup = 16;
constexpr float kConst = -1.0f;
#ifndef ZG_SCAN_FT
#define ZG_SCAN_FT 16
#endif
#ifndef ZG_SCAN_BT
#define ZG_SCAN_BT 8
#endif
#ifndef ZG_SCAN_FB
#define ZG_SCAN_FB 2
#endif
#ifndef ZG_SCAN_BB
#define ZG_SCAN_BB 1
#endif

// ------------------------------------------------------------------ elements

// Two elements as they lie in memory, so that bf16 pairs take one register.
template <class T, bool PAIR>
struct Raw;
template <bool PAIR>
struct Raw<uint16_t, PAIR> {
    uint32_t w;
    __device__ __forceinline__ void load(const uint16_t *p, int64_t c0, int64_t c1, bool ok0, bool ok1)
    {
        if (PAIR)
            w = ok0 ? __ldcs(reinterpret_cast<const uint32_t *>(p + c0)) : 0u;
        else
            w = (ok0 ? uint32_t(__ldcs(p + c0)) : 0u) | ((ok1 ? uint32_t(__ldcs(p + c1)) : 0u) << 16);
    }
    __device__ __forceinline__ void zero() { w = 0u; }
    __device__ __forceinline__ float2 get() const { return make_float2(bf16_lo(w), bf16_hi(w)); }
};
template <bool PAIR>
struct Raw<float, PAIR> {
    float2 w;
    __device__ __forceinline__ void load(const float *p, int64_t c0, int64_t c1, bool ok0, bool ok1)
    {
        if (PAIR)
            w = ok0 ? __ldcs(reinterpret_cast<const float2 *>(p + c0)) : make_float2(0.0f, 0.0f);
        else
            w = make_float2(ok0 ? __ldcs(p + c0) : 0.0f, ok1 ? __ldcs(p + c1) : 0.0f);
    }
    __device__ __forceinline__ void zero() { w = make_float2(0.0f, 0.0f); }
    __device__ __forceinline__ float2 get() const { return w; }
};

template <bool PAIR>
__device__ __forceinline__ void store2(uint16_t *p, int64_t c0, int64_t c1, bool ok0, bool ok1, float2 v)
{
    const uint32_t w = pack_bf16x2(v.x, v.y);
    if (PAIR) {
        if (ok0) __stcs(reinterpret_cast<uint32_t *>(p + c0), w);
    } else {
        if (ok0) __stcs(p + c0, uint16_t(w));
        if (ok1) __stcs(p + c1, uint16_t(w >> 16));
    }
}
template <bool PAIR>
__device__ __forceinline__ void store2(float *p, int64_t c0, int64_t c1, bool ok0, bool ok1, float2 v)
{
    if (PAIR) {
        if (ok0) __stcs(reinterpret_cast<float2 *>(p + c0), v);
    } else {
        if (ok0) __stcs(p + c0, v.x);
        if (ok1) __stcs(p + c1, v.y);
    }
}

// ------------------------------------------------------------------ gates

// The smaller of sigmoid(f) and sigmoid(-f), at most a half, with its sign
// set when it is sigmoid(-f): the larger one is one minus it, exactly rounded,
// so one register keeps both gates to a few units in the last place.
__device__ __forceinline__ float gate(float f)
{
    const float e = __expf(-fabsf(f));
    const float small = __fdividef(e, 1.0f + e);
    return copysignf(small, -f);
}
__device__ __forceinline__ float keep_of(float v) { return signbit(v) ? 1.0f + v : v; }  // sigmoid(f)
__device__ __forceinline__ float take_of(float v) { return signbit(v) ? -v : 1.0f - v; }  // sigmoid(-f)
__device__ __forceinline__ float2 keep_of(float2 v) { return make_float2(keep_of(v.x), keep_of(v.y)); }
__device__ __forceinline__ float2 take_of(float2 v) { return make_float2(take_of(v.x), take_of(v.y)); }

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return make_float2(a.x - b.x, a.y - b.y); }

// A map of the state, for a lane's two channels.
struct Map {
    float2 a, b;
};
__device__ __forceinline__ Map identity() { return Map{make_float2(1.0f, 1.0f), make_float2(0.0f, 0.0f)}; }
// `first`, then `second`. Both channels of a constant map are marked.
__device__ __forceinline__ Map then(const Map &first, const Map &second)
{
    if (second.a.x < 0.0f) return second;
    const float2 b = fma2(second.a, first.b, second.b);
    if (first.a.x < 0.0f) return Map{first.a, b};
    return Map{mul2(second.a, first.a), b};
}
__device__ __forceinline__ float2 apply(const Map &m, float2 h) { return m.a.x < 0.0f ? m.b : fma2(m.a, h, m.b); }

// ------------------------------------------------------------------ the workspace
//
// Every binary32 goes with a 32-bit tag in one 64-bit word, which is written
// and read whole: a word whose tag is the launch's epoch holds that launch's
// value, so nothing has to be cleared between launches and no fence orders
// data and flag. ctl holds the epoch (high half) and how many blocks have
// taken a place (low half).

struct Work {
    unsigned long long *ctl;
    ulonglong2 *chunk;  // per chunk, tile and lane: a.x, b.x and a.y, b.y
    ulonglong2 *group;  // the same per group
    ulonglong2 *span;   // per span, tile and lane: the state after it
    int *status;
    long long wait_limit;
};

__device__ __forceinline__ void put(ulonglong2 *p, float x, float y, uint32_t tag)
{
    const unsigned long long t = (unsigned long long)(tag) << 32;
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p), "l"(t | __float_as_uint(x)),
                 "l"(t | __float_as_uint(y))
                 : "memory");
}
__device__ __forceinline__ bool got(const ulonglong2 *p, uint32_t tag, float &x, float &y)
{
    unsigned long long u, v;
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(u), "=l"(v) : "l"(p) : "memory");
    x = __uint_as_float(uint32_t(u));
    y = __uint_as_float(uint32_t(v));
    return uint32_t(u >> 32) == tag && uint32_t(v >> 32) == tag;
}

// Another try at a word that is not there yet; false when the wait ran out,
// here or in another block (which then must not be waited for).
__device__ __noinline__ bool try_on(const Work &w, long long &polls)
{
    if (++polls > w.wait_limit) {
        atomicExch(w.status, ZG_ERR_DEVICE_TIMEOUT);
        return false;
    }
    return (polls & 63) || *reinterpret_cast<volatile int *>(w.status) == 0;
}

__device__ __forceinline__ Map wait_map(const ulonglong2 *p, uint32_t tag, const Work &w)
{
    Map m;
    long long polls = 0;
    while (!(got(p, tag, m.a.x, m.b.x) & got(p + 1, tag, m.a.y, m.b.y)))
        if (!try_on(w, polls)) return identity();
    return m;
}
__device__ __forceinline__ void put_map(ulonglong2 *p, const Map &m, uint32_t tag)
{
    put(p, m.a.x, m.b.x, tag);
    put(p + 1, m.a.y, m.b.y, tag);
}

// ------------------------------------------------------------------ packed sequences

// First index in the non-decreasing v[0, n) whose value is at least `key` (n
// if there is none), by all lanes of a warp, 32 probes at a time.
__device__ __forceinline__ int64_t lower_bound(const int64_t *v, int64_t n, int64_t key)
{
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
        const int m = __popc(__ballot_sync(0xffffffffu, at < hi && v[at] < key));
        const int64_t end = lo + m * step;
        hi = end < hi ? end : hi;
        lo = m ? lo + (m - 1) * step + 1 : lo;
        if (!m) hi = lo;
    }
    return lo;
}

// Where sequences begin and end in a chunk: their number by token, or -1.
struct Cuts {
    int first[kChunk];
    int last[kChunk];
    int64_t range[2];
};

// Fills `cuts` for the tokens [c0, c0 + kChunk) and copies the state of the
// empty sequences that lie there. All threads of the block; ends with a
// barrier.
template <int W>
__device__ __forceinline__ void find_cuts(Cuts &cuts, const ScanArgs &a, int64_t c0, int64_t ch0, int64_t ch1, bool ok0,
                                          bool ok1, const float *from, float *to)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int64_t c1 = c0 + kChunk < a.tokens ? c0 + kChunk : a.tokens;
    for (int i = threadIdx.x; i < kChunk; i += 32 * W) cuts.first[i] = cuts.last[i] = -1;
    if (warp == 0) {
        const int64_t lo = lower_bound(a.seq_start, a.n_seq, c0);
        if (lane == 0) cuts.range[0] = lo > 0 ? lo - 1 : 0;
    }
    if (warp == W - 1) {
        const int64_t hi = c1 == a.tokens ? a.n_seq : lower_bound(a.seq_start, a.n_seq, c1);
        if (lane == 0) cuts.range[1] = hi;
    }
    __syncthreads();
    for (int64_t s = cuts.range[0] + warp; s < cuts.range[1]; s += W) {
        const int64_t lo = a.seq_start[s], hi = a.seq_start[s + 1];
        if (hi > lo) {
            if (lane == 0 && lo >= c0 && lo < c1) cuts.first[lo - c0] = int(s);
            if (lane == 0 && hi > c0 && hi <= c1) cuts.last[hi - 1 - c0] = int(s);
        } else if (to && lo >= c0 && (lo < c1 || c1 == a.tokens)) {
            if (ok0) to[s * a.channels + ch0] = from ? from[s * a.channels + ch0] : 0.0f;
            if (ok1) to[s * a.channels + ch1] = from ? from[s * a.channels + ch1] : 0.0f;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ float2 state2(const float *p, int64_t s, int64_t channels, int64_t c0, int64_t c1, bool ok0,
                                         bool ok1)
{
    if (!p) return make_float2(0.0f, 0.0f);
    return make_float2(ok0 ? p[s * channels + c0] : 0.0f, ok1 ? p[s * channels + c1] : 0.0f);
}
__device__ __forceinline__ void put_state2(float *p, int64_t s, int64_t channels, int64_t c0, int64_t c1, bool ok0,
                                           bool ok1, float2 v)
{
    if (ok0) p[s * channels + c0] = v.x;
    if (ok1) p[s * channels + c1] = v.y;
}

// ------------------------------------------------------------------ a block's place and its predecessors

struct Place {
    int64_t k, rest;  // chunk in scan order, and batch row x tile
    uint32_t epoch;
};

// Blocks take their places in scan order as they start, so the ones that a
// block waits for have all started before it.
__device__ __forceinline__ Place take_place(const Work &w, int64_t width, bool alone, unsigned long long *shared)
{
    if (alone) return Place{0, int64_t(blockIdx.x), 0u};
    if (threadIdx.x == 0) {
        const unsigned long long got = atomicAdd(w.ctl, 1ull);
        if (uint32_t(got) == gridDim.x - 1)  // the last place: the next launch has another epoch
            atomicExch(w.ctl, ((got >> 32) + 1ull) << 32);
        *shared = got;
    }
    __syncthreads();
    const unsigned long long got = *shared;
    const uint32_t n = uint32_t(got);
    return Place{int64_t(n) / width, int64_t(n) % width, uint32_t(got >> 32)};
}

template <int W>
struct Shared {
    float4 warp_map[W][32];  // a.x, a.y, b.x, b.y
    float4 part[8][32];
    unsigned long long place;
};

__device__ __forceinline__ float4 pack(const Map &m) { return make_float4(m.a.x, m.a.y, m.b.x, m.b.y); }
__device__ __forceinline__ Map unpack(float4 v) { return Map{make_float2(v.x, v.y), make_float2(v.z, v.w)}; }

// Publishes this block's map and returns the state before its first token (in
// scan order) from the blocks before it. sh.warp_map holds the warps' maps in
// scan order and has been fenced by a barrier. `slot`: index of the record of
// chunk k at this tile; chunks, groups and spans of a tile are `width` records
// of 32 lanes apart.
template <int W>
__device__ __forceinline__ float2 state_before(Shared<W> &sh, const Work &w, const Place &at, int64_t chunks, int64_t width)
{
    static_assert(W >= 8, "four warps compose the groups and four the chunks");
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int in_group = int(at.k % kGroup), group = int(at.k / kGroup % kGroup);
    const int64_t first_chunk = at.k - in_group, this_group = at.k / kGroup, first_group = this_group - group;
    auto chunk_at = [&](int64_t k) { return w.chunk + 2 * ((k * width + at.rest) * 32 + lane); };
    auto group_at = [&](int64_t g) { return w.group + 2 * ((g * width + at.rest) * 32 + lane); };
    auto span_at = [&](int64_t s) { return w.span + (s * width + at.rest) * 32 + lane; };
    const bool ends_group = in_group == kGroup - 1 && at.k + 1 < chunks;
    Map mine = identity();
    if (warp == 4) {
#pragma unroll
        for (int v = 0; v < W; ++v) mine = then(mine, unpack(sh.warp_map[v][lane]));
        if (!ends_group && at.k + 1 < chunks) put_map(chunk_at(at.k), mine, at.epoch);
    }
    if (warp < 8) {
        Map m = identity();
        if (warp >= 4) {  // chunks of this group, four to a warp
            const int lo = 4 * (warp - 4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lo + i < in_group) m = then(m, wait_map(chunk_at(first_chunk + lo + i), at.epoch, w));
        } else {  // the span before, then groups of this span
            const int lo = 4 * warp - 1;
            if (warp == 0 && first_group > 0) {
                long long polls = 0;
                float2 s;
                while (!got(span_at(first_group / kGroup - 1), at.epoch, s.x, s.y))
                    if (!try_on(w, polls)) {
                        s = make_float2(0.0f, 0.0f);
                        break;
                    }
                m = Map{make_float2(kConst, kConst), s};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lo + i >= 0 && lo + i < group) m = then(m, wait_map(group_at(first_group + lo + i), at.epoch, w));
        }
        sh.part[warp][lane] = pack(m);
        if (warp >= 4 && ends_group) {
            // the group's map must not wait for the groups before it
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (warp == 4) {
                Map g = unpack(sh.part[4][lane]);
#pragma unroll
                for (int v = 5; v < 8; ++v) g = then(g, unpack(sh.part[v][lane]));
                if (group < kGroup - 1) put_map(group_at(this_group), then(g, mine), at.epoch);
            }
        }
    }
    __syncthreads();
    float2 h = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int v = 0; v < 8; ++v) h = apply(unpack(sh.part[v][lane]), h);
    if (warp == 4 && ends_group && group == kGroup - 1) {
        const float2 s = apply(mine, h);
        put(span_at(this_group / kGroup), s.x, s.y, at.epoch);
    }
    return h;
}

// ------------------------------------------------------------------ forward

template <class T, bool PAIR, bool PACKED, int TPT, int W>
__global__ void __launch_bounds__(32 * W, W == 1 ? 8 : W == 8 ? ZG_SCAN_FB : 1) scan_kernel(ScanArgs a, Work w, int64_t chunks, int64_t tiles)
{
    __shared__ Shared<W> sh;
    __shared__ Cuts cuts;  // unused, and not allocated, unless PACKED
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const Place at = take_place(w, a.batch * tiles, chunks == 1, &sh.place);
    const int64_t row = at.rest / tiles, tile = at.rest % tiles;
    const int64_t ch0 = tile * kTile + (PAIR ? 2 * lane : lane), ch1 = ch0 + (PAIR ? 1 : 32);
    const bool ok0 = ch0 < a.channels, ok1 = ch1 < a.channels;
    const int64_t c0 = at.k * (TPT * W), t0 = c0 + warp * TPT;

    Raw<T, PAIR> x[TPT], f[TPT];
    {
        const T *px = static_cast<const T *>(a.x.ptr) + row * a.x.sb + t0 * a.x.st;
        const T *pf = static_cast<const T *>(a.f.ptr) + row * a.f.sb + t0 * a.f.st;
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const bool in = t0 + i < a.tokens;
            f[i].load(pf + i * a.f.st, ch0, ch1, in && ok0, in && ok1);
            x[i].load(px + i * a.x.st, ch0, ch1, in && ok0, in && ok1);
        }
    }
    int64_t end = a.tokens;
    uint32_t first = !PACKED && t0 == 0, last = 0;
    if (PACKED) {
        end = a.seq_start[a.n_seq];
        end = end < a.tokens ? end : a.tokens;
        find_cuts<W>(cuts, a, c0, ch0, ch1, ok0, ok1, a.h0, a.h_last);
        first = __ballot_sync(0xffffffffu, lane < TPT && cuts.first[warp * TPT + (lane < TPT ? lane : 0)] >= 0);
        last = __ballot_sync(0xffffffffu, lane < TPT && cuts.last[warp * TPT + (lane < TPT ? lane : 0)] >= 0);
    } else if (t0 < end && t0 + TPT >= end) {
        last = 1u << (end - 1 - t0);
    }
    auto first_seq = [&](int i) { return PACKED ? int64_t(cuts.first[warp * TPT + i]) : row; };
    auto last_seq = [&](int i) { return PACKED ? int64_t(cuts.last[warp * TPT + i]) : row; };

    float2 keep[TPT], add[TPT];
    Map m = identity();
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const float2 ff = f[i].get();
        const float2 v = make_float2(gate(ff.x), gate(ff.y));
        keep[i] = keep_of(v);
        add[i] = mul2(take_of(v), x[i].get());
        if (first >> i & 1) {
            m.b = fma2(keep[i], state2(a.h0, first_seq(i), a.channels, ch0, ch1, ok0, ok1), add[i]);
            m.a = make_float2(kConst, kConst);
        } else if (t0 + i < a.tokens) {
            m.b = fma2(keep[i], m.b, add[i]);
            if (m.a.x >= 0.0f) m.a = mul2(m.a, keep[i]);
        }
    }
    float2 h = make_float2(0.0f, 0.0f);
    if (W > 1) {
        sh.warp_map[warp][lane] = pack(m);
        __syncthreads();
        if constexpr (W >= 8) {
            if (chunks > 1) h = state_before<W>(sh, w, at, chunks, a.batch * tiles);
        }
    }
    if (a.states && warp == 0)
        put_state2(a.states + (row * chunks + at.k) * a.channels, 0, 0, ch0, ch1, ok0, ok1, h);
    for (int v = 0; v < warp; ++v) h = apply(unpack(sh.warp_map[v][lane]), h);
    T *py = static_cast<T *>(a.y.ptr) + row * a.y.sb + t0 * a.y.st;
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        if (first >> i & 1) h = state2(a.h0, first_seq(i), a.channels, ch0, ch1, ok0, ok1);
        h = fma2(keep[i], h, add[i]);
        const bool in = t0 + i < end;
        store2<PAIR>(py + i * a.y.st, ch0, ch1, in && ok0, in && ok1, h);
        if (a.h_last && (last >> i & 1)) put_state2(a.h_last, last_seq(i), a.channels, ch0, ch1, ok0, ok1, h);
    }
}

// ------------------------------------------------------------------ backward

template <class T, bool PAIR, bool PACKED, int TPT, int W>
__global__ void __launch_bounds__(32 * W, W == 1 ? 8 : W == 16 ? ZG_SCAN_BB : 1) scan_bwd_kernel(ScanArgs a, Work w, int64_t chunks, int64_t tiles)
{
    __shared__ Shared<W> sh;
    __shared__ float4 fwd[W][32];
    __shared__ Cuts cuts;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const Place at = take_place(w, a.batch * tiles, chunks == 1, &sh.place);
    const int64_t row = at.rest / tiles, tile = at.rest % tiles;
    const int64_t ch0 = tile * kTile + (PAIR ? 2 * lane : lane), ch1 = ch0 + (PAIR ? 1 : 32);
    const bool ok0 = ch0 < a.channels, ok1 = ch1 < a.channels;
    const int64_t k = chunks - 1 - at.k;  // the scan goes from the end
    const int64_t c0 = k * (TPT * W), t0 = c0 + warp * TPT;

    Raw<T, PAIR> x[TPT], f[TPT], dy[TPT];
    {
        const T *px = static_cast<const T *>(a.x.ptr) + row * a.x.sb + t0 * a.x.st;
        const T *pf = static_cast<const T *>(a.f.ptr) + row * a.f.sb + t0 * a.f.st;
        const T *pd = static_cast<const T *>(a.y.ptr) + row * a.y.sb + t0 * a.y.st;
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const bool in = t0 + i < a.tokens;
            f[i].load(pf + i * a.f.st, ch0, ch1, in && ok0, in && ok1);
            dy[i].load(pd + i * a.y.st, ch0, ch1, in && ok0, in && ok1);
            x[i].load(px + i * a.x.st, ch0, ch1, in && ok0, in && ok1);
        }
    }
    float2 h = make_float2(0.0f, 0.0f);
    if (k > 0) h = state2(a.states + (row * chunks + k) * a.channels, 0, 0, ch0, ch1, ok0, ok1);
    int64_t end = a.tokens;
    uint32_t first = !PACKED && t0 == 0, last = 0;
    if (PACKED) {
        end = a.seq_start[a.n_seq];
        end = end < a.tokens ? end : a.tokens;
        find_cuts<W>(cuts, a, c0, ch0, ch1, ok0, ok1, a.dh_last, a.dh0);
        first = __ballot_sync(0xffffffffu, lane < TPT && cuts.first[warp * TPT + (lane < TPT ? lane : 0)] >= 0);
        last = __ballot_sync(0xffffffffu, lane < TPT && cuts.last[warp * TPT + (lane < TPT ? lane : 0)] >= 0);
    } else if (t0 < end && t0 + TPT >= end) {
        last = 1u << (end - 1 - t0);
    }
    auto first_seq = [&](int i) { return PACKED ? int64_t(cuts.first[warp * TPT + i]) : row; };
    auto last_seq = [&](int i) { return PACKED ? int64_t(cuts.last[warp * TPT + i]) : row; };

    float2 gates[TPT], slope[TPT];
    Map m = identity(), r = identity();
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const float2 ff = f[i].get();
        gates[i] = make_float2(gate(ff.x), gate(ff.y));
        const float2 keep = keep_of(gates[i]), add = mul2(take_of(gates[i]), x[i].get());
        if (first >> i & 1) {
            m.b = fma2(keep, state2(a.h0, first_seq(i), a.channels, ch0, ch1, ok0, ok1), add);
            m.a = make_float2(kConst, kConst);
        } else {
            m.b = fma2(keep, m.b, add);
            if (m.a.x >= 0.0f) m.a = mul2(m.a, keep);
        }
    }
#pragma unroll
    for (int i = TPT - 1; i >= 0; --i) {
        if (t0 + i >= end) continue;
        const float2 keep = keep_of(gates[i]);
        if (last >> i & 1) {
            r.b = mul2(keep, add2(dy[i].get(), state2(a.dh_last, last_seq(i), a.channels, ch0, ch1, ok0, ok1)));
            r.a = make_float2(kConst, kConst);
        } else {
            r.b = mul2(keep, add2(dy[i].get(), r.b));
            if (r.a.x >= 0.0f) r.a = mul2(r.a, keep);
        }
    }
    float2 g = make_float2(0.0f, 0.0f);
    if (W > 1) {
        sh.warp_map[W - 1 - warp][lane] = pack(r);
        fwd[warp][lane] = pack(m);
        __syncthreads();
        if constexpr (W >= 8) {
            if (chunks > 1) g = state_before<W>(sh, w, at, chunks, a.batch * tiles);
        }
        for (int v = 0; v < warp; ++v) h = apply(unpack(fwd[v][lane]), h);
        for (int v = 0; v < W - 1 - warp; ++v) g = apply(unpack(sh.warp_map[v][lane]), g);
    }
    // forward once more: x gives way to (h_{t-1} - x_t) a_t (1 - a_t)
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        if (first >> i & 1) h = state2(a.h0, first_seq(i), a.channels, ch0, ch1, ok0, ok1);
        const float2 keep = keep_of(gates[i]), take = take_of(gates[i]), xx = x[i].get();
        slope[i] = mul2(sub2(h, xx), mul2(keep, take));
        h = fma2(keep, h, mul2(take, xx));
    }
    T *px = static_cast<T *>(a.dx.ptr) + row * a.dx.sb + t0 * a.dx.st;
    T *pf = static_cast<T *>(a.df.ptr) + row * a.df.sb + t0 * a.df.st;
#pragma unroll
    for (int i = TPT - 1; i >= 0; --i) {
        if (t0 + i >= end) continue;
        if (last >> i & 1) g = state2(a.dh_last, last_seq(i), a.channels, ch0, ch1, ok0, ok1);
        g = add2(dy[i].get(), g);
        store2<PAIR>(px + i * a.dx.st, ch0, ch1, ok0, ok1, mul2(take_of(gates[i]), g));
        store2<PAIR>(pf + i * a.df.st, ch0, ch1, ok0, ok1, mul2(slope[i], g));
        g = mul2(keep_of(gates[i]), g);
        if (a.dh0 && (first >> i & 1)) put_state2(a.dh0, first_seq(i), a.channels, ch0, ch1, ok0, ok1, g);
    }
}

// ------------------------------------------------------------------ launches

bool pairs(const ScanView &v, int size, int64_t channels)
{
    return channels % 2 == 0 && v.sb % 2 == 0 && v.st % 2 == 0 && reinterpret_cast<uintptr_t>(v.ptr) % (2 * size) == 0;
}

template <class T, bool PAIR, bool PACKED, int TPT, int W, bool BWD>
cudaError_t launch(const ScanArgs &a, const ScanWork &sw, cudaStream_t st)
{
    const int64_t tiles = (a.channels + kTile - 1) / kTile, chunks = (a.tokens + TPT * W - 1) / (TPT * W);
    const int64_t blocks = a.batch * tiles * chunks;
    if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    Work w{};
    w.ctl = sw.ctl;
    w.status = sw.status;
    w.wait_limit = sw.wait_limit;
    w.chunk = reinterpret_cast<ulonglong2 *>(sw.records);
    w.group = w.chunk + 2 * 32 * (a.batch * tiles * chunks);
    w.span = w.group + 2 * 32 * (a.batch * tiles * (chunks / kGroup));
    if (BWD)
        scan_bwd_kernel<T, PAIR, PACKED, TPT, W><<<unsigned(blocks), 32 * W, 0, st>>>(a, w, chunks, tiles);
    else
        scan_kernel<T, PAIR, PACKED, TPT, W><<<unsigned(blocks), 32 * W, 0, st>>>(a, w, chunks, tiles);
    return cudaGetLastError();
}

template <class T, bool PAIR, bool BWD>
cudaError_t pick(const ScanArgs &a, const ScanWork &w, cudaStream_t st)
{
    // One warp walks a short row alone, its tokens all in registers; packed
    // rows always take whole chunks, in whose tables their sequences are found.
    constexpr int TPT = BWD ? ZG_SCAN_BT : ZG_SCAN_FT;
    if (a.seq_start) return launch<T, PAIR, true, TPT, kChunk / TPT, BWD>(a, w, st);
    if (a.tokens == 1) return launch<T, PAIR, false, 1, 1, BWD>(a, w, st);
    if (a.tokens <= 8) return launch<T, PAIR, false, 8, 1, BWD>(a, w, st);
    return launch<T, PAIR, false, TPT, kChunk / TPT, BWD>(a, w, st);
}

template <bool BWD>
cudaError_t by_type(const ScanArgs &a, const ScanWork &w, cudaStream_t st)
{
    const int size = a.dtype == ZG_DTYPE_BF16 ? 2 : 4;
    bool pair = pairs(a.x, size, a.channels) && pairs(a.f, size, a.channels) && pairs(a.y, size, a.channels);
    if (BWD) pair = pair && pairs(a.dx, size, a.channels) && pairs(a.df, size, a.channels);
    if (size == 2) return pair ? pick<uint16_t, true, BWD>(a, w, st) : pick<uint16_t, false, BWD>(a, w, st);
    return pair ? pick<float, true, BWD>(a, w, st) : pick<float, false, BWD>(a, w, st);
}

}  // namespace

int64_t scan_record_bytes(int64_t batch, int64_t tokens, int64_t channels)
{
    const int64_t width = batch * ((channels + kTile - 1) / kTile), chunks = (tokens + kChunk - 1) / kChunk;
    if (chunks == 1) return 0;
    return width * 32 * 16 * (2 * chunks + 2 * (chunks / kGroup) + chunks / (kGroup * kGroup));
}

cudaError_t launch_scan(const ScanArgs &a, const ScanWork &w, cudaStream_t st) { return by_type<false>(a, w, st); }
cudaError_t launch_scan_bwd(const ScanArgs &a, const ScanWork &w, cudaStream_t st) { return by_type<true>(a, w, st); }

}  // namespace zg
