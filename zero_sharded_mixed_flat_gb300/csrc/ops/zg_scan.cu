// The gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t with
// a_t = sigmoid(f_t), forward and backward, in one pass over the data.
//
// The recurrence is a scan over affine maps: a run of tokens takes the state
// h to A h + B, with A the product of its gates, and two runs compose to
// (A2 A1, A2 B1 + B2). Backward is the same scan from the end, of
// r -> a_t (dy_t + r). A tile is kChunk tokens by kTile channels: each half
// warp holds a run of kRun tokens in registers, four channels to a lane, and
// reduces it to one map; the runs' maps are composed through shared memory, and
// the chunks' maps through a workspace in global memory, where a block waits
// for the chunks before its own. With the state at its first token known, each
// run goes through its tokens again from the registers and stores.
//
// So x and f are read once and y is written once: 6 bytes per element in
// bf16 (10 in backward, with dy, dx and df) and about 0.3 in the workspace.
// Blocks stay on their SM and take tile after tile; the next tile's copies
// into shared memory are in flight while a tile is worked on, so memory stays
// busy through the waits.
//
// The maps of earlier chunks are composed in a fixed order, by a tree of
// kGroup chunks to a group and kGroup groups to a span, whatever the order
// in which blocks run: the same inputs give the same bits. Only the state at
// the end of a span hangs on the span before it, so the chain of waits is one
// step per kGroup^2 chunks.
//
// Packed sequences that begin inside a chunk cut the scan: a run that holds a
// beginning has a constant map, marked by A = kConst (every real A is >= 0, or a
// NaN), so nothing before it, a NaN included, is multiplied into what follows.
// (The mark is asked for as A < 0, which a NaN is not.)
//
// Measured: 8 x 4096 x 1536 in bf16 forward 66 us (4.6 TB/s of x, f and y),
// backward 104 (4.9 TB/s of five). Neither the bytes (44.5 and 74 us) nor the issue
// of 25 and 45 instructions an element (31 and 55 us) is the limit: with two blocks
// of eight warps to an SM, which is what 128 registers allow, issue is active in 50
// and 56 % of the cycles and DRAM in 41 and 48 %, and warps wait at barriers most of
// all (profile of 8 x 2048 x 1536). Three blocks to an SM, tried with what is kept in
// registers now, spill and are slower. Rows at odd channels (1535 of them) 97 and
// 160, with stores of two bytes; 1 x 65536 x 768 90 and 123 (twelve tiles to a chunk,
// so a block waits for records that blocks beside it are only writing); 8 x 1024 x
// 768 13.5 and 19.6, two tiles to a block; binary32, 1 x 20000 x 768 45 and 62, 8 x
// 4096 x 1536 98 and 159. Packed: 9001 x 771 in binary32 31 and 48, in bf16 24 and 40
// (three full waves of blocks and a part of a fourth, and a last tile of 3 channels);
// bf16 65536 x 768 107 and 180, 32768 x 4096 247 and 420.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "zg_launch.h"
#include "zg_ops.h"

namespace zg {
namespace {

constexpr int kTile = 64;  // channels of a tile: four to a lane of a half warp
constexpr int kChunk = ZG_SCAN_CHUNK;
constexpr int kWarps = 8;
constexpr int kRun = kChunk / (2 * kWarps);  // tokens of a half warp
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 16;
constexpr float kConst = -1.0f;

// ------------------------------------------------------------------ arithmetic

// Four channels of a lane, two to a packed operation.
struct F4 {
    float2 lo, hi;
};
__device__ __forceinline__ F4 all(float v) { return F4{make_float2(v, v), make_float2(v, v)}; }
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t *>(&a)), "l"(*reinterpret_cast<const uint64_t *>(&b)));
    return *reinterpret_cast<const float2 *>(&d);
}
__device__ __forceinline__ float2 neg(float2 v) { return make_float2(-v.x, -v.y); }
__device__ __forceinline__ F4 mul(F4 a, F4 b) { return F4{mul_f32x2(a.lo, b.lo), mul_f32x2(a.hi, b.hi)}; }
__device__ __forceinline__ F4 add(F4 a, F4 b) { return F4{add_f32x2(a.lo, b.lo), add_f32x2(a.hi, b.hi)}; }
__device__ __forceinline__ F4 fma(F4 a, F4 b, F4 c)
{
    return F4{fma_f32x2(a.lo, b.lo, c.lo), fma_f32x2(a.hi, b.hi, c.hi)};
}
__device__ __forceinline__ F4 sub(F4 a, F4 b) { return fma(b, all(-1.0f), a); }

__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float exp2_approx(float v)
{
    float d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
    return d;
}
__device__ __forceinline__ float rcp_approx(float v)
{
    float d;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
    return d;
}

// keep = sigmoid(f) = 1 / (1 + e) and take = sigmoid(-f) = e / (1 + e) with
// e = exp(-f): neither is a difference, so both hold to a few units in the
// last place however near to one the other is. f is held above kLowest, where
// e and its sum are still finite, and keep is taken down by just less than its
// value there, so that it ends at zero, never below; a NaN stays. That is an error
// below 3e-38, which shows in keep itself where f is below about -70 (its last
// place there, 1.5e-3 of it at -80). For binary32 data the exponent's argument is reduced first
// (as Cody and Waite do it: n log 2 taken off in two parts), which keeps its rounding
// out of e; for bf16 data that rounding (|f| 2^-24 of e) is far below the data's own.
constexpr float kLowest = -86.5f;
constexpr float kKeepAtLowest = 2.71337577e-38f;  // exp(kLowest), less 4e-5 of itself for the roundings on the way
constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f;

template <class T>
__device__ __forceinline__ float2 decay(float2 f)  // f at least kLowest, or NaN
{
    float2 e;
    if (sizeof(T) == 2) {
        const float2 t = mul_f32x2(f, make_float2(-kLog2e, -kLog2e));
        e = make_float2(exp2_approx(t.x), exp2_approx(t.y));
    } else {
        const float2 t = mul_f32x2(f, make_float2(-kLog2e, -kLog2e));
        // whole part of the exponent; a multiplication by 2^n at or above 2^-126
        const float2 n = make_float2(rintf(max_nan(t.x, -126.0f)), rintf(max_nan(t.y, -126.0f)));
        float2 r = fma_f32x2(f, make_float2(-kLog2e, -kLog2e), neg(n));
        r = fma_f32x2(make_float2(fminf(f.x, 1e30f), fminf(f.y, 1e30f)), make_float2(-kLog2eRest, -kLog2eRest), r);
        e = mul_f32x2(make_float2(exp2_approx(r.x), exp2_approx(r.y)),
                      make_float2(__int_as_float((__float2int_rn(n.x) + 127) << 23),
                                  __int_as_float((__float2int_rn(n.y) + 127) << 23)));
    }
    return e;
}
template <class T>
__device__ __forceinline__ F4 decay(F4 f)
{
    return F4{decay<T>(f.lo), decay<T>(f.hi)};
}
// The reciprocal once more, in a pass that is not to find the first one's kept
// in registers.
__device__ __forceinline__ float rcp_again(float v)
{
    float d;
    asm volatile("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
    return d;
}
__device__ __forceinline__ void gates_again(float2 e, float2 &keep, float2 &take)
{
    const float2 d = add_f32x2(e, make_float2(1.0f, 1.0f));
    const float2 r = make_float2(rcp_again(d.x), rcp_again(d.y));
    keep = add_f32x2(r, make_float2(-kKeepAtLowest, -kKeepAtLowest));
    take = mul_f32x2(e, r);
}
__device__ __forceinline__ void gates(float2 e, float2 &keep, float2 &take)
{
    const float2 d = add_f32x2(e, make_float2(1.0f, 1.0f));
    const float2 r = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    keep = add_f32x2(r, make_float2(-kKeepAtLowest, -kKeepAtLowest));
    take = mul_f32x2(e, r);
}
__device__ __forceinline__ void gates(F4 e, F4 &keep, F4 &take)
{
    gates(e.lo, keep.lo, take.lo);
    gates(e.hi, keep.hi, take.hi);
}

__device__ __forceinline__ void gates_again(F4 e, F4 &keep, F4 &take)
{
    gates_again(e.lo, keep.lo, take.lo);
    gates_again(e.hi, keep.hi, take.hi);
}

// A map of the state, h -> a h + b: for a lane's four channels of a run, and for
// one slot (x = a, y = b). A constant one is marked in all channels; there are
// none unless sequences are packed (CUT).
struct Map {
    F4 a, b;
};
// `first`, then `second`.
template <bool CUT>
__device__ __forceinline__ float2 then(float2 first, float2 second)
{
    if (CUT && second.x < 0.0f) return second;
    return make_float2(CUT && first.x < 0.0f ? first.x : second.x * first.x, fmaf(second.x, first.y, second.y));
}
template <bool CUT>
__device__ __forceinline__ float apply(float2 m, float h)
{
    return CUT && m.x < 0.0f ? m.y : fmaf(m.x, h, m.y);
}

// ------------------------------------------------------------------ the workspace
//
// Every binary32 goes with a 32-bit tag in one 64-bit word, which is written
// and read whole: a word whose tag is the launch's epoch holds that launch's
// value, so nothing has to be cleared between launches and no fence orders
// data and flag. ctl holds the epoch (high half) and how many places have been
// taken (low half).

struct Work {
    unsigned long long *ctl;
    ulonglong2 *chunk;  // per chunk, tile and slot: a, b
    ulonglong2 *group;  // the same per group
    ulonglong2 *span;   // per span, tile and slot: the state after it (twice)
    int *status;
    uint32_t *gave_up;  // the epoch of the last launch in which a wait ran out
    long long wait_limit;
};

__device__ __forceinline__ void put(ulonglong2 *p, float x, float y, uint32_t tag)
{
    const unsigned long long t = (unsigned long long)(tag) << 32;
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p), "l"(t | __float_as_uint(x)),
                 "l"(t | __float_as_uint(y))
                 : "memory");
}
__device__ __forceinline__ ulonglong2 look(const ulonglong2 *p)
{
    ulonglong2 v;
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ bool there(ulonglong2 v, uint32_t tag)
{
    return uint32_t(v.x >> 32) == tag && uint32_t(v.y >> 32) == tag;
}
__device__ __forceinline__ float2 values(ulonglong2 v)
{
    return make_float2(__uint_as_float(uint32_t(v.x)), __uint_as_float(uint32_t(v.y)));
}

// Whether to ask again for words that are not there yet; false when the wait ran
// out, here or in another block of this launch (which then must not be waited for).
// The status stays until it is asked for, over launches that are not concerned.
__device__ __forceinline__ bool go_on(const Work &w, uint32_t tag, long long polls)
{
    if (polls >= w.wait_limit) {
        atomicExch(w.status, kStatusTimeout);
        atomicExch(w.gave_up, tag);
        return false;
    }
    return (polls & 63) != 63 || *reinterpret_cast<volatile uint32_t *>(w.gave_up) != tag;
}

// Up to four maps of one slot, asked for together and composed in order. The
// places past the last are filled with it again, which takes no branch and
// counts for nothing; without any, nothing is asked for.
struct Four {
    const ulonglong2 *p;
    int64_t step;
    int count;  // the same in all lanes of a warp
    ulonglong2 v[4];
    __device__ __forceinline__ void ask()
    {
        if (count <= 0) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = look(p + min(i, count - 1) * step);
    }
    // Where the wait runs out, what is not there is undefined.
    template <bool CUT>
    __device__ __forceinline__ float2 get(uint32_t tag, const Work &w)
    {
        if (count <= 0) return make_float2(1.0f, 0.0f);
        for (long long polls = 0;; ++polls) {
            uint32_t off = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) off |= (uint32_t(v[i].x >> 32) ^ tag) | (uint32_t(v[i].y >> 32) ^ tag);
            if (off == 0u || !go_on(w, tag, polls)) break;
            ask();
        }
        float2 m = values(v[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const float2 n = values(v[i]), both = then<CUT>(m, n);
            m = make_float2(i < count ? both.x : m.x, i < count ? both.y : m.y);
        }
        return m;
    }
};

// ------------------------------------------------------------------ a tile's place

struct Grid {
    int64_t tiles;   // of channels
    int64_t width;   // batch rows x tiles: the tiles of one chunk
    int64_t chunks;
    int64_t places;  // width x chunks
};

// Places are taken in scan order, chunk by chunk, as blocks become free, and
// each block works through the ones it took in that order. So whoever waits
// for a chunk waits for one whose place was taken earlier, and the lowest place
// not yet done never waits: the waits end. Without anything to wait for (one
// chunk) the places are dealt out by block number.
struct Places {
    unsigned long long *ctl;
    int64_t next;  // used where nothing waits
    __device__ __forceinline__ unsigned long long take(const Grid &g)
    {
        if (g.chunks == 1) {
            const int64_t n = next;
            next += gridDim.x;
            return (unsigned long long)(n < g.places ? n : 0xffffffffll);
        }
        const unsigned long long got = atomicAdd(ctl, 1ull);
        // every block stops at its first place past the end, so that many are
        // taken in all; the last one leaves ctl ready for the next launch,
        // under another epoch
        if (uint32_t(got) == uint32_t(g.places) + gridDim.x - 1) atomicExch(ctl, ((got >> 32) + 1ull) << 32);
        return got;
    }
};

struct Tile {
    bool valid;
    uint32_t k;     // chunk in scan order
    uint32_t rest;  // batch row x tiles + tile
    uint32_t row;
    uint32_t chunk;
    int64_t ch;     // first channel
};

template <bool BWD>
__device__ __forceinline__ Tile tile_at(unsigned long long taken, const Grid &g)
{
    const uint32_t place = uint32_t(taken), width = uint32_t(g.width), tiles = uint32_t(g.tiles);
    Tile t;
    t.valid = place < uint32_t(g.places);
    t.k = place / width;
    t.rest = place % width;
    t.row = t.rest / tiles;
    t.ch = int64_t(t.rest % tiles) * kTile;
    t.chunk = BWD ? uint32_t(g.chunks) - 1 - t.k : t.k;
    return t;
}

// ------------------------------------------------------------------ shared memory

struct Cuts {  // where sequences begin and end in a chunk: their number by token, or -1
    int first[kChunk];
    int last[kChunk];
    int64_t range[2];
};

constexpr int kRuns = 2 * kWarps;

// The runs' maps, in scan order; slot 4 l + j of a run is channel j of lane l
// of its half warp. b gives way to the state before each run.
struct Runs {
    float a[kRuns][kTile], b[kRuns][kTile];
};

// What composes a tile's maps. Maps of four runs, and of the chunks and groups
// before, by fours: a, b.
template <bool BWD>
struct Maps {
    Runs runs;
    float2 quarters[4][kTile], chunks[4][kTile], groups[4][kTile];
    float span[kTile];
};
template <>
struct Maps<true> {
    Runs runs;
    union {
        Runs fwd;  // of h; when the maps of chunks and groups come, its a has been read
        struct {
            float2 chunks[4][kTile], groups[4][kTile];
        };
    };
    float2 quarters[4][kTile], fwd_quarters[4][kTile];
    float span[kTile];
};
static_assert(sizeof(Maps<true>::chunks) + sizeof(Maps<true>::groups) <= sizeof(Runs::a), "chunks and groups lie on fwd.a");

struct Shared {
    Tile tile;
    uint32_t tag;
    Cuts cuts;
};

__device__ __forceinline__ F4 lds4(const float *p)
{
    const float4 v = *reinterpret_cast<const float4 *>(p);
    return F4{make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
__device__ __forceinline__ void sts4(float *p, F4 v)
{
    *reinterpret_cast<float4 *>(p) = make_float4(v.lo.x, v.lo.y, v.hi.x, v.hi.y);
}

// N bytes, of which the first `bytes` are read and the others become zero.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, int bytes)
{
    if (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// How a tile's rows lie in memory, and how they are copied. WHOLE: all begin at
// multiples of 16 bytes. ANY: anywhere. Copies are of 16 bytes from 16-byte
// boundaries all the same, from the one at or before a row's first channel, which
// so stands up to kUnit - 1 channels into its row of the buffer (copies of 4 bytes,
// or plain loads of 2: 179 us for 8 x 4096 x 1535 in bf16 forward and 310 backward,
// against 97 and 160). Rows of bf16 at multiples of 8 bytes are loaded and stored
// four channels at a time as WHOLE is, and copied as ANY (FOURS, backward: 131 us
// for 8 x 4096 x 1540 against 175) or in units of 8 bytes (EIGHTS, forward: 74
// against 82; such copies pass through L1, for which backward's buffers leave no
// room).
enum { ANY, FOURS, EIGHTS, WHOLE };
template <int ROWS>
constexpr bool kShifted = ROWS <= FOURS;
template <class T>
constexpr int kUnit = 16 / int(sizeof(T));
template <class T, int ROWS>
constexpr int kPitch = kShifted<ROWS> ? kTile + kUnit<T> : kTile;
// For ANY, whose lanes read single channels, every odd run stands another kSkew
// channels on, so that the two half warps read different banks (binary32, packed,
// 9001 x 771: 34.1 us against 35.1).
template <int ROWS>
constexpr int kSkew = ROWS == ANY ? 16 : 0;
template <class T, int ROWS>
constexpr int kBuffer = kChunk * kPitch<T, ROWS> + kRuns / 2 * kSkew<ROWS>;
template <class T, int ROWS>
__device__ __forceinline__ constexpr int place_of(int r)
{
    return r * kPitch<T, ROWS> + (r / kRun + 1) / 2 * kSkew<ROWS>;
}

// Where the tokens of a run begin in their 16 bytes, one after another. A chunk's
// first token, and every kRun-th, is at the same place, and so is every tile of a
// row.
static_assert(kRun % 8 == 0 && kTile % 8 == 0, "shifts repeat");
template <class T, int ROWS>
struct Walk {
    uint32_t at;
    __device__ __forceinline__ Walk(const ScanView &v, const Tile &t, int i)
    {
        if (!kShifted<ROWS>) return;
        at = uint32_t(reinterpret_cast<uintptr_t>(v.ptr) / sizeof(T)) + t.row * uint32_t(v.sb) + uint32_t(i) * uint32_t(v.st);
        asm volatile("" : "+r"(at));  // not formed again for every token
    }
    __device__ __forceinline__ int shift() const { return kShifted<ROWS> ? int(at % kUnit<T>) : 0; }
    // Token i of a run in a buffer, then on to the next or the last token.
    __device__ __forceinline__ const T *next(const T *buffer, const ScanView &v, int run, int i)
    {
        const T *const row = buffer + place_of<T, ROWS>(run * kRun) + i * kPitch<T, ROWS> + shift();
        if (kShifted<ROWS>) at += uint32_t(v.st);
        return row;
    }
    __device__ __forceinline__ const T *last(const T *buffer, const ScanView &v, int run, int i)
    {
        const T *const row = buffer + place_of<T, ROWS>(run * kRun) + i * kPitch<T, ROWS> + shift();
        if (kShifted<ROWS>) at -= uint32_t(v.st);
        return row;
    }
};

// The unit of v's first element, for copies that read nothing.
template <class T>
__device__ __forceinline__ const T *unit_zero(const ScanView &v)
{
    return reinterpret_cast<const T *>(reinterpret_cast<uintptr_t>(v.ptr) & ~uintptr_t(15));
}

// Copies a tile of v into dst[token][shift + channel]; what lies past the tensor
// becomes zero. Nothing is read past a row's last channel. Up to 15 bytes before
// its first are, in the same 16: memory is allocated from such a boundary on.
template <class T, int ROWS>
__device__ __forceinline__ void start_copy(T *dst, const ScanView &v, const Tile &t, const ScanArgs &a)
{
    constexpr int N = ROWS == EIGHTS ? 8 : 16, kEach = N / int(sizeof(T)), kPerRow = kTile / kEach, kRows = kThreads / kPerRow;
    constexpr int kStep = place_of<T, ROWS>(kRows) * int(sizeof(T));
    static_assert(kRows % (2 * kRun) == 0, "each step is as far as the first");
    const int r0 = threadIdx.x / kPerRow, e = threadIdx.x % kPerRow * kEach;
    const int64_t c0 = int64_t(t.chunk) * kChunk;
    const int shift = Walk<T, ROWS>(v, t, r0).shift();
    const T *const first = static_cast<const T *>(v.ptr) + t.row * v.sb + c0 * v.st + t.ch;
    const T *src = first + r0 * v.st + e - shift;
    const uint32_t base = uint32_t(__cvta_generic_to_shared(dst)), to = base + (place_of<T, ROWS>(r0) + e) * int(sizeof(T));
    const int64_t far = kRows * v.st;
    const bool inside = c0 + kChunk <= a.tokens && t.ch + kTile <= a.channels;
    if (inside) {
#pragma unroll
        for (int i = 0; i < kChunk / kRows; ++i) {
            copy_async<N>(to + i * kStep, src, N);
            src += far;
        }
        if (!kShifted<ROWS>) return;
    }
    const int wide = int(a.channels - t.ch < kTile ? a.channels - t.ch : kTile);
    const int rows = int(a.tokens - c0 < kChunk ? a.tokens - c0 : kChunk);
    if (!inside) {
        const int left = (shift + wide - e) * int(sizeof(T)), bytes = left <= 0 ? 0 : left < N ? left : N;
#pragma unroll 1
        for (int i = 0; i < kChunk / kRows; ++i) {
            const int n = r0 + i * kRows < rows ? bytes : 0;
            copy_async<N>(to + i * kStep, n ? src : unit_zero<T>(v), n);
            src += far;
        }
    }
    if (kShifted<ROWS> && threadIdx.x < kChunk) {  // what the shift moved past a row's last unit
        const int r = threadIdx.x, over = Walk<T, ROWS>(v, t, r).shift() + wide - kTile;
        const bool any = over > 0 && r < rows;
        copy_async<16>(base + (place_of<T, ROWS>(r) + kTile) * int(sizeof(T)), any ? first + r * v.st + (wide - over) : unit_zero<T>(v),
                       any ? over * int(sizeof(T)) : 0);
    }
}
// Asks for a tile of v to be brought into L2, a line for each row (two in
// binary32). Blocks that take their places late cannot copy ahead, but where the
// GPU's next tiles lie is known, whoever takes them: one grid on. Without this
// memory idles while all wait for one another (in bf16, 1 x 65536 x 768 forward 92
// against 97 us and backward 122 against 130; from two grids on, 93 and 126).
template <class T>
__device__ __forceinline__ void bring(const ScanView &v, const Tile &t, const ScanArgs &a)
{
    constexpr int kEach = 128 / int(sizeof(T)), kPieces = kTile / kEach;
    const int64_t c0 = int64_t(t.chunk) * kChunk;
    if (threadIdx.x >= kChunk * kPieces) return;
    const int r = threadIdx.x / kPieces, e = threadIdx.x % kPieces * kEach;
    if (c0 + r < a.tokens && t.ch + e < a.channels)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T *>(v.ptr) + t.row * v.sb + (c0 + r) * v.st + t.ch + e));
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// A lane's channels: four neighbours (VEC) or every sixteenth, so that rows
// whose alignment forbids wide stores are written in whole sectors all the same.
template <bool VEC>
__device__ __forceinline__ int channel_of(int l, int j) { return VEC ? 4 * l + j : l + 16 * j; }

// Lane l's four channels of a row in shared memory.
template <bool VEC>
__device__ __forceinline__ F4 read4(const uint16_t *row, int l)
{
    if (VEC) {
        const uint2 w = *reinterpret_cast<const uint2 *>(row + 4 * l);
        return F4{make_float2(bf16_lo(w.x), bf16_hi(w.x)), make_float2(bf16_lo(w.y), bf16_hi(w.y))};
    }
    return F4{make_float2(bf16_lo(row[l]), bf16_lo(row[l + 16])), make_float2(bf16_lo(row[l + 32]), bf16_lo(row[l + 48]))};
}
// The same of f, held above kLowest.
template <bool VEC>
__device__ __forceinline__ F4 read_f4(const uint16_t *row, int l)
{
    uint2 w;
    if (VEC)
        w = *reinterpret_cast<const uint2 *>(row + 4 * l);
    else
        w = make_uint2(row[l] | uint32_t(row[l + 16]) << 16, row[l + 32] | uint32_t(row[l + 48]) << 16);
    constexpr uint32_t kLowest2 = 0xc2adc2adu;  // kLowest twice in bf16
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.x) : "r"(kLowest2));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.y) : "r"(kLowest2));
    return F4{make_float2(bf16_lo(w.x), bf16_hi(w.x)), make_float2(bf16_lo(w.y), bf16_hi(w.y))};
}
template <bool VEC>
__device__ __forceinline__ F4 read4(const float *row, int l)
{
    if (VEC) return lds4(row + 4 * l);
    return F4{make_float2(row[l], row[l + 16]), make_float2(row[l + 32], row[l + 48])};
}

template <bool VEC>
__device__ __forceinline__ F4 read_f4(const float *row, int l)
{
    const F4 f = read4<VEC>(row, l);
    return F4{make_float2(max_nan(f.lo.x, kLowest), max_nan(f.lo.y, kLowest)),
              make_float2(max_nan(f.hi.x, kLowest), max_nan(f.hi.y, kLowest))};
}

// Lane l's four channels of a row of a tile, `n` of whose channels exist.
template <bool VEC>
__device__ __forceinline__ void store4(uint16_t *row, int l, int n, F4 v)
{
    const uint32_t w0 = pack_bf16x2(v.lo.x, v.lo.y), w1 = pack_bf16x2(v.hi.x, v.hi.y);
    if (VEC) {
        if (4 * l < n) __stcs(reinterpret_cast<uint2 *>(row + 4 * l), make_uint2(w0, w1));
    } else {
        if (l < n) __stcs(row + l, uint16_t(w0));
        if (l + 16 < n) __stcs(row + l + 16, uint16_t(w0 >> 16));
        if (l + 32 < n) __stcs(row + l + 32, uint16_t(w1));
        if (l + 48 < n) __stcs(row + l + 48, uint16_t(w1 >> 16));
    }
}
template <bool VEC>
__device__ __forceinline__ void store4(float *row, int l, int n, F4 v)
{
    if (VEC) {
        if (4 * l < n) __stcs(reinterpret_cast<float4 *>(row + 4 * l), make_float4(v.lo.x, v.lo.y, v.hi.x, v.hi.y));
    } else {
        if (l < n) __stcs(row + l, v.lo.x);
        if (l + 16 < n) __stcs(row + l + 16, v.lo.y);
        if (l + 32 < n) __stcs(row + l + 32, v.hi.x);
        if (l + 48 < n) __stcs(row + l + 48, v.hi.y);
    }
}

// Rows of binary32 states (contiguous, of any alignment), from a tile's first channel.
template <bool VEC>
__device__ __forceinline__ F4 state4(const float *row, int l, int n)
{
    F4 v = all(0.0f);
    if (!row) return v;
    if (channel_of<VEC>(l, 0) < n) v.lo.x = row[channel_of<VEC>(l, 0)];
    if (channel_of<VEC>(l, 1) < n) v.lo.y = row[channel_of<VEC>(l, 1)];
    if (channel_of<VEC>(l, 2) < n) v.hi.x = row[channel_of<VEC>(l, 2)];
    if (channel_of<VEC>(l, 3) < n) v.hi.y = row[channel_of<VEC>(l, 3)];
    return v;
}
template <bool VEC>
__device__ __forceinline__ void put_state4(float *row, int l, int n, F4 v)
{
    if (channel_of<VEC>(l, 0) < n) row[channel_of<VEC>(l, 0)] = v.lo.x;
    if (channel_of<VEC>(l, 1) < n) row[channel_of<VEC>(l, 1)] = v.lo.y;
    if (channel_of<VEC>(l, 2) < n) row[channel_of<VEC>(l, 2)] = v.hi.x;
    if (channel_of<VEC>(l, 3) < n) row[channel_of<VEC>(l, 3)] = v.hi.y;
}

// Zeros to a run's tokens of an output past `end`, where no sequence lies.
template <class T, bool VEC>
__device__ __forceinline__ void clear_rest(const ScanView &v, const Tile &t, int64_t t0, int64_t end, const ScanArgs &a, int l, int n)
{
    T *const p = static_cast<T *>(v.ptr) + t.row * v.sb + t.ch;
    const int64_t stop = t0 + kRun < a.tokens ? t0 + kRun : a.tokens;
#pragma unroll 1
    for (int64_t i = t0 > end ? t0 : end; i < stop; ++i) store4<VEC>(p + i * v.st, l, n, all(0.0f));
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
        if (m)
            lo = lo + (m - 1) * step + 1;
        else
            hi = lo;
    }
    return lo;
}

// Fills `cuts` for the chunk at c0 and copies the state of the empty sequences
// that lie there, for the tile's n channels. All threads; ends with a barrier.
__device__ __forceinline__ void find_cuts(Cuts &cuts, const ScanArgs &a, const Tile &t, int n, const float *from, float *to)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int64_t c0 = int64_t(t.chunk) * kChunk, c1 = c0 + kChunk < a.tokens ? c0 + kChunk : a.tokens;
    if (threadIdx.x < kChunk) cuts.first[threadIdx.x] = cuts.last[threadIdx.x] = -1;
    if (warp == 0) {
        const int64_t lo = lower_bound(a.seq_start, a.n_seq, c0);
        if (lane == 0) cuts.range[0] = lo > 0 ? lo - 1 : 0;
    }
    if (warp == 1) {
        const int64_t hi = c1 == a.tokens ? a.n_seq : lower_bound(a.seq_start, a.n_seq, c1);
        if (lane == 0) cuts.range[1] = hi;
    }
    __syncthreads();
    for (int64_t s = cuts.range[0] + warp; s < cuts.range[1]; s += kWarps) {
        const int64_t lo = a.seq_start[s], hi = a.seq_start[s + 1];
        if (hi > lo) {
            if (lane == 0 && lo >= c0 && lo < c1) cuts.first[lo - c0] = int(s);
            if (lane == 0 && hi > c0 && hi <= c1) cuts.last[hi - 1 - c0] = int(s);
        } else if (to && lo >= c0 && (lo < c1 || c1 == a.tokens)) {
            for (int c = lane; c < n; c += 32)
                to[s * a.channels + t.ch + c] = from ? from[s * a.channels + t.ch + c] : 0.0f;
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------------ the chunks before

// Four runs of one slot: their maps, and the state before each in place of
// the runs' b.
struct Quarter {
    float2 m[4];
    __device__ __forceinline__ void load(const Runs &runs, int part, int slot)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = make_float2(runs.a[4 * part + i][slot], runs.b[4 * part + i][slot]);
    }
    template <bool CUT>
    __device__ __forceinline__ float2 whole() const
    {
        return then<CUT>(then<CUT>(m[0], m[1]), then<CUT>(m[2], m[3]));
    }
    template <bool CUT>
    __device__ __forceinline__ float run(Runs &runs, int part, int slot, float h) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            runs.b[4 * part + i][slot] = h;
            h = apply<CUT>(m[i], h);
        }
        return h;
    }
};

// The chunks before a tile: what a thread waits for, which is four chunks and
// four groups at one slot (and, for the last four, the span), all asked for
// before the first is looked at.
struct Before {
    Four chunks, groups;
    uint32_t in_group, group, first_group;
    __device__ __forceinline__ void ask(const Work &w, const Tile &t, const Grid &g)
    {
        const int slot = threadIdx.x % kTile, part = threadIdx.x / kTile;
        in_group = t.k % kGroup;
        group = t.k / kGroup % kGroup;
        first_group = t.k / kGroup - group;
        const int64_t step = g.width * kTile, at = int64_t(t.rest) * kTile + slot;
        chunks = Four{w.chunk + (t.k - in_group + 4 * part) * step + at, step, int(in_group) - 4 * part};
        groups = Four{w.group + (first_group + 4 * part) * step + at, step, int(group) - 4 * part};
        chunks.ask();
        groups.ask();
    }
};

// Publishes this chunk's map, waits for the chunks before it, and leaves the
// state before each run in maps.runs.b. The chunk's own map never waits for
// others, nor does the group's for earlier groups. `start` is the state before
// the row's first token, at the thread's slot. The runs' maps are behind a
// barrier; ends with one. Records of kTile slots lie by chunk (group, span) and
// then by tile.
template <bool CUT, class M>
__device__ __forceinline__ void solve(M &maps, Before &before, const Work &w, const Tile &t, const Grid &g, uint32_t tag,
                                      float start)
{
    const int slot = threadIdx.x % kTile, part = threadIdx.x / kTile;
    Quarter mine;
    mine.load(maps.runs, part, slot);
    maps.quarters[part][slot] = mine.whole<CUT>();
    if (g.chunks == 1) {
        __syncthreads();
        float h = start;
        for (int i = 0; i < part; ++i) h = apply<CUT>(maps.quarters[i][slot], h);
        mine.run<CUT>(maps.runs, part, slot, h);
        __syncthreads();
        return;
    }
    // Through shared memory, so that it has been read before this chunk's map is
    // published: the row's last block may write its final state over it after that.
    maps.span[slot] = start;
    const bool followed = t.k + 1 < uint32_t(g.chunks), ends_group = before.in_group == kGroup - 1 && followed;
    const int64_t step = g.width * kTile, at = int64_t(t.rest) * kTile + slot;
    const uint32_t this_group = t.k / kGroup;
    __syncthreads();
    float2 all_runs = make_float2(1.0f, 0.0f);
    if (part == 0 && followed) {
#pragma unroll
        for (int i = 0; i < 4; ++i) all_runs = then<CUT>(all_runs, maps.quarters[i][slot]);
        if (!ends_group) put(w.chunk + t.k * step + at, all_runs.x, all_runs.y, tag);
    }
    maps.chunks[part][slot] = before.chunks.get<CUT>(tag, w);
    if (ends_group && before.group < kGroup - 1) {
        __syncthreads();
        if (part == 0) {
            float2 m = make_float2(1.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) m = then<CUT>(m, maps.chunks[i][slot]);
            m = then<CUT>(m, all_runs);
            put(w.group + this_group * step + at, m.x, m.y, tag);
        }
    }
    maps.groups[part][slot] = before.groups.get<CUT>(tag, w);
    if (part == 3 && before.first_group > 0) {
        const ulonglong2 *p = w.span + (before.first_group / kGroup - 1) * step + at;
        ulonglong2 v = look(p);
        for (long long polls = 0; !there(v, tag) && go_on(w, tag, polls); ++polls) v = look(p);
        maps.span[slot] = values(v).x;
    }
    __syncthreads();
    float h = maps.span[slot];
#pragma unroll
    for (int i = 0; i < 4; ++i) h = apply<CUT>(maps.groups[i][slot], h);
#pragma unroll
    for (int i = 0; i < 4; ++i) h = apply<CUT>(maps.chunks[i][slot], h);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const float next = apply<CUT>(maps.quarters[i][slot], h);
        h = i < part ? next : h;
    }
    h = mine.run<CUT>(maps.runs, part, slot, h);
    if (part == 3 && ends_group && before.group == kGroup - 1) put(w.span + this_group / kGroup * step + at, h, h, tag);
    __syncthreads();
}

// The masks of a run's tokens (bit i: token i) at which packed sequences begin and end.
struct Marks {
    uint32_t first, last;
};
__device__ __forceinline__ Marks marks_of(const Cuts &cuts)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, half = lane >> 4;
    const int at = warp * 2 * kRun + (lane & 15);
    const uint32_t f = __ballot_sync(0xffffffffu, cuts.first[at] >= 0);
    const uint32_t l = __ballot_sync(0xffffffffu, cuts.last[at] >= 0);
    return Marks{(f >> (kRun * half)) & 0xffu, (l >> (kRun * half)) & 0xffu};
}

// State row `row` of p (null: zeros) at the thread's slot.
template <bool VEC>
__device__ __forceinline__ float state1(const float *p, int64_t row, const ScanArgs &a, const Tile &t)
{
    const int slot = threadIdx.x % kTile;
    const int64_t c = t.ch + channel_of<VEC>(slot >> 2, slot & 3);
    return p && c < a.channels ? p[row * a.channels + c] : 0.0f;
}

// ------------------------------------------------------------------ forward

// Backward's buffers of x and dy per block: with two, the next tile's copies
// start when a tile is begun; with one (binary32, where two would leave one block
// to an SM) when it is done. Then f's buffer, read once, gives way to the maps, or
// they would leave one block to an SM all the same.
template <class T, bool BWD>
constexpr int kBuffers = BWD && sizeof(T) == 2 ? 2 : 1;
template <class T, int ROWS, bool BWD>
constexpr size_t kTileBytes = (BWD ? 2 * kBuffers<T, BWD> + 1 : 2) * kBuffer<T, ROWS> * sizeof(T);

// A block's places. Where rows and tiles of channels alone fill the GPU (EARLY; not
// with packed sequences) the next place is taken when a tile is begun, so that its
// copies can start at once; a block's second place then waits for its first tile's
// copies, when all blocks have begun and taken their first. Where blocks work side
// by side on few rows, a place that is taken but not begun holds up every block
// after it, so the next one is taken only when a tile waits for nothing more.
template <bool BWD, bool EARLY>
struct Ahead {
    Shared &sh;
    Places places;
    unsigned long long next;
    bool begun;
    __device__ __forceinline__ Ahead(Shared &s, const Work &w, const Grid &g) : sh(s), places{w.ctl, int64_t(blockIdx.x)}, next(0), begun(false)
    {
        if (threadIdx.x == 0) {
            const unsigned long long taken = places.take(g);
            sh.tile = tile_at<BWD>(taken, g);
            sh.tag = uint32_t(taken >> 32);
        }
    }
    // Before the barrier that opens a tile.
    __device__ __forceinline__ void open(const Grid &g)
    {
        if (EARLY && threadIdx.x == 0 && !begun) sh.tile = tile_at<BWD>(places.take(g), g);
        begun = true;
    }
    // Early: the tile after the one just opened, whose successor is asked for.
    __device__ __forceinline__ Tile after_open(const Grid &g)
    {
        const Tile u = sh.tile;
        if (threadIdx.x == 0 && u.valid) next = places.take(g);
        return u;
    }
    __device__ __forceinline__ void done(const Tile &u, const Grid &g)
    {
        if (threadIdx.x == 0 && u.valid) sh.tile = tile_at<BWD>(next, g);
    }
    // Late: around the second pass.
    __device__ __forceinline__ void ask(const Grid &g)
    {
        if (!EARLY && threadIdx.x == 0) next = places.take(g);
    }
    __device__ __forceinline__ Tile close(const Grid &g)
    {
        if (threadIdx.x == 0) sh.tile = tile_at<BWD>(next, g);
        __syncthreads();
        return sh.tile;
    }
};

template <class T, int ROWS, bool PACKED, bool EARLY>
__global__ void __launch_bounds__(kThreads, 2) scan_kernel(ScanArgs a, Work w, Grid g)
{
    extern __shared__ __align__(128) unsigned char raw[];
    static_assert(!(PACKED && EARLY), "the cuts are found between two tiles");
    constexpr bool VEC = ROWS != ANY;
    constexpr int kSize = kBuffer<T, ROWS>;
    T *const bf = reinterpret_cast<T *>(raw), *const bx = bf + kSize;
    __shared__ struct { __align__(128) Maps<false> m; Shared s; } both;  // wide accesses to unaligned banks cost a tenth
    Maps<false> &maps = both.m;
    Shared &sh = both.s;
    const int l = threadIdx.x & 15, run = threadIdx.x / 16;
    Ahead<false, EARLY> ahead(sh, w, g);
    __syncthreads();
    Tile t = sh.tile;
    const uint32_t tag = sh.tag;
    if (t.valid) {
        start_copy<T, ROWS>(bf, a.f, t, a);
        start_copy<T, ROWS>(bx, a.x, t, a);
    }
    commit_copies();
    int64_t end = a.tokens;
    if (PACKED) {
        end = a.seq_start[a.n_seq];
        end = end < 0 ? 0 : end < a.tokens ? end : a.tokens;
    }
    __syncthreads();
    while (t.valid) {
        const int n = int(a.channels - t.ch < kTile ? a.channels - t.ch : kTile);
        const int64_t t0 = int64_t(t.chunk) * kChunk + run * kRun;
        const float start = PACKED ? 0.0f : state1<VEC>(a.h0, t.row, a, t);
        if (PACKED) find_cuts(sh.cuts, a, t, n, a.h0, a.h_last);  // while the copies are under way
        wait_copies();
        ahead.open(g);
        __syncthreads();
        if (!EARLY) {
            const Tile soon = tile_at<false>(t.k * uint32_t(g.width) + t.rest + gridDim.x, g);
            if (soon.valid) {
                bring<T>(a.f, soon, a);
                bring<T>(a.x, soon, a);
            }
        }
        Tile u;
        if (EARLY) u = ahead.after_open(g);
        Before before;
        if (EARLY) before.ask(w, t, g);
        Marks mk{0u, 0u};
        if (PACKED) mk = marks_of(sh.cuts);
        auto initial = [&](int i) {
            return state4<VEC>(a.h0 ? a.h0 + sh.cuts.first[run * kRun + i] * a.channels + t.ch : nullptr, l, n);
        };

        F4 keep[kRun], in[kRun];
        Walk<T, ROWS> at_f(a.f, t, 0), at_x(a.x, t, 0);
        Map m;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            F4 take;
            gates(decay<T>(read_f4<VEC>(at_f.next(bf, a.f, run, i), l)), keep[i], take);
            in[i] = mul(take, read4<VEC>(at_x.next(bx, a.x, run, i), l));
            if (PACKED && (mk.first >> i & 1)) {
                // the state after the first token stands for its input: h0 is not read
                // again, since h_last may be the same memory, and the block that has the
                // sequence's last token writes there once this tile's map is known
                m.b = fma(keep[i], initial(i), in[i]);
                m.a = all(kConst);
                in[i] = m.b;
            } else if (i == 0) {
                m = Map{keep[0], in[0]};
            } else {
                m.b = fma(keep[i], m.b, in[i]);
                if (!PACKED || !(m.a.lo.x < 0.0f)) m.a = mul(keep[i], m.a);
            }
        }
        if (!EARLY) before.ask(w, t, g);
        sts4(&maps.runs.a[run][4 * l], m.a);
        sts4(&maps.runs.b[run][4 * l], m.b);
        __syncthreads();
        if (EARLY) {
            if (u.valid) {
                start_copy<T, ROWS>(bf, a.f, u, a);
                start_copy<T, ROWS>(bx, a.x, u, a);
            }
            commit_copies();
        }
        solve<PACKED>(maps, before, w, t, g, tag, start);
        ahead.ask(g);
        F4 h = lds4(&maps.runs.b[run][4 * l]);
        if (a.states && run == 0)
            put_state4<VEC>(a.states + (t.row * g.chunks + t.chunk) * a.channels + t.ch, l, n, h);
        T *py = static_cast<T *>(a.y.ptr) + t.row * a.y.sb + t0 * a.y.st + t.ch;
        if (t0 + kRun < end && (!PACKED || !(mk.first | mk.last))) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                h = fma(keep[i], h, in[i]);
                store4<VEC>(py, l, n, h);
                py += a.y.st;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                if (PACKED && (mk.first >> i & 1)) h = all(-0.0f);  // then in[i], to the bit
                h = fma(keep[i], h, in[i]);
                if (t0 + i < end) store4<VEC>(py, l, n, h);
                py += a.y.st;
                if (a.h_last && (PACKED ? mk.last >> i & 1 : t0 + i == end - 1))
                    put_state4<VEC>(a.h_last + (PACKED ? int64_t(sh.cuts.last[run * kRun + i]) : int64_t(t.row)) * a.channels + t.ch,
                                    l, n, h);
            }
            if (PACKED && a.clear_rest) clear_rest<T, VEC>(a.y, t, t0, end, a, l, n);
        }
        if (EARLY) {
            ahead.done(u, g);
            t = u;
        } else {
            t = ahead.close(g);
            if (t.valid) {
                start_copy<T, ROWS>(bf, a.f, t, a);
                start_copy<T, ROWS>(bx, a.x, t, a);
            }
            commit_copies();
        }
    }
}

// ------------------------------------------------------------------ backward

template <class T, int ROWS, bool PACKED, bool EARLY>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(ScanArgs a, Work w, Grid g)
{
    extern __shared__ __align__(128) unsigned char raw[];
    static_assert(!(PACKED && EARLY), "the cuts are found between two tiles");
    constexpr bool VEC = ROWS != ANY;
    constexpr int kSize = kBuffer<T, ROWS>;
    constexpr bool kTwo = kBuffers<T, true> == 2;
    T *const bf = reinterpret_cast<T *>(raw), *bx = bf + kSize, *other = kTwo ? bx + 2 * kSize : bx;  // dy behind x
    static_assert(kTwo || sizeof(Maps<true>) <= kSize * sizeof(T), "the maps fit into f's buffer");
    __shared__ struct { __align__(128) unsigned char own[kTwo ? sizeof(Maps<true>) : 16]; Shared s; } both;
    Maps<true> &maps = *reinterpret_cast<Maps<true> *>(kTwo ? both.own : raw);
    Shared &sh = both.s;
    const int l = threadIdx.x & 15, run = threadIdx.x / 16;
    Ahead<true, EARLY> ahead(sh, w, g);
    __syncthreads();
    Tile t = sh.tile;
    const uint32_t tag = sh.tag;
    if (t.valid) {
        start_copy<T, ROWS>(bf, a.f, t, a);
        start_copy<T, ROWS>(bx, a.x, t, a);
        start_copy<T, ROWS>(bx + kSize, a.y, t, a);
    }
    commit_copies();
    int64_t end = a.tokens;
    if (PACKED) {
        end = a.seq_start[a.n_seq];
        end = end < 0 ? 0 : end < a.tokens ? end : a.tokens;
    }
    __syncthreads();
    while (t.valid) {
        const int n = int(a.channels - t.ch < kTile ? a.channels - t.ch : kTile);
        const int64_t t0 = int64_t(t.chunk) * kChunk + run * kRun;
        const float start = PACKED ? 0.0f : state1<VEC>(a.dh_last, t.row, a, t);
        const float h_start = t.chunk > 0 ? state1<VEC>(a.states, t.row * g.chunks + t.chunk, a, t)
                              : PACKED    ? 0.0f
                                          : state1<VEC>(a.h0, t.row, a, t);
        if (PACKED) find_cuts(sh.cuts, a, t, n, a.dh_last, a.dh0);  // while the copies are under way
        wait_copies();
        ahead.open(g);
        __syncthreads();
        if (!EARLY) {
            const Tile soon = tile_at<true>(t.k * uint32_t(g.width) + t.rest + gridDim.x, g);
            if (soon.valid) {
                bring<T>(a.f, soon, a);
                bring<T>(a.x, soon, a);
                bring<T>(a.y, soon, a);
            }
        }
        Tile u;
        Before before;
        if (EARLY) before.ask(w, t, g);
        if (EARLY) {
            u = ahead.after_open(g);
            if (u.valid) {
                start_copy<T, ROWS>(other, a.x, u, a);
                start_copy<T, ROWS>(other + kSize, a.y, u, a);
            }
        }
        Marks mk{0u, 0u};
        if (PACKED) mk = marks_of(sh.cuts);
        auto side = [&](const float *p, const int *table, int i) {
            return state4<VEC>(p ? p + table[run * kRun + i] * a.channels + t.ch : nullptr, l, n);
        };

        // dh_last of the sequences that end in the run, in order. It is not read after
        // this tile's map is known, since dh0 may be the same memory, and the block that
        // has a sequence's first token writes there then. Indexed when running, so that
        // it lies in local memory and takes no registers where nothing ends.
        F4 ends[PACKED ? kRun : 1];
        if (PACKED) {
            int ended = 0;
#pragma unroll 1
            for (uint32_t left = mk.last; left; left &= left - 1u)
                ends[ended++] = side(a.dh_last, sh.cuts.last, __ffs(int(left)) - 1);
        }

        // Both maps in one pass over the tokens: the later tokens' gradient
        // comes in through the product of the gates so far. exp(-f) alone is
        // kept of the gates, which are formed again from it where they are
        // needed (a reciprocal each), to hold the tile in 128 registers.
        F4 e[kRun];
        Walk<T, ROWS> at_f(a.f, t, 0), at_x(a.x, t, 0), at_dy(a.y, t, 0);
        Map m, r;
        F4 weight = all(1.0f);  // of a token's dy in the run's gradient
        bool cut = false;       // a packed sequence ended: the later tokens do not count
        r.b = all(0.0f);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            F4 keep, take;
            e[i] = decay<T>(read_f4<VEC>(at_f.next(bf, a.f, run, i), l));
            gates(e[i], keep, take);
            const F4 in = mul(take, read4<VEC>(at_x.next(bx, a.x, run, i), l));
            if (PACKED && (mk.first >> i & 1)) {
                m.b = fma(keep, side(a.h0, sh.cuts.first, i), in);
                m.a = all(kConst);
            } else if (i == 0) {
                m = Map{keep, in};
            } else {
                m.b = fma(keep, m.b, in);
                if (!PACKED || !(m.a.lo.x < 0.0f)) m.a = mul(keep, m.a);
            }
            const T *const row_dy = at_dy.next(bx + kSize, a.y, run, i);
            // tokens past the end have no gradient: what comes in there is zero or dh_last, unchanged
            if (PACKED ? !cut && t0 + i < end : t0 + i < a.tokens) {
                weight = mul(weight, keep);
                r.b = fma(weight, read4<VEC>(row_dy, l), r.b);
                if (PACKED && (mk.last >> i & 1)) {
                    r.b = fma(weight, ends[0], r.b);
                    cut = true;
                }
            }
        }
        r.a = cut ? all(kConst) : weight;
        if (!EARLY) before.ask(w, t, g);
        if (!kTwo) __syncthreads();  // all of f has been read
        sts4(&maps.fwd.a[run][4 * l], m.a);
        sts4(&maps.fwd.b[run][4 * l], m.b);
        sts4(&maps.runs.a[kRuns - 1 - run][4 * l], r.a);
        sts4(&maps.runs.b[kRuns - 1 - run][4 * l], r.b);
        __syncthreads();
        if (EARLY) {
            if (u.valid) start_copy<T, ROWS>(bf, a.f, u, a);
            commit_copies();
        }
        {
            const int slot = threadIdx.x % kTile, part = threadIdx.x / kTile;
            Quarter q;
            q.load(maps.fwd, part, slot);
            maps.fwd_quarters[part][slot] = q.whole<PACKED>();
            __syncthreads();
            float h = h_start;
            for (int i = 0; i < part; ++i) h = apply<PACKED>(maps.fwd_quarters[i][slot], h);
            q.run<PACKED>(maps.fwd, part, slot, h);
        }
        solve<PACKED>(maps, before, w, t, g, tag, start);
        ahead.ask(g);
        F4 h = lds4(&maps.fwd.b[run][4 * l]), gr = lds4(&maps.runs.b[kRuns - 1 - run][4 * l]);
        // forward once more, for h_{t-1} - x_t
        F4 over[kRun];
        Walk<T, ROWS> at_x2(a.x, t, 0);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            if (PACKED && (mk.first >> i & 1)) h = side(a.h0, sh.cuts.first, i);
            F4 keep, take;
            gates_again(e[i], keep, take);
            const F4 xx = read4<VEC>(at_x2.next(bx, a.x, run, i), l);
            over[i] = sub(h, xx);
            h = fma(keep, h, mul(take, xx));
        }
        T *px = static_cast<T *>(a.dx.ptr) + t.row * a.dx.sb + (t0 + kRun - 1) * a.dx.st + t.ch;
        T *pf = static_cast<T *>(a.df.ptr) + t.row * a.df.sb + (t0 + kRun - 1) * a.df.st + t.ch;
        Walk<T, ROWS> at_dy2(a.y, t, kRun - 1);
        auto back = [&](int i, const T *row_dy) {
            F4 keep, take;
            gates_again(e[i], keep, take);
            gr = add(read4<VEC>(row_dy, l), gr);
            const F4 dx = mul(take, gr);
            store4<VEC>(px, l, n, dx);
            gr = mul(keep, gr);
            store4<VEC>(pf, l, n, mul(mul(over[i], keep), dx));
        };
        if (t0 + kRun <= end && (!PACKED || !(mk.first | mk.last))) {
#pragma unroll
            for (int i = kRun - 1; i >= 0; --i) {
                back(i, at_dy2.last(bx + kSize, a.y, run, i));
                px -= a.dx.st;
                pf -= a.df.st;
            }
        } else {
#pragma unroll
            for (int i = kRun - 1; i >= 0; --i) {
                const T *const row_dy = at_dy2.last(bx + kSize, a.y, run, i);
                if (t0 + i < end) {
                    if (PACKED && (mk.last >> i & 1)) gr = ends[__popc(mk.last & ((1u << i) - 1u))];
                    back(i, row_dy);
                    if (PACKED && a.dh0 && (mk.first >> i & 1))
                        put_state4<VEC>(a.dh0 + sh.cuts.first[run * kRun + i] * a.channels + t.ch, l, n, gr);
                }
                px -= a.dx.st;
                pf -= a.df.st;
            }
            if (PACKED && a.clear_rest) {
                clear_rest<T, VEC>(a.dx, t, t0, end, a, l, n);
                clear_rest<T, VEC>(a.df, t, t0, end, a, l, n);
            }
        }
        if (!PACKED && a.dh0 && t0 == 0) put_state4<VEC>(a.dh0 + t.row * a.channels + t.ch, l, n, gr);
        if (EARLY) {
            ahead.done(u, g);
            t = u;
            T *const swap = bx;
            bx = other;
            other = swap;
        } else {
            t = ahead.close(g);
            if (t.valid) {
                start_copy<T, ROWS>(bf, a.f, t, a);
                start_copy<T, ROWS>(bx, a.x, t, a);
                start_copy<T, ROWS>(bx + kSize, a.y, t, a);
            }
            commit_copies();
        }
    }
}

// ------------------------------------------------------------------ a few tokens

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = uint16_t(pack_bf16x2(v, 0.0f)); }

constexpr int kFew = 16;

// Rows of at most kFew tokens: a thread to a channel, all its loads at once, the
// tokens one after another, so that a call for several tokens has the bits of
// calls for each. One token of 32 rows of 768 channels takes 1.7 us, the launch's
// own time. The scan would fill an eighth of its tiles' rows: 64 x 12 x 768 in
// bf16 forward 4.1 us against 10.6 in the scan, backward 5.6 against 15.8;
// 512 x 16 x 768 27 against 64, and 59 against 94.
template <class T, int N, bool BWD>
__global__ void __launch_bounds__(128) few_kernel(ScanArgs a)
{
    const int64_t i0 = int64_t(blockIdx.x) * 128 + threadIdx.x;
    if (i0 >= a.batch * a.channels) return;
    const int64_t row = i0 / a.channels, c = i0 % a.channels;
    const T *px = static_cast<const T *>(a.x.ptr) + row * a.x.sb + c;
    const T *pf = static_cast<const T *>(a.f.ptr) + row * a.f.sb + c;
    const T *pd = static_cast<const T *>(a.y.ptr) + row * a.y.sb + c;
    float x[N], f[N], dy[N], before[N], take[N];
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const bool in = t < a.tokens;
        f[t] = in ? load1(pf + t * a.f.st) : 0.0f;
        x[t] = in ? load1(px + t * a.x.st) : 0.0f;
        if (BWD) dy[t] = in ? load1(pd + t * a.y.st) : 0.0f;
    }
    float h = a.h0 ? a.h0[i0] : 0.0f;
    float r = BWD && a.dh_last ? a.dh_last[i0] : 0.0f;
    if (!BWD && a.states) a.states[i0] = h;
    T *py = static_cast<T *>(a.y.ptr) + row * a.y.sb + c;
#pragma unroll
    for (int t = 0; t < N; ++t) {
        float2 k, u;
        const float ft = max_nan(f[t], kLowest);
        gates(decay<T>(make_float2(ft, ft)), k, u);
        before[t] = h;
        f[t] = k.x;
        take[t] = u.x;
        if (t < a.tokens) {
            h = fmaf(k.x, h, u.x * x[t]);
            if (!BWD) store1(py + t * a.y.st, h);
        }
    }
    if (!BWD) {
        if (a.h_last) a.h_last[i0] = h;
        return;
    }
    T *dx = static_cast<T *>(a.dx.ptr) + row * a.dx.sb + c, *df = static_cast<T *>(a.df.ptr) + row * a.df.sb + c;
#pragma unroll
    for (int t = N - 1; t >= 0; --t) {
        if (t >= a.tokens) continue;
        const float g = dy[t] + r;
        store1(dx + t * a.dx.st, take[t] * g);
        store1(df + t * a.df.st, g * (before[t] - x[t]) * (f[t] * take[t]));
        r = f[t] * g;
    }
    if (a.dh0) a.dh0[i0] = r;
}

// ------------------------------------------------------------------ launches

// How the rows of v lie.
int rows_of(const ScanView &v, int size, int64_t channels)
{
    const uintptr_t bits = reinterpret_cast<uintptr_t>(v.ptr) | uintptr_t(v.sb * size) | uintptr_t(v.st * size);
    return bits % 16 == 0 && channels % 4 == 0 ? WHOLE : bits % (4 * size) == 0 && channels % 4 == 0 ? FOURS : ANY;
}

Grid grid_of(const ScanArgs &a)
{
    Grid g{};
    g.tiles = (a.channels + kTile - 1) / kTile;
    g.width = a.batch * g.tiles;
    g.chunks = (a.tokens + kChunk - 1) / kChunk;
    g.places = g.width * g.chunks;
    return g;
}

// (The kernel is a template argument: all of a direction have one type, and each
// has a flag of its own for the shared memory that it was allowed.)
template <class T, int ROWS, bool BWD, auto kernel>
cudaError_t launch(const ScanArgs &a, const ScanWork &sw, const Grid &g, cudaStream_t st)
{
    constexpr size_t smem = kTileBytes<T, ROWS, BWD>;
    if (g.places >= int64_t(0xf0000000)) return cudaErrorInvalidConfiguration;
    // the driver is asked once for each kernel and device
    static std::atomic<bool> allowed[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !allowed[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed[dev].store(true, std::memory_order_relaxed);
    }
    Work w{};
    w.ctl = sw.ctl;
    w.status = sw.status;
    w.gave_up = sw.gave_up;
    w.wait_limit = sw.wait_limit;
    w.chunk = reinterpret_cast<ulonglong2 *>(sw.records);
    w.group = w.chunk + kTile * g.width * g.chunks;
    w.span = w.group + kTile * g.width * (g.chunks / kGroup);
    const int64_t wave = wave_blocks(reinterpret_cast<const void *>(kernel), kThreads, smem);
    kernel<<<unsigned(g.places < wave ? g.places : wave), kThreads, smem, st>>>(a, w, g);
    return cudaGetLastError();
}

template <class T, int ROWS, bool PACKED, bool BWD>
cudaError_t choose(const ScanArgs &a, const ScanWork &sw, cudaStream_t st)
{
    const Grid g = grid_of(a);
    // A place taken a tile ahead has its copies in flight early, but others wait
    // the longer for its records. Measured in bf16, a tile ahead against at the
    // end of a tile, tiles of a chunk x chunks: 192 x 32 forward 65 against 68 us,
    // backward 103 against 101; 768 x 2 19.5 against 20.3, 29.0 against 30.3;
    // 96 x 16 22.7 against 21.1, 32.5 against 31.7; 48 x 32 24.6 against 22.6, 36
    // against 34; 12 x 512 105 against 92, 153 against 122. In long rows forward
    // gains from fewer tiles on: 64 x 512 367 against 400, 568 against 574;
    // 32 x 512 208 against 222, 312 against 305; 24 x 512 168 against 172, 245
    // against 232. Forward in binary32: 192 x 32 97 against 99; 768 x 3 38.5 against
    // 40.8; 96 x 16 32.6 against 30.5; 48 x 32 35.4 against 35.0; 12 x 512 143 against
    // 124; 64 x 256 266 against 287; 32 x 256 151 against 158. Packed sequences never
    // gain, since finding the cuts then has no copies to hide behind: in bf16, 192 x 32
    // 99.7 against 93.4, backward 189 against 166; 64 x 256 267 against 246, 552
    // against 418; 32 x 512 285 against 254, 575 against 416; 12 x 512 141 against 106,
    // 244 against 178; binary32, 192 x 64 forward 244 against 235; 32 x 512 364 against
    // 327.
    if constexpr (!PACKED && (!BWD || kBuffers<T, true> == 2)) {
        const bool early = g.width >= 128 || (!BWD && g.width >= 32 && g.chunks >= 256);
        if constexpr (BWD) {
            if (early) return launch<T, ROWS, BWD, &scan_bwd_kernel<T, ROWS, PACKED, true>>(a, sw, g, st);
        } else {
            if (early) return launch<T, ROWS, BWD, &scan_kernel<T, ROWS, PACKED, true>>(a, sw, g, st);
        }
    }
    if constexpr (BWD)
        return launch<T, ROWS, BWD, &scan_bwd_kernel<T, ROWS, PACKED, false>>(a, sw, g, st);
    else
        return launch<T, ROWS, BWD, &scan_kernel<T, ROWS, PACKED, false>>(a, sw, g, st);
}

template <class T, bool BWD>
cudaError_t launch_few(const ScanArgs &a, cudaStream_t st)
{
    const int64_t blocks = (a.batch * a.channels + 127) / 128;
    if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    if (a.tokens == 1)
        few_kernel<T, 1, BWD><<<unsigned(blocks), 128, 0, st>>>(a);
    else
        few_kernel<T, kFew, BWD><<<unsigned(blocks), 128, 0, st>>>(a);
    return cudaGetLastError();
}

template <class T, bool BWD>
cudaError_t pick(const ScanArgs &a, const ScanWork &w, cudaStream_t st)
{
    if (!a.seq_start && a.tokens <= kFew) return launch_few<T, BWD>(a, st);
    auto lie = [&](const ScanView &v) { return rows_of(v, int(sizeof(T)), a.channels); };
    int rows = std::min({lie(a.x), lie(a.f), lie(a.y)});
    if (BWD) rows = std::min({rows, lie(a.dx), lie(a.df)});
    if (rows == WHOLE) return a.seq_start ? choose<T, WHOLE, true, BWD>(a, w, st) : choose<T, WHOLE, false, BWD>(a, w, st);
    if constexpr (sizeof(T) == 2)
        if (rows == FOURS) {
            constexpr int how = BWD ? FOURS : EIGHTS;
            return a.seq_start ? choose<T, how, true, BWD>(a, w, st) : choose<T, how, false, BWD>(a, w, st);
        }
    return a.seq_start ? choose<T, ANY, true, BWD>(a, w, st) : choose<T, ANY, false, BWD>(a, w, st);
}

template <bool BWD>
cudaError_t by_type(const ScanArgs &a, const ScanWork &w, cudaStream_t st)
{
    return a.dtype == ZG_DTYPE_BF16 ? pick<uint16_t, BWD>(a, w, st) : pick<float, BWD>(a, w, st);
}

}  // namespace

int64_t scan_record_bytes(int64_t batch, int64_t tokens, int64_t channels)
{
    const int64_t width = batch * ((channels + kTile - 1) / kTile), chunks = (tokens + kChunk - 1) / kChunk;
    if (chunks == 1) return 0;
    return width * kTile * int64_t(sizeof(ulonglong2)) * (chunks + chunks / kGroup + chunks / (kGroup * kGroup));
}

cudaError_t launch_scan(const ScanArgs &a, const ScanWork &w, cudaStream_t st) { return by_type<false>(a, w, st); }
cudaError_t launch_scan_bwd(const ScanArgs &a, const ScanWork &w, cudaStream_t st) { return by_type<true>(a, w, st); }

}  // namespace zg
