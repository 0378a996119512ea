// The token embedding and its gradient.
//
// Lookup: out row i = scale * table row tokens[i]. Gradient: dtable row v = add
// row v + scale * the sum of the drows rows whose token is v.
//
// Both are bound by memory: the lookup reads and writes each row once; the gradient
// reads each drows row once, and writes the whole table, of which most rows have no
// token. Rows of one token must be added in an order that does not depend on the
// run, so the tokens are sorted first, stably by (token, position):
//
//   sort   one cluster sorts by counting, 8 or 9 bits of the token at a time, its
//          blocks exchanging their counts through distributed shared memory.
//   fill   at the same time the first blocks of the next launch write the rows without
//          a token, which each finds by looking all tokens through.
//   sum    in that launch's other blocks a warp to a tile of the sorted list and 256 columns adds rows up in
//          binary32 registers; where a token's rows end inside the tile it writes the
//          table's row, else a partial row.
//   join   adds the partial rows of tokens that reach over several tiles, in their
//          order.
//
// Measured, a table of 50257 x 768 in bf16: the lookup of 8192 tokens 4.5 us, of 65536 17 us. The gradient of 8192
// tokens 25 us for 90 MB: the sort 14 us, beside which most rows without a token are written, then sum and join; of
// 65536 tokens 78 us; of 8192 at 4096 columns 82 us (479 MB, 5.8 TB/s). Added to another gradient in place, 20011
// tokens at 771 columns in binary32, 51 us, beside it 89 (at 768 columns 78). All 8192 tokens the same: 41 us. The sort
// is a cluster's, however many tokens there are: from some 65536 on it takes the longer, the more of them. 262144
// tokens take 256 us, of which the sort 133, 1048576 885, of which 498.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

namespace cg = cooperative_groups;

// VEC neighbouring elements, `n` of which are there.
template <class T, int VEC>
__device__ __forceinline__ void store(T *p, int n, const float (&v)[VEC])
{
    if constexpr (VEC == 1) {
        if (n > 0) store1(p, v[0]);
    } else {
        constexpr int N = Unit<T>::kN;
        if (n >= VEC && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
            for (int i = 0; i < VEC; i += N) {
                float2 f[N / 2];
#pragma unroll
                for (int j = 0; j < N / 2; ++j) f[j] = make_float2(v[i + 2 * j], v[i + 2 * j + 1]);
                Unit<T> u;
                u.set(f);
                *reinterpret_cast<uint4 *>(p + i) = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (i < n) store1(p + i, v[i]);
        }
    }
}

__device__ __forceinline__ int64_t token_of(const void *tokens, bool wide, int64_t i)
{
    return wide ? static_cast<const int64_t *>(tokens)[i] : static_cast<const int32_t *>(tokens)[i];
}

// ------------------------------------------------------------------ lookup

constexpr int kRows = 2;  // of a warp at a time

// A warp copies kRows rows side by side, U units of each at a time: their loads are in
// flight together, as they are in memory. Places past a row's end repeat its last unit.
template <class T, bool WHOLE, int U>
__global__ void __launch_bounds__(128) lookup_kernel(EmbedArgs a)
{
    using Word = typename std::conditional<WHOLE, uint4, T>::type;
    constexpr int N = int(sizeof(Word) / sizeof(T));
    const int lane = threadIdx.x % 32;
    const int64_t first = (int64_t(blockIdx.x) * 4 + threadIdx.x / 32) * kRows;
    if (first >= a.n) return;
    const int words = int(a.width) / N;
    bool there[kRows];
    const Word *row[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int64_t t = token_of(a.tokens, a.token_bytes == 8, min(first + j, a.n - 1));
        there[j] = t >= 0 && t < a.vocab;
        row[j] = reinterpret_cast<const Word *>(static_cast<const T *>(a.table) + (there[j] ? t * a.table_stride : 0));
    }
    for (int c0 = lane; c0 < words; c0 += U * 32) {
        Word w[kRows][U];
#pragma unroll
        for (int j = 0; j < kRows; ++j)
#pragma unroll
            for (int u = 0; u < U; ++u) w[j][u] = row[j][min(c0 + u * 32, words - 1)];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            if (first + j >= a.n) break;
            T *const out = static_cast<T *>(a.out) + (first + j) * a.out_stride;
            const float k = there[j] ? a.scale : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * 32;
                if (c >= words) break;
                if constexpr (WHOLE) {
                    Unit<T> x;
                    x.w = w[j][u];
                    float2 f[N / 2];
                    x.get(f);
                    // zeros even where row 0 holds an infinity
#pragma unroll
                    for (int i = 0; i < N / 2; ++i)
                        f[i] = there[j] ? make_float2(f[i].x * k, f[i].y * k) : make_float2(0.0f, 0.0f);
                    x.set(f);
                    reinterpret_cast<uint4 *>(out)[c] = x.w;
                } else {
                    store1(out + c, there[j] ? load1(&w[j][u]) * k : 0.0f);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ sort

constexpr int kSort = 1024;          // threads of a block
constexpr int kEach = 8;             // tokens of a thread at a time
constexpr int kMostBins = 512;
constexpr int kMostBlocks = 8;       // of the cluster

struct SortPlan {
    int blocks;      // of the sorting cluster
    int passes, bits;
    uint2 *pair[2];  // (token, position): pass p writes pair[p & 1]
};

struct SortShared {
    uint16_t of_warp[kSort / 32][kMostBins];  // counts, then places, of a warp's tokens in a tile
    uint32_t count[kMostBins];  // of the block's tokens; read by the cluster
    uint32_t at[kMostBins];     // place of the tile's first token
    uint32_t total[kMostBins / 32];
};

__device__ __forceinline__ uint2 sort_input(const EmbedArgs &a, const SortPlan &p, int pass, int64_t i)
{
    if (pass) return p.pair[(pass - 1) & 1][i];
    const int64_t t = token_of(a.tokens, a.token_bytes == 8, i);
    return make_uint2(t >= 0 && t < a.vocab ? uint32_t(t) : uint32_t(a.vocab), uint32_t(i));
}

__global__ void __launch_bounds__(kSort, 1) sort_kernel(EmbedArgs a, SortPlan p)
{
    __shared__ SortShared sh;
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, rank = blockIdx.x;
    const int bins = 1 << p.bits;  // at most as many as threads
    const int64_t each = (a.n + p.blocks - 1) / p.blocks;
    const int64_t lo = min(rank * each, a.n), hi = min(lo + each, a.n);
    // a warp takes 32 tokens in each of `rounds`; of a single tile they stay in registers between the two looks
    const int rounds = int(min((each + kSort - 1) / kSort, int64_t(kEach)));
    const int64_t whole_tile = int64_t(rounds) * kSort;
    const bool once = hi - lo <= whole_tile;
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.bits;
        uint2 *const out = p.pair[pass & 1];
        uint32_t key[kEach], at[kEach];
        int place[kEach];
        auto digit = [&](uint32_t k) { return int(k >> shift) & (bins - 1); };
        auto index = [&](int64_t tile, int r) { return tile + (warp * rounds + r) * 32 + lane; };
        auto take = [&](int64_t tile) {
#pragma unroll
            for (int r = 0; r < kEach; ++r) {
                key[r] = at[r] = 0;
                if (r >= rounds || index(tile, r) >= hi) continue;
                const uint2 x = sort_input(a, p, pass, index(tile, r));
                key[r] = x.x;
                at[r] = x.y;
            }
        };
        // Each token's place among its warp's of the same digit; of_warp: how many of a digit
        // before a warp in the tile. Returns the tile's count of digit `tid`. Lanes of one digit
        // find each other by a vote for each bit (a match instruction took 1 us a round more).
        auto rank_tile = [&](int64_t tile) {
            for (int i = tid; i < kSort / 32 * bins / 2; i += kSort)
                reinterpret_cast<uint32_t *>(sh.of_warp[i / (bins / 2)])[i % (bins / 2)] = 0;
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kEach; ++r) {
                place[r] = 0;
                if (r >= rounds) continue;
                const bool there = index(tile, r) < hi;
                const int d = digit(key[r]);
                uint32_t same = __ballot_sync(0xffffffffu, there);
                for (int bit = 0; bit < p.bits; ++bit) {
                    const bool set = d >> bit & 1;
                    const uint32_t vote = __ballot_sync(0xffffffffu, set);
                    same &= set ? vote : ~vote;
                }
                const int earlier = there ? sh.of_warp[warp][d] : 0;
                place[r] = earlier + __popc(same & ((1u << lane) - 1u));
                __syncwarp();
                if (there && lane == __ffs(same) - 1) sh.of_warp[warp][d] = uint16_t(earlier + __popc(same));
                __syncwarp();
            }
            __syncthreads();
            uint32_t so_far = 0;
            if (tid < bins) {
                uint32_t c[kSort / 32];
#pragma unroll
                for (int w = 0; w < kSort / 32; ++w) c[w] = sh.of_warp[w][tid];
#pragma unroll
                for (int w = 0; w < kSort / 32; ++w) {
                    sh.of_warp[w][tid] = uint16_t(so_far);
                    so_far += c[w];
                }
            }
            return so_far;
        };
        auto put = [&](int64_t tile) {
#pragma unroll
            for (int r = 0; r < kEach; ++r) {
                if (r >= rounds || index(tile, r) >= hi) continue;
                const int d = digit(key[r]);
                out[sh.at[d] + sh.of_warp[warp][d] + place[r]] = make_uint2(key[r], at[r]);
            }
        };
        if (once) {
            take(lo);
            const uint32_t n = rank_tile(lo);
            if (tid < bins) sh.count[tid] = n;
        } else {
            if (tid < bins) sh.count[tid] = 0;
            __syncthreads();
            for (int64_t tile = lo; tile < hi; tile += whole_tile) {
                take(tile);
#pragma unroll
                for (int r = 0; r < kEach; ++r)
                    if (r < rounds && index(tile, r) < hi) atomicAdd(&sh.count[digit(key[r])], 1u);
            }
        }
        cluster.sync();
        // places: of all tokens with lower digits, and of the same digit in earlier blocks
        uint32_t all = 0, before = 0, sum;
        if (tid < bins) {
            uint32_t c[kMostBlocks];  // all asked for before one is used
#pragma unroll
            for (int b = 0; b < kMostBlocks; ++b) c[b] = b < p.blocks ? *cluster.map_shared_rank(&sh.count[tid], b) : 0;
#pragma unroll
            for (int b = 0; b < kMostBlocks; ++b) {
                all += c[b];
                if (b < rank) before += c[b];
            }
        }
        sum = all;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (tid < bins && lane == 31) sh.total[warp] = sum;
        __syncthreads();
        uint32_t next = 0;
        if (tid < bins) {
            for (int w = 0; w < warp; ++w) sum += sh.total[w];
            next = sum - all + before;
        }
        if (once) {
            if (tid < bins) sh.at[tid] = next;
            __syncthreads();
            put(lo);
        } else {
            for (int64_t tile = lo; tile < hi; tile += whole_tile) {
                take(tile);
                __syncthreads();  // of_warp is free
                const uint32_t n = rank_tile(tile);
                if (tid < bins) sh.at[tid] = next;
                next += n;
                __syncthreads();
                put(tile);
            }
        }
        cluster.sync();  // all of the pass is written, and count is free
    }
}

// ------------------------------------------------------------------ fill

constexpr int kFill = 256;               // threads of a block
constexpr int kFillBlocks = 608;         // that share the rows
constexpr uint32_t kFillRows = 1 << 13;  // rows whose marks a block holds at once

// Rows [lo, hi) of the table without a mark, a warp to each: add's row, or zeros, in 16-byte units
// counted from the boundary that out's row has, and single elements at its ends. All that a
// lane asks for is in flight before it stores: out and add may be one memory for all that the
// compiler knows.
template <class T>
__device__ void fill_rows(const EmbedArgs &a, const uint32_t *marks, int64_t lo, int64_t hi)
{
    constexpr int N = Unit<T>::kN, U = 8;
    const int lane = threadIdx.x % 32, width = int(a.width);
    for (uint32_t r = threadIdx.x / 32; r < uint32_t(hi - lo); r += kFill / 32) {
        if (marks[r / 32] >> (r % 32) & 1u) continue;
        T *const out = static_cast<T *>(a.out) + (lo + r) * a.out_stride;
        const T *const add = a.table ? static_cast<const T *>(a.table) + (lo + r) * a.table_stride : nullptr;
        const bool alike = !add || ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(add)) & 15u) == 0;
        if (!alike) {
            for (int c0 = lane; c0 < width; c0 += U * 32) {
                T e[U];
#pragma unroll
                for (int i = 0; i < U; ++i) e[i] = add[min(c0 + i * 32, width - 1)];
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (c0 + i * 32 < width) out[c0 + i * 32] = e[i];
            }
            continue;
        }
        const int head = min(int((16 - (reinterpret_cast<uintptr_t>(out) & 15u)) % 16 / sizeof(T)), width);
        const int units = (width - head) / N, tail = head + units * N;
        if (lane < head) out[lane] = add ? add[lane] : T(0);
        if (lane < width - tail) out[tail + lane] = add ? add[tail + lane] : T(0);
        uint4 *const to = reinterpret_cast<uint4 *>(out + head);
        const uint4 *const from = reinterpret_cast<const uint4 *>(add + head);
        for (int u0 = lane; u0 < units; u0 += U * 32) {
            uint4 w[U];
#pragma unroll
            for (int i = 0; i < U; ++i) w[i] = add ? __ldcs(from + min(u0 + i * 32, units - 1)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (u0 + i * 32 < units) __stcs(to + u0 + i * 32, w[i]);
        }
    }
}

// The tokens of `n` within a block's rows, marked: eight loads of a thread at a time.
template <class I>
__device__ __forceinline__ void mark_tokens(const I *tokens, int64_t n, int64_t lo, int64_t hi, uint32_t *marks)
{
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += 8 * kFill) {
        I t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = tokens[min(i0 + j * kFill, n - 1)];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (t[j] >= lo && t[j] < hi) atomicOr(&marks[uint32_t(t[j] - lo) / 32], 1u << (uint32_t(t[j] - lo) % 32));
    }
}

// Block `block` of `blocks`. `looks`: it looks all tokens through for those of its rows, beside
// the sort; otherwise it finds its part of the sorted list.
template <class T>
__device__ void fill(const EmbedArgs &a, const uint2 *sorted, bool looks, int64_t block, int64_t blocks)
{
    __shared__ uint32_t marks[kFillRows / 32];
    __shared__ int64_t edge[2];
    const int64_t each = (a.vocab + blocks - 1) / blocks, end = min((block + 1) * each, a.vocab);
    for (int64_t lo = block * each; lo < end; lo += kFillRows) {
        const int64_t hi = min(lo + int64_t(kFillRows), end);
        for (uint32_t i = threadIdx.x; i < uint32_t(hi - lo + 31) / 32; i += kFill) marks[i] = 0;
        if (!looks && threadIdx.x < 2) {  // the first token of at least lo, and of at least hi
            const uint32_t key = uint32_t(threadIdx.x ? hi : lo);
            int64_t from = 0, to = a.n;
            while (from < to) {
                const int64_t mid = (from + to) / 2;
                if (sorted[mid].x < key)
                    from = mid + 1;
                else
                    to = mid;
            }
            edge[threadIdx.x] = from;
        }
        __syncthreads();
        if (looks) {
            if (a.token_bytes == 8)
                mark_tokens(static_cast<const int64_t *>(a.tokens), a.n, lo, hi, marks);
            else
                mark_tokens(static_cast<const int32_t *>(a.tokens), a.n, lo, hi, marks);
        } else {
            for (int64_t i = edge[0] + threadIdx.x; i < edge[1]; i += kFill)
                atomicOr(&marks[uint32_t(sorted[i].x - lo) / 32], 1u << (uint32_t(sorted[i].x - lo) % 32));
        }
        __syncthreads();
        fill_rows<T>(a, marks, lo, hi);
        __syncthreads();
    }
}

// ------------------------------------------------------------------ sum and join

constexpr int kSlab = 256;      // columns of a warp
constexpr int kSumThreads = kFill;

struct SumPlan {
    const uint2 *sorted;
    float *part;       // (tile, whether the token begins in it, slab): kSlab sums, element j of lane l at j * 32 + l
    int rows;          // of a tile
    int64_t tiles;
    int slabs;
    int fills;         // blocks that fill, before the others
    bool looks;        // they do not wait for the sorted list
};

__device__ __forceinline__ float *part_of(const SumPlan &p, int64_t tile, int slot, int slab)
{
    return p.part + ((tile * 2 + slot) * p.slabs + slab) * kSlab;
}

// A thread's columns of a row, K times VEC neighbouring ones, as they are in memory.
template <class T, int VEC, int K>
struct Cols {
    static constexpr int N = VEC == 1 ? 1 : Unit<T>::kN;
    using Word = typename std::conditional<VEC == 1, T, uint4>::type;
    Word w[K * VEC / N];
    // `row` at the slab's first column, of which `n` >= 1 are there (a multiple of N). Columns past
    // them repeat the last ones, so that no load waits for a condition: loads under conditions of
    // their own came back one row at a time (20011 x 771 in binary32, add's rows among them:
    // 103 us for 43).
    template <bool FULL>
    __device__ __forceinline__ void fetch(const T *row, int n, int lane)
    {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC / N; ++i)
                w[k * VEC / N + i] = *reinterpret_cast<const Word *>(row + (FULL ? (k * 32 + lane) * VEC + i * N
                                                                         : min((k * 32 + lane) * VEC + i * N, n - N)));
    }
    __device__ __forceinline__ void get(float (&v)[K * VEC]) const
    {
        if constexpr (VEC == 1) {
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] = load1(&w[k]);
        } else {
#pragma unroll
            for (int k = 0; k < K * VEC / N; ++k) {
                Unit<T> u;
                u.w = w[k];
                float2 f[N / 2];
                u.get(f);
#pragma unroll
                for (int j = 0; j < N; ++j) v[k * N + j] = j & 1 ? f[j / 2].y : f[j / 2].x;
            }
        }
    }
};
template <class T, int VEC, int K>
__device__ __forceinline__ void write_row(const EmbedArgs &a, uint32_t v, int c0, int lane, const float (&sum)[K * VEC],
                                          const Cols<T, VEC, K> *add)
{
    T *const out = static_cast<T *>(a.out) + int64_t(v) * a.out_stride + c0;
    float x[K * VEC];
    if (add) {
        add->get(x);
#pragma unroll
        for (int i = 0; i < K * VEC; ++i) x[i] = fmaf(a.scale, sum[i], x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < K * VEC; ++i) x[i] = a.scale * sum[i];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * 32 + lane) * VEC;
        float y[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) y[i] = x[k * VEC + i];
        store<T, VEC>(out + c, int(a.width) - c0 - c, y);
    }
}

// kAhead rows at a time: they, and add's rows where a token ends, are asked for
// together; then each is added to the one before it where that is the same token's.
template <class T, class D, int VEC, int K, int kAhead, bool ADD, bool FULL>
__device__ __forceinline__ void sum_tile(const EmbedArgs &a, const SumPlan &p, uint32_t tile, int slab)
{
    static_assert(VEC * K * 32 == kSlab && kAhead <= 8, "a warp has a slab");
    constexpr int C = VEC * K;
    const int lane = threadIdx.x % 32, c0 = slab * kSlab, n = int(a.width) - c0;
    const int64_t lo = int64_t(tile) * p.rows, hi = min(lo + p.rows, a.n);
    const uint32_t none = uint32_t(a.vocab);
    uint32_t last = lo > 0 ? p.sorted[lo - 1].x : 0xffffffffu;  // the token before
    bool early = true;                                          // it began in an earlier tile
    float sum[C];
    for (int64_t base = lo; base < hi; base += kAhead) {
        // entry j in lane j, and the token after the last
        const uint2 mine = lane <= kAhead && base + lane < a.n ? p.sorted[base + lane] : make_uint2(0xffffffffu, 0u);
        uint32_t key[kAhead + 1];
        Cols<D, VEC, K> v[kAhead];
        Cols<T, VEC, K> add[ADD ? kAhead : 1];
#pragma unroll
        for (int j = 0; j <= kAhead; ++j) key[j] = __shfl_sync(0xffffffffu, mine.x, j);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            // what is not there, and add's row of a token that goes on, is read from row 0 instead
            const uint32_t at = __shfl_sync(0xffffffffu, mine.y, j);
            const bool there = base + j < hi && key[j] < none;
            v[j].template fetch<FULL>(static_cast<const D *>(a.drows) + (there ? int64_t(at) * a.drow_stride : 0) + c0, n, lane);
            if (ADD)
                add[ADD ? j : 0].template fetch<FULL>(static_cast<const T *>(a.table) +
                                           (there && key[j] != key[j + 1] ? int64_t(key[j]) * a.table_stride : 0) + c0,
                                       n, lane);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (base + j >= hi || key[j] >= none) return;  // absent tokens come last
            early = early && key[j] == last;
            const bool same = key[j] == last && base + j > lo;
            last = key[j];
            float x[C];
            v[j].get(x);
#pragma unroll
            for (int i = 0; i < C; ++i) sum[i] = same ? sum[i] + x[i] : x[i];
            const bool ends = key[j] != key[j + 1];
            if (ends && !early) {
                write_row<T, VEC, K>(a, key[j], c0, lane, sum, ADD ? &add[ADD ? j : 0] : nullptr);
            } else if (ends || base + j == hi - 1) {
                float *const to = part_of(p, tile, early ? 0 : 1, slab) + lane;
#pragma unroll
                for (int i = 0; i < C; ++i) to[i * 32] = sum[i];
            }
        }
    }
}

template <class T, class D, int VEC, int K, int kAhead, bool ADD>
__global__ void __launch_bounds__(kSumThreads, 2) sum_kernel(EmbedArgs a, SumPlan p)
{
    pdl_trigger();
    if (int(blockIdx.x) < p.fills) {
        if (!p.looks) pdl_wait();
        fill<T>(a, p.sorted, p.looks, blockIdx.x, p.fills);
        return;
    }
    pdl_wait();
    const uint32_t number = (blockIdx.x - p.fills) * (kSumThreads / 32) + threadIdx.x / 32;
    const uint32_t tile = number / uint32_t(p.slabs);
    if (tile >= p.tiles) return;
    const int slab = int(number - tile * p.slabs);
    if ((slab + 1) * kSlab <= a.width)
        sum_tile<T, D, VEC, K, kAhead, ADD, true>(a, p, tile, slab);
    else
        sum_tile<T, D, VEC, K, kAhead, ADD, false>(a, p, tile, slab);
}

constexpr int kJoinWarps = 8;

// A warp looks at a tile: where a token begins in it and goes on, the partial rows from
// there on are added up, many of them by the whole block.
template <class T, int VEC, int K>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(EmbedArgs a, SumPlan p)
{
    __shared__ float sh[kJoinWarps][kSlab];
    __shared__ int64_t count[kJoinWarps];
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, slab = blockIdx.y;
    const int64_t tile = int64_t(blockIdx.x) * kJoinWarps + warp;
    int64_t more = 0;  // tiles that the token reaches into
    uint32_t key = 0xffffffffu;
    if ((tile + 1) * p.rows < a.n) {
        const int64_t lo = tile * p.rows, hi = lo + p.rows;
        key = p.sorted[hi - 1].x;
        const bool goes_on = key < uint32_t(a.vocab) && p.sorted[hi].x == key;
        const bool began_before = lo > 0 && p.sorted[lo - 1].x == key;
        if (goes_on && !began_before) {
            // the last tile that starts with the token: the next 32 first, then 32 looks at a time
            const int64_t most = p.tiles - tile - 1;
            int64_t from, to = most, step;  // tile + from does
            const int64_t near = tile + min(int64_t(lane) + 1, most);
            from = __popc(__ballot_sync(0xffffffffu, p.sorted[near * p.rows].x == key));
            if (from < 32 || most <= 32) {
                from = min(from, most);
                to = from;
            }
            while (from < to) {
                step = (to - from + 31) / 32;
                const int64_t at = min(from + (lane + 1) * step, to);
                const int hits = __popc(__ballot_sync(0xffffffffu, p.sorted[(tile + at) * p.rows].x == key));  // a prefix
                if (hits == 32) {
                    from = to;
                } else {
                    to = min(from + (hits + 1) * step, to) - 1;
                    from += hits * step;
                    to = max(to, from);
                }
            }
            more = from;
        }
    }
    auto add_up = [&](int64_t t, int64_t lo, int64_t hi, float (&sum)[kSlab / 32]) {
        // pieces [lo, hi) of the token that begins in tile t
#pragma unroll
        for (int j = 0; j < kSlab / 32; ++j) sum[j] = 0.0f;
        for (int64_t i0 = lo; i0 < hi; i0 += 4) {
            float x[4][kSlab / 32];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int64_t i = min(i0 + m, hi - 1);
                const float *const from = part_of(p, t + i, i == 0 ? 1 : 0, slab) + lane;
#pragma unroll
                for (int j = 0; j < kSlab / 32; ++j) x[m][j] = from[j * 32];
            }
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int j = 0; j < kSlab / 32; ++j)
                    if (i0 + m < hi) sum[j] += x[m][j];
        }
    };
    auto write = [&](uint32_t k, const float (&sum)[kSlab / 32]) {
        const int c0 = slab * kSlab;
        Cols<T, VEC, K> add;
        if (a.table)
            add.template fetch<false>(static_cast<const T *>(a.table) + int64_t(k) * a.table_stride + c0, int(a.width) - c0, lane);
        write_row<T, VEC, K>(a, k, c0, lane, sum, a.table ? &add : nullptr);
    };
    constexpr int64_t kAlone = 8;
    if (more && more <= kAlone) {
        float sum[kSlab / 32];
        add_up(tile, 0, more + 1, sum);
        write(key, sum);
    }
    if (lane == 0) count[warp] = more;
    __syncthreads();
    for (int w = 0; w < kJoinWarps; ++w) {
        const int64_t n = count[w] + 1;
        if (n <= kAlone + 1) continue;
        const int64_t each = (n + kJoinWarps - 1) / kJoinWarps;
        float sum[kSlab / 32];
        add_up(int64_t(blockIdx.x) * kJoinWarps + w, min(warp * each, n), min((warp + 1) * each, n), sum);
#pragma unroll
        for (int j = 0; j < kSlab / 32; ++j) sh[warp][j * 32 + lane] = sum[j];
        __syncthreads();
        if (warp == w) {
#pragma unroll
            for (int j = 0; j < kSlab / 32; ++j) {
                sum[j] = 0.0f;
                for (int i = 0; i < kJoinWarps; ++i) sum[j] += sh[i][j * 32 + lane];
            }
            write(key, sum);
        }
        __syncthreads();
    }
}

// Rows to a tile: 8, or more where that still leaves work for every SM.
int tile_rows(int64_t n, int64_t slabs)
{
    int rows = 8;
    while (rows < 1024 && n / rows * slabs > 152 * 64) rows *= 2;
    return rows;
}

bool whole(const void *p, int64_t stride, int size)
{
    return (reinterpret_cast<uintptr_t>(p) | uintptr_t(stride * size)) % 16 == 0;
}

template <class T, class D, int VEC>
cudaError_t sum_and_join(const EmbedArgs &a, const SumPlan &p, cudaStream_t st)
{
    constexpr int K = kSlab / 32 / VEC, kAhead = VEC == 1 || sizeof(D) == 4 ? 4 : 8;
    constexpr int kAheadAdd = VEC == 1 ? 3 : kAhead;
    const int64_t blocks = p.fills + (p.tiles * p.slabs + kSumThreads / 32 - 1) / (kSumThreads / 32);
    if (blocks * 8 >= (int64_t(1) << 31) || p.slabs > 65535) return cudaErrorInvalidConfiguration;
    auto *sum = a.table ? &sum_kernel<T, D, VEC, K, kAheadAdd, true> : &sum_kernel<T, D, VEC, K, kAhead, false>;
    if (cudaError_t e = launch_dependent(sum, int(blocks), kSumThreads, 0, st, a, p)) return e;
    if (p.tiles < 2) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((p.tiles + kJoinWarps - 1) / kJoinWarps), unsigned(p.slabs));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = ZG_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, &join_kernel<T, VEC, K>, a, p);
}

// Tokens up to which the blocks that fill look them all through, beside the sort. (50257 x 768 in bf16, looking and from the
// sorted list: 8192 tokens 32 and 44 us with a graph's replay, 20011 46 and 59, 65536 85 and 91, 262144 251 and 263,
// 1048576 912 and 892. A larger bound would gain a little up to some 262144: 262144 x 768 there 296 and 351.)
constexpr int64_t kLooks = 65536;

template <class T, class D>
cudaError_t gradient_of(const EmbedArgs &a, cudaStream_t st)
{
    SortPlan s{};
    int bits = 1;
    while (bits < 31 && (int64_t(1) << bits) <= a.vocab) ++bits;  // holds vocab itself, the key of absent tokens
    s.passes = (bits + 8) / 9;
    s.bits = (bits + s.passes - 1) / s.passes;
    s.blocks = 1;
    while (s.blocks < kMostBlocks && a.n > int64_t(s.blocks) * kSort) s.blocks *= 2;
    s.pair[0] = static_cast<uint2 *>(a.work);
    s.pair[1] = s.pair[0] + a.n + (a.n & 1);
    const uint2 *const sorted = s.pair[(s.passes - 1) & 1];
    if (a.n) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(unsigned(s.blocks));
        cfg.blockDim = dim3(kSort);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(s.blocks);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaError_t e = cudaLaunchKernelEx(&cfg, &sort_kernel, a, s)) return e;
    }
    SumPlan p{};
    p.sorted = sorted;
    p.slabs = int((a.width + kSlab - 1) / kSlab);
    p.rows = tile_rows(a.n, p.slabs);
    p.tiles = (a.n + p.rows - 1) / p.rows;
    p.part = reinterpret_cast<float *>(s.pair[1] + a.n + (a.n & 1));
    if (a.table != a.out) p.fills = int(std::min(int64_t(kFillBlocks), (a.vocab + kFill / 32 - 1) / (kFill / 32)));
    p.looks = a.n > 0 && a.n <= kLooks;
    if (p.fills + p.tiles == 0) return cudaSuccess;
    if (whole(a.drows, a.drow_stride, int(sizeof(D))) && a.width % 8 == 0 &&
        (!a.table || whole(a.table, a.table_stride, int(sizeof(T)))))
        return sum_and_join<T, D, 8>(a, p, st);
    return sum_and_join<T, D, 1>(a, p, st);
}

template <class T>
cudaError_t lookup_of(const EmbedArgs &a, cudaStream_t st)
{
    const int64_t blocks = (a.n + 4 * kRows - 1) / (4 * kRows);
    if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    if (whole(a.table, a.table_stride, int(sizeof(T))) && whole(a.out, a.out_stride, int(sizeof(T))) &&
        a.width % Unit<T>::kN == 0)
        lookup_kernel<T, true, 4><<<unsigned(blocks), 128, 0, st>>>(a);
    else
        lookup_kernel<T, false, 8><<<unsigned(blocks), 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs &a, cudaStream_t st)
{
    return a.dtype == ZG_DTYPE_BF16 ? lookup_of<uint16_t>(a, st) : lookup_of<float>(a, st);
}

int64_t embed_grad_workspace(int64_t n, int64_t, int64_t width)
{
    const int64_t slabs = (width + kSlab - 1) / kSlab, rows = tile_rows(n, slabs);
    return 2 * (n + (n & 1)) * int64_t(sizeof(uint2)) + (n + rows - 1) / rows * 2 * slabs * kSlab * 4;
}

cudaError_t launch_embed_grad(const EmbedArgs &a, cudaStream_t st)
{
    const bool bf = a.dtype == ZG_DTYPE_BF16, dbf = a.drow_dtype == ZG_DTYPE_BF16;
    if (bf) return dbf ? gradient_of<uint16_t, uint16_t>(a, st) : gradient_of<uint16_t, float>(a, st);
    return dbf ? gradient_of<float, uint16_t>(a, st) : gradient_of<float, float>(a, st);
}

}  // namespace zg
