// The k largest of each row of logits, largest first, ties to the lowest index.
//
// Bound by memory: a row is read once. It is cut into kShares shares, whose
// maxima are taken as it streams through registers. The k-th largest of these
// maxima is no more than the row's k-th largest logit (k shares each hold one
// at least as large), so it is a bound below which nothing has to be looked at:
// only shares whose maximum reaches it are read again, out of L2, and about k
// logits pass. Those are put in order by counting, for each, how many come
// before it (a longer list by sorted runs, and searches in the others). Rows in
// which too many pass (many equal values) have their k-th largest found bit by
// bit. Few rows take a cluster of blocks to a row, whose lists are merged
// through distributed shared memory.
//
// Measured at 4096 x 50257 in bf16: k = 64 84 us (4.9 TB/s), k = 256 146. What
// is above the 61 us of the bytes is each row's end (bound, shares read again,
// order), during which its block asks for nothing; other blocks of the SM fill
// in for it. At k = 256 the bound is the median share's maximum, and half of the row
// is looked at again. In binary32 186 us (4.4 TB/s) for 121: the rows in flight, 183
// MB, do not fit L2, and a third of the logits comes from DRAM again. 7 rows, k = 100,
// 8 us, all latency.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "zg_launch.h"
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

namespace cg = cooperative_groups;

constexpr int kMost = 1024;  // logits that may pass the bound

// Unsigned keys in the order of the values, NaN above everything, -0 = +0, none
// zero: 16 bits for bf16, 32 for binary32. `bits` are the value's as binary32.
template <class T>
__device__ __forceinline__ uint32_t key_of(uint32_t bits)
{
    uint32_t key = (bits & 0x80000000u) ? ~bits : (bits | 0x80000000u);
    if (bits == 0x80000000u) key = 0x80000000u;
    if ((bits & 0x7fffffffu) > 0x7f800000u) key = 0xffffffffu;
    return sizeof(T) == 2 ? key >> 16 : key;
}
// A binary32 that no value whose key is at least `key` is less than.
template <class T>
__device__ __forceinline__ float value_of(uint32_t key)
{
    if (sizeof(T) == 2) key <<= 16;
    if (key == 0u) return -INFINITY;
    if (key > 0xff800000u) return INFINITY;  // NaNs alone reach it: they are less than nothing
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ uint32_t bits_at(const float *p) { return __float_as_uint(*p); }
__device__ __forceinline__ uint32_t bits_at(const uint16_t *p) { return uint32_t(*p) << 16; }
template <class T>
__device__ __forceinline__ uint32_t bits_in(const Unit<T> &x, int i)
{
    const uint32_t w[4] = {x.w.x, x.w.y, x.w.z, x.w.w};
    if (sizeof(T) == 4) return w[i & 3];
    return (i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16;
}

// The same for an i that is not known when compiling.
template <class T>
__device__ __forceinline__ uint32_t bits_of(const Unit<T> &x, int i)
{
    const int word = sizeof(T) == 2 ? i >> 1 : i;
    const uint32_t lo = word & 1 ? x.w.y : x.w.x, hi = word & 1 ? x.w.w : x.w.z, w = word & 2 ? hi : lo;
    if (sizeof(T) == 4) return w;
    return i & 1 ? w & 0xffff0000u : w << 16;
}

// Larger keys first, then lower indices: one number, larger first. Its lowest
// bit marks a -0, so that all but a NaN's bits can be had back from it.
__device__ __forceinline__ uint64_t entry(uint32_t key, int v, uint32_t bits)
{
    return (uint64_t(key) << 32) | uint32_t(0x3fffffff - v) << 1 | uint32_t(bits == 0x80000000u);
}
__device__ __forceinline__ int index_of(uint64_t e) { return 0x3fffffff - int(uint32_t(e) >> 1); }
template <class T>
__device__ __forceinline__ T value_in(uint64_t e, const T *z)
{
    const uint32_t key = uint32_t(e >> 32), top = sizeof(T) == 2 ? 0x8000u : 0x80000000u;
    if (key == top * 2u - 1u) return z[index_of(e)];  // a NaN
    const uint32_t bits = (key & top) ? ((key & ~top) | ((e & 1u) ? top : 0u)) : ~key;
    if constexpr (sizeof(T) == 2)
        return T(bits);
    else
        return __uint_as_float(bits);
}

struct Shared {
    uint64_t list[kMost];
    uint64_t top[ZG_TOPK_MAX];  // this part's, in order; read by the others
    uint16_t hot[512];  // threads whose maximum reaches the bound
    uint32_t bound;
    int hots, count, tops;
    int warps[16];
};

template <int WARPS>
__device__ __forceinline__ int block_sum(int v, int *red)
{
    v = __reduce_add_sync(0xffffffffu, v);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) v += red[i];
    __syncthreads();
    return v;
}

constexpr int kShares = 512;  // of a block's part: unit u belongs to share u mod kShares

template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1536 / THREADS) topk_kernel(const T *logits, int vocab, int64_t row_stride, int k,
                                                                      T *values, int32_t *index, int blocks, int each)
{
    extern __shared__ uint64_t lists[];  // the parts' lists, where a row has several
    __shared__ Shared sh;
    constexpr int N = Unit<T>::kN, kWarps = THREADS / 32, kBits = 8 * int(sizeof(T)), kOwn = kShares / THREADS;
    const int tid = threadIdx.x;
    const unsigned number = blockIdx.x / unsigned(blocks);
    const int64_t r = number;
    const int rank = int(blockIdx.x - number * unsigned(blocks));
    const T *const z = logits + r * row_stride;
    const Row<T> row(z, vocab, each, rank);
    const Part &part = row.part;
    const uint4 *const from = row.from();
    const int units = row.units;
    auto unit_at = [&](int u) {
        Unit<T> x;
        x.w = from[u];
        return x;
    };
    const int base = part.u0 * N - part.head;  // vocabulary index of unit 0's first element
    int ragged = row.ragged(tid);
    if (ragged >= 0) ragged -= part.head;
    const uint32_t ragged_bits = ragged >= 0 ? bits_at(z + ragged) : 0u;
    const uint32_t ragged_key = ragged >= 0 ? key_of<T>(ragged_bits) : 0u;

    // a thread has the shares tid, tid + THREADS, ...
    typename Unit<T>::Top most[kOwn];
    constexpr int kRounds = 4 / kOwn;  // four units asked for before the first is looked at
    int u = tid;
    for (; u + kRounds * kShares - THREADS < units; u += kRounds * kShares) {
        Unit<T> x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = unit_at(u + i * THREADS);
#pragma unroll
        for (int i = 0; i < 4; ++i) most[i % kOwn].add(x[i]);
    }
    {
        Unit<T> x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (u + i * THREADS < units) x[i] = unit_at(u + i * THREADS);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (u + i * THREADS < units) most[i % kOwn].add(x[i]);
    }
    uint32_t best[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) best[i] = tid + i * THREADS < units ? key_of<T>(__float_as_uint(most[i].get())) : 0u;
    const uint32_t units_best = best[0];  // without the ragged element
    best[0] = max(best[0], ragged_key);

    // the largest bound, to 16 bits, that k of the threads' maxima reach: one
    // warp looks for it between the least and the largest of them
    uint32_t *const bests = reinterpret_cast<uint32_t *>(sh.list);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) bests[tid + i * THREADS] = best[i] >> (kBits - 16);
    __syncthreads();
    if (tid < 32) {
        uint32_t v[kShares / 32], lo = 0xffffffffu, hi = 0u;
        int some = 0;
#pragma unroll
        for (int i = 0; i < kShares / 32; ++i) {
            v[i] = bests[tid + 32 * i];
            some += v[i] != 0u;
            lo = min(lo, v[i] ? v[i] : 0xffffffffu);
            hi = max(hi, v[i]);
        }
        some = __reduce_add_sync(0xffffffffu, some);
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (some < k) {
            lo = 0u;  // everything passes
        } else {
            while (lo < hi) {  // lo is reached by k, hi + 1 is not
                const uint32_t mid = lo + (hi - lo + 1) / 2;
                int n = 0;
#pragma unroll
                for (int i = 0; i < kShares / 32; ++i) n += v[i] >= mid;
                if (__reduce_add_sync(0xffffffffu, n) >= k)
                    lo = mid;
                else
                    hi = mid - 1;
            }
        }
        if (tid == 0) {
            sh.bound = lo << (kBits - 16);
            sh.hots = 0;
            sh.count = 0;
        }
    }
    __syncthreads();
    const uint32_t bound = sh.bound;
    const float least = value_of<T>(bound);
    // what reaches it: the shares of the threads whose maximum does, spread over all threads
    auto put = [&](uint32_t bits, int v) {
        const int n = atomicAdd(&sh.count, 1);
        if (n < kMost) sh.list[n] = entry(key_of<T>(bits), v, bits);
    };
    if (ragged >= 0 && ragged_key >= bound) put(ragged_bits, ragged);
    best[0] = units_best;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
        if (best[i] && best[i] >= bound) sh.hot[atomicAdd(&sh.hots, 1)] = uint16_t(tid + i * THREADS);
    __syncthreads();
    {
        const int hots = sh.hots, per = (units + kShares - 1) / kShares;
        int side = 0;  // lanes to a share that reaches it: a power of two, at most a warp
        while (side < 5 && (1 << side) < per) ++side;
        auto look = [&](const Unit<T> &x, int u) {
            typename Unit<T>::Top top;
            top.add(x);
            if (top.get() < least) return;
            uint32_t hits = 0u;
#pragma unroll
            for (int j = 0; j < N; ++j) hits |= uint32_t(!(__uint_as_float(bits_in(x, j)) < least)) << j;
            while (hits) {
                const int j = __ffs(int(hits)) - 1;
                hits &= hits - 1u;
                put(bits_of(x, j), base + u * N + j);
            }
        };
        // two units asked for before the first is looked at (one: 85 us for 83 above, four: 85)
        const int lanes = 1 << side;
        for (int i = tid & (lanes - 1); i < per; i += lanes) {
            for (int h = tid >> side; h < hots; h += 2 * THREADS >> side) {
                Unit<T> x[2];
                int at[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int share = h + (j * THREADS >> side);
                    at[j] = share < hots ? sh.hot[share] + i * kShares : units;
                    if (at[j] < units) x[j] = unit_at(at[j]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (at[j] < units) look(x[j], at[j]);
            }
        }
    }
    __syncthreads();
    if (sh.count > kMost) {
        // The k-th largest key itself, bit by bit: then all above it, and of its
        // equals the first ones by index.
        const int size = part.last - part.first, want = min(k, size);
        auto reaching = [&](uint32_t key) {
            int n = ragged >= 0 && ragged_key >= key;
            for (int u = tid; u < units; u += THREADS) {
                const Unit<T> x = unit_at(u);
#pragma unroll
                for (int i = 0; i < N; ++i) n += key_of<T>(bits_in(x, i)) >= key;
            }
            return block_sum<kWarps>(n, sh.warps);
        };
        uint32_t kth = 0u;
        for (int b = kBits - 1; b >= 0; --b) {
            const uint32_t with = kth | (1u << b);
            if (reaching(with) >= want) kth = with;
        }
        if (tid == 0) sh.count = 0;
        __syncthreads();
        if (ragged >= 0 && ragged_key > kth) put(ragged_bits, ragged);
        for (int u = tid; u < units; u += THREADS) {
            const Unit<T> x = unit_at(u);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t bits = bits_in(x, i);
                if (key_of<T>(bits) > kth) put(bits, base + u * N + i);
            }
        }
        __syncthreads();
        // the equals, in the order of their indices: the head, the units, the tail
        int have = sh.count;
        __syncthreads();
        auto equals = [&](int n, auto each_one) {  // n of this thread's, after those of the threads before it
            int before = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, before, o);
                if (tid % 32 >= o) before += v;
            }
            if (tid % 32 == 31) sh.warps[tid / 32] = before;
            __syncthreads();
            int all = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w == tid / 32) before += all;
                all += sh.warps[w];
            }
            if (n) each_one(have + before - n);
            have += all;
            __syncthreads();
        };
        const bool head = ragged >= 0 && ragged < base, tail = ragged >= 0 && !head;
        equals(head && ragged_key == kth, [&](int at) {
            if (at < want) sh.list[at] = entry(kth, ragged, ragged_bits);
        });
        for (int u0 = 0; u0 < units && have < want; u0 += THREADS) {
            const int u = u0 + tid;
            Unit<T> x;
            int n = 0;
            if (u < units) {
                x = unit_at(u);
#pragma unroll
                for (int i = 0; i < N; ++i) n += key_of<T>(bits_in(x, i)) == kth;
            }
            equals(n, [&](int at) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (key_of<T>(bits_in(x, i)) == kth) {
                        if (at < want) sh.list[at] = entry(kth, base + u * N + i, bits_in(x, i));
                        ++at;
                    }
            });
        }
        if (have < want)
            equals(tail && ragged_key == kth, [&](int at) {
                if (at < want) sh.list[at] = entry(kth, ragged, ragged_bits);
            });
        if (tid == 0) sh.count = min(have, want);
        __syncthreads();
    }
    const int count = sh.count;
    auto settle = [&](uint64_t e, int place) {
        if (blocks == 1) {
            values[r * k + place] = value_in(e, z);
            index[r * k + place] = index_of(e);
        } else {
            sh.top[place] = e;
        }
    };
    if (count <= 128) {
        // An entry's place is the number of those before it, counted by the
        // threads that share it.
        int share = 1;
        while (share < 32 && count * share * 2 <= THREADS) share *= 2;
        for (int e0 = 0; e0 < count; e0 += THREADS / share) {
            const int e = e0 + tid / share;
            const uint64_t mine = e < count ? sh.list[e] : 0u;
            int place = 0;
            for (int j = tid % share; j < count; j += share) place += sh.list[j] > mine;
            for (int o = share / 2; o; o >>= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
            if (e < count && tid % share == 0 && place < k) settle(mine, place);
        }
    } else {
        // More than counting is good for: runs of 32 are sorted by a warp each,
        // and an entry's place is the sum of its places among the runs.
        const int runs = (count + 31) / 32;
        for (int n = tid / 32; n < runs; n += kWarps) {
            const int e = n * 32 + tid % 32;
            uint64_t m = e < count ? sh.list[e] : 0u;
#pragma unroll
            for (int size = 2; size <= 32; size *= 2)
#pragma unroll
                for (int o = size / 2; o; o /= 2) {
                    const uint64_t other = __shfl_xor_sync(0xffffffffu, m, o);
                    const bool larger = ((tid & o) == 0) == ((tid & 31 & size) == 0);  // this lane takes the larger
                    if ((other > m) == larger) m = other;
                }
            sh.list[e] = m;
        }
        __syncthreads();
        for (int n = tid / 32; n < runs; n += kWarps) {
            const uint64_t m = sh.list[n * 32 + tid % 32];
            int place = tid % 32;
            for (int b = 0; b < runs; ++b) {
                if (b == n) continue;
                int at = 0;
#pragma unroll
                for (int step = 16; step; step /= 2)
                    if (sh.list[b * 32 + at + step - 1] > m) at += step;
                place += at + (at == 31 && sh.list[b * 32 + 31] > m);
            }
            if (m && place < k) settle(m, place);
        }
    }
    if (blocks == 1) return;

    // Several parts: all their lists, each in order, into this block's shared
    // memory; an entry's place is then the sum of its places among them.
    cg::cluster_group cluster = cg::this_cluster();
    const int mine = min(count, k);
    if (tid == 0) sh.tops = mine;
    cluster.sync();
    __shared__ int counts[8];
    if (tid < blocks) counts[tid] = cluster.map_shared_rank(&sh, tid)->tops;
    for (int i = tid; i < blocks * k; i += THREADS) {
        const int b = i / k, j = i - b * k;
        lists[i] = cluster.map_shared_rank(&sh, b)->top[j];
    }
    cluster.barrier_arrive();  // its reads are done; nobody leaves before all are
    __syncthreads();
    // eight lanes to an entry, a list to each
    for (int e0 = 0; e0 < mine; e0 += THREADS / 8) {
        const int e = e0 + tid / 8, b = tid % 8;
        const uint64_t m = e < mine ? sh.top[e] : 0u;
        int lo = 0, hi = b < blocks && e < mine ? counts[b] : 0;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (lists[b * k + mid] > m)
                lo = mid + 1;
            else
                hi = mid;
        }
#pragma unroll
        for (int o = 4; o; o >>= 1) lo += __shfl_xor_sync(0xffffffffu, lo, o);
        if (e < mine && b == 0 && lo < k) {
            values[r * k + lo] = value_in(m, z);
            index[r * k + lo] = index_of(m);
        }
    }
    cluster.barrier_wait();
}

template <class T, int THREADS>
cudaError_t launch(const T *logits, int64_t rows, int vocab, int64_t stride, int k, T *values, int32_t *index,
                   int64_t blocks, int64_t units, cudaStream_t st)
{
    auto *kernel = &topk_kernel<T, THREADS>;
    if (rows * blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(rows * blocks));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = blocks > 1 ? size_t(blocks) * k * sizeof(uint64_t) : 0;  // at most 16 KB
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(blocks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, logits, vocab, stride, k, values, index, int(blocks),
                              int((units + blocks - 1) / blocks));
}

template <class T>
cudaError_t by_size(const T *logits, int64_t rows, int vocab, int64_t stride, int k, T *values, int32_t *index, cudaStream_t st)
{
    // Small blocks keep most rows in flight, at different places at once, so that
    // the ends of some do not leave memory idle; too small ones are long at the
    // candidates: of 4096 x 50257 in bf16, k = 64, 128 threads to a row take
    // 101 us, 256 90, 512 113; k = 256 206, 177 and 196 (at 1024 threads to an SM;
    // with 1536, as it is, 256 take 85 and 153). Short rows need fewer, and
    // rows too few to fill half the GPU take more threads, then more blocks.
    const int64_t units = (int64_t(vocab) * int64_t(sizeof(T)) + 30) / 16;
    int threads = units <= 2048 ? 128 : 256;
    int64_t blocks = 1;
    while (rows * blocks * threads < 152 * 512 && units / blocks > 4 * threads) {
        if (threads < 512)
            threads *= 2;
        else if (blocks < 8)
            blocks *= 2;
        else
            break;
    }
    if (threads == 128) return launch<T, 128>(logits, rows, vocab, stride, k, values, index, blocks, units, st);
    if (threads == 256) return launch<T, 256>(logits, rows, vocab, stride, k, values, index, blocks, units, st);
    return launch<T, 512>(logits, rows, vocab, stride, k, values, index, blocks, units, st);
}

}  // namespace

cudaError_t launch_topk(const void *logits, int dtype, int64_t rows, int vocab, int64_t stride, int k, void *values,
                        int32_t *index, cudaStream_t st)
{
    if (dtype == ZG_DTYPE_BF16)
        return by_size(static_cast<const uint16_t *>(logits), rows, vocab, stride, k, static_cast<uint16_t *>(values), index, st);
    return by_size(static_cast<const float *>(logits), rows, vocab, stride, k, static_cast<float *>(values), index, st);
}

}  // namespace zg
