// zg_block.cuh -- the norms before and after a block, with its gate and the residual's scale.
//
// Forward, for a row: b = w1 o s1, x' = r x + gate b, n = w2 x' s2, where s1 and s2
// are 1 / sqrt(mean square + eps) of o and of x'.
// Backward forms x' again from x and o in binary32, so that nothing of its rounding
// enters. With xh = x' s2, oh = o s1, u = gate w1, e = dn w2 and y = dx_new:
//   dX = y + s2 (e - xh c2),      c2 = mean(e xh),
//   dx = r dX,  do = s1 (u dX - oh c1),  c1 = mean(u oh dX)
//                                           = mean(u oh (y + s2 e)) - s2 c2 mean(u oh xh),
// so a row takes one joint sum of three values. Of the weights' gradients
// dw2 = Q = sum dn xh, and with P = sum of dX oh over a gate's rows, dgate = w1 P
// and dw1 = sum over gates of gate P: two sums to a column.
//
// Bound by memory: forward reads two rows and writes two, backward reads four and
// writes two, of which each is moved once. A team of warps works on a row; it copies its next
// rows into shared memory while it computes (cp.async: an aligned row's units are
// copied and read by the same thread, and by no other, so they need no barrier), and goes
// over the row in shared memory again where a sum has to be known first.
//
// Measured at 16384 x 4096 in bf16: forward 94 us (5.7 TB/s), backward 151 (5.3 TB/s) and some 6 to 10 for the sums of
// the weights' gradients after it; with a gate for each of 64 sequences 184, of 512 231, of every row 720. In binary32 172
// and 252 us (6.2 and 6.4 TB/s). Issue is active in 45 to 49 % of the cycles at 16 warps to an SM: what is left are
// the dependent sums of a row. 32768 x 2048 in bf16 91 and 147 us (5.9 and 5.5 TB/s). 9001 x 771 in binary32, rows at any
// alignment: 23 and 44 us (4.8 and 3.8 TB/s); 2000 x 4099 35 and 80. Of 16384 columns in bf16 the backward pass has
// no room in shared memory for its rows and weights and reads rows from memory twice (4096 rows 562 us, forward 137).
#pragma once

#include <atomic>

#include "zg_async.cuh"
#include "zg_launch.h"
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

constexpr int kMost = 512;     // threads of a block
constexpr int kBlocks = 152;   // SMs
// Blocks to an SM: two where a thread's few columns fit half of the registers. (Not so in the backward pass of aligned
// rows, whose threads hold whole units of four tensors: 32768 x 768 there in bf16 106 us with two and 79 with one, in
// binary32 128 and 100.)
template <int COLUMNS, bool ALL>
constexpr int kToSm = ALL && COLUMNS <= 8 ? 2 : 1;
constexpr int kStages = 4;     // rows of a team in shared memory, at most
constexpr int kTeams = 8;      // of a block, at most
constexpr int kMemory = 224 * 1024;  // of an SM's blocks

// The threads that share a row: whole warps of a block.
struct Team {
    int id, count;     // of the block's teams
    int tid, threads;  // of the team's threads
    int parity = 0;
    __device__ __forceinline__ Team(int team_threads)
    {
        threads = team_threads;
        count = blockDim.x / team_threads;
        id = threadIdx.x / team_threads;
        tid = threadIdx.x - id * team_threads;
    }
    __device__ __forceinline__ void sync() const
    {
        team_sync(id, threads);
    }
    // Sums over the team, the same in all of its threads. Two buffers, so that one
    // barrier is enough: nobody is two sums ahead of another. A team has 16 places of each,
    // those that it has no warp for zero, which are read all at once.
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N], float *sh)
    {
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (threads == 32) return;
        float *const mine = sh + (id * 2 + parity) * (kMost / 32 * N);
        parity ^= 1;
        if (tid % 32 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) mine[i * (kMost / 32) + tid / 32] = v[i];
        sync();
        // a lane takes its half's place of one value, and 16 lanes add up
        float x[(N + 1) / 2];
        const int lane = tid % 32;
#pragma unroll
        for (int i = 0; i < (N + 1) / 2; ++i) x[i] = mine[min(2 * i + lane / 16, N - 1) * 16 + lane % 16];
#pragma unroll
        for (int o = 8; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < (N + 1) / 2; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x[i / 2], i % 2 * 16);
    }
};
// Before the first sum.
template <int N>
__device__ __forceinline__ void clear_sums(float *sh)
{
    for (int i = threadIdx.x; i < N; i += blockDim.x) sh[i] = 0.0f;
    __syncthreads();
}

// How a block's teams keep rows in shared memory: `stages` of them, each of some tensors
// whose rows take `slot` bytes. Without stages rows are read from memory itself.
struct Ring {
    int stages, slot;
};

// A thread has K chunks of E columns: chunk k is VEC = E neighbouring columns of a row whose
// tensors all lie on 16 bytes, or (VEC = 1) E columns one team apart. With TEAM, the
// team's size is known, and a row in shared memory has zeros behind it up to the last column of
// the team, so that nothing but the stores asks whether a column is the row's.
template <int VEC, int E, int TEAM>
__device__ __forceinline__ int column(const Team &team, int k, int i)
{
    const int threads = TEAM ? TEAM : team.threads;
    return VEC == 1 ? team.tid + (k * E + i) * threads : (team.tid + k * threads) * VEC + i;
}

__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }
__device__ __forceinline__ float total(float2 v) { return v.x + v.y; }

// The rows of one tensor as a team reads them. Whole warps have places past an aligned row's end, whose units no
// thread copies. ZEROS: they count as zero in a row's sums. A unit that another thread copies would not do there: its
// copy may still be on its way, and a NaN found in its place stays one times a weight of zero.
template <class T, int VEC, int E, int K, int TEAM, bool ZEROS>
struct Source {
    const T *ptr;
    int64_t stride;
    uint32_t at;  // shared address of the team's first stage; stages are `step` bytes apart
    int step;
    __device__ __forceinline__ Source(const RowsView &v, uint32_t first, int tensor, const Ring &ring, int tensors)
        : ptr(static_cast<const T *>(v.ptr)), stride(v.stride), at(first + tensor * ring.slot), step(ring.slot * tensors)
    {
    }
    __device__ __forceinline__ int head(int64_t r) const  // elements between a 16-byte boundary and the row
    {
        return VEC == 1 ? int((reinterpret_cast<uintptr_t>(ptr + r * stride) & 15u) / sizeof(T)) : 0;
    }
    // Row r on its way into a stage. Of aligned rows a thread copies what it reads itself.
    __device__ __forceinline__ void copy(const Team &team, int64_t r, int stage, int width) const
    {
        const T *const row = ptr + r * stride;
        const uint32_t to = at + stage * step;
        if constexpr (VEC == 1) {
            constexpr int N = Unit<T>::kN;
            const int h = head(r), units = (h + width + N - 1) / N;
            const char *const from = reinterpret_cast<const char *>(row - h);
            for (int u = team.tid; u < units; u += TEAM ? TEAM : team.threads) copy16(to + u * 16, from + u * 16);
        } else {
            const T *const mine = row + team.tid * VEC;
            const uint32_t there = to + team.tid * 16;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (column<VEC, E, TEAM>(team, k, 0) < width)
                    copy16(there + k * team.threads * 16, mine + k * team.threads * VEC);
        }
    }
    // Once its own copies are here, and before the team's barrier: zeros from a row's end on, over what
    // its last unit has behind it and the unit after that, which an earlier row may have reached.
    __device__ __forceinline__ void close(const Team &team, int64_t r, int stage, int width) const
    {
        if constexpr (TEAM != 0) {
            constexpr int N = Unit<T>::kN;
            const int end = head(r) + width, units = (end + N - 1) / N;
            if (team.tid != (units - 1) % TEAM) return;  // the thread that copied the last unit
            const uint32_t to = at + stage * step;
            for (int i = end; i < (units + 1) * N; ++i) {
                if constexpr (sizeof(T) == 2)
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + i * 2), "h"(uint16_t(0)) : "memory");
                else
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + i * 4), "r"(0u) : "memory");
            }
        }
    }
    // Before the first row: zeros in the thread's own places past the row's end, which no copy reaches. (16384 x 2048 in
    // binary32, backward: 132 us; with loads under a condition 138, with zeros by a condition after them 144, and 4096 x
    // 8192 183 for 153. The places take room: at 9217 to 9556 columns in binary32 none is left for a row, 495 us for 339.)
    __device__ __forceinline__ void open(const Team &team, int stages, int width) const
    {
        if constexpr (VEC != 1 && ZEROS) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = column<VEC, E, TEAM>(team, k, 0);
                if (c < width) continue;
                for (int i = 0; i < stages; ++i)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + i * step + c * int(sizeof(T))), "r"(0u)
                                 : "memory");
            }
        }
    }
    // Chunk k of row r. Of aligned rows, places past the width are zero, or without ZEROS the thread's own first place
    // again; of others, where the team's barrier has made every copy visible, they are (without TEAM) column 0 again.
    __device__ __forceinline__ void get(const Team &team, int64_t r, int stage, bool staged, int k, int width,
                                        float2 (&v)[E / 2]) const
    {
        if constexpr (VEC == 1) {
            const uint32_t row = at + stage * step + head(r) * uint32_t(sizeof(T));
            float e[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = column<VEC, E, TEAM>(team, k, i), at_c = TEAM || c < width ? c : 0;
                if (!TEAM && !staged) {
                    e[i] = load1(ptr + r * stride + at_c);
                } else if constexpr (sizeof(T) == 2) {
                    uint16_t w;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(row + at_c * 2));
                    e[i] = __uint_as_float(uint32_t(w) << 16);
                } else {
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(e[i]) : "r"(row + at_c * 4));
                }
            }
#pragma unroll
            for (int i = 0; i < E / 2; ++i) v[i] = make_float2(e[2 * i], e[2 * i + 1]);
        } else {
            const int place = column<VEC, E, TEAM>(team, k, 0), own = place < width ? place : column<VEC, E, TEAM>(team, 0, 0);
            const int c = ZEROS ? place : own;
            Unit<T> u;
            if (!staged)
                u.w = *reinterpret_cast<const uint4 *>(ptr + r * stride + min(own, (width - 1) / VEC * VEC));
            else
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(u.w.x), "=r"(u.w.y), "=r"(u.w.z), "=r"(u.w.w)
                             : "r"(at + stage * step + c * int(sizeof(T))));
            u.get(v);
            if (c + VEC > width) {
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    if (c + 2 * i >= width) v[i].x = 0.0f;
                    if (c + 2 * i + 1 >= width) v[i].y = 0.0f;
                }
            }
        }
    }
};

// Chunk k of a row of an output.
template <class T, int VEC, int E, int TEAM>
__device__ __forceinline__ void store(const Team &team, T *row, int k, int width, const float2 (&v)[E / 2])
{
    if constexpr (VEC != 1) {
        const int c = column<VEC, E, TEAM>(team, k, 0);
        if (c + VEC <= width) {
            Unit<T> u;
            u.set(v);
            *reinterpret_cast<uint4 *>(row + c) = u.w;
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = column<VEC, E, TEAM>(team, k, i);
        if ((TEAM && (k * E + i + 1) * TEAM <= width) || c < width) store1(row + c, i & 1 ? v[i / 2].y : v[i / 2].x);
    }
}
template <class T>
__device__ __forceinline__ T *out_row(const RowsView &v, int64_t r)
{
    return static_cast<T *>(v.ptr) + r * v.stride;
}

// A thread's columns of a weight: ones without one, zeros past the width.
template <class T, int VEC, int E, int K, int TEAM>
__device__ __forceinline__ void weights(const void *w, int64_t at, const Team &team, int width, float2 (&v)[K][E / 2])
{
    const T *const from = static_cast<const T *>(w) + at;
    const bool whole = VEC != 1 && w && (reinterpret_cast<uintptr_t>(from) & 15u) == 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if constexpr (VEC != 1) {
            const int c = column<VEC, E, TEAM>(team, k, 0);
            if (whole && c + VEC <= width) {
                Unit<T> u;
                u.w = *reinterpret_cast<const uint4 *>(from + c);
                u.get(v[k]);
                continue;
            }
        }
        float e[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = column<VEC, E, TEAM>(team, k, i);
            e[i] = c >= width ? 0.0f : w ? load1(from + c) : 1.0f;
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i) v[k][i] = make_float2(e[2 * i], e[2 * i + 1]);
    }
}

// A weight of the block's, binary32 in shared memory, laid out so that a warp's loads of 16 bytes
// are neighbours: of chunks of eight columns the first halves come before the second ones.
template <int VEC, int E, int K, int TEAM>
struct Wide {
    uint32_t at;
    int chunks;  // of a row
    __host__ __device__ __forceinline__ static int size(int width)
    {
        return TEAM ? TEAM * E * K : VEC == 1 ? (width + 3) / 4 * 4 : (width + VEC - 1) / VEC * VEC;
    }
    __device__ __forceinline__ Wide(const float *p, int width)
        : at(uint32_t(__cvta_generic_to_shared(p))), chunks(VEC == 1 ? 0 : (width + VEC - 1) / VEC)
    {
    }
    __device__ __forceinline__ int index(int c) const
    {
        return VEC == 8 ? ((c % 8 / 4) * chunks + c / 8) * 4 + c % 4 : c;
    }
    __device__ __forceinline__ void get(const Team &team, int k, int width, float2 (&v)[E / 2]) const
    {
        if constexpr (VEC == 1) {
            float e[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = column<VEC, E, TEAM>(team, k, i);
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(e[i]) : "r"(at + (TEAM || c < width ? c : 0) * 4));
                if (!TEAM && c >= width) e[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < E / 2; ++i) v[i] = make_float2(e[2 * i], e[2 * i + 1]);
        } else {
            const int n = team.tid + k * team.threads, chunk = n < chunks ? n : 0;
#pragma unroll
            for (int h = 0; h < E / 4; ++h) {
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(v[2 * h].x), "=f"(v[2 * h].y), "=f"(v[2 * h + 1].x), "=f"(v[2 * h + 1].y)
                             : "r"(at + (h * chunks + chunk) * 16));
            }
            if (n >= chunks)  // a chunk that is none of the row's counts for nothing
#pragma unroll
                for (int i = 0; i < E / 2; ++i) v[i] = make_float2(0.0f, 0.0f);
        }
    }
};

// A chunk's sum of squares, of the columns that are the row's.
template <int VEC, int E, int TEAM>
__device__ __forceinline__ float squares(const Team &team, int k, int width, const float2 (&v)[E / 2])
{
    float2 s = pair(0.0f);
    if constexpr (VEC == 1 && !TEAM) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float x = i & 1 ? v[i / 2].y : v[i / 2].x;
            sum = column<VEC, E, TEAM>(team, k, i) < width ? fmaf(x, x, sum) : sum;
        }
        return sum;
    } else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) s = fma_f32x2(v[i], v[i], s);
        return TEAM || column<VEC, E, TEAM>(team, k, 0) < width ? total(s) : 0.0f;
    }
}

// Shared memory cleared, so that with TEAM there are zeros behind every row.
__device__ __forceinline__ void clear(char *p, int bytes)
{
    for (int i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16) *reinterpret_cast<uint4 *>(p + i) = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
}

// ALL: x_new, o and w_pre are there, and rows are staged.
template <class T, int VEC, int E, int K, int TEAM, bool ALL>
__global__ void __launch_bounds__(kMost, (kToSm<E * K, ALL>)) forward_kernel(BlockArgs a, int team_threads, Ring ring)
{
    __shared__ __align__(16) float sh[kTeams * 2 * kMost / 32];
    extern __shared__ __align__(16) char rows[];
    Team team(TEAM ? TEAM : team_threads);
    if (TEAM) clear(rows, team.count * 2 * ring.slot * ring.stages);
    clear_sums<kTeams * 2 * kMost / 32>(sh);
    const int width = a.width, stages = ring.stages > 0 ? ring.stages : 1;
    const bool staged = TEAM || ALL || ring.stages > 0, block = ALL || a.o.ptr, has_n = ALL || a.w_pre, has_x = ALL || a.x_new.ptr;
    const uint32_t mine = uint32_t(__cvta_generic_to_shared(rows)) + team.id * (2 * ring.slot * ring.stages);
    const Source<T, VEC, E, K, TEAM, false> x_in(a.x, mine, 0, ring, 2), o_in(a.o, mine, 1, ring, 2);
    const int64_t teams = int64_t(gridDim.x) * team.count, each = (a.rows + teams - 1) / teams;
    const int64_t lo = min((int64_t(blockIdx.x) * team.count + team.id) * each, a.rows), hi = min(lo + each, a.rows);
    const int64_t in_group = a.rows / a.groups;
    auto ask = [&](int64_t r, int stage) {
        if (staged && r < hi) {
            x_in.copy(team, r, stage, width);
            if (block) o_in.copy(team, r, stage, width);
        }
        commit_copies();
    };
    for (int i = 0; i < stages; ++i) ask(lo + i, i);
    float2 u[K][E / 2], w2[K][E / 2];
    weights<T, VEC, E, K, TEAM>(a.w_pre, 0, team, width, w2);
    int64_t next_group = lo;  // where u changes
    const float mean = 1.0f / float(width);
    int stage = 0;
    for (int64_t r = lo; r < hi; ++r) {
        if (r == next_group && block) {
            const int64_t g = r / in_group;
            float2 gate[K][E / 2];
            weights<T, VEC, E, K, TEAM>(a.w_post, 0, team, width, u);
            weights<T, VEC, E, K, TEAM>(a.gate, g * width, team, width, gate);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < E / 2; ++i) u[k][i] = mul_f32x2(u[k][i], gate[k][i]);
            next_group = (g + 1) * in_group;
        }
        wait_copies(stages - 1);
        if (VEC == 1) {
            x_in.close(team, r, stage, width);
            if (block) o_in.close(team, r, stage, width);
            team.sync();
        }
        float s[1] = {0.0f}, s1 = 1.0f, s2 = 1.0f;
        float2 y[K][E / 2];
        if (a.w_post) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float2 o[E / 2];
                o_in.get(team, r, stage, staged, k, width, o);
                s[0] += squares<VEC, E, TEAM>(team, k, width, o);
            }
            team.sum<1>(s, sh);
            s1 = rsqrtf(fmaf(s[0], mean, a.eps));
            s[0] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float2 o[E / 2];
            x_in.get(team, r, stage, staged, k, width, y[k]);
            if (block) o_in.get(team, r, stage, staged, k, width, o);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                y[k][i] = mul_f32x2(y[k][i], pair(a.res_scale));
                if (block) y[k][i] = fma_f32x2(mul_f32x2(u[k][i], pair(s1)), o[i], y[k][i]);
            }
            s[0] += squares<VEC, E, TEAM>(team, k, width, y[k]);
        }
        if (VEC == 1) team.sync();  // the row has been read
        ask(r + stages, stage);
        if (has_x)
#pragma unroll
            for (int k = 0; k < K; ++k) store<T, VEC, E, TEAM>(team, out_row<T>(a.x_new, r), k, width, y[k]);
        if (has_n) {
            team.sum<1>(s, sh);
            s2 = rsqrtf(fmaf(s[0], mean, a.eps));
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int i = 0; i < E / 2; ++i) y[k][i] = mul_f32x2(y[k][i], mul_f32x2(w2[k][i], pair(s2)));
                store<T, VEC, E, TEAM>(team, out_row<T>(a.n, r), k, width, y[k]);
            }
        }
        if (a.kept && team.tid == 0) {
            a.kept[r] = s1;
            a.kept[a.rows + r] = s2;
        }
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
    wait_copies(0);
}

// How the rows are shared out: `segments` blocks to each gate, a block's teams taking
// its rows in turn; or, with segments 0, whole gates to a team, in turn. A block that has all of a gate's
// rows finishes its gradient itself.
struct Shares {
    int segments;
    int64_t blocks, each;  // rows to a segment
};
inline Shares shares_of(int64_t rows, int64_t groups, int wave)
{
    Shares s;
    const int64_t in_group = rows / groups;
    if (groups >= 2 * wave && in_group < 16) {  // too few rows to a gate for a block's beginning and end
        s.segments = 0;
        s.blocks = wave;
        s.each = 0;
        return s;
    }
    // Blocks come in waves: of the numbers of segments that fill one to four waves, that for which the
    // rows of all waves are fewest. (16384 x 4096 in bf16, backward, 64 gates: three segments, a wave and a quarter,
    // 237 us, seven 190.)
    int64_t best = 0, least = 0;
    for (int waves = 1; waves <= 4; ++waves) {
        int64_t n = waves * wave / groups;
        n = n < 1 ? 1 : n > in_group ? in_group : n;
        const int64_t each = (in_group + n - 1) / n, blocks = groups * ((in_group + each - 1) / each);
        const int64_t cost = (blocks + wave - 1) / wave * (each + 2);  // a block's own beginning and end, in rows
        if (!best || cost < least) {
            best = n;
            least = cost;
        }
    }
    s.each = (in_group + best - 1) / best;
    s.segments = int((in_group + s.each - 1) / s.each);
    s.blocks = groups * s.segments;
    return s;
}

// A thread's sums over its columns, added up over the block's teams in their order: finish(column, sum).
template <int VEC, int E, int K, int TEAM, class F>
__device__ __forceinline__ void hand_in(const Team &team, const float2 (&v)[K][E / 2], float *sh, int width, F finish)
{
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = column<VEC, E, TEAM>(team, k, i);
            const float mine = i & 1 ? v[k][i / 2].y : v[k][i / 2].x;
            if (c >= width) continue;
            if (team.count == 1)
                finish(c, mine);
            else
                sh[team.id * width + c] = mine;
        }
    if (team.count == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < width; c += blockDim.x) {
        float s = sh[c];
        for (int t = 1; t < team.count; ++t) s += sh[t * width + c];
        finish(c, s);
    }
    __syncthreads();
}

// MANY: whole gates to a team (segments is 0), whose sums it finishes itself. ALL: every tensor of
// rows is there and staged, which leaves a third of the instructions out.
template <class T, int VEC, int E, int K, int TEAM, bool MANY, bool ALL>
__global__ void __launch_bounds__(kMost, (kToSm<E * K, ALL && VEC == 1>)) backward_kernel(BlockArgs a, int team_threads, Ring ring, Shares shares)
{
    __shared__ __align__(16) float sh[kTeams * 6 * kMost / 32];
    extern __shared__ __align__(16) char rows[];
    static_assert(!TEAM || (ALL && !MANY), "a known team has all of its rows");
    Team team(TEAM ? TEAM : team_threads);
    pdl_trigger();
    if (TEAM) clear(rows, team.count * 4 * ring.slot * ring.stages);
    clear_sums<kTeams * 6 * kMost / 32>(sh);
    const int width = a.width, stages = ring.stages > 0 ? ring.stages : 1;
    const bool staged = ALL || ring.stages > 0, block = ALL || a.o.ptr, has_n = ALL || a.w_pre, has_y = ALL || a.x_new.ptr,
               has_w1 = a.w_post != nullptr;
    const uint32_t mine = uint32_t(__cvta_generic_to_shared(rows)) + team.id * (4 * ring.slot * ring.stages);
    float *const wide = reinterpret_cast<float *>(rows + team.count * (4 * ring.slot * ring.stages));
    const Wide<VEC, E, K, TEAM> u_of(wide, width), w2_of(wide + Wide<VEC, E, K, TEAM>::size(width), width);
    using In = Source<T, VEC, E, K, TEAM, true>;
    const In x_in(a.x, mine, 0, ring, 4), o_in(a.o, mine, 1, ring, 4), dn_in(a.n, mine, 2, ring, 4), y_in(a.x_new, mine, 3, ring, 4);
    const int64_t in_group = a.rows / a.groups, group_step = int64_t(gridDim.x) * team.count;
    // The team's rows, one after another: of one gate's segment every count-th, or all of
    // every gate that is the team's.
    struct At {
        int64_t row, end, group;
    } now;
    if (MANY) {
        now.group = int64_t(blockIdx.x) * team.count + team.id;
        now.row = now.group * in_group;
        now.end = now.group < a.groups ? now.row + in_group : now.row;
    } else {
        now.group = blockIdx.x / shares.segments;
        const int64_t lo = (blockIdx.x - now.group * shares.segments) * shares.each;
        now.end = now.group * in_group + min(lo + shares.each, in_group);
        now.row = now.group * in_group + lo + team.id;
    }
    auto advance = [&](At &p) {
        p.row += MANY ? 1 : team.count;
        if (MANY && p.row >= p.end && p.group < a.groups) {
            p.group += group_step;
            p.row = p.group * in_group;
            p.end = p.group < a.groups ? p.row + in_group : p.row;
        }
    };
    At asked = now;
    auto ask = [&](int stage) {
        if (staged && asked.row < asked.end) {
            x_in.copy(team, asked.row, stage, width);
            if (block) o_in.copy(team, asked.row, stage, width);
            if (has_n) dn_in.copy(team, asked.row, stage, width);
            if (has_y) y_in.copy(team, asked.row, stage, width);
            advance(asked);
        }
        commit_copies();
    };
    x_in.open(team, ring.stages, width);
    o_in.open(team, ring.stages, width);
    dn_in.open(team, ring.stages, width);
    y_in.open(team, ring.stages, width);
    for (int i = 0; i < stages; ++i) ask(i);
    constexpr int R = MANY ? K : 1;  // what a gate's change or end concerns is a team's own, in registers
    float2 q[K][E / 2], p[K][E / 2], dw1[R][E / 2], u_here[R][E / 2], w2_here[R][E / 2];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < E / 2; ++i) q[k][i] = p[k][i] = pair(0.0f);
    if constexpr (MANY) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < E / 2; ++i) dw1[k][i] = pair(0.0f);
        weights<T, VEC, E, K, TEAM>(a.w_pre, 0, team, width, w2_here);
    } else {
        // gate w1 and w2 are the block's: in registers they cost a team its place beside another
        for (int c = threadIdx.x; c < Wide<VEC, E, K, TEAM>::size(width); c += blockDim.x) {
            const bool in = c < width;
            const float w1 = in && a.w_post ? load1(static_cast<const T *>(a.w_post) + c) : 1.0f;
            const float g = in && a.gate ? load1(static_cast<const T *>(a.gate) + now.group * width + c) : 1.0f;
            wide[u_of.index(c)] = in ? w1 * g : 0.0f;
            const float w2 = in && a.w_pre ? load1(static_cast<const T *>(a.w_pre) + c) : 1.0f;
            (wide + Wide<VEC, E, K, TEAM>::size(width))[w2_of.index(c)] = in ? w2 : 0.0f;
        }
        __syncthreads();
    }
    auto u_at = [&](int k, float2 (&v)[E / 2]) {
        if constexpr (MANY) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) v[i] = u_here[k][i];
        } else {
            u_of.get(team, k, width, v);
        }
    };
    auto w2_at = [&](int k, float2 (&v)[E / 2]) {
        if constexpr (MANY) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) v[i] = w2_here[k][i];
        } else {
            w2_of.get(team, k, width, v);
        }
    };
    const float mean = 1.0f / float(width);
    float s1 = now.row < now.end ? a.kept[now.row] : 0.0f, s2 = now.row < now.end ? a.kept[a.rows + now.row] : 0.0f;
    int64_t of = -1;  // the gate that u is of
    int stage = 0;
    while (now.row < now.end) {
        if constexpr (MANY) {
            if (now.group != of && block) {
                float2 gate[K][E / 2];
                weights<T, VEC, E, K, TEAM>(a.w_post, 0, team, width, u_here);
                weights<T, VEC, E, K, TEAM>(a.gate, now.group * width, team, width, gate);
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) u_here[k][i] = mul_f32x2(u_here[k][i], gate[k][i]);
            }
        }
        of = now.group;
        const int64_t r = now.row;
        advance(now);
        // of the row after this one, before they are needed
        const float next1 = now.row < now.end ? a.kept[now.row] : 0.0f;
        const float next2 = now.row < now.end ? a.kept[a.rows + now.row] : 0.0f;
        wait_copies(stages - 1);
        if (VEC == 1) {
            if (TEAM) {
                x_in.close(team, r, stage, width);
                o_in.close(team, r, stage, width);
                dn_in.close(team, r, stage, width);
                y_in.close(team, r, stage, width);
            }
            team.sync();
        }
        // x' s2, o s1, dn and y of a chunk
        auto chunk = [&](int k, float2 (&xh)[E / 2], float2 (&oh)[E / 2], float2 (&dn)[E / 2], float2 (&y)[E / 2],
                         float2 (&u)[E / 2], float2 (&w2)[E / 2]) {
            if (block) u_at(k, u);
            if (has_n) w2_at(k, w2);
            x_in.get(team, r, stage, staged, k, width, xh);
            if (!ALL)
#pragma unroll
                for (int i = 0; i < E / 2; ++i) oh[i] = dn[i] = y[i] = pair(0.0f);
            if (!block)
#pragma unroll
                for (int i = 0; i < E / 2; ++i) u[i] = pair(0.0f);
            if (!has_n)
#pragma unroll
                for (int i = 0; i < E / 2; ++i) w2[i] = pair(0.0f);
            if (block) o_in.get(team, r, stage, staged, k, width, oh);
            if (has_n) dn_in.get(team, r, stage, staged, k, width, dn);
            if (has_y) y_in.get(team, r, stage, staged, k, width, y);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                xh[i] = mul_f32x2(xh[i], pair(a.res_scale * s2));
                if (block) {
                    oh[i] = mul_f32x2(oh[i], pair(s1));
                    xh[i] = fma_f32x2(mul_f32x2(u[i], pair(s2)), oh[i], xh[i]);
                }
            }
        };
        float s[3] = {0.0f, 0.0f, 0.0f};
        if (has_n || has_w1) {
            float2 sum[3] = {pair(0.0f), pair(0.0f), pair(0.0f)};
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float2 xh[E / 2], oh[E / 2], dn[E / 2], y[E / 2], u[E / 2], w2[E / 2];
                chunk(k, xh, oh, dn, y, u, w2);
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    q[k][i] = fma_f32x2(dn[i], xh[i], q[k][i]);
                    const float2 e = mul_f32x2(dn[i], w2[i]), uo = mul_f32x2(u[i], oh[i]);
                    sum[0] = fma_f32x2(e, xh[i], sum[0]);
                    if (ALL || has_w1) {
                        sum[1] = fma_f32x2(uo, fma_f32x2(pair(s2), e, y[i]), sum[1]);
                        sum[2] = fma_f32x2(uo, xh[i], sum[2]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 3; ++i) s[i] = total(sum[i]);
            team.sum<3>(s, sh);
        }
        const float c2 = has_n ? s[0] * mean : 0.0f, c1 = has_w1 ? (s[1] - s2 * c2 * s[2]) * mean : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float2 xh[E / 2], oh[E / 2], dn[E / 2], y[E / 2], u[E / 2], w2[E / 2];
            chunk(k, xh, oh, dn, y, u, w2);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 d = fma_f32x2(pair(s2), fma_f32x2(xh[i], pair(-c2), mul_f32x2(dn[i], w2[i])), y[i]);
                p[k][i] = fma_f32x2(d, oh[i], p[k][i]);
                xh[i] = mul_f32x2(d, pair(a.res_scale));
                if (block) oh[i] = mul_f32x2(pair(s1), fma_f32x2(oh[i], pair(-c1), mul_f32x2(u[i], d)));
            }
            store<T, VEC, E, TEAM>(team, out_row<T>(a.dx, r), k, width, xh);
            if (block) store<T, VEC, E, TEAM>(team, out_row<T>(a.d_o, r), k, width, oh);
        }
        if (VEC == 1) team.sync();  // the row has been read
        ask(stage);
        stage = stage + 1 == stages ? 0 : stage + 1;
        s1 = next1;
        s2 = next2;
        if constexpr (MANY) {
            if (now.row < now.end && now.group == of) continue;
            float2 w[K][E / 2], gate[K][E / 2];
            weights<T, VEC, E, K, TEAM>(a.w_post, 0, team, width, w);
            weights<T, VEC, E, K, TEAM>(a.gate, of * width, team, width, gate);
            T *const dgate = static_cast<T *>(a.dgate) + of * width;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    dw1[k][i] = fma_f32x2(gate[k][i], p[k][i], dw1[k][i]);
                    w[k][i] = mul_f32x2(w[k][i], p[k][i]);
                    p[k][i] = pair(0.0f);
                    const int c0 = column<VEC, E, TEAM>(team, k, 2 * i), c1 = column<VEC, E, TEAM>(team, k, 2 * i + 1);
                    if (c0 < width) store1(dgate + c0, w[k][i].x);
                    if (c1 < width) store1(dgate + c1, w[k][i].y);
                }
        }
    }
    wait_copies(0);
    __syncthreads();  // the rows' memory is free
    float *const joint = reinterpret_cast<float *>(rows);
    float *const q_out = a.work + int64_t(blockIdx.x) * width, *const p_out = q_out + shares.blocks * width;
    if (a.w_pre) hand_in<VEC, E, K, TEAM>(team, q, joint, width, [&](int c, float sum) { q_out[c] = sum; });
    if constexpr (MANY) {
        if (a.w_post) hand_in<VEC, E, K, TEAM>(team, dw1, joint, width, [&](int c, float sum) { p_out[c] = sum; });
    } else {
        if (a.gate && shares.segments == 1) {
            const int64_t at = (blockIdx.x / shares.segments) * int64_t(width);
            hand_in<VEC, E, K, TEAM>(team, p, joint, width, [&](int c, float sum) {
                const float w1 = a.w_post ? load1(static_cast<const T *>(a.w_post) + c) : 1.0f;
                store1(static_cast<T *>(a.dgate) + at + c, w1 * sum);
                p_out[c] = load1(static_cast<const T *>(a.gate) + at + c) * sum;
            });
        } else if (a.w_post || a.gate) {
            hand_in<VEC, E, K, TEAM>(team, p, joint, width, [&](int c, float sum) { p_out[c] = sum; });
        }
    }
}

// Every step-th of `count` rows from `first` on, eight loads at a time.
__device__ __forceinline__ float sum_rows(const float *p, int width, int first, int count, int step)
{
    float s = 0.0f;
    for (int b = first; b < count; b += 8 * step) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p[int64_t(min(b + i * step, count - 1)) * width];
#pragma unroll
        for (int i = 0; i < 8; ++i) s += b + i * step < count ? v[i] : 0.0f;
    }
    return s;
}

// A block to 32 columns of dw2 (blockIdx.y 0), or of dw1 and dgate: a warp adds up every 32nd block's sums, then
// they are added up.
template <class T>
__global__ void __launch_bounds__(1024) weights_kernel(BlockArgs a, Shares shares)
{
    __shared__ float sh[32][33];
    pdl_wait();
    const int lane = threadIdx.x % 32, row = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    const bool there = c < a.width;
    const int blocks = int(shares.blocks);
    auto total = [&](float v) {  // in the first warp
        sh[row][lane] = v;
        __syncthreads();
        float s = 0.0f;
        if (row == 0)
#pragma unroll
            for (int i = 0; i < 32; ++i) s += sh[i][lane];
        return s;
    };
    if (blockIdx.y == 0) {
        if (!a.w_pre) return;
        const float s = total(there ? sum_rows(a.work + c, a.width, row, blocks, 32) : 0.0f);
        if (there && row == 0) store1(static_cast<T *>(a.dw_pre) + c, s);
        return;
    }
    const bool done = !a.gate || shares.segments <= 1;  // the sums are dw1's own
    if (!a.w_post && done) return;
    const float *const sums = a.work + shares.blocks * a.width;
    if (done || a.groups == 1) {
        const float s = total(there ? sum_rows(sums + c, a.width, row, blocks, 32) : 0.0f);
        if (!there || row) return;
        if (done) {
            store1(static_cast<T *>(a.dw_post) + c, s);
            return;
        }
        store1(static_cast<T *>(a.dgate) + c, a.w_post ? s * load1(static_cast<const T *>(a.w_post) + c) : s);
        if (a.w_post) store1(static_cast<T *>(a.dw_post) + c, s * load1(static_cast<const T *>(a.gate) + c));
        return;
    }
    const float w = there && a.w_post ? load1(static_cast<const T *>(a.w_post) + c) : 1.0f;
    float dw1 = 0.0f;
    // few gates: several warps to each
    const int share = a.groups <= 16 ? 32 / int(a.groups) : 1, part = row % share;
    for (int64_t g = row / share; g < a.groups; g += 32 / share) {
        float s = there ? sum_rows(sums + g * shares.segments * a.width + c, a.width, part, shares.segments, share) : 0.0f;
        if (share > 1) {  // once around: the first 32 / share gates are all
            sh[row][lane] = s;
            asm volatile("bar.sync 1, %0;" ::"r"(int(a.groups) * share * 32) : "memory");
            s = 0.0f;
            for (int i = 0; i < share; ++i) s += sh[row - part + i][lane];
        }
        if (!there || part) continue;
        store1(static_cast<T *>(a.dgate) + g * a.width + c, w * s);
        dw1 = fmaf(s, load1(static_cast<const T *>(a.gate) + g * a.width + c), dw1);
    }
    __syncthreads();
    dw1 = total(dw1);
    if (a.w_post && there && row == 0) store1(static_cast<T *>(a.dw_post) + c, dw1);
}

inline bool whole(const RowsView &v, int size)
{
    return (reinterpret_cast<uintptr_t>(v.ptr) | uintptr_t(v.stride * size)) % 16 == 0;
}

// Every row of every tensor starts on 16 bytes.
bool in_units(const BlockArgs &a, bool backward)
{
    const int size = a.dtype == ZG_DTYPE_BF16 ? 2 : 4;
    const bool ok = whole(a.x, size) && whole(a.o, size) && whole(a.x_new, size) && whole(a.n, size);
    return ok && (!backward || (whole(a.dx, size) && whole(a.d_o, size)));
}

// Threads of a team, teams of a block (an SM has one), and the rows that its shared memory holds.
struct Shape {
    int team, teams;
    Ring ring;
    size_t bytes;
};
// `places`: what a thread has of an aligned row in shared memory, at least.
Shape shape_of(const BlockArgs &a, int vec, int columns, int team, int tensors, bool wide, int places, int to_sm)
{
    const int size = a.dtype == ZG_DTYPE_BF16 ? 2 : 4;
    Shape s;
    s.team = team ? team : ((a.width + columns - 1) / columns + 31) / 32 * 32;
    s.teams = kMost / s.team;
    if (s.teams > kTeams) s.teams = kTeams;
    const int64_t blocks = kBlocks * to_sm;
    if (a.rows < s.teams * blocks) s.teams = int((a.rows + blocks - 1) / blocks);  // few rows: all SMs
    // columns of a stage
    const int held = team ? team * columns : vec != 1 && a.width < s.team * places ? s.team * places : a.width;
    s.ring.slot = (held * size + (vec == 1 ? 48 : 0) + 15) / 16 * 16;  // a head, and two units that are cleared
    const size_t row = size_t(s.teams) * tensors * s.ring.slot;
    const size_t beside = wide ? size_t((team ? held : a.width) + 7) / 8 * 64 : 0;  // two weights in binary32
    s.ring.stages = beside < size_t(kMemory / to_sm) ? int((size_t(kMemory / to_sm) - (to_sm - 1) * 4096 - beside) / row) : 0;
    if (s.ring.stages > kStages) s.ring.stages = kStages;
    s.bytes = row * s.ring.stages + beside;
    const size_t joint = s.teams > 1 ? size_t(s.teams) * a.width * 4 : 0;  // of the weights' sums
    if (s.bytes < joint) s.bytes = joint;
    return s;
}

// The most shared memory that any shape takes is allowed once for each kernel and device.
template <class F>
cudaError_t allow(F *kernel, std::atomic<uint64_t> &devices)
{
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (devices.load(std::memory_order_acquire) & bit) return cudaSuccess;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMemory)) return e;
    devices.fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
}

template <class T, int VEC, int E, int K, int TEAM>
cudaError_t forward(const BlockArgs &a, cudaStream_t st)
{
    const bool every = a.o.ptr && a.x_new.ptr && a.w_pre;
    int to_sm = kToSm<E * K, true>;
    Shape s = shape_of(a, VEC, E * K, TEAM, 2, false, E, to_sm);
    const bool all = every && s.ring.stages > 0;
    if (!all) s = shape_of(a, VEC, E * K, TEAM, 2, false, E, to_sm = 1);
    auto *kernel = all ? &forward_kernel<T, VEC, E, K, TEAM, true> : &forward_kernel<T, VEC, E, K, TEAM, false>;
    static std::atomic<uint64_t> allowed[2];
    if (cudaError_t e = allow(kernel, allowed[all])) return e;
    const int64_t want = (a.rows + s.teams - 1) / s.teams;
    kernel<<<unsigned(want < kBlocks * to_sm ? want : kBlocks * to_sm), s.team * s.teams, s.bytes, st>>>(a, s.team, s.ring);
    return cudaGetLastError();
}

template <class T, int VEC, int E, int K, int TEAM>
cudaError_t backward(const BlockArgs &a, cudaStream_t st)
{
    constexpr int kMany = kToSm<E * K, VEC == 1>;
    static std::atomic<uint64_t> allowed[3];
    auto *kernel = &backward_kernel<T, VEC, E, K, 0, false, false>;
    int which = 0;
    Shares shares = shares_of(a.rows, a.groups, kBlocks * kMany);
    Shape s = shape_of(a, VEC, E * K, TEAM, 4, true, E * K, kMany);
    if (a.o.ptr && a.n.ptr && a.x_new.ptr && shares.segments && s.ring.stages > 0) {
        kernel = &backward_kernel<T, VEC, E, K, TEAM, false, true>;
        which = 2;
    } else {
        shares = shares_of(a.rows, a.groups, kBlocks);
        s = shape_of(a, VEC, E * K, 0, 4, shares.segments > 0, E * K, 1);
        if (!shares.segments) {
            kernel = &backward_kernel<T, VEC, E, K, 0, true, false>;
            which = 1;
        }
    }
    if (shares.blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    if (cudaError_t e = allow(kernel, allowed[which])) return e;
    kernel<<<unsigned(shares.blocks), s.team * s.teams, s.bytes, st>>>(a, s.team, s.ring, shares);
    if (cudaError_t e = cudaGetLastError()) return e;
    if (!a.w_pre && !a.w_post && !(a.gate && shares.segments > 1)) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((a.width + 31) / 32), 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = ZG_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, &weights_kernel<T>, a, shares);
}

template <class T, bool BACK>
cudaError_t of_type(const BlockArgs &a, cudaStream_t st)
{
    // chunks of E columns, K of them to a thread, and at most MOST threads to a row (backward, aligned rows, 8 columns to
    // a thread against 16, in us with a graph's replay: in bf16 8192 x 768 32 and 36, 32768 x 768 79 and 93, 32768 x 1024
    // 95 and 85, 32768 x 2048 181 and 155; in binary32 8192 x 768 34 and 42, 32768 x 768 100 and 114, 32768 x 1024 132 and
    // 130, 16384 x 2048 132 both)
#define ZG_CASE(MOST, VEC, E, K, TEAM) \
    if (a.width <= (E) * (K) * (MOST)) return BACK ? backward<T, VEC, E, K, TEAM>(a, st) : forward<T, VEC, E, K, TEAM>(a, st);
    constexpr int N = Unit<T>::kN;
    if (in_units(a, BACK)) {
        ZG_CASE(BACK ? 96 : 256, N, N, 8 / N, 0) ZG_CASE(kMost, N, N, 16 / N, 0) ZG_CASE(kMost, N, N, 32 / N, 0)
    } else {
        ZG_CASE(64, 1, 8, 1, 64) ZG_CASE(128, 1, 8, 1, 128) ZG_CASE(256, 1, 8, 1, 256) ZG_CASE(512, 1, 8, 1, 512)
        ZG_CASE(kMost, 1, 8, 2, 512) ZG_CASE(kMost, 1, 8, 4, 0)
    }
#undef ZG_CASE
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace zg
