// The norms before and after a block, with its gate and the residual's scale.
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
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

constexpr int kMost = 512;     // threads of a block
constexpr int kBlocks = 304;   // blocks that share the rows of the backward pass

// VEC neighbouring elements, `n` of which are there.
template <class T, int VEC>
__device__ __forceinline__ void load(const T *p, int n, float (&v)[VEC])
{
    if constexpr (VEC == 1) {
        v[0] = n > 0 ? load1(p) : 0.0f;
    } else {
        if (n >= VEC) {
            Unit<T> u;
            u.w = *reinterpret_cast<const uint4 *>(p);
            float2 f[VEC / 2];
            u.get(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = i & 1 ? f[i / 2].y : f[i / 2].x;
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = i < n ? load1(p + i) : 0.0f;
        }
    }
}
template <class T, int VEC>
__device__ __forceinline__ void store(T *p, int n, const float (&v)[VEC])
{
    if constexpr (VEC == 1) {
        if (n > 0) store1(p, v[0]);
    } else {
        if (n >= VEC) {
            float2 f[VEC / 2];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) f[i] = make_float2(v[2 * i], v[2 * i + 1]);
            Unit<T> u;
            u.set(f);
            *reinterpret_cast<uint4 *>(p) = u.w;
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (i < n) store1(p + i, v[i]);
        }
    }
}

// The threads that share a row: whole warps of a block.
struct Team {
    int id, count;       // of the block's teams
    int tid, threads;    // of the team's threads
    int parity = 0;
    __device__ __forceinline__ Team(int team_threads)
    {
        threads = team_threads;
        count = blockDim.x / team_threads;
        id = threadIdx.x / team_threads;
        tid = threadIdx.x - id * team_threads;
    }
    // Sums over the team, the same in all of its threads. Two buffers, so that one
    // barrier is enough: nobody is two sums ahead of another.
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N], float *sh)
    {
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (threads == 32) return;
        float *const mine = sh + parity * (kMost / 32 * N) + id * (threads / 32) * N;
        parity ^= 1;
        if (tid % 32 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) mine[tid / 32 * N + i] = v[i];
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
        for (int w = 0; w < threads / 32; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += mine[w * N + i];
    }
};

template <class T>
__device__ __forceinline__ const T *row_of(const RowsView &v, int64_t r)
{
    return static_cast<const T *>(v.ptr) + r * v.stride;
}
template <class T>
__device__ __forceinline__ T *out_row(const RowsView &v, int64_t r)
{
    return static_cast<T *>(v.ptr) + r * v.stride;
}
// A weight's unit at column c, or ones.
template <class T, int VEC>
__device__ __forceinline__ void weight(const void *w, int64_t at, int n, float (&v)[VEC])
{
    if (w) {
        load<T, VEC>(static_cast<const T *>(w) + at, n, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 1.0f;
}

template <class T, int VEC, int K>
__global__ void __launch_bounds__(kMost) forward_kernel(BlockArgs a, int team_threads)
{
    __shared__ float sh[2 * kMost / 32];
    Team team(team_threads);
    const int64_t r = int64_t(blockIdx.x) * team.count + team.id;
    if (r >= a.rows) return;
    const int64_t group = r / (a.rows / a.groups);
    const int width = a.width;
    float x[K][VEC], o[K][VEC];
    float s[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (team.tid + k * team.threads) * VEC;
        load<T, VEC>(row_of<T>(a.x, r) + c, width - c, x[k]);
        if (!a.o.ptr) continue;
        load<T, VEC>(row_of<T>(a.o, r) + c, width - c, o[k]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[0] = fmaf(o[k][i], o[k][i], s[0]);
    }
    float s1 = 1.0f;
    if (a.w_post) {
        team.sum<1>(s, sh);
        s1 = 1.0f / sqrtf(s[0] / float(width) + a.eps);
    }
    s[0] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (team.tid + k * team.threads) * VEC, n = width - c;
        float w[VEC], g[VEC];
        if (a.o.ptr) {
            weight<T, VEC>(a.w_post, c, n, w);
            weight<T, VEC>(a.gate, group * width + c, n, g);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            x[k][i] *= a.res_scale;
            if (a.o.ptr) x[k][i] = i < n ? fmaf(g[i] * w[i], o[k][i] * s1, x[k][i]) : 0.0f;
            s[0] = fmaf(x[k][i], x[k][i], s[0]);
        }
        if (a.x_new.ptr) store<T, VEC>(out_row<T>(a.x_new, r) + c, n, x[k]);
    }
    float s2 = 1.0f;
    if (a.w_pre) {
        team.sum<1>(s, sh);
        s2 = 1.0f / sqrtf(s[0] / float(width) + a.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (team.tid + k * team.threads) * VEC, n = width - c;
            float w[VEC];
            weight<T, VEC>(a.w_pre, c, n, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[k][i] *= s2 * w[i];
            store<T, VEC>(out_row<T>(a.n, r) + c, n, x[k]);
        }
    }
    if (a.kept && team.tid == 0) {
        a.kept[r] = s1;
        a.kept[a.rows + r] = s2;
    }
}

// How the rows are shared out: `segments` blocks to each gate, a block's teams taking
// its rows in turn; or, with segments 0, whole gates to a team, in turn.
struct Shares {
    int segments;
    int64_t blocks, each;  // rows to a segment
};
__host__ __device__ inline Shares shares_of(int64_t rows, int64_t groups)
{
    Shares s;
    if (groups >= 2 * kBlocks) {
        s.segments = 0;
        s.blocks = kBlocks;
        s.each = 0;
        return s;
    }
    const int64_t in_group = rows / groups;
    int64_t n = (kBlocks + groups - 1) / groups;
    if (n > in_group) n = in_group;
    s.each = (in_group + n - 1) / n;
    s.segments = int((in_group + s.each - 1) / s.each);
    s.blocks = groups * s.segments;
    return s;
}

// A thread's sums over its columns, added up over the block's teams in their order.
template <int VEC, int K>
__device__ __forceinline__ void hand_in(const Team &team, float (&v)[K][VEC], float *sh, float *out, int width)
{
    for (int t = 0; t < team.count; ++t) {
        if (team.id == t) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int c = (team.tid + k * team.threads) * VEC + i;
                    if (c >= width) continue;
                    const float sum = t ? sh[c] + v[k][i] : v[k][i];
                    if (t == team.count - 1)
                        out[c] = sum;
                    else
                        sh[c] = sum;
                }
        }
        __syncthreads();
    }
}

template <class T, int VEC, int K>
__global__ void __launch_bounds__(kMost) backward_kernel(BlockArgs a, int team_threads, Shares shares)
{
    __shared__ float sh[6 * kMost / 32];
    extern __shared__ float joint[];
    Team team(team_threads);
    const int width = a.width;
    const int64_t in_group = a.rows / a.groups;
    float q[K][VEC], p[K][VEC], dw1[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) q[k][i] = p[k][i] = dw1[k][i] = 0.0f;

    auto one_row = [&](int64_t r, int64_t group) {
        float xh[K][VEC], oh[K][VEC], e[K][VEC], y[K][VEC];
        const float s1 = a.kept[r], s2 = a.kept[a.rows + r];
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (team.tid + k * team.threads) * VEC, n = width - c;
            float u[VEC], w[VEC], dn[VEC];
            load<T, VEC>(row_of<T>(a.x, r) + c, n, xh[k]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) oh[k][i] = y[k][i] = e[k][i] = 0.0f;
            if (a.o.ptr) load<T, VEC>(row_of<T>(a.o, r) + c, n, oh[k]);
            if (a.x_new.ptr) load<T, VEC>(row_of<T>(a.x_new, r) + c, n, y[k]);
            weight<T, VEC>(a.w_post, c, n, u);
            weight<T, VEC>(a.gate, group * width + c, n, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                u[i] *= w[i];
                oh[k][i] *= s1;
                xh[k][i] = fmaf(u[i], oh[k][i], a.res_scale * xh[k][i]) * s2;
            }
            if (a.w_pre) {
                load<T, VEC>(row_of<T>(a.n, r) + c, n, dn);
                weight<T, VEC>(a.w_pre, c, n, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    q[k][i] = fmaf(dn[i], xh[k][i], q[k][i]);
                    e[k][i] = dn[i] * w[i];
                    s[0] = fmaf(e[k][i], xh[k][i], s[0]);
                }
            }
            if (a.w_post)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float uo = u[i] * oh[k][i];
                    s[1] = fmaf(uo, fmaf(s2, e[k][i], y[k][i]), s[1]);
                    s[2] = fmaf(uo, xh[k][i], s[2]);
                }
        }
        team.sum<3>(s, sh);
        const float mean = 1.0f / float(width), c2 = a.w_pre ? s[0] * mean : 0.0f;
        const float c1 = a.w_post ? (s[1] - s2 * c2 * s[2]) * mean : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (team.tid + k * team.threads) * VEC, n = width - c;
            float u[VEC], w[VEC], dx[VEC];
            weight<T, VEC>(a.w_post, c, n, u);
            weight<T, VEC>(a.gate, group * width + c, n, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = a.w_pre ? fmaf(s2, fmaf(-xh[k][i], c2, e[k][i]), y[k][i]) : y[k][i];
                p[k][i] = fmaf(d, oh[k][i], p[k][i]);
                dx[i] = a.res_scale * d;
                e[k][i] = s1 * fmaf(u[i] * w[i], d, -oh[k][i] * c1);
            }
            store<T, VEC>(out_row<T>(a.dx, r) + c, n, dx);
            if (a.o.ptr) store<T, VEC>(out_row<T>(a.d_o, r) + c, n, e[k]);
        }
    };

    if (shares.segments) {
        const int64_t group = blockIdx.x / shares.segments;
        const int64_t lo = (blockIdx.x - group * shares.segments) * shares.each;
        const int64_t hi = min(lo + shares.each, in_group);
        for (int64_t i = lo + team.id; i < hi; i += team.count) one_row(group * in_group + i, group);
    } else {
        for (int64_t g = int64_t(blockIdx.x) * team.count + team.id; g < a.groups; g += int64_t(gridDim.x) * team.count) {
            for (int64_t i = 0; i < in_group; ++i) one_row(g * in_group + i, g);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (team.tid + k * team.threads) * VEC, n = width - c;
                float w[VEC], gate[VEC];
                weight<T, VEC>(a.w_post, c, n, w);
                weight<T, VEC>(a.gate, g * width + c, n, gate);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    dw1[k][i] = fmaf(gate[i], p[k][i], dw1[k][i]);
                    w[i] *= p[k][i];
                    p[k][i] = 0.0f;
                }
                if (a.dgate) store<T, VEC>(static_cast<T *>(a.dgate) + g * width + c, n, w);
            }
        }
    }
    if (a.w_pre) hand_in<VEC, K>(team, q, joint, a.work + int64_t(blockIdx.x) * width, width);
    if (a.w_post || (a.gate && shares.segments))
        hand_in<VEC, K>(team, shares.segments ? p : dw1, joint, a.work + (shares.blocks + blockIdx.x) * width, width);
}

// The sums of the weights' gradients over the blocks.
template <class T>
__global__ void __launch_bounds__(512) weights_kernel(BlockArgs a, Shares shares)
{
    __shared__ float sh[16][33];
    const int lane = threadIdx.x % 32, row = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    const bool there = c < a.width;
    auto total = [&](float v) {
        sh[row][lane] = v;
        __syncthreads();
        float s = 0.0f;
        for (int i = 0; i < 16; ++i) s += sh[i][lane];
        __syncthreads();
        return s;
    };
    if (a.w_pre) {
        float s = 0.0f;
        if (there)
            for (int64_t b = row; b < shares.blocks; b += 16) s += a.work[b * a.width + c];
        s = total(s);
        if (there && row == 0) store1(static_cast<T *>(a.dw_pre) + c, s);
    }
    const float *const sums = a.work + shares.blocks * a.width;
    if (!shares.segments || !a.gate) {
        if (!a.w_post) return;
        float s = 0.0f;
        if (there)
            for (int64_t b = row; b < shares.blocks; b += 16) s += sums[b * a.width + c];
        s = total(s);
        if (there && row == 0) store1(static_cast<T *>(a.dw_post) + c, s);
        return;
    }
    const float w = there && a.w_post ? load1(static_cast<const T *>(a.w_post) + c) : 1.0f;
    float dw1 = 0.0f;
    if (a.groups == 1) {
        float s = 0.0f;
        if (there)
            for (int64_t b = row; b < shares.blocks; b += 16) s += sums[b * a.width + c];
        s = total(s);
        if (there && row == 0) {
            store1(static_cast<T *>(a.dgate) + c, w * s);
            if (a.w_post) store1(static_cast<T *>(a.dw_post) + c, s * load1(static_cast<const T *>(a.gate) + c));
        }
        return;
    }
    for (int64_t g = row; there && g < a.groups; g += 16) {
        float s = 0.0f;
        for (int i = 0; i < shares.segments; ++i) s += sums[(g * shares.segments + i) * a.width + c];
        store1(static_cast<T *>(a.dgate) + g * a.width + c, w * s);
        dw1 = fmaf(s, load1(static_cast<const T *>(a.gate) + g * a.width + c), dw1);
    }
    dw1 = total(dw1);
    if (a.w_post && there && row == 0) store1(static_cast<T *>(a.dw_post) + c, dw1);
}

bool whole(const RowsView &v, int size)
{
    return (reinterpret_cast<uintptr_t>(v.ptr) | uintptr_t(v.stride * size)) % 16 == 0;
}
bool aligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Every row of every tensor starts on 16 bytes.
bool in_units(const BlockArgs &a, bool backward)
{
    const int size = a.dtype == ZG_DTYPE_BF16 ? 2 : 4;
    bool ok = whole(a.x, size) && whole(a.o, size) && whole(a.x_new, size) && whole(a.n, size) && aligned(a.w_post) &&
              aligned(a.w_pre) && aligned(a.gate) && (a.groups == 1 || a.width * size % 16 == 0);
    if (backward) ok = ok && whole(a.dx, size) && whole(a.d_o, size) && aligned(a.dgate);
    return ok;
}

int team_of(int width, int vec, int k) { return ((width + vec * k - 1) / (vec * k) + 31) / 32 * 32; }

template <class T, int VEC, int K>
cudaError_t forward(const BlockArgs &a, cudaStream_t st)
{
    const int team = team_of(a.width, VEC, K), teams = team >= 128 ? 1 : 128 / team;
    const int64_t blocks = (a.rows + teams - 1) / teams;
    if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
    forward_kernel<T, VEC, K><<<unsigned(blocks), team * teams, 0, st>>>(a, team);
    return cudaGetLastError();
}

template <class T, int VEC, int K>
cudaError_t backward(const BlockArgs &a, cudaStream_t st)
{
    const int team = team_of(a.width, VEC, K), teams = kMost / team > 8 ? 8 : kMost / team;
    const Shares s = shares_of(a.rows, a.groups);
    const size_t joint = teams > 1 ? size_t(a.width) * 4 : 0;
    backward_kernel<T, VEC, K><<<unsigned(s.blocks), team * teams, joint, st>>>(a, team, s);
    if (cudaError_t e = cudaGetLastError()) return e;
    if (a.w_pre || a.w_post || (a.gate && s.segments)) weights_kernel<T><<<(a.width + 31) / 32, 512, 0, st>>>(a, s);
    return cudaGetLastError();
}

template <class T, bool BACK>
cudaError_t of_type(const BlockArgs &a, cudaStream_t st)
{
#define ZG_CASE(VEC, K) \
    if (a.width <= (VEC) * (K) * kMost) return BACK ? backward<T, VEC, K>(a, st) : forward<T, VEC, K>(a, st);
    constexpr int N = Unit<T>::kN;
    if (in_units(a, BACK)) {
        ZG_CASE(N, 1) ZG_CASE(N, 2) ZG_CASE(N, 4) ZG_CASE(N, 8)
    } else {
        ZG_CASE(1, 2) ZG_CASE(1, 8) ZG_CASE(1, 32)
    }
#undef ZG_CASE
    return cudaErrorInvalidValue;
}

}  // namespace

int64_t block_norm_workspace(int64_t rows, int64_t width, int64_t groups)
{
    return 2 * shares_of(rows, groups).blocks * width * 4;
}

cudaError_t launch_block_norm(const BlockArgs &a, cudaStream_t st)
{
    return a.dtype == ZG_DTYPE_BF16 ? of_type<uint16_t, false>(a, st) : of_type<float, false>(a, st);
}

cudaError_t launch_block_norm_grad(const BlockArgs &a, cudaStream_t st)
{
    return a.dtype == ZG_DTYPE_BF16 ? of_type<uint16_t, true>(a, st) : of_type<float, true>(a, st);
}

}  // namespace zg
