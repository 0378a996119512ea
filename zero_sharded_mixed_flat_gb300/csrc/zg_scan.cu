// The gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t with
// a_t = sigmoid(f_t), forward and backward.
#include <cuda_bf16.h>

#include "zg_launch.h"
#include "zg_ops.h"

namespace zg {
namespace {

template <class T>
__device__ __forceinline__ float load1(const T *p);
template <>
__device__ __forceinline__ float load1(const float *p) { return *p; }
template <>
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// sigmoid(f) and sigmoid(-f), each to a few ulp: the smaller one is never
// formed as a difference from one.
__device__ __forceinline__ void gates(float f, float &a, float &u)
{
    const float e = expf(-fabsf(f));
    const float big = 1.0f / (1.0f + e);
    const float small = e * big;
    a = f >= 0.0f ? big : small;
    u = f >= 0.0f ? small : big;
    if (f != f) a = u = f;
}

struct Range {
    int64_t row, lo, hi;  // batch row and its tokens
};

__device__ __forceinline__ Range sequence(const ScanArgs &a, int64_t s)
{
    if (!a.seq_start) return Range{s, 0, a.tokens};
    int64_t lo = a.seq_start[s], hi = a.seq_start[s + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > a.tokens ? a.tokens : hi;
    return Range{0, lo, hi};
}

// One thread walks one channel of one sequence.
template <class T>
__global__ void __launch_bounds__(128) scan_kernel(ScanArgs a)
{
    const int64_t c = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= a.channels) return;
    const int64_t chunks = (a.tokens + ZG_SCAN_CHUNK - 1) / ZG_SCAN_CHUNK;
    for (int64_t s = blockIdx.y; s < a.n_seq; s += gridDim.y) {
        const Range q = sequence(a, s);
        const T *x = static_cast<const T *>(a.x.ptr) + q.row * a.x.sb + c;
        const T *f = static_cast<const T *>(a.f.ptr) + q.row * a.f.sb + c;
        T *y = static_cast<T *>(a.y.ptr) + q.row * a.y.sb + c;
        float h = a.h0 ? a.h0[s * a.channels + c] : 0.0f;
        for (int64_t t = q.lo; t < q.hi; ++t) {
            if (a.states && t % ZG_SCAN_CHUNK == 0)
                a.states[(q.row * chunks + t / ZG_SCAN_CHUNK) * a.channels + c] = h;
            float g, u;
            gates(load1(f + t * a.f.st), g, u);
            h = fmaf(g, h, u * load1(x + t * a.x.st));
            store1(y + t * a.y.st, h);
        }
        if (a.h_last) a.h_last[s * a.channels + c] = h;
    }
}

template <class T>
__global__ void __launch_bounds__(128) scan_bwd_kernel(ScanArgs a)
{
    const int64_t c = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= a.channels) return;
    const int64_t chunks = (a.tokens + ZG_SCAN_CHUNK - 1) / ZG_SCAN_CHUNK;
    for (int64_t s = blockIdx.y; s < a.n_seq; s += gridDim.y) {
        const Range q = sequence(a, s);
        const T *x = static_cast<const T *>(a.x.ptr) + q.row * a.x.sb + c;
        const T *f = static_cast<const T *>(a.f.ptr) + q.row * a.f.sb + c;
        const T *dy = static_cast<const T *>(a.y.ptr) + q.row * a.y.sb + c;
        T *dx = static_cast<T *>(a.dx.ptr) + q.row * a.dx.sb + c;
        T *df = static_cast<T *>(a.df.ptr) + q.row * a.df.sb + c;
        float r = a.dh_last ? a.dh_last[s * a.channels + c] : 0.0f;
        for (int64_t end = q.hi; end > q.lo;) {
            const int64_t k = (end - 1) / ZG_SCAN_CHUNK;
            const int64_t lo = k * ZG_SCAN_CHUNK > q.lo ? k * ZG_SCAN_CHUNK : q.lo;
            float before[ZG_SCAN_CHUNK];
            float h = lo == q.lo ? (a.h0 ? a.h0[s * a.channels + c] : 0.0f)
                                 : a.states[(q.row * chunks + k) * a.channels + c];
            for (int64_t t = lo; t < end; ++t) {
                float g, u;
                before[t - lo] = h;
                gates(load1(f + t * a.f.st), g, u);
                h = fmaf(g, h, u * load1(x + t * a.x.st));
            }
            for (int64_t t = end - 1; t >= lo; --t) {
                float g, u;
                gates(load1(f + t * a.f.st), g, u);
                const float d = load1(dy + t * a.y.st) + r;
                store1(dx + t * a.dx.st, u * d);
                store1(df + t * a.df.st, d * (before[t - lo] - load1(x + t * a.x.st)) * (g * u));
                r = g * d;
            }
            end = lo;
        }
        if (a.dh0) a.dh0[s * a.channels + c] = r;
    }
}

dim3 grid_of(const ScanArgs &a)
{
    return dim3(unsigned((a.channels + 127) / 128), unsigned(a.n_seq < 65535 ? a.n_seq : 65535));
}

}  // namespace

cudaError_t launch_scan(const ScanArgs &a, cudaStream_t st)
{
    if (a.dtype == ZG_DTYPE_BF16)
        scan_kernel<uint16_t><<<grid_of(a), 128, 0, st>>>(a);
    else
        scan_kernel<float><<<grid_of(a), 128, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_scan_bwd(const ScanArgs &a, cudaStream_t st)
{
    if (a.dtype == ZG_DTYPE_BF16)
        scan_bwd_kernel<uint16_t><<<grid_of(a), 128, 0, st>>>(a);
    else
        scan_bwd_kernel<float><<<grid_of(a), 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace zg
