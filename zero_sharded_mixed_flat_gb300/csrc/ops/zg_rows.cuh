// zg_rows.cuh -- rows of logits shared out over blocks: how a row of any
// alignment is cut into parts of whole 16-byte units and ragged ends.
#pragma once

#include "zg_kernels.cuh"

namespace zg {

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = uint16_t(pack_bf16x2(v, 0.0f)); }

// max that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Sixteen bytes of logits: eight bf16 or four binary32.
template <class T>
struct Unit;
template <>
struct Unit<uint16_t> {
    static constexpr int kN = 8;
    uint4 w;
    // Running maxima of the low and the high halves.
    struct Top {
        uint32_t m = 0xff80ff80u;  // -inf
        __device__ __forceinline__ void add(const Unit &x) { m = max2(max2(m, max2(x.w.x, x.w.y)), max2(x.w.z, x.w.w)); }
        __device__ __forceinline__ float get() const { return max_nan(bf16_lo(m), bf16_hi(m)); }
        __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
        {
            uint32_t d;
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
            return d;
        }
    };
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
    struct Top {
        float m = -INFINITY;
        __device__ __forceinline__ void add(const Unit &x)
        {
            m = max_nan(max_nan(m, max_nan(__uint_as_float(x.w.x), __uint_as_float(x.w.y))),
                        max_nan(__uint_as_float(x.w.z), __uint_as_float(x.w.w)));
        }
        __device__ __forceinline__ float get() const { return m; }
    };
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

// A block's part of a row. Elements are counted from the 16-byte boundary at
// or below the row's first, so the row is [head, head + vocab); the part is the
// elements [first, last), and units [u0, u1) are whole in it.
struct Part {
    int head, lo, first, last, u0, u1;
};
template <class T>
__device__ __forceinline__ Part part_of(const T *row, int vocab, int each, int rank)
{
    constexpr int N = Unit<T>::kN;
    Part p;
    p.head = int((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int end = p.head + vocab;  // vocab is at most 2^30
    p.lo = rank * each;
    p.first = max(min(p.lo * N, end), p.head);
    p.last = p.lo + each < (end + N - 1) / N ? (p.lo + each) * N : end;
    p.last = max(p.last, p.first);
    p.u0 = (p.first + N - 1) / N;
    p.u1 = max(p.last / N, p.u0);
    return p;
}

// A block's part of a row, and how it lies in memory.
template <class T>
struct Row {
    const T *z;     // the row
    const T *base;  // element 0 of the part's count: only [head, head + vocab) is touched
    Part part;
    int units;      // whole ones
    __device__ __forceinline__ Row(const T *first, int vocab, int each, int rank)
    {
        z = first;
        part = part_of(z, vocab, each, rank);
        base = z - part.head;
        units = part.u1 - part.u0;
    }
    __device__ __forceinline__ const uint4 *from() const { return reinterpret_cast<const uint4 *>(base) + part.u0; }
    // A thread's one element of the part's ragged ends (less than a unit each), or -1.
    __device__ __forceinline__ int ragged(int tid) const
    {
        constexpr int N = Unit<T>::kN;
        const int head_end = min(part.u0 * N, part.last), tail = max(part.u1 * N, head_end);
        if (part.first + tid < head_end) return part.first + tid;
        return tid >= 32 && tail + tid - 32 < part.last ? tail + tid - 32 : -1;
    }
};

}  // namespace zg
