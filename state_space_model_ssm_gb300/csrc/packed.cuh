// Arithmetic on pairs of fp32 values, and pairs of neighbouring elements of a row, shared by the
// selective scan and the short causal convolution.  One packed instruction does two
// fp32 operations in one issue slot; exponentials and reciprocals are the hardware's approximate
// ones (2^x and 1/x, each within 2 ulp, denormals taken as zero).
#pragma once

#include "layer_common.cuh"

namespace ssm {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<unsigned long long &>(d))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)),
          "l"(reinterpret_cast<unsigned long long &>(c)));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long &>(d))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long &>(d))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
    return d;
}

__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }

__device__ __forceinline__ float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float2 rcp2(float2 v) { return make_float2(rcp(v.x), rcp(v.y)); }

// sigmoid(v), within (2|v| + 8) 2^-24 of it: the rounded argument of 2^x, and the two approximations.  v times it is 0 times
// v where exp(-v) overflows (v below -88).
__device__ __forceinline__ float2 sigmoid2(float2 v)
{
    return rcp2(make_float2(1.f + ex2(-v.x * kLog2e), 1.f + ex2(-v.y * kLog2e)));
}

// Two neighbouring channels of a row as they lie in memory.
template <class T>
struct RawPair { uint32_t w; };
template <>
struct RawPair<float> { float2 w; };

template <class T>
__device__ __forceinline__ float2 pair_of(const RawPair<T> &r)
{
    Vec<T, 2> v;
    *reinterpret_cast<uint32_t *>(&v) = r.w;
    return make_float2(to_float(v.v[0]), to_float(v.v[1]));
}
template <>
__device__ __forceinline__ float2 pair_of<float>(const RawPair<float> &r) { return r.w; }

template <class T>
__device__ __forceinline__ RawPair<T> join_pair(T a, T b)
{
    RawPair<T> r;
    const Vec<T, 2> v{{a, b}};
    if constexpr (sizeof(T) == 4)
        r.w = make_float2(a, b);
    else
        r.w = *reinterpret_cast<const uint32_t *>(&v);
    return r;
}

// Of an aligned pair in memory.
template <class T>
__device__ __forceinline__ RawPair<T> load_pair(const T *p)
{
    RawPair<T> r;
    if constexpr (sizeof(T) == 4)
        r.w = *reinterpret_cast<const float2 *>(p);
    else
        r.w = *reinterpret_cast<const uint32_t *>(p);
    return r;
}

template <class T>
__device__ __forceinline__ void store_word(T *p, float2 v)
{
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float2 *>(p) = v;
    } else {
        const Vec<T, 2> o{{from_float<T>(v.x), from_float<T>(v.y)}};
        *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(&o);
    }
}

}  // namespace ssm
