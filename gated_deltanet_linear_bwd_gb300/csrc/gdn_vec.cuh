// gdn_vec.cuh -- what the convolution and the state space scan share: neighbouring
// elements as one load, activations, and the token ranges of sequences.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

// VEC neighbouring elements of T at an address that is a multiple of their size.
template <int BYTES>
struct RawBytes;
template <>
struct RawBytes<2> {
    using type = uint16_t;
};
template <>
struct RawBytes<4> {
    using type = uint32_t;
};
template <>
struct RawBytes<8> {
    using type = uint2;
};
template <>
struct RawBytes<16> {
    using type = uint4;
};
template <typename T, int VEC>
struct Vec {
    using Raw = typename RawBytes<VEC * (int)sizeof(T)>::type;
    static __device__ __forceinline__ Raw raw(const T *p) { return *reinterpret_cast<const Raw *>(p); }
    static __device__ __forceinline__ void get(const Raw &r, float *v) {
        const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = to_f(e[i]);
    }
    static __device__ __forceinline__ void load(const T *p, float *v) { get(raw(p), v); }
    static __device__ __forceinline__ void store(T *p, const float *v) {
        Raw r;
        T *e = reinterpret_cast<T *>(&r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) from_f(e + i, v[i]);
        *reinterpret_cast<Raw *>(p) = r;
    }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The logistic function.  fp32 tensors take the accurate functions; of bf16 ones, whose results
// are rounded to 2^-8 of themselves, the hardware's exponential and reciprocal (2^-21).
template <typename T>
__device__ __forceinline__ float logistic(float x) {
    if (sizeof(T) == 4) return 1.f / (1.f + expf(-x));
    return rcp(1.f + ex2(x * -1.4426950408889634f));
}
template <typename T>
__device__ __forceinline__ float2 logistic2(float2 x) {
    if (sizeof(T) == 4) return make_float2(logistic<T>(x.x), logistic<T>(x.y));
    const float2 y = __fmul2_rn(x, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    const float2 e = __fadd2_rn(make_float2(ex2(y.x), ex2(y.y)), make_float2(1.f, 1.f));
    return make_float2(rcp(e.x), rcp(e.y));
}
// d(x logistic(x)) / dx, s = logistic(x).
__device__ __forceinline__ float silu_slope(float x, float s) { return s * (1.f + x * (1.f - s)); }

// log(1 + e^x).  Of bf16 tensors with the hardware's exponential and logarithm, but for e = e^-|x| <
// 1/8, where the logarithm of the rounded 1 + e would lose what a small step is made of: there e p(e),
// p the polynomial through log2(1 + e) / e at the four Chebyshev points of 0 .. 1/8 (3.1e-7 of itself).
template <typename T>
__device__ __forceinline__ float2 softplus2(float2 x) {
    if (sizeof(T) == 4)
        return make_float2(fmaxf(x.x, 0.f) + log1pf(expf(-fabsf(x.x))), fmaxf(x.y, 0.f) + log1pf(expf(-fabsf(x.y))));
    const auto both = [](float v) { return make_float2(v, v); };
    const float2 y = __fmul2_rn(make_float2(fabsf(x.x), fabsf(x.y)), both(-1.4426950408889634f));
    const float2 e = make_float2(ex2(y.x), ex2(y.y));
    float2 p = __ffma2_rn(e, both(-2.9770274392e-1f), both(4.7618794121e-1f));
    p = __ffma2_rn(p, e, both(-7.2123178461e-1f));
    p = __fmul2_rn(__ffma2_rn(p, e, both(1.4426945903f)), e);
    const float2 u = __fadd2_rn(e, both(1.f));
    return __ffma2_rn(make_float2(e.x < 0.125f ? p.x : __log2f(u.x), e.y < 0.125f ? p.y : __log2f(u.y)),
                      both(0.6931471805599453f), make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}
template <typename T>
__device__ __forceinline__ float softplus(float x) {
    return softplus2<T>(make_float2(x, x)).x;
}

// Sequences: rows of T tokens, or (cu) a packed batch of T tokens in all.
struct Seqs {
    const int32_t *cu;
    long long T;
    int N;
};

// Token range of sequence n; false for an impossible one, whose tokens are then left alone.
__device__ __forceinline__ bool seq_tokens(const Seqs &s, int n, long long &bos, long long &len) {
    if (!s.cu) {
        bos = (long long)n * s.T;
        len = s.T;
        return true;
    }
    const long long lo = s.cu[n], hi = s.cu[n + 1];
    const bool bad = lo < 0 || hi < lo || hi > s.T || (n == 0 && lo != 0) || (n == s.N - 1 && hi != s.T);
    bos = bad ? 0 : lo;
    len = bad ? 0 : hi - lo;
    return !bad;
}

// The sequence of token t (of a packed batch the last that begins at or before it).
__device__ __forceinline__ int seq_of(const Seqs &s, long long t) {
    if (!s.cu) return (int)(t / s.T);
    int lo = 0, hi = s.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

}  // namespace gdn
