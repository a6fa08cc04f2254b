// gdn_mx_strip.cuh -- quantising a strip of a row to MXFP8 / MXFP4, a warp at a time.
#pragma once

#include <cuda_bf16.h>

#include "gdn_mx.cuh"

namespace gdn {
namespace mx {

// Eight elements of a row, and the bits of their largest magnitude.
struct Eight {
    float2 v[4];
    uint32_t amax;
};
__device__ __forceinline__ Eight unpack(uint4 r) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    Eight e;
    uint32_t m = 0;                // bf16 magnitudes compare as 16-bit numbers, two at a time
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    }
    e.amax = max(m << 16, m & 0xffff0000u);
    return e;
}
struct Floats {
    float4 a, b;
};
__device__ __forceinline__ Eight unpack(Floats r) {
    Eight e;
    e.v[0] = make_float2(r.a.x, r.a.y), e.v[1] = make_float2(r.a.z, r.a.w);
    e.v[2] = make_float2(r.b.x, r.b.y), e.v[3] = make_float2(r.b.z, r.b.w);
    e.amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) e.amax = max(e.amax, max(abs_bits(e.v[i].x), abs_bits(e.v[i].y)));
    return e;
}
template <typename T>
struct Load8;
template <>
struct Load8<__nv_bfloat16> {
    using Raw = uint4;
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
};
template <>
struct Load8<float> {
    using Raw = Floats;
    static __device__ __forceinline__ Raw zero() { return Floats{make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)}; }
};

// A warp takes spans of 256 columns of a row, 8 to a lane, kSpans of them at a time so
// that their loads are in flight together (of kSpans rows where a row is one span: ROWS);
// a block is four lanes, and the four blocks of a scale tile's word are sixteen.  Spans
// [first, end) of `row`; rows and blocks past the end, up to whole scale tiles, are walked
// for their zero scales.  Addresses move by constants within a row: with a division and
// 64-bit products for every span the pass was bound by arithmetic.
constexpr int kSpans = 4;

template <typename T, bool FP4, bool ROWS>
__device__ __forceinline__ void quantize_strip(const T *x, uint8_t *data, uint8_t *scales, long long row, int first,
                                               int end, int rows, int K, int ktiles) {
    using Raw = typename Load8<T>::Raw;
    const int lane = threadIdx.x & 31;
    // from one of the kSpans to the next
    const int dx = ROWS ? K : 256, dd = FP4 ? dx / 2 : dx, dsc = ROWS ? 16 : 1024;
    const long long at = row * K + first * 256 + lane * 8;
    const T *px = x + at;
    uint8_t *pd = data + (FP4 ? at / 2 : at);
    uint8_t *ps = scales + scale_offset(row, 0, ktiles) + (2ll * first + (lane >> 4)) * 512;
    for (int span = first; span < end; span += kSpans) {
        const int col = span * 256 + lane * 8;
        auto inside = [&](int u) { return ROWS ? row + u < rows && col < K : row < rows && col + 256 * u < K; };
        Raw raw[kSpans];
#pragma unroll
        for (int u = 0; u < kSpans; ++u)
            raw[u] = inside(u) ? *reinterpret_cast<const Raw *>(px + dx * u) : Load8<T>::zero();
#pragma unroll
        for (int u = 0; u < kSpans; ++u) {
            const Eight e = unpack(raw[u]);
            uint32_t amax = max(e.amax, __shfl_xor_sync(0xffffffffu, e.amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int byte = scale_byte<FP4>(amax);        // 0 where nothing is
            uint32_t word = (uint32_t)byte << (8 * ((lane >> 2) & 3));
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            word |= __shfl_xor_sync(0xffffffffu, word, 8);
            if ((lane & 15) == 0 && col + (ROWS ? 0 : 256 * u) < ktiles * 128)
                *reinterpret_cast<uint32_t *>(ps + dsc * u) = word;
            if (!inside(u)) continue;
            const float f = scale_factor(byte);
            float2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(e.v[j], make_float2(f, f));
            const bool bad = byte == 255;                  // the elements of a NaN block are zeros
            if (FP4) {
                const uint32_t q = e2m1x8(v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y);
                *reinterpret_cast<uint32_t *>(pd + dd * u) = bad ? 0u : q;
            } else {
                const uint32_t q0 = e4m3x4(v[0].x, v[0].y, v[1].x, v[1].y), q1 = e4m3x4(v[2].x, v[2].y, v[3].x, v[3].y);
                *reinterpret_cast<uint2 *>(pd + dd * u) = make_uint2(bad ? 0u : q0, bad ? 0u : q1);
            }
        }
        px += 256 * kSpans;
        pd += (FP4 ? 128 : 256) * kSpans;
        ps += 1024 * kSpans;
    }
}

}  // namespace mx
}  // namespace gdn
