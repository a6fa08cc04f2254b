// gdn_mx_quant.cu -- quantisation to MXFP8 / MXFP4 and back.
#include <algorithm>

#include "gdn_layer_internal.h"
#include "gdn_mx.cuh"

namespace gdn {
namespace mx {
namespace {

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *v) {
    const uint4 r = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float *v) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float *v) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A warp takes 256 columns of a row, 8 to a lane; a block is four lanes, and the
// four blocks of a scale tile's word are sixteen.  Rows and blocks past the end, up
// to whole scale tiles, are walked for their zero scales.
template <typename T, bool FP4>
__global__ void __launch_bounds__(256) quantize_kernel(const T *x, uint8_t *data, uint8_t *scales,
                                                       int rows, int K, int ktiles) {
    pdl_enter();
    const int lane = threadIdx.x & 31, spans = (ktiles + 1) / 2;
    const long long items = (rows + 127ll) / 128 * 128 * spans;
    for (long long i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < items; i += gridDim.x * 8ll) {
        const long long row = i / spans;
        const int col = (int)(i % spans) * 256 + lane * 8;
        const bool in = row < rows && col < K;
        float v[8];
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
        if (in) load8(x + row * K + col, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(v[j]));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int byte = in ? scale_byte<FP4>(amax) : 0;
        uint32_t word = (uint32_t)byte << (8 * ((lane >> 2) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if ((lane & 15) == 0 && col < ktiles * 128)
            *reinterpret_cast<uint32_t *>(scales + scale_offset(row, col / 32, ktiles)) = word;
        if (!in) continue;
        const float f = scale_factor(byte);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = byte == 255 ? 0.f : v[j] * f;
        if (FP4)
            *reinterpret_cast<uint32_t *>(data + (row * K + col) / 2) = e2m1x8(v);
        else
            *reinterpret_cast<uint2 *>(data + row * K + col) =
                make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
    }
}

__device__ __forceinline__ float from_e4m3(uint32_t b) {
    const uint32_t e = (b >> 3) & 15, m = b & 7;
    const float v = e == 15 && m == 7 ? __uint_as_float(0x7fc00000u)
                    : e == 0          ? (float)m * 0x1p-9f
                                      : __uint_as_float(((e + 120) << 23) | (m << 20));
    return b & 0x80 ? -v : v;
}
__device__ __forceinline__ float from_e2m1(uint32_t b) {
    const uint32_t e = (b >> 1) & 3, m = b & 1;
    const float v = e == 0 ? 0.5f * (float)m : __uint_as_float(((e + 126) << 23) | (m << 22));
    return b & 8 ? -v : v;
}

template <typename T, bool FP4>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t *data, const uint8_t *scales,
                                                         T *x, int rows, int K, int ktiles) {
    pdl_enter();
    const long long per = K / 8, items = rows * per;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < items; i += gridDim.x * 256ll) {
        const long long row = i / per;
        const int col = (int)(i % per) * 8;
        const int byte = scales[scale_offset(row, col / 32, ktiles)];
        // 2^(byte - 127) in two factors, as 2^-127 alone is no normal number
        const float s1 = byte == 255 ? __uint_as_float(0x7fc00000u)
                                     : __uint_as_float((uint32_t)(byte / 2 + 64) << 23);
        const float s2 = __uint_as_float((uint32_t)(byte - byte / 2 + 63) << 23);
        float v[8];
        if (FP4) {
            const uint32_t q = *reinterpret_cast<const uint32_t *>(data + (row * K + col) / 2);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = from_e2m1((q >> (4 * j)) & 15) * s1 * s2;
        } else {
            const uint2 q = *reinterpret_cast<const uint2 *>(data + row * K + col);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = from_e4m3(((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 255) * s1 * s2;
        }
        store8(x + row * K + col, v);
    }
}

gdn_status check(int rows, int K, int dtype, int format) {
    if (rows < 0 || K < 0) return fail(GDN_ERR_INVALID_ARG, "bad sizes rows=%d K=%d", rows, K);
    if (K % 32 != 0) return fail(GDN_ERR_UNSUPPORTED, "K = %d (a multiple of 32)", K);
    if (dtype != GDN_FP32 && dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_FP32 or GDN_BF16", dtype);
    if (format != GDN_MXFP8 && format != GDN_MXFP4)
        return fail(GDN_ERR_UNSUPPORTED, "format %d is not GDN_MXFP8 or GDN_MXFP4", format);
    return GDN_OK;
}

}  // namespace
}  // namespace mx
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_mx_scale_bytes(int32_t rows, int32_t K) {
    return rows > 0 && K > 0 ? (size_t)((rows + 127ll) / 128) * (size_t)((K + 127ll) / 128) * 512 : 0;
}

gdn_status gdn_mx_quantize(const gdn_mx_quantize_args *a, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = mx::check(a->rows, a->K, a->dtype, a->format);
    if (st != GDN_OK) return st;
    if (a->rows == 0 || a->K == 0) return GDN_OK;
    if (!a->x || !a->data || !a->scales) return fail(GDN_ERR_INVALID_ARG, "x, data and scales are required");
    if (misaligned(a->x) || misaligned(a->data) || misaligned(a->scales))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    const int ktiles = (a->K + 127) / 128;
    const long long items = (a->rows + 127ll) / 128 * 128 * ((ktiles + 1) / 2);
    const unsigned grid = (unsigned)std::min<long long>((items + 7) / 8, 8ll * dev.sms);
    cudaStream_t q = (cudaStream_t)stream;
    prof_before("mx_quantize", q);
    cudaError_t e;
    if (a->dtype == GDN_BF16) {
        auto k = a->format == GDN_MXFP4 ? mx::quantize_kernel<__nv_bfloat16, true>
                                        : mx::quantize_kernel<__nv_bfloat16, false>;
        e = launch_pdl(k, dim3(grid), dim3(256), 0, q, (const __nv_bfloat16 *)a->x, (uint8_t *)a->data,
                       a->scales, a->rows, a->K, ktiles);
    } else {
        auto k = a->format == GDN_MXFP4 ? mx::quantize_kernel<float, true>
                                        : mx::quantize_kernel<float, false>;
        e = launch_pdl(k, dim3(grid), dim3(256), 0, q, (const float *)a->x, (uint8_t *)a->data,
                       a->scales, a->rows, a->K, ktiles);
    }
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "mx quantise launch");
}

gdn_status gdn_mx_dequantize(const gdn_mx_dequantize_args *a, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = mx::check(a->rows, a->K, a->dtype, a->format);
    if (st != GDN_OK) return st;
    if (a->rows == 0 || a->K == 0) return GDN_OK;
    if (!a->x || !a->data || !a->scales) return fail(GDN_ERR_INVALID_ARG, "x, data and scales are required");
    if (misaligned(a->x) || misaligned(a->data) || misaligned(a->scales))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    const int ktiles = (a->K + 127) / 128;
    const long long items = (long long)a->rows * (a->K / 8);
    const unsigned grid = (unsigned)std::min<long long>((items + 255) / 256, 8ll * dev.sms);
    cudaStream_t q = (cudaStream_t)stream;
    prof_before("mx_dequantize", q);
    cudaError_t e;
    if (a->dtype == GDN_BF16) {
        auto k = a->format == GDN_MXFP4 ? mx::dequantize_kernel<__nv_bfloat16, true>
                                        : mx::dequantize_kernel<__nv_bfloat16, false>;
        e = launch_pdl(k, dim3(grid), dim3(256), 0, q, (const uint8_t *)a->data, a->scales,
                       (__nv_bfloat16 *)a->x, a->rows, a->K, ktiles);
    } else {
        auto k = a->format == GDN_MXFP4 ? mx::dequantize_kernel<float, true>
                                        : mx::dequantize_kernel<float, false>;
        e = launch_pdl(k, dim3(grid), dim3(256), 0, q, (const uint8_t *)a->data, a->scales,
                       (float *)a->x, a->rows, a->K, ktiles);
    }
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "mx dequantise launch");
}

}  // extern "C"
