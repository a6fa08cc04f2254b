// gdn_mx_quant.cu -- quantisation to MXFP8 / MXFP4 and back.
#include <algorithm>

#include "gdn_layer_internal.h"
#include "gdn_mx_strip.cuh"

namespace gdn {
namespace mx {
namespace {

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

// A row's spans are shared out over 2^log_parts warps, as many as fill the GPU when rows
// are few.  Bound by memory: 32768 x 4096 bf16 to MXFP4 52 us, 97% of the measured copy
// rate.  Clears `words` words at `work` for a product that follows.
template <typename T, bool FP4, bool ROWS>
__global__ void __launch_bounds__(256) quantize_kernel(const T *x, uint8_t *data, uint8_t *scales,
                                                       int rows, int K, int ktiles, int log_parts,
                                                       uint32_t *work, int words) {
    // the kernel behind may start once all before this one has ended: a product that
    // follows loads its weight under the quantisation
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = blockIdx.x * 256 + threadIdx.x; i < words; i += gridDim.x * 256) work[i] = 0;
    const int spans = (ktiles + 1) / 2, parts = 1 << log_parts;
    const int per = ((spans + parts - 1) / parts + kSpans - 1) / kSpans * kSpans;
    const long long padded = (rows + 127ll) / 128 * 128;
    const long long items = ROWS ? padded / kSpans : padded << log_parts;
    for (long long i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < items; i += gridDim.x * 8ll) {
        const long long row = ROWS ? i * kSpans : i >> log_parts;
        const int first = ROWS ? 0 : (int)(i & (parts - 1)) * per, end = min(first + per, spans);
        quantize_strip<T, FP4, ROWS>(x, data, scales, row, first, end, rows, K, ktiles);
    }
}

template <typename T>
auto quantize_of(bool fp4, bool by_rows) {
    return fp4 ? (by_rows ? quantize_kernel<T, true, true> : quantize_kernel<T, true, false>)
               : (by_rows ? quantize_kernel<T, false, true> : quantize_kernel<T, false, false>);
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
    if (K > kMaxExtent) return fail(GDN_ERR_INVALID_ARG, "problem too large: K=%d", K);
    if (K % 32 != 0) return fail(GDN_ERR_UNSUPPORTED, "K = %d (a multiple of 32)", K);
    if (dtype != GDN_FP32 && dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_FP32 or GDN_BF16", dtype);
    if (format != GDN_MXFP8 && format != GDN_MXFP4)
        return fail(GDN_ERR_UNSUPPORTED, "format %d is not GDN_MXFP8 or GDN_MXFP4", format);
    return GDN_OK;
}

}  // namespace
}  // namespace mx

gdn_status check_quantize(const gdn_mx_quantize_args *a) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    const gdn_status st = mx::check(a->rows, a->K, a->dtype, a->format);
    if (st != GDN_OK || a->rows == 0 || a->K == 0) return st;
    if (!a->x || !a->data || !a->scales) return fail(GDN_ERR_INVALID_ARG, "x, data and scales are required");
    if (misaligned(a->x) || misaligned(a->data) || misaligned(a->scales))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    return GDN_OK;
}

gdn_status mx_quantize(const gdn_mx_quantize_args *a, uint32_t *work, int words, void *stream) {
    gdn_status st = check_quantize(a);
    if (st != GDN_OK || a->rows == 0 || a->K == 0) return st;
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    const int ktiles = (a->K + 127) / 128, spans = (ktiles + 1) / 2;
    // warps to a row: doubled while rows x warps are fewer than 16 to an SM and each has kSpans
    int log_parts = 0;
    while (((long long)a->rows << log_parts) < 16ll * dev.sms && (mx::kSpans << log_parts) < spans) ++log_parts;
    const bool by_rows = spans == 1;
    const long long padded = (a->rows + 127ll) / 128 * 128, items = by_rows ? padded / mx::kSpans : padded << log_parts;
    const unsigned grid = (unsigned)std::min<long long>((items + 7) / 8, 16ll * dev.sms);
    cudaStream_t q = (cudaStream_t)stream;
    prof_before("mx_quantize", q);
    cudaError_t e;
    if (a->dtype == GDN_BF16)
        e = launch_pdl(mx::quantize_of<__nv_bfloat16>(a->format == GDN_MXFP4, by_rows), dim3(grid), dim3(256), 0, q,
                       (const __nv_bfloat16 *)a->x, (uint8_t *)a->data, a->scales, a->rows, a->K, ktiles, log_parts, work, words);
    else
        e = launch_pdl(mx::quantize_of<float>(a->format == GDN_MXFP4, by_rows), dim3(grid), dim3(256), 0, q,
                       (const float *)a->x, (uint8_t *)a->data, a->scales, a->rows, a->K, ktiles, log_parts, work, words);
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "mx quantise launch");
}

}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_mx_scale_bytes(int32_t rows, int32_t K) {
    return rows > 0 && K > 0 ? (size_t)((rows + 127ll) / 128) * (size_t)((K + 127ll) / 128) * 512 : 0;
}

gdn_status gdn_mx_quantize(const gdn_mx_quantize_args *a, void *stream) { return mx_quantize(a, nullptr, 0, stream); }

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
