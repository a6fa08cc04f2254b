// gdn_layer_util.cu -- what the layer operators share: the sum over rows that their
// weight gradients end with, and the shared-memory limits of their kernels.
#include <algorithm>
#include <mutex>

#include "gdn_layer_internal.h"

namespace gdn {
namespace {

// out[d] = sum over rows of partial[row][d], in a fixed order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *partial, int rows, int D,
                                                          float *out) {
    __shared__ float strip[32][33];
    pdl_enter();
    const int lane = threadIdx.x & 31, strip_no = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (d < D)
        for (int r = strip_no; r < rows; r += 32) t += partial[(long long)r * D + d];
    strip[strip_no][lane] = t;
    __syncthreads();
    if (strip_no == 0 && d < D) {
        t = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) t += strip[k][lane];
        out[d] = t;
    }
}

}  // namespace

cudaError_t allow_smem(const void *kernel, size_t bytes) {
    // what has been granted; a kernel for which no entry is left is granted it on every call
    struct Grant {
        const void *kernel;
        int dev;
        size_t bytes;
    };
    static std::mutex mu;
    static Grant granted[256];
    static int n = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    Grant *g = std::find_if(granted, granted + n, [&](const Grant &h) { return h.kernel == kernel && h.dev == dev; });
    if (g < granted + n && g->bytes >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    if (g < granted + n) g->bytes = bytes;
    else if (n < 256) granted[n++] = {kernel, dev, bytes};
    return cudaSuccess;
}

cudaError_t column_sum(const float *partial, int rows, int D, float *out, cudaStream_t s) {
    prof_before("column_sum", s);
    const cudaError_t e = launch_pdl(column_sum_kernel, dim3((D + 31) / 32), dim3(1024), 0, s, partial,
                                     rows, D, out);
    prof_after(s);
    return e;
}

}  // namespace gdn
