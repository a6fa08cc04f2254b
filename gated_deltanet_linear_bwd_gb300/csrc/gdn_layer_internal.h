// gdn_layer_internal.h -- what the layer operators' translation units share:
// error reporting and device set-up (both in gdn_api.cu).  Not part of the ABI.
#pragma once

#include "gdn_internal.h"
#include "gdn_layer.h"

namespace gdn {

// Records the message behind gdn_last_error() and returns `code`.
gdn_status fail(gdn_status code, const char *fmt, ...);
gdn_status cuda_fail(cudaError_t e, const char *what);

// The current device's SM count and status word (device memory); refuses
// devices other than sm_103a.
struct LayerDevice {
    int sms = 0;
    int *status = nullptr;
    long long spin_limit = 0;
};
gdn_status layer_device(LayerDevice *out);

// launch_pdl with thread-block clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                               int cluster, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Lets `kernel` take `bytes` of dynamic shared memory on the current device; asks the
// runtime once for each kernel, device and larger size.
cudaError_t allow_smem(const void *kernel, size_t bytes);

// out[d] = sum over `rows` of partial[row][d], in a fixed order.
cudaError_t column_sum(const float *partial, int rows, int D, float *out, cudaStream_t s);

// The refusals of gdn_mx_quantize.
gdn_status check_quantize(const gdn_mx_quantize_args *a);
// gdn_mx_quantize that also clears `words` words at `work`.
gdn_status mx_quantize(const gdn_mx_quantize_args *a, uint32_t *work, int words, void *stream);

// Rows and columns of a microscaled matrix: what is rounded up to whole tiles, and walked past
// by one, stays an int.
constexpr int kMaxExtent = (int)((1ll << 31) - (1 << 16));

inline bool misaligned(const void *p) { return ((uintptr_t)p & 15u) != 0; }

}  // namespace gdn
