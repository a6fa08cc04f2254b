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

inline bool misaligned(const void *p) { return ((uintptr_t)p & 15u) != 0; }

}  // namespace gdn
