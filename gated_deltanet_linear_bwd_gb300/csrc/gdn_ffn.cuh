// gdn_ffn.cuh -- what the feed-forward block's translation units share: the activations, and the
// backward pass of few tokens.
#pragma once

#include "gdn_layer_internal.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace ffn {

// The activation f(g) and its derivative; gelu is its tanh form, g logistic(2 c (g + 0.044715 g^3))
// with c = sqrt(2 / pi).
constexpr float kGelu2c = 1.5957691216057308f, kGeluCube = 0.044715f;
template <bool GELU>
__device__ __forceinline__ float activation(float g) {
    return g * logistic<__nv_bfloat16>(GELU ? kGelu2c * g * fmaf(kGeluCube, g * g, 1.f) : g);
}
template <bool GELU>
__device__ __forceinline__ float activation(float g, float &slope) {
    if (!GELU) {
        const float s = logistic<__nv_bfloat16>(g);
        slope = silu_slope(g, s);
        return g * s;
    }
    // past 2^60 the slope is 0 or 1 and g^2 might overflow, of which 0 times would be NaN
    const float g2 = fminf(g * g, 0x1p120f), s = logistic<__nv_bfloat16>(kGelu2c * g * fmaf(kGeluCube, g2, 1.f));
    slope = fmaf(g * s * (1.f - s), kGelu2c * fmaf(3.f * kGeluCube, g2, 1.f), s);
    return g * s;
}

// So few tokens keep what passes between the products in more than bf16's 8 bits: over few
// tokens such roundings do not average out (a gradient of one token was up to 1.6 times as far from its
// 64-bit value as its own rounding takes it), and the weights' bytes bound the products anyway.
constexpr int kFewTokens = 8;      // backward: by CUDA cores
constexpr int kLowTokens = 64;     // forward: h as two rows, both in a tile of 128

// The backward pass of up to kFewTokens tokens (and sizes whose rows, of both weights together, an int
// counts), whose arguments are checked.
inline bool few_bwd_fits(int M, int K, int F) { return M <= kFewTokens && K <= 1 << 29 && F <= 1 << 29; }
size_t few_bwd_bytes(int M, int K, int F);
cudaError_t few_bwd(const gdn_ffn_bwd_args *a, float *ws, cudaStream_t q);

}  // namespace ffn
}  // namespace gdn
