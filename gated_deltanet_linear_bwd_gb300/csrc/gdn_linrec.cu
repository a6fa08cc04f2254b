// gdn_linrec.cu -- per-channel gated linear recurrence h_t = a_t h_{t-1} + x_t,
// its backward pass and its one-token step.
//
// A token's map h -> a h + x composes as (A, B) then (A', B') = (A A', A' B + B'),
// so a run of tokens is one pair per channel.  A CTA takes 32 or 64 channels (one
// 128-byte row per warp load) of one sequence and walks it in tiles of kWarps x R
// tokens.  Each warp reduces its R tokens to a pair, the pairs meet in shared
// memory, and every warp, knowing the value before its first token, forms its R
// results from the tile it still holds in registers: one pass over memory.
#include <algorithm>

#include "gdn_layer_internal.h"

namespace gdn {
namespace linrec {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;          // tokens a warp holds in registers
constexpr int kTile = kWarps * kRows;

// The channels a lane carries: VC elements of T as one load.
template <typename T, int VC>
struct Lane;
template <>
struct Lane<__nv_bfloat16, 2> {
    using Raw = uint32_t;
    static __device__ __forceinline__ void get(Raw r, float (&v)[2]) {
        v[0] = __uint_as_float(r << 16);
        v[1] = __uint_as_float(r & 0xffff0000u);
    }
    static __device__ __forceinline__ Raw put(const float (&v)[2]) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[0], v[1]);
        return *reinterpret_cast<const uint32_t *>(&b);
    }
};
template <>
struct Lane<__nv_bfloat16, 1> {
    using Raw = unsigned short;
    static __device__ __forceinline__ void get(Raw r, float (&v)[1]) {
        v[0] = __uint_as_float((uint32_t)r << 16);
    }
    static __device__ __forceinline__ Raw put(const float (&v)[1]) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    }
};
template <>
struct Lane<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ void get(Raw r, float (&v)[1]) { v[0] = r; }
    static __device__ __forceinline__ Raw put(const float (&v)[1]) { return v[0]; }
};

// Functions of an element, in full single precision for fp32 tensors.  For bf16
// ones softplus and its derivative come from the hardware approximations, whose
// errors (about 1e-7, in the log decay) lie far below the 2^-9 of the input's own
// rounding; with the accurate functions the gated pass would be bound by
// arithmetic instead of memory.  The decay itself is always the accurate expf: a
// slow channel multiplies a thousand decays near 1 together, so that a relative
// error of 2e-7 that always points the same way (the approximation's) would grow
// to 2e-4 in the fp32 states.
template <typename T>
struct Fn {
    static __device__ __forceinline__ float gate_exp(float x) { return expf(x); }
    static __device__ __forceinline__ float softplus(float x, float e) {
        return fmaxf(x, 0.f) + log1pf(e);
    }
    static __device__ __forceinline__ float rcp(float x) { return 1.f / x; }
};
template <>
struct Fn<__nv_bfloat16> {
    static __device__ __forceinline__ float gate_exp(float x) { return __expf(x); }
    static __device__ __forceinline__ float softplus(float x, float e) {
        return fmaxf(x, 0.f) + __logf(1.f + e);
    }
    static __device__ __forceinline__ float rcp(float x) { return __fdividef(1.f, x); }
};

// a = exp(g), or exp(-s softplus(g)); fmaxf drops a NaN, so a NaN gate is put back.
template <typename T, bool GATED>
__device__ __forceinline__ float decay(float g, float s) {
    if (!GATED) return expf(g);
    const float a = expf(-s * Fn<T>::softplus(g, Fn<T>::gate_exp(-fabsf(g))));
    return g != g ? g : a;
}

struct Shape {
    const int32_t *cu;
    long long T;               // tokens per row, or of the packed batch
    int N, D, groups;          // sequences, channels, channel groups
    int lanes_n;               // clusters that share a channel group's sequences
    int *status;
};

// Token range of sequence n; an impossible cu_seqlens is recorded and reads as empty.
__device__ __forceinline__ void range(const Shape &s, int n, long long &bos, long long &len) {
    if (!s.cu) {
        bos = (long long)n * s.T;
        len = s.T;
        return;
    }
    const long long lo = s.cu[n], hi = s.cu[n + 1];
    const bool bad = lo < 0 || hi < lo || hi > s.T || (n == 0 && lo != 0) ||
                     (n == s.N - 1 && hi != s.T);
    if (bad && threadIdx.x == 0) set_status(s.status, GDN_ERR_BAD_SEQLENS);
    bos = bad ? 0 : lo;
    len = bad ? 0 : hi - lo;
}

struct FwdArgs {
    const void *x, *g;
    const float *scale, *h0;
    void *h;
    float *ht;
};

template <typename T, int VC, bool GATED>
__global__ void __launch_bounds__(kThreads, 2) fwd_kernel(FwdArgs a, Shape s) {
    using L = Lane<T, VC>;
    using Raw = typename L::Raw;
    __shared__ float2 pairs[2][kWarps][32 * VC];
    pdl_enter();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = blockIdx.x % s.groups, first_n = blockIdx.x / s.groups;
    const int ch = group * 32 * VC + lane * VC;
    const bool live = ch < s.D;
    float sc[VC];
#pragma unroll
    for (int j = 0; j < VC; ++j) sc[j] = GATED && live ? a.scale[ch + j] : 0.f;

    int buf = 0;
    for (int n = first_n; n < s.N; n += s.lanes_n) {
        long long bos, len;
        range(s, n, bos, len);
        const Raw *x = reinterpret_cast<const Raw *>(reinterpret_cast<const T *>(a.x) + bos * s.D + ch);
        const Raw *g = reinterpret_cast<const Raw *>(reinterpret_cast<const T *>(a.g) + bos * s.D + ch);
        Raw *h = reinterpret_cast<Raw *>(reinterpret_cast<T *>(a.h) + bos * s.D + ch);
        const long long pitch = s.D / VC;
        float carry[VC];
#pragma unroll
        for (int j = 0; j < VC; ++j)
            carry[j] = a.h0 && live ? a.h0[(long long)n * s.D + ch + j] : 0.f;

        for (long long t0 = 0; t0 < len; t0 += kTile, buf ^= 1) {
            const long long tw = t0 + warp * kRows;
            const int rows = live ? (int)max(0ll, min((long long)kRows, len - tw)) : 0;
            Raw xr[kRows], gr[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                xr[r] = r < rows ? x[(tw + r) * pitch] : Raw(0);
                gr[r] = r < rows ? g[(tw + r) * pitch] : Raw(0);
            }
            float al[kRows][VC], A[VC], Bv[VC];
#pragma unroll
            for (int j = 0; j < VC; ++j) A[j] = 1.f, Bv[j] = 0.f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float xv[VC], gv[VC];
                L::get(xr[r], xv);
                L::get(gr[r], gv);
#pragma unroll
                for (int j = 0; j < VC; ++j) {
                    al[r][j] = r < rows ? decay<T, GATED>(gv[j], sc[j]) : 1.f;
                    A[j] *= al[r][j];
                    Bv[j] = al[r][j] * Bv[j] + xv[j];
                }
            }
#pragma unroll
            for (int j = 0; j < VC; ++j) pairs[buf][warp][lane * VC + j] = make_float2(A[j], Bv[j]);
            __syncthreads();      // two buffers: one barrier per tile is enough
            float hv[VC];
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
#pragma unroll
                for (int j = 0; j < VC; ++j) {
                    if (w == warp) hv[j] = carry[j];
                    const float2 p = pairs[buf][w][lane * VC + j];
                    carry[j] = p.x * carry[j] + p.y;
                }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float xv[VC];
                L::get(xr[r], xv);
#pragma unroll
                for (int j = 0; j < VC; ++j) hv[j] = al[r][j] * hv[j] + xv[j];
                if (r < rows) h[(tw + r) * pitch] = L::put(hv);
            }
        }
        if (a.ht && warp == 0 && live)
#pragma unroll
            for (int j = 0; j < VC; ++j) a.ht[(long long)n * s.D + ch + j] = carry[j];
    }
}

struct BwdArgs {
    const void *dh, *g, *h;
    const float *scale, *h0, *dht;
    void *dx, *dg;
    float *dh0, *partial;      // partial: [lanes_n][D], or null
};

// The same walk from the last token to the first: with e_t = dh_t + c_t, a token's
// map on the carried gradient is c -> a (dh + c), the pair (a, a dh).
template <typename T, int VC, bool GATED>
__global__ void __launch_bounds__(kThreads, 2) bwd_kernel(BwdArgs a, Shape s) {
    using L = Lane<T, VC>;
    using Raw = typename L::Raw;
    __shared__ float2 pairs[2][kWarps][32 * VC];
    pdl_enter();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = blockIdx.x % s.groups, first_n = blockIdx.x / s.groups;
    const int ch = group * 32 * VC + lane * VC;
    const bool live = ch < s.D;
    float sc[VC], dscale[VC];
#pragma unroll
    for (int j = 0; j < VC; ++j) {
        sc[j] = GATED && live ? a.scale[ch + j] : 0.f;
        dscale[j] = 0.f;
    }

    int buf = 0;
    for (int n = first_n; n < s.N; n += s.lanes_n) {
        long long bos, len;
        range(s, n, bos, len);
        const long long base = bos * s.D + ch, pitch = s.D / VC;
        const Raw *dh = reinterpret_cast<const Raw *>(reinterpret_cast<const T *>(a.dh) + base);
        const Raw *g = reinterpret_cast<const Raw *>(reinterpret_cast<const T *>(a.g) + base);
        const Raw *h = reinterpret_cast<const Raw *>(reinterpret_cast<const T *>(a.h) + base);
        Raw *dx = reinterpret_cast<Raw *>(reinterpret_cast<T *>(a.dx) + base);
        Raw *dg = reinterpret_cast<Raw *>(reinterpret_cast<T *>(a.dg) + base);
        float carry[VC], h0[VC];
#pragma unroll
        for (int j = 0; j < VC; ++j) {
            carry[j] = a.dht && live ? a.dht[(long long)n * s.D + ch + j] : 0.f;
            h0[j] = a.h0 && live ? a.h0[(long long)n * s.D + ch + j] : 0.f;
        }

        for (long long u0 = 0; u0 < len; u0 += kTile, buf ^= 1) {
            // token of row r: tw - r
            const long long tw = len - 1 - (u0 + warp * kRows);
            const int rows = live ? (int)max(0ll, min((long long)kRows, tw + 1)) : 0;
            Raw dr[kRows], gr[kRows], hr[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                dr[r] = r < rows ? dh[(tw - r) * pitch] : Raw(0);
                gr[r] = r < rows ? g[(tw - r) * pitch] : Raw(0);
                hr[r] = r < rows && r < tw ? h[(tw - r - 1) * pitch] : Raw(0);
            }
            float al[kRows][VC], A[VC], Bv[VC];
#pragma unroll
            for (int j = 0; j < VC; ++j) A[j] = 1.f, Bv[j] = 0.f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float dv[VC], gv[VC];
                L::get(dr[r], dv);
                L::get(gr[r], gv);
#pragma unroll
                for (int j = 0; j < VC; ++j) {
                    al[r][j] = r < rows ? decay<T, GATED>(gv[j], sc[j]) : 1.f;
                    A[j] *= al[r][j];
                    Bv[j] = al[r][j] * (Bv[j] + dv[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < VC; ++j) pairs[buf][warp][lane * VC + j] = make_float2(A[j], Bv[j]);
            __syncthreads();
            float c[VC];
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
#pragma unroll
                for (int j = 0; j < VC; ++j) {
                    if (w == warp) c[j] = carry[j];
                    const float2 p = pairs[buf][w][lane * VC + j];
                    carry[j] = p.x * carry[j] + p.y;
                }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float dv[VC], gv[VC], hv[VC], e[VC], dl[VC];
                L::get(dr[r], dv);
                L::get(gr[r], gv);
                L::get(hr[r], hv);
#pragma unroll
                for (int j = 0; j < VC; ++j) {
                    if (r == tw) hv[j] = h0[j];        // the token before the first is h0
                    e[j] = dv[j] + c[j];
                    c[j] = al[r][j] * e[j];
                    dl[j] = c[j] * hv[j];
                    if (GATED && r < rows) {
                        // d softplus = logistic(g) = 1 / (1 + e^-|g|), or e^-|g| times that
                        const float q = Fn<T>::gate_exp(-fabsf(gv[j]));
                        dscale[j] -= dl[j] * Fn<T>::softplus(gv[j], q);
                        dl[j] *= -sc[j] * (gv[j] >= 0.f ? 1.f : q) * Fn<T>::rcp(1.f + q);
                    }
                }
                if (r < rows) {
                    dx[(tw - r) * pitch] = L::put(e);
                    dg[(tw - r) * pitch] = L::put(dl);
                }
            }
        }
        if (a.dh0 && warp == 0 && live)
#pragma unroll
            for (int j = 0; j < VC; ++j) a.dh0[(long long)n * s.D + ch + j] = carry[j];
    }
    if (GATED && a.partial) {
        __syncthreads();
        float *sum = reinterpret_cast<float *>(pairs);
#pragma unroll
        for (int j = 0; j < VC; ++j) sum[(warp * 32 + lane) * VC + j] = dscale[j];
        __syncthreads();
        if (warp == 0 && live)
#pragma unroll
            for (int j = 0; j < VC; ++j) {
                float t = 0.f;
                for (int w = 0; w < kWarps; ++w) t += sum[(w * 32 + lane) * VC + j];
                a.partial[(long long)first_n * s.D + ch + j] = t;
            }
    }
}

// One token: a channel per thread.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256) step_kernel(const T *x, const T *g, const float *scale,
                                                   const float *state, T *h, float *out,
                                                   long long total, int D) {
    pdl_enter();
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const float a = decay<T, GATED>(to_f(g[i]), GATED ? scale[i % D] : 0.f);
        const float v = a * state[i] + to_f(x[i]);
        out[i] = v;
        from_f(h + i, v);
    }
}

// Channels a lane carries: bf16 pairs where every row starts on 4 bytes.
int lane_channels(int dtype, int D) { return dtype == GDN_BF16 && D % 2 == 0 ? 2 : 1; }

// Clusters (here single CTAs) that share a channel group's sequences: one each,
// but no more than fill the GPU several times over, so that the per-CTA partial
// sums of d(gate_scale) stay small beside the data.
int group_lanes(int N, int groups) {
    const int most = std::max(1, 4096 / groups);
    return std::min(N, std::max(most, 64));
}

gdn_status check(int B, int T, int D, int N, int dtype, bool packed) {
    if (B < 1 || T < 0 || D < 1) return fail(GDN_ERR_INVALID_ARG, "bad sizes B=%d T=%d D=%d", B, T, D);
    if (dtype != GDN_FP32 && dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_FP32 or GDN_BF16", dtype);
    if (packed && (B != 1 || N < 1))
        return fail(GDN_ERR_INVALID_ARG, "cu_seqlens needs B == 1 and N >= 1 (B=%d N=%d)", B, N);
    if ((long long)B * T >= (1ll << 31) || (long long)(packed ? N : B) * D >= (1ll << 40))
        return fail(GDN_ERR_INVALID_ARG, "problem too large");
    return GDN_OK;
}

Shape shape_of(const int32_t *cu, int B, int T, int D, int N, int dtype, int *status) {
    Shape s;
    s.cu = cu;
    s.T = T;
    s.N = cu ? N : B;
    s.D = D;
    const int width = 32 * lane_channels(dtype, D);
    s.groups = (D + width - 1) / width;
    s.lanes_n = group_lanes(s.N, s.groups);
    s.status = status;
    return s;
}

template <typename Args, typename K>
cudaError_t launch(const char *name, K kernel, const Args &a, const Shape &s, cudaStream_t st) {
    prof_before(name, st);
    const cudaError_t e = launch_pdl(kernel, dim3((unsigned)(s.groups * s.lanes_n)), dim3(kThreads),
                                     0, st, a, s);
    prof_after(st);
    return e;
}

#define GDN_LINREC_KERNEL(kernel)                                                               \
    (dtype == GDN_FP32 ? (gated ? kernel<float, 1, true> : kernel<float, 1, false>)             \
     : vc == 2 ? (gated ? kernel<__nv_bfloat16, 2, true> : kernel<__nv_bfloat16, 2, false>)     \
               : (gated ? kernel<__nv_bfloat16, 1, true> : kernel<__nv_bfloat16, 1, false>))

size_t bwd_workspace(const gdn_linrec_bwd_args *a) {
    if (!a->gate_scale || !a->d_gate_scale) return 256;
    const Shape s = shape_of(a->cu_seqlens, a->B, a->T, a->D, a->N, a->dtype, nullptr);
    return std::max<size_t>(256, (size_t)s.lanes_n * s.D * sizeof(float));
}

}  // namespace
}  // namespace linrec
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_linrec_fwd(const gdn_linrec_fwd_args *a, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = linrec::check(a->B, a->T, a->D, a->N, a->dtype, a->cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (a->T > 0 && (!a->x || !a->g || !a->h))
        return fail(GDN_ERR_INVALID_ARG, "x, g and h are required");
    if (misaligned(a->x) || misaligned(a->g) || misaligned(a->h) || misaligned(a->gate_scale) ||
        misaligned(a->initial_state) || misaligned(a->cu_seqlens) || misaligned(a->final_state))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    const linrec::Shape s = linrec::shape_of(a->cu_seqlens, a->B, a->T, a->D, a->N, a->dtype, dev.status);
    const int dtype = a->dtype, vc = linrec::lane_channels(dtype, a->D);
    const bool gated = a->gate_scale != nullptr;
    const linrec::FwdArgs f{a->x, a->g, a->gate_scale, a->initial_state, a->h, a->final_state};
    const cudaError_t e = linrec::launch("linrec_fwd", GDN_LINREC_KERNEL(linrec::fwd_kernel), f, s,
                                         (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "linear recurrence launch");
}

size_t gdn_linrec_bwd_workspace_size(const gdn_linrec_bwd_args *a) {
    if (!a) {
        fail(GDN_ERR_INVALID_ARG, "null args");
        return 0;
    }
    if (linrec::check(a->B, a->T, a->D, a->N, a->dtype, a->cu_seqlens != nullptr) != GDN_OK) return 0;
    return linrec::bwd_workspace(a);
}

gdn_status gdn_linrec_bwd(const gdn_linrec_bwd_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = linrec::check(a->B, a->T, a->D, a->N, a->dtype, a->cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (a->T > 0 && (!a->d_h || !a->g || !a->h || !a->dx || !a->dg))
        return fail(GDN_ERR_INVALID_ARG, "d_h, g, h, dx and dg are required");
    if (misaligned(a->d_h) || misaligned(a->g) || misaligned(a->h) || misaligned(a->gate_scale) ||
        misaligned(a->initial_state) || misaligned(a->cu_seqlens) || misaligned(a->d_final_state) ||
        misaligned(a->dx) || misaligned(a->dg) || misaligned(a->d_initial_state) ||
        misaligned(a->d_gate_scale))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    const bool gated = a->gate_scale != nullptr, sums = gated && a->d_gate_scale;
    if (sums && (!ws || misaligned(ws) || ws_bytes < linrec::bwd_workspace(a)))
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0,
                    linrec::bwd_workspace(a));
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    const linrec::Shape s = linrec::shape_of(a->cu_seqlens, a->B, a->T, a->D, a->N, a->dtype, dev.status);
    const int dtype = a->dtype, vc = linrec::lane_channels(dtype, a->D);
    const linrec::BwdArgs b{a->d_h, a->g, a->h, a->gate_scale, a->initial_state, a->d_final_state,
                            a->dx, a->dg, a->d_initial_state, sums ? (float *)ws : nullptr};
    cudaStream_t q = (cudaStream_t)stream;
    cudaError_t e = linrec::launch("linrec_bwd", GDN_LINREC_KERNEL(linrec::bwd_kernel), b, s, q);
    if (e == cudaSuccess && sums) {
        e = column_sum((const float *)ws, s.lanes_n, a->D, a->d_gate_scale, q);
    }
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "linear recurrence backward launch");
}

gdn_status gdn_linrec_step(const gdn_linrec_step_args *a, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    if (a->N < 0 || a->D < 1) return fail(GDN_ERR_INVALID_ARG, "bad sizes N=%d D=%d", a->N, a->D);
    if (a->dtype != GDN_FP32 && a->dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_FP32 or GDN_BF16", a->dtype);
    if (a->N == 0) return GDN_OK;
    if (!a->x || !a->g || !a->state || !a->h || !a->out_state)
        return fail(GDN_ERR_INVALID_ARG, "x, g, state, h and out_state are required");
    if (misaligned(a->x) || misaligned(a->g) || misaligned(a->gate_scale) || misaligned(a->state) ||
        misaligned(a->h) || misaligned(a->out_state))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    LayerDevice dev;
    const gdn_status st = layer_device(&dev);
    if (st != GDN_OK) return st;
    const long long total = (long long)a->N * a->D;
    const unsigned grid = (unsigned)std::min<long long>((total + 255) / 256, 8ll * dev.sms);
    cudaStream_t q = (cudaStream_t)stream;
    prof_before("linrec_step", q);
    cudaError_t e;
    if (a->dtype == GDN_BF16) {
        auto k = a->gate_scale ? linrec::step_kernel<__nv_bfloat16, true>
                               : linrec::step_kernel<__nv_bfloat16, false>;
        e = launch_pdl(k, dim3(grid), dim3(256), 0, q, (const __nv_bfloat16 *)a->x,
                       (const __nv_bfloat16 *)a->g, a->gate_scale, a->state, (__nv_bfloat16 *)a->h,
                       a->out_state, total, a->D);
    } else {
        auto k = a->gate_scale ? linrec::step_kernel<float, true> : linrec::step_kernel<float, false>;
        e = launch_pdl(k, dim3(grid), dim3(256), 0, q, (const float *)a->x, (const float *)a->g,
                       a->gate_scale, a->state, (float *)a->h, a->out_state, total, a->D);
    }
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "linear recurrence step launch");
}

}  // extern "C"
