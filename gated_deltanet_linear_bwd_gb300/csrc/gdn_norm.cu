// gdn_norm.cu -- residual addition with the RMS norm, to the input's type or to
// MXFP8 with its scales, and the backward pass.
//
// A row is held in registers, PER elements to a thread, by `tpr` threads (a power
// of two): loaded once, reduced by shuffles (and through shared memory where a row
// spans warps), scaled and written, while the next row's loads are in flight.  Rows of
// few columns share a CTA.  Bound by memory: 32768 x 4096 bf16
// with a residual to MXFP8 151 us, 92% of the measured copy rate (to bf16 161 us, 98%);
// backward of 16384 x 4096 89 us, 89%.
#include <algorithm>

#include "gdn_layer_internal.h"
#include "gdn_mx.cuh"

namespace gdn {
namespace norm {
namespace {

constexpr int kMaxD = 1024 * 16;

// VEC elements of T as one 16-byte load (or one element where rows do not start
// on 16 bytes).
template <typename T, int VEC>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ void get(Raw r, float *v) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ Raw put(const float *v) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Chunk<float, 4> {
    using Raw = float4;
    static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
    static __device__ __forceinline__ void get(Raw r, float *v) { v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w; }
    static __device__ __forceinline__ Raw put(const float *v) { return make_float4(v[0], v[1], v[2], v[3]); }
};
template <typename T>
struct Chunk<T, 1> {
    using Raw = T;
    static __device__ __forceinline__ Raw zero() { return T(0.f); }
    static __device__ __forceinline__ void get(Raw r, float *v) { v[0] = to_f(r); }
    static __device__ __forceinline__ Raw put(const float *v) {
        T r;
        from_f(&r, v[0]);
        return r;
    }
};

// A thread's share of a row: NV chunks, chunk v at column (v tpr + tid) VEC.
template <typename T, int VEC, int PER>
struct Share {
    using C = Chunk<T, VEC>;
    static constexpr int NV = PER / VEC;
    typename C::Raw raw[NV];
    __device__ __forceinline__ void load(const void *base, long long at, int tid, int tpr, int D, bool live) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = (v * tpr + tid) * VEC;
            raw[v] = live && col < D
                         ? *reinterpret_cast<const typename C::Raw *>(reinterpret_cast<const T *>(base) + at + col)
                         : C::zero();
        }
    }
};
template <typename T, int VEC>
__device__ __forceinline__ void store_chunk(void *base, long long at, const float *v) {
    using C = Chunk<T, VEC>;
    *reinterpret_cast<typename C::Raw *>(reinterpret_cast<T *>(base) + at) = C::put(v);
}

// Sum over a row's `tpr` threads; every one of them gets it.  `red` holds one float
// per warp, two of them used in turn so that one barrier a row is enough; the whole
// CTA calls.
__device__ __forceinline__ float row_sum(float x, int tpr, float *red) {
    for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (tpr <= 32) return x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = tpr >> 5;      // a power of two
    if (lane == 0) red[warp] = x;
    __syncthreads();
    x = red[(warp & ~(per - 1)) + (lane & (per - 1))];
    for (int o = per >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// The larger magnitude, or NaN if there is one.
__device__ __forceinline__ float max_abs(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

struct FwdArgs {
    const void *x, *res, *w;
    void *y, *sum;
    uint8_t *scales;
    float *rstd;
    float eps, inv_d;
    int rows, D, tpr, ktiles;
};

template <typename T, int VEC, int PER, bool MX, int THREADS>
__global__ void __launch_bounds__(THREADS) fwd_kernel(FwdArgs a) {
    using C = Chunk<T, VEC>;
    constexpr int NV = PER / VEC;
    __shared__ float red[2][32];
    pdl_enter();

    const int tid = threadIdx.x & (a.tpr - 1), per_cta = blockDim.x / a.tpr;
    const int group = threadIdx.x / a.tpr;
    const bool words = a.tpr >= 128 / VEC;           // a scale tile's four blocks are neighbouring lanes
    Share<T, VEC, PER> w, x, r;
    w.load(a.w, 0, tid, a.tpr, a.D, true);
    // with MX scales the last tile's rows past the end are walked too: their scales are zeros
    const long long last = MX ? (a.rows + 127ll) / 128 * 128 : a.rows, step = (long long)gridDim.x * per_cta;
    long long row = (long long)blockIdx.x * per_cta + group, base = row * a.D;
    auto fetch = [&](long long at, bool in) {
        x.load(a.x, at, tid, a.tpr, a.D, in);
        if (a.res) r.load(a.res, at, tid, a.tpr, a.D, in);
    };
    if (VEC > 1) fetch(base, row < a.rows);
    int turn = 0;
    for (; row - group < last; row += step, base += step * a.D, turn ^= 1) {
        const bool live = row < a.rows;
        if (VEC == 1) fetch(base, live);
        // pairs of neighbouring columns (VEC 1: a column and one that is not there)
        constexpr int P = VEC > 1 ? VEC / 2 : 1;
        float2 s[NV][P], ss2 = both(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = (v * a.tpr + tid) * VEC;
            float *sv = reinterpret_cast<float *>(s[v]);
            if (VEC == 1) s[v][0].y = 0.f;
            C::get(x.raw[v], sv);
            if (a.res) {
                float2 q[P];
                if (VEC == 1) q[0].y = 0.f;
                C::get(r.raw[v], reinterpret_cast<float *>(q));
#pragma unroll
                for (int i = 0; i < P; ++i) s[v][i] = __fadd2_rn(s[v][i], q[i]);
                if (live && col < a.D) store_chunk<T, VEC>(a.sum, base + col, sv);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) ss2 = __ffma2_rn(s[v][i], s[v][i], ss2);
        }
        if (VEC > 1) fetch(base + step * a.D, row + step < a.rows);
        const float rstd = rsqrtf(row_sum(ss2.x + ss2.y, a.tpr, red[turn]) * a.inv_d + a.eps);
        if (live && a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = (v * a.tpr + tid) * VEC;
            float2 y[P];
            if (VEC == 1) y[0].y = 0.f;
            C::get(w.raw[v], reinterpret_cast<float *>(y));
#pragma unroll
            for (int i = 0; i < P; ++i) y[i] = __fmul2_rn(__fmul2_rn(s[v][i], both(rstd)), y[i]);
            if constexpr (!MX) {
                if (live && col < a.D) store_chunk<T, VEC>(a.y, base + col, reinterpret_cast<float *>(y));
            } else {
                // a block of 32 columns is 32 / VEC neighbouring lanes
                float big = 0.f;
#pragma unroll
                for (int i = 0; i < P; ++i) big = max_abs(max_abs(big, y[i].x), y[i].y);
                uint32_t amax = mx::abs_bits(big);
#pragma unroll
                for (int o = 1; o < 32 / VEC; o <<= 1)
                    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                // 0 where nothing is, whose zeros an infinite or NaN rstd makes NaN
                const int byte = live && col < a.D ? mx::scale_byte<false>(amax) : 0;
                if (words) {
                    uint32_t word = (uint32_t)byte << (8 * (col / 32 & 3));
#pragma unroll
                    for (int o = 32 / VEC; o < 128 / VEC; o <<= 1)
                        word |= __shfl_xor_sync(0xffffffffu, word, o);
                    if (col < a.ktiles * 128 && col % 128 == 0 && row < last)
                        *reinterpret_cast<uint32_t *>(a.scales + mx::scale_offset(row, col / 32, a.ktiles)) = word;
                } else if (col < a.ktiles * 128 && col % 32 == 0 && row < last) {
                    a.scales[mx::scale_offset(row, col / 32, a.ktiles)] = (uint8_t)byte;
                }
                if (live && col < a.D) {
                    const float2 f = both(mx::scale_factor(byte));
                    const bool bad = byte == 255;                    // the elements of a NaN block are zeros
#pragma unroll
                    for (int i = 0; i < P; ++i) y[i] = __fmul2_rn(y[i], f);
                    uint32_t *o = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(a.y) + base + col);
                    const uint32_t q0 = mx::e4m3x4(y[0].x, y[0].y, y[1].x, y[1].y);
                    if constexpr (VEC == 8) {
                        const uint32_t q1 = mx::e4m3x4(y[2].x, y[2].y, y[3].x, y[3].y);
                        *reinterpret_cast<uint2 *>(o) = make_uint2(bad ? 0u : q0, bad ? 0u : q1);
                    } else {
                        *o = bad ? 0u : q0;
                    }
                }
            }
        }
    }
}

struct BwdArgs {
    const void *dy, *s, *w, *dsum;
    const float *rstd;
    void *ds;
    float *partial;                // [gridDim.x][D]
    float inv_d;
    int rows, D, tpr;
};

template <typename T, int VEC, int PER, int THREADS>
__global__ void __launch_bounds__(THREADS) bwd_kernel(BwdArgs a) {
    using C = Chunk<T, VEC>;
    constexpr int NV = PER / VEC;
    extern __shared__ float sums[];          // [rows per CTA][D], where a CTA holds several rows
    __shared__ float red[2][32];
    pdl_enter();

    const int tid = threadIdx.x & (a.tpr - 1), per_cta = blockDim.x / a.tpr;
    const int group = threadIdx.x / a.tpr;
    Share<T, VEC, PER> w, dy, s, up;
    w.load(a.w, 0, tid, a.tpr, a.D, true);
    float dw[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) dw[i] = 0.f;
    const long long step = (long long)gridDim.x * per_cta;
    long long row = (long long)blockIdx.x * per_cta + group;
    float rs;
    auto fetch = [&](long long at) {
        const bool in = at < a.rows;
        dy.load(a.dy, at * a.D, tid, a.tpr, a.D, in);
        s.load(a.s, at * a.D, tid, a.tpr, a.D, in);
        if (a.dsum) up.load(a.dsum, at * a.D, tid, a.tpr, a.D, in);
        rs = in ? a.rstd[at] : 0.f;
    };
    if (VEC > 1) fetch(row);
    int turn = 0;
    for (; row - group < a.rows; row += step, turn ^= 1) {
        const bool live = row < a.rows;
        if (VEC == 1) fetch(row);
        const long long base = row * a.D;
        const float rstd = rs;
        float xh[PER], wdy[PER], dot = 0.f;
        Share<T, VEC, PER> dsum = up;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float g[VEC];
            C::get(s.raw[v], xh + v * VEC);
            C::get(dy.raw[v], wdy + v * VEC);
            C::get(w.raw[v], g);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = v * VEC + i;
                xh[k] *= rstd;
                dw[k] += wdy[k] * xh[k];
                wdy[k] *= g[i];
                dot += wdy[k] * xh[k];
            }
        }
        if (VEC > 1) fetch(row + step);
        const float c = row_sum(dot, a.tpr, red[turn]) * a.inv_d;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = (v * a.tpr + tid) * VEC;
            if (!live || col >= a.D) continue;
            float d[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) d[i] = 0.f;
            if (a.dsum) C::get(dsum.raw[v], d);
#pragma unroll
            for (int i = 0; i < VEC; ++i) d[i] += rstd * (wdy[v * VEC + i] - xh[v * VEC + i] * c);
            store_chunk<T, VEC>(a.ds, base + col, d);
        }
    }
    // the CTA's sum of dy xh over its rows, the row groups added in order
    float *out = a.partial + (long long)blockIdx.x * a.D;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int col = (v * a.tpr + tid) * VEC + i;
            if (col < a.D) (per_cta > 1 ? sums + group * a.D : out)[col] = dw[v * VEC + i];
        }
    if (per_cta > 1) {
        __syncthreads();
        for (int col = threadIdx.x; col < a.D; col += blockDim.x) {
            float t = 0.f;
            for (int k = 0; k < per_cta; ++k) t += sums[k * a.D + col];
            out[col] = t;
        }
    }
}

// Whole 16-byte chunks in every row.
bool vector_rows(int dtype, int D) { return D % (dtype == GDN_BF16 ? 8 : 4) == 0; }

// Elements to a thread: 16, or 8 of rows that are read one by one (a register each).  Us with 8 |
// 16: 16000 x 4095 bf16 forward 164 | 208, backward 229 | 168; 60000 x 1001 128 | 187, 151 | 153; in
// fp32 8000 x 4095 126 | 138, 132 | 155, 30000 x 1001 102 | 127, 89 | 142.  (The backward pass of wide
// bf16 rows is the exception, and of rows of over 4096 columns, 9224 x 7275 228 | 201.)
int per_thread(int dtype, int D) { return vector_rows(dtype, D) || D > 8192 ? 16 : 8; }
// Threads of a row: the least power of two that holds it; 8 with MX scales, so that a
// scale tile's blocks have threads.
int row_threads(int dtype, int D, bool mx) {
    int t = mx ? 8 : 1;
    while (t * per_thread(dtype, D) < D) t *= 2;
    return t;
}
int cta_threads(int tpr) { return std::max(tpr, 256); }

// CTAs of the backward pass: as many as run at once (2 of 256 threads per SM, 3 where rows
// are read one by one), since each leaves a row of partial sums of dweight.
int bwd_ctas(int rows, int dtype, int D, int sms) {
    const int tpr = row_threads(dtype, D, false), threads = cta_threads(tpr), per = threads / tpr;
    const long long most = (long long)sms * std::max(1, (vector_rows(dtype, D) ? 2 : 3) * 256 / threads);
    return (int)std::max(1ll, std::min((rows - 1ll + per) / per, most));
}

template <typename T, int VEC, int PER, bool MX>
auto fwd_of(int threads) {
    return threads <= 256   ? fwd_kernel<T, VEC, PER, MX, 256>
           : threads <= 512 ? fwd_kernel<T, VEC, PER, MX, 512>
                            : fwd_kernel<T, VEC, PER, MX, 1024>;
}
template <typename T, int VEC, int PER>
auto bwd_of(int threads) {
    return threads <= 256   ? bwd_kernel<T, VEC, PER, 256>
           : threads <= 512 ? bwd_kernel<T, VEC, PER, 512>
                            : bwd_kernel<T, VEC, PER, 1024>;
}
// Rows read one by one; PER 16 has a row of over 8192 columns, hence 1024 threads.
template <typename T>
auto odd_fwd_of(int D, int threads) {
    return D > 8192 ? fwd_kernel<T, 1, 16, false, 1024> : fwd_of<T, 1, 8, false>(threads);
}
template <typename T>
auto odd_bwd_of(int D, int threads) {
    return D > 8192 ? bwd_kernel<T, 1, 16, 1024> : bwd_of<T, 1, 8>(threads);
}

// The GPU's SM count enters the workspace's size, which is asked for without a
// device: sized for the most SMs of an sm_103a part.
constexpr int kMaxSms = 160;

gdn_status check(int rows, int D, int dtype) {
    if (rows < 0 || D < 1) return fail(GDN_ERR_INVALID_ARG, "bad sizes rows=%d D=%d", rows, D);
    if (D > kMaxD) return fail(GDN_ERR_UNSUPPORTED, "D = %d (at most %d)", D, kMaxD);
    if (dtype != GDN_FP32 && dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_FP32 or GDN_BF16", dtype);
    return GDN_OK;
}

}  // namespace
}  // namespace norm
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_rms_norm_fwd(const gdn_rms_norm_fwd_args *a, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = norm::check(a->rows, a->D, a->dtype);
    if (st != GDN_OK) return st;
    if (a->mx != 0 && a->mx != 1) return fail(GDN_ERR_INVALID_ARG, "mx = %d (0 or 1)", a->mx);
    if (a->mx && a->D % 32 != 0)
        return fail(GDN_ERR_UNSUPPORTED, "D = %d: MXFP8 output takes multiples of 32", a->D);
    if (a->rows == 0) return GDN_OK;
    if (!a->x || !a->weight || !a->y || (a->mx && !a->scales) || (a->residual && !a->sum))
        return fail(GDN_ERR_INVALID_ARG, "x, weight, y, scales (for MXFP8) and sum (with a residual) are required");
    if (misaligned(a->x) || misaligned(a->residual) || misaligned(a->weight) || misaligned(a->y) ||
        misaligned(a->scales) || misaligned(a->sum) || misaligned(a->rstd))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    norm::FwdArgs f{a->x, a->residual, a->weight, a->y, a->sum, a->scales, a->rstd, a->eps,
                    1.f / (float)a->D, a->rows, a->D, norm::row_threads(a->dtype, a->D, a->mx != 0), (a->D + 127) / 128};
    const int threads = norm::cta_threads(f.tpr), per = threads / f.tpr;
    const long long rows = a->mx ? (a->rows + 127ll) / 128 * 128 : a->rows;
    const long long ctas = std::min<long long>((rows + per - 1) / per, (long long)dev.sms * (8 * 256 / threads));
    const bool vec = norm::vector_rows(a->dtype, a->D);
    auto k = a->dtype == GDN_BF16 ? (a->mx ? norm::fwd_of<__nv_bfloat16, 8, 16, true>(threads)
                                     : vec ? norm::fwd_of<__nv_bfloat16, 8, 16, false>(threads)
                                           : norm::odd_fwd_of<__nv_bfloat16>(a->D, threads))
                                  : (a->mx ? norm::fwd_of<float, 4, 16, true>(threads)
                                     : vec ? norm::fwd_of<float, 4, 16, false>(threads)
                                           : norm::odd_fwd_of<float>(a->D, threads));
    cudaStream_t q = (cudaStream_t)stream;
    prof_before("rms_norm_fwd", q);
    const cudaError_t e = launch_pdl(k, dim3((unsigned)ctas), dim3(threads), 0, q, f);
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "rms norm launch");
}

size_t gdn_rms_norm_bwd_workspace_size(const gdn_rms_norm_bwd_args *a) {
    if (!a) {
        fail(GDN_ERR_INVALID_ARG, "null args");
        return 0;
    }
    if (norm::check(a->rows, a->D, a->dtype) != GDN_OK) return 0;
    return std::max<size_t>(256, (size_t)norm::bwd_ctas(a->rows, a->dtype, a->D, norm::kMaxSms) * a->D * 4);
}

gdn_status gdn_rms_norm_bwd(const gdn_rms_norm_bwd_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = norm::check(a->rows, a->D, a->dtype);
    if (st != GDN_OK) return st;
    if ((a->rows > 0 && (!a->dy || !a->sum || !a->rstd || !a->ds)) || !a->weight || !a->dweight)
        return fail(GDN_ERR_INVALID_ARG, "dy, sum, weight, rstd, ds and dweight are required");
    if (misaligned(a->dy) || misaligned(a->sum) || misaligned(a->weight) || misaligned(a->rstd) ||
        misaligned(a->d_sum) || misaligned(a->ds) || misaligned(a->dweight))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    const size_t need = gdn_rms_norm_bwd_workspace_size(a);
    if (!ws || misaligned(ws) || ws_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    const int ctas = norm::bwd_ctas(a->rows, a->dtype, a->D, std::min(dev.sms, norm::kMaxSms));
    const int tpr = norm::row_threads(a->dtype, a->D, false), threads = norm::cta_threads(tpr), per = threads / tpr;
    const norm::BwdArgs b{a->dy, a->sum, a->weight, a->d_sum, a->rstd, a->ds, (float *)ws,
                          1.f / (float)a->D, a->rows, a->D, tpr};
    const bool vec = norm::vector_rows(a->dtype, a->D);
    auto k = a->dtype == GDN_BF16
                 ? (vec ? norm::bwd_of<__nv_bfloat16, 8, 16>(threads) : norm::odd_bwd_of<__nv_bfloat16>(a->D, threads))
                 : (vec ? norm::bwd_of<float, 4, 16>(threads) : norm::odd_bwd_of<float>(a->D, threads));
    // rows that share a CTA: 256 / tpr of at most 16 tpr columns, 16 KB of sums
    const size_t smem = per > 1 ? (size_t)per * a->D * sizeof(float) : 0;
    cudaStream_t q = (cudaStream_t)stream;
    prof_before("rms_norm_bwd", q);
    cudaError_t e = launch_pdl(k, dim3(ctas), dim3(threads), smem, q, b);
    prof_after(q);
    if (e == cudaSuccess) e = column_sum((const float *)ws, ctas, a->D, a->dweight, q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "rms norm backward launch");
}

}  // extern "C"
