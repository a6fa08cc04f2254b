// gdn_ffn_few.cu -- the feed-forward block's backward pass for a few tokens, in fp32 on the CUDA cores.
//
//     rows     out[m][c] = sum over r of v[m][r] W[r][c]:  dh from dy and Wd; dx from dg, Wg and du, Wu
//     outer    out[r][c] = sum over m of a[m][r] b[m][c]:  dWg, dWu, dWd
//
// Each weight is read once and each gradient written once; with eight tokens at most the arithmetic
// (64 multiply-adds for 16 bytes) keeps within their time, and dg, du and h stay fp32.
#include <algorithm>

#include "gdn_ffn.cuh"

namespace gdn {
namespace ffn {
namespace {

constexpr int kThreads = 128, kCols = 8 * kThreads;  // eight columns to a thread
constexpr int kRows = 64;                            // whose v are in shared memory at once
constexpr int kCtas = kSms * 4;                      // that are enough to fill the GPU

struct RowsArgs {
    const __nv_bfloat16 *w, *w2;   // [R, C]; w2: the rows from R on
    const __nv_bfloat16 *v16;      // [M, R], or
    const float *v, *v2;           // [M, R] each
    float *partial;                // [splits][M][C]
    int M, R, C, rows;             // rows of a split, of one or both matrices
};
__global__ void __launch_bounds__(kThreads) rows_kernel(RowsArgs a) {
    __shared__ __align__(16) float v[kRows][kFewTokens];
    pdl_enter();
    const int col = blockIdx.x * kCols + 8 * threadIdx.x, all = a.w2 ? 2 * a.R : a.R;
    const int r0 = blockIdx.y * a.rows, r1 = min(r0 + a.rows, all);
    const bool in = col < a.C;
    float2 acc[kFewTokens][4];
#pragma unroll
    for (int m = 0; m < kFewTokens; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = make_float2(0.f, 0.f);
    for (int base = r0; base < r1; base += kRows) {
        const int n = min(kRows, r1 - base);
        __syncthreads();
        for (int k = threadIdx.x; k < kRows * kFewTokens; k += kThreads) {
            const int r = base + k % kRows, m = k / kRows;
            float x = 0.f;
            if (m < a.M && r < r1) {
                const int at = r < a.R ? r : r - a.R;
                x = a.v16 ? to_f(a.v16[(long long)m * a.R + at]) : (r < a.R ? a.v : a.v2)[(long long)m * a.R + at];
            }
            v[k % kRows][m] = x;
        }
        __syncthreads();
        constexpr int kAhead = 8;                    // rows whose loads are in flight
        for (int k = 0; k < n; k += kAhead) {
            uint4 raw[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int r = base + k + j;
                raw[j] = make_uint4(0, 0, 0, 0);
                if (in && r < r1)
                    raw[j] = *reinterpret_cast<const uint4 *>((r < a.R ? a.w + (long long)r * a.C : a.w2 + (long long)(r - a.R) * a.C) + col);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                float w[8];
                Vec<__nv_bfloat16, 8>::get(raw[j], w);
                const float4 lo = *reinterpret_cast<const float4 *>(&v[k + j][0]), hi = *reinterpret_cast<const float4 *>(&v[k + j][4]);
                const float t[kFewTokens] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int m = 0; m < kFewTokens; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[m][i] = __ffma2_rn(make_float2(t[m], t[m]), make_float2(w[2 * i], w[2 * i + 1]), acc[m][i]);
            }
        }
    }
    if (!in) return;
#pragma unroll
    for (int m = 0; m < kFewTokens; ++m) {
        if (m >= a.M) break;
        float4 *to = reinterpret_cast<float4 *>(a.partial + ((long long)blockIdx.y * a.M + m) * a.C + col);
        to[0] = make_float4(acc[m][0].x, acc[m][0].y, acc[m][1].x, acc[m][1].y);
        to[1] = make_float4(acc[m][2].x, acc[m][2].y, acc[m][3].x, acc[m][3].y);
    }
}

// The splits' sums, in order; with gate and up: dh, of which dg, du and h are made, else dx.
struct FinishArgs {
    const float *partial;
    int splits;
    long long n;                   // M C
    const __nv_bfloat16 *gate, *up;
    float *dg, *du, *h;
    __nv_bfloat16 *dx;
    int gelu;
};
__global__ void __launch_bounds__(256) finish_kernel(FinishArgs a) {
    pdl_enter();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= a.n) return;
    float t = 0.f;
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) t += a.partial[s * a.n + i];
    if (!a.gate) {
        a.dx[i] = __float2bfloat16_rn(t);
        return;
    }
    const float g = to_f(a.gate[i]), u = to_f(a.up[i]);
    float slope;
    const float f = a.gelu ? activation<true>(g, slope) : activation<false>(g, slope);
    a.dg[i] = t * u * slope;
    a.du[i] = t * f;
    a.h[i] = f * u;
}

// A thread has eight columns of b and walks kRows rows of a.
struct OuterArgs {
    struct {
        const float *a, *b;        // [M, R], [M, C], or
        const __nv_bfloat16 *a16, *b16;
        __nv_bfloat16 *out;        // [R, C]
        int R, C;
    } p[3];
    int M;
};
__global__ void __launch_bounds__(kThreads) outer_kernel(const __grid_constant__ OuterArgs a) {
    __shared__ __align__(16) float v[kRows][kFewTokens];
    pdl_enter();
    const auto &p = a.p[blockIdx.z];
    const int col = blockIdx.x * kCols + 8 * threadIdx.x;
    if (blockIdx.x * kCols >= p.C) return;
    const bool in = col < p.C;
    float2 b[kFewTokens][4];
#pragma unroll
    for (int m = 0; m < kFewTokens; ++m) {
        float f[8] = {};
        if (in && m < a.M) {
            const long long at = (long long)m * p.C + col;
            if (p.b16) Vec<__nv_bfloat16, 8>::load(p.b16 + at, f);
            else Vec<float, 4>::load(p.b + at, f), Vec<float, 4>::load(p.b + at + 4, f + 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) b[m][i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
    for (int base = blockIdx.y * kRows; base < p.R; base += gridDim.y * kRows) {
        __syncthreads();
        for (int k = threadIdx.x; k < kRows * kFewTokens; k += kThreads) {
            const int r = base + k % kRows, m = k / kRows;
            const long long at = (long long)m * p.R + r;
            v[k % kRows][m] = m < a.M && r < p.R ? (p.a16 ? to_f(p.a16[at]) : p.a[at]) : 0.f;
        }
        __syncthreads();
        const int n = min(kRows, p.R - base);
        if (!in) continue;
        for (int k = 0; k < n; ++k) {
            const float4 lo = *reinterpret_cast<const float4 *>(&v[k][0]), hi = *reinterpret_cast<const float4 *>(&v[k][4]);
            const float t[kFewTokens] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            float2 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[i] = __fmul2_rn(make_float2(t[0], t[0]), b[0][i]);
#pragma unroll
                for (int m = 1; m < kFewTokens; ++m) o[i] = __ffma2_rn(make_float2(t[m], t[m]), b[m][i], o[i]);
            }
            const float f[8] = {o[0].x, o[0].y, o[1].x, o[1].y, o[2].x, o[2].y, o[3].x, o[3].y};
            Vec<__nv_bfloat16, 8>::store(p.out + (long long)(base + k) * p.C + col, f);
        }
    }
}

// Rows of a split: as few splits as fill the GPU, of whole kRows.
struct Split {
    int across, splits, rows;
};
Split split_of(int rows, int C) {
    const int across = (C + kCols - 1) / kCols;
    const int most = (rows + kRows - 1) / kRows, splits = std::max(1, std::min(most, std::min(kCtas / across + 1, 65535)));
    const int each = ((rows + splits - 1) / splits + kRows - 1) / kRows * kRows;
    return {across, (rows + each - 1) / each, each};
}
size_t partial_floats(int M, int K, int F) {
    return std::max((size_t)split_of(K, F).splits * M * F, (size_t)split_of(2 * F, K).splits * M * K);
}

cudaError_t launch_rows(RowsArgs r, cudaStream_t q) {
    const Split s = split_of(r.w2 ? 2 * r.R : r.R, r.C);
    r.rows = s.rows;
    prof_before("ffn_rows", q);
    const cudaError_t e = launch_pdl(rows_kernel, dim3(s.across, s.splits), dim3(kThreads), 0, q, r);
    prof_after(q);
    return e;
}
cudaError_t launch_finish(const FinishArgs &f, cudaStream_t q) {
    prof_before("ffn_finish", q);
    const cudaError_t e = launch_pdl(finish_kernel, dim3((unsigned)((f.n + 255) / 256)), dim3(256), 0, q, f);
    prof_after(q);
    return e;
}

}  // namespace

size_t few_bwd_bytes(int M, int K, int F) { return 4 * (3 * (size_t)M * F + partial_floats(M, K, F)); }

cudaError_t few_bwd(const gdn_ffn_bwd_args *a, float *ws, cudaStream_t q) {
    const auto bf = [](const void *p) { return (const __nv_bfloat16 *)p; };
    const long long n = (long long)a->M * a->F;
    float *dg = ws, *du = dg + n, *h = du + n, *partial = h + n;
    cudaError_t e = launch_rows({bf(a->w_down), nullptr, bf(a->d_y), nullptr, nullptr, partial, a->M, a->K, a->F, 0}, q);
    if (e == cudaSuccess)
        e = launch_finish({partial, split_of(a->K, a->F).splits, n, bf(a->gate), bf(a->up), dg, du, h, nullptr,
                           a->activation == GDN_ACT_GELU}, q);
    if (e == cudaSuccess)
        e = launch_rows({bf(a->w_gate), bf(a->w_up), nullptr, dg, du, partial, a->M, a->F, a->K, 0}, q);
    if (e == cudaSuccess)
        e = launch_finish({partial, split_of(2 * a->F, a->K).splits, (long long)a->M * a->K, nullptr, nullptr, nullptr,
                           nullptr, nullptr, (__nv_bfloat16 *)a->dx, 0}, q);
    if (e != cudaSuccess) return e;
    OuterArgs o{};
    o.p[0] = {dg, nullptr, nullptr, bf(a->x), (__nv_bfloat16 *)a->dw_gate, a->F, a->K};
    o.p[1] = {du, nullptr, nullptr, bf(a->x), (__nv_bfloat16 *)a->dw_up, a->F, a->K};
    o.p[2] = {nullptr, h, bf(a->d_y), nullptr, (__nv_bfloat16 *)a->dw_down, a->K, a->F};
    o.M = a->M;
    const int across = (std::max(a->K, a->F) + kCols - 1) / kCols, most = (std::max(a->K, a->F) + kRows - 1) / kRows;
    prof_before("ffn_outer", q);
    e = launch_pdl(outer_kernel, dim3(across, std::max(1, std::min(most, 4 * kCtas / across)), 3), dim3(kThreads), 0, q, o);
    prof_after(q);
    return e;
}

}  // namespace ffn
}  // namespace gdn
