// gdn_mx_gemm.cu -- C = A B^T of microscaled matrices on the block-scaled tcgen05
// MMAs.
//
// One CTA makes 128 rows of B (features) x `nt` rows of A (tokens) of C: the weight
// is the MMA's 128-row operand, so that few tokens cost a narrow MMA and not idle
// rows.  A producer warp feeds a ring of stages with TMA (both operand tiles and
// both scale tiles, 128 bytes of K at a time), one warp copies scales to TMEM and
// issues the MMAs, and the fp32 tile leaves TMEM through shared memory so that
// rows of C are written 128 features at a time.
#include <algorithm>

#include "gdn_layer_internal.h"
#include "tc_mx_ptx.cuh"

namespace gdn {
namespace mx {
namespace {

constexpr int kFeat = 128;         // features of a tile
constexpr int kThreads = 192;      // producer, MMA and four epilogue warps
constexpr int kMaxStages = 8;

struct GemmArgs {
    const uint8_t *sx, *sw;        // scales of tokens and features
    void *c;
    int tokens, feats, K;
    int nt, token_tiles;
    int kblocks, ktiles;           // 128-byte blocks of K, scale tiles along K
    int stages, stage_bytes, tmem_cols;
    int c_fp32;
    int *status;
    long long spin_limit;
};

struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages], done;
    uint32_t tmem;
    int failed, issued;
};

__device__ __forceinline__ void store_c4(const GemmArgs &a, long long row, int col, float4 v) {
    const long long at = row * a.feats + col;
    if ((a.feats & 3) == 0) {
        if (col >= a.feats) return;
        const float x[4] = {v.x, v.y, v.z, v.w};
        if (a.c_fp32) tc::st4(reinterpret_cast<float *>(a.c) + at, x);
        else tc::st4(reinterpret_cast<__nv_bfloat16 *>(a.c) + at, x);
        return;
    }
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (col + j < a.feats) {
            if (a.c_fp32) reinterpret_cast<float *>(a.c)[at + j] = x[j];
            else reinterpret_cast<__nv_bfloat16 *>(a.c)[at + j] = __float2bfloat16_rn(x[j]);
        }
}

template <bool FP4>
__global__ void __launch_bounds__(kThreads) gemm_kernel(const __grid_constant__ CUtensorMap map_x,
                                                        const __grid_constant__ CUtensorMap map_w,
                                                        const GemmArgs a) {
    constexpr int kStep = FP4 ? 64 : 32;            // K of one MMA
    constexpr int kBlock = 4 * kStep;               // K of a stage
    constexpr int kScaleTiles = kBlock / 128;       // scale tiles of a stage: 1 or 2
    extern __shared__ uint8_t raw[];
    __shared__ Control ctl;
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_rank(), splits = (int)tc::cluster_size();
    const int tile = blockIdx.x / splits;
    const int f0 = tile / a.token_tiles * kFeat, t0 = tile % a.token_tiles * a.nt;
    const int kb0 = (int)((long long)a.kblocks * rank / splits);
    const int kb1 = (int)((long long)a.kblocks * (rank + 1) / splits);

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            tc::mbar_init(&ctl.full[s], 1);
            tc::mbar_init(&ctl.empty[s], 1);
        }
        tc::mbar_init(&ctl.done, 1);
        ctl.failed = 0;
        tc::fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&ctl.tmem, (uint32_t)a.tmem_cols);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    pdl_enter();

    const uint32_t x_off = kFeat * 128, sw_off = x_off + a.nt * 128, sx_off = sw_off + kScaleTiles * 512;
    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int kb = kb0;
            for (; kb < kb1; ++kb) {
                const int i = kb - kb0, s = i % a.stages;
                if (i >= a.stages)
                    ok = tc::mbar_wait(&ctl.empty[s], (i / a.stages - 1) & 1, a.spin_limit, a.status);
                if (!ok) break;
                uint8_t *st = ring + s * a.stage_bytes;
                const uint32_t sb = 512u * (uint32_t)min(kScaleTiles, a.ktiles - kb * kScaleTiles);
                tc::mbar_arrive_expect_tx(&ctl.full[s], (uint32_t)(kFeat + a.nt) * 128u + 2u * sb);
                tc::tma_load_2d(st, &map_w, &ctl.full[s], kb * 128, f0);
                tc::tma_load_2d(st + x_off, &map_x, &ctl.full[s], kb * 128, t0);
                tc::bulk_load(st + sw_off, a.sw + ((long long)(f0 / 128) * a.ktiles + kb * kScaleTiles) * 512,
                              sb, &ctl.full[s]);
                tc::bulk_load(st + sx_off, a.sx + ((long long)(t0 / 128) * a.ktiles + kb * kScaleTiles) * 512,
                              sb, &ctl.full[s]);
            }
            if (!ok) ctl.failed = 1;
            ctl.issued = kb - kb0;
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t tsw = tmem + a.nt, tsx = tsw + 4 * kScaleTiles;
        for (int kb = kb0; kb < kb1; ++kb) {
            const int i = kb - kb0, s = i % a.stages;
            const bool full = tc::mbar_wait(&ctl.full[s], (i / a.stages) & 1, a.spin_limit, a.status);
            if (!__all_sync(0xffffffffu, full)) {
                ctl.failed = 1;
                break;
            }
            tc::tc_fence_after();
            const uint32_t st = tc::smem_u32(ring + s * a.stage_bytes);
            const int tiles = min(kScaleTiles, a.ktiles - kb * kScaleTiles);
            for (int k = 0; k < tiles; ++k) {
                tc::copy_scales(tsw + 4 * k, tc::desc_scales(st + sw_off + 512 * k));
                tc::copy_scales(tsx + 4 * k, tc::desc_scales(st + sx_off + 512 * k));
            }
            const uint64_t dw = tc::desc_sw128(st, 0, 1024), dx = tc::desc_sw128(st + x_off, 0, 1024);
            const int steps = min(4, (a.K - kb * kBlock + kStep - 1) / kStep);
            for (int j = 0; j < steps; ++j) {
                const int id = FP4 ? 2 * (j & 1) : j, col = FP4 ? 4 * (j >> 1) : 0;
                tc::mma_mx<FP4>(tmem, dw + 2 * j, dx + 2 * j, tc::idesc_mx(FP4, kFeat, a.nt, id),
                                tsw + col, tsx + col, i > 0 || j > 0);
            }
            tc::mma_commit(&ctl.empty[s]);
        }
        tc::mma_commit(&ctl.done);
    }
    __syncwarp();
    // every MMA done: the ring is free and the tile is whole
    if (!tc::mbar_wait(&ctl.done, 0, a.spin_limit, a.status)) {
        ctl.failed = 1;
        tc::mbar_drain(&ctl.done, 0);
    }
    tc::tc_fence_after();
    __syncthreads();
    const bool ok = ctl.failed == 0;
    if (!ok && threadIdx.x == 0)   // a wait gave up: nothing may land after the CTA has gone
        for (int j = max(0, ctl.issued - a.stages); j < ctl.issued; ++j)
            tc::mbar_drain(&ctl.full[j % a.stages], (j / a.stages) & 1);
    float *out = reinterpret_cast<float *>(ring);    // [nt][128]
    if (ok && warp >= 2) {
        for (int c = 0; c < a.nt; c += 16) {
            float v[16];
            tc::tmem_ld8x2(tc::tmem_addr(tmem, warp, c), tc::tmem_addr(tmem, warp, c + 8), v, v + 8);
#pragma unroll
            for (int j = 0; j < 16; ++j) out[(c + j) * kFeat + 32 * (warp & 3) + lane] = v[j];
        }
    }
    tc::tc_fence_before();
    if (splits > 1) tc::cluster_sync();
    else __syncthreads();
    tc::tc_fence_after();
    if (ok) {
        const uint32_t base = tc::smem_u32(out);
        for (int j = rank * (kThreads / 32) + warp; j < a.nt && t0 + j < a.tokens; j += splits * (kThreads / 32)) {
            const uint32_t at = base + (uint32_t)(j * kFeat + 4 * lane) * 4u;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < splits; ++r) {
                const float4 p = tc::ld_cluster4(tc::map_rank(at, r));
                v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
            }
            store_c4(a, t0 + j, f0 + 4 * lane, v);
        }
    }
    if (splits > 1) tc::cluster_sync();              // the others have read this CTA's tile
    if (warp == 1) tc::tmem_dealloc(tmem, (uint32_t)a.tmem_cols);
}

gdn_status run(const gdn_mx_matmul_args *a, const LayerDevice &dev, cudaStream_t q) {
    const bool fp4 = a->format == GDN_MXFP4;
    cudaError_t e = tc::encoder();
    if (e != cudaSuccess) return cuda_fail(e, "cuTensorMapEncodeTiled lookup");
    GemmArgs g{};
    g.sx = a->a_scales;
    g.sw = a->b_scales;
    g.c = a->c;
    g.tokens = a->M, g.feats = a->N, g.K = a->K;
    g.nt = 16;
    while (g.nt < 128 && g.nt < a->M) g.nt *= 2;
    g.token_tiles = (a->M + g.nt - 1) / g.nt;
    g.kblocks = (a->K + (fp4 ? 255 : 127)) / (fp4 ? 256 : 128);
    g.ktiles = (a->K + 127) / 128;
    g.stage_bytes = (kFeat + g.nt) * 128 + (fp4 ? 2048 : 1024);
    g.stages = std::min(kMaxStages, 96 * 1024 / g.stage_bytes);
    g.tmem_cols = 32;
    while (g.tmem_cols < g.nt + 16) g.tmem_cols *= 2;
    g.c_fp32 = a->out_dtype == GDN_FP32;
    g.status = dev.status;
    g.spin_limit = dev.spin_limit;
    const long long bytes = fp4 ? a->K / 2 : a->K;
    CUtensorMap mapx, mapw;
    if ((e = tc::make_map_bytes(&mapx, a->a, a->M, bytes, g.nt)) != cudaSuccess ||
        (e = tc::make_map_bytes(&mapw, a->b, a->N, bytes, kFeat)) != cudaSuccess)
        return cuda_fail(e, "tensor map of an operand");
    const size_t smem = std::max(g.stages * g.stage_bytes, g.nt * kFeat * 4) + 1024;
    auto k = fp4 ? gemm_kernel<true> : gemm_kernel<false>;
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
        return cuda_fail(e, "shared memory of the product");
    const int splits = 1;
    const long long ctas = (long long)((a->N + kFeat - 1) / kFeat) * g.token_tiles * splits;
    if (ctas >= (1ll << 31)) return fail(GDN_ERR_INVALID_ARG, "problem too large");
    prof_before("mx_gemm", q);
    e = launch_pdl_cluster(k, dim3((unsigned)ctas), dim3(kThreads), smem, splits, q, mapx, mapw, g);
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "mx product launch");
}

}  // namespace
}  // namespace mx
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_mx_matmul(const gdn_mx_matmul_args *a, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    if (a->M < 0 || a->N < 0 || a->K < 0)
        return fail(GDN_ERR_INVALID_ARG, "bad sizes M=%d N=%d K=%d", a->M, a->N, a->K);
    if (a->K % 32 != 0) return fail(GDN_ERR_UNSUPPORTED, "K = %d (a multiple of 32)", a->K);
    if (a->format != GDN_MXFP8 && a->format != GDN_MXFP4)
        return fail(GDN_ERR_UNSUPPORTED, "format %d is not GDN_MXFP8 or GDN_MXFP4", a->format);
    if (a->out_dtype != GDN_FP32 && a->out_dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "out_dtype %d is not GDN_FP32 or GDN_BF16", a->out_dtype);
    if (a->M == 0 || a->N == 0) return GDN_OK;
    if (!a->c || (a->K > 0 && (!a->a || !a->a_scales || !a->b || !a->b_scales)))
        return fail(GDN_ERR_INVALID_ARG, "a, b, their scales and c are required");
    if (misaligned(a->a) || misaligned(a->a_scales) || misaligned(a->b) || misaligned(a->b_scales) ||
        misaligned(a->c))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    LayerDevice dev;
    const gdn_status st = layer_device(&dev);
    if (st != GDN_OK) return st;
    if (a->K == 0) {
        const cudaError_t e = cudaMemsetAsync(a->c, 0, (size_t)a->M * a->N * (a->out_dtype == GDN_FP32 ? 4 : 2),
                                              (cudaStream_t)stream);
        return e == cudaSuccess ? GDN_OK : cuda_fail(e, "clearing c");
    }
    return mx::run(a, dev, (cudaStream_t)stream);
}

// Bytes of X's elements in the workspace, its scales following.
static size_t linear_data_bytes(const gdn_mx_linear_args *a) {
    const size_t n = (size_t)a->M * a->K;
    return ((a->format == GDN_MXFP4 ? n / 2 : n) + 255) / 256 * 256;
}

extern "C" size_t gdn_mx_linear_workspace_size(const gdn_mx_linear_args *a) {
    if (!a || a->M < 0 || a->K < 0) {
        fail(GDN_ERR_INVALID_ARG, "null args or bad sizes");
        return 0;
    }
    return std::max<size_t>(256, linear_data_bytes(a) + gdn_mx_scale_bytes(a->M, a->K));
}

extern "C" gdn_status gdn_mx_linear(const gdn_mx_linear_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    const size_t need = gdn_mx_linear_workspace_size(a);
    if (need == 0) return GDN_ERR_INVALID_ARG;
    if (!ws || misaligned(ws) || ws_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    uint8_t *data = (uint8_t *)ws, *scales = data + linear_data_bytes(a);
    const gdn_mx_quantize_args q{a->x, a->M, a->K, a->dtype, a->format, data, scales};
    const gdn_status st = gdn_mx_quantize(&q, stream);
    if (st != GDN_OK) return st;
    const gdn_mx_matmul_args m{data, scales, a->w, a->w_scales, a->M, a->N, a->K, a->format, a->out_dtype, a->c};
    return gdn_mx_matmul(&m, stream);
}
