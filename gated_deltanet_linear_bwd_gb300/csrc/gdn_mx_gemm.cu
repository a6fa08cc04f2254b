// gdn_mx_gemm.cu -- C = A B^T of microscaled matrices on the block-scaled tcgen05
// MMAs.
//
// Small and middling products: one CTA makes 128 rows of B (features) x `nt` rows of A
// (tokens) of C: the weight is the MMA's 128-row operand, so that few tokens cost a narrow
// MMA and not idle rows.  A producer warp feeds a ring of stages with TMA (both operand
// tiles and both scale tiles, 128 bytes of K at a time), one warp copies scales to TMEM
// and issues the MMAs, and the fp32 tile leaves TMEM through shared memory so that rows of
// C are written 128 features at a time.  Where tiles are too few for the GPU the CTAs of a
// cluster share K: each leaves its fp32 tile in its shared memory, and after the cluster's
// barrier each adds up its share of the rows, in rank order.  Bound by the weight's bytes:
// 7 x 12288 x 4096 MXFP4 8.4 us (6.7 with the weight in L2), of which its 27 MB take 4.0 at the
// measured copy rate.
#include <algorithm>

#include "gdn_layer_internal.h"
#include "gdn_mx_strip.cuh"
#include "tc_mx_ptx.cuh"

namespace gdn {
namespace mx {
namespace {

constexpr int kFeat = 128;         // features of a tile
constexpr int kThreads = 192;      // producer, MMA and four epilogue warps
constexpr int kTmemBarrier = 1;    // named: TMEM is there, and waits with a limit may begin
constexpr int kMaxStages = 10;
constexpr int kMaxSplits = 8;

struct GemmArgs {
    const uint8_t *sx, *sw;        // scales of tokens and features
    void *c;
    int tokens, feats, K;
    int nt, token_tiles;
    int kblocks, ktiles;           // 128-byte blocks of K, scale tiles along K
    int stages, stage_bytes, tmem_cols;
    int c_fp32;
    int early_w;                   // the kernel ahead of this one began when all before it, the weight's
                                   // writers among them, had ended, and takes no TMEM
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

    if (threadIdx.x == 32) {
        tc::prefetch_map(&map_x);
        tc::prefetch_map(&map_w);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            tc::mbar_init(&ctl.full[s], 1);
            tc::mbar_init(&ctl.empty[s], 1);
        }
        tc::mbar_init(&ctl.done, 1);
        ctl.failed = 0;
        tc::fence_barrier_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const uint32_t x_off = kFeat * 128, sw_off = x_off + a.nt * 128, sx_off = sw_off + kScaleTiles * 512;
    if (warp == 0) {
        const int n = kb1 - kb0;
        const uint32_t ring0 = tc::smem_u32(ring), full0 = tc::smem_u32(ctl.full), empty0 = tc::smem_u32(ctl.empty);
        const uint8_t *sw = a.sw + (long long)(f0 / 128) * a.ktiles * 512, *sx = a.sx + (long long)(t0 / 128) * a.ktiles * 512;
        auto tile_bytes = [&](int kb) { return 512u * (uint32_t)min(kScaleTiles, a.ktiles - kb * kScaleTiles); };
        auto load_w = [&](int kb, uint32_t st, uint32_t bar) {       // arms the stage for all it gets
            const uint32_t sb = tile_bytes(kb);
            tc::expect_bytes(bar, (uint32_t)(kFeat + a.nt) * 128u + 2u * sb, true);
            tc::load_operand(st, &map_w, kb * 128, f0, st + sw_off, sw + kb * (512ll * kScaleTiles), sb, bar);
        };
        auto load_x = [&](int kb, uint32_t st, uint32_t bar) {
            tc::load_operand(st + x_off, &map_x, kb * 128, t0, st + sx_off, sx + kb * (512ll * kScaleTiles), tile_bytes(kb), bar);
        };
        // a ring's worth of weights may come before the kernel ahead has written the tokens
        const int ahead = a.early_w ? min(n, a.stages) : 0;
        for (int i = 0; i < ahead; ++i) load_w(kb0 + i, ring0 + i * a.stage_bytes, full0 + 8 * i);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        int i = 0, s = 0;
        uint32_t parity = 1;                         // of the stage's last release; the first round has none
        auto fill = [&] {
            const uint32_t st = ring0 + s * a.stage_bytes, bar = full0 + 8 * s;
            if (i >= ahead) load_w(kb0 + i, st, bar);
            load_x(kb0 + i, st, bar);
            if (++s == a.stages) s = 0, parity ^= 1;
        };
        for (; i < min(n, a.stages); ++i) fill();
        tc::named_sync(kTmemBarrier, kThreads);
        for (; i < n; ++i) {
            if (!tc::mbar_spin(empty0 + 8 * s, parity, a.spin_limit, a.status)) {
                ctl.failed = 1;
                break;
            }
            fill();
        }
        if (lane == 0) ctl.issued = i;
    } else if (warp == 1) {
        // TMEM is taken once the kernel ahead has ended: if CTAs of that one have yet to take
        // theirs, they would wait for this one's, and this kernel waits for their end.  With
        // early_w the kernel ahead takes none, and those before it have ended.
        if (!a.early_w) asm volatile("griddepcontrol.wait;" ::: "memory");
        tc::tmem_alloc(&ctl.tmem, (uint32_t)a.tmem_cols);
        tc::tmem_relinquish();
        asm volatile("griddepcontrol.wait;" ::: "memory");           // waits with a limit begin when work does
        tc::tc_fence_before();
        tc::named_sync(kTmemBarrier, kThreads);
        tc::tc_fence_after();
        const uint32_t tmem = ctl.tmem, tsw = tmem + a.nt, tsx = tsw + 4 * kScaleTiles;
        for (int kb = kb0; kb < kb1; ++kb) {
            const int i = kb - kb0, s = i % a.stages;
            if (!tc::mbar_spin(tc::smem_u32(&ctl.full[s]), (i / a.stages) & 1, a.spin_limit, a.status)) {
                ctl.failed = 1;
                break;
            }
            const uint32_t st = tc::smem_u32(ring + s * a.stage_bytes);
            const uint64_t dw = tc::desc_sw128(st, 0, 1024), dx = tc::desc_sw128(st + x_off, 0, 1024);
            if ((kb + 1) * kBlock <= a.K) {
                tc::mma_mx_stage<FP4>(tmem, dw, dx, tc::desc_scales(st + sw_off), tsw, tsx,
                                      tc::idesc_mx(FP4, kFeat, a.nt, 0), i > 0, &ctl.empty[s]);
                continue;
            }
            // the last block of a K that is not whole stages
            const int tiles = min(kScaleTiles, a.ktiles - kb * kScaleTiles);
            for (int k = 0; k < tiles; ++k) {
                tc::copy_scales(tsw + 4 * k, tc::desc_scales(st + sw_off + 512 * k));
                tc::copy_scales(tsx + 4 * k, tc::desc_scales(st + sx_off + 512 * k));
            }
            const int steps = (a.K - kb * kBlock + kStep - 1) / kStep;
            for (int j = 0; j < steps; ++j) {
                const int id = FP4 ? 2 * (j & 1) : j, col = FP4 ? 4 * (j >> 1) : 0;
                tc::mma_mx<FP4>(tmem, dw + 2 * j, dx + 2 * j, tc::idesc_mx(FP4, kFeat, a.nt, id),
                                tsw + col, tsx + col, i > 0 || j > 0);
            }
            tc::mma_commit(&ctl.empty[s]);
        }
        tc::mma_commit(&ctl.done);
    }
    if (warp > 1) {
        asm volatile("griddepcontrol.wait;" ::: "memory");              // C may be written
        tc::named_sync(kTmemBarrier, kThreads);
    }
    __syncwarp();
    // every MMA done: the ring is free and the tile is whole
    if (!tc::mbar_wait(&ctl.done, 0, a.spin_limit, a.status)) {
        ctl.failed = 1;
        tc::mbar_drain(&ctl.done, 0);
    }
    tc::tc_fence_after();
    __syncthreads();
    const uint32_t tmem = ctl.tmem;
    const bool ok = ctl.failed == 0;
    if (!ok && threadIdx.x == 0)   // a wait gave up: nothing may land after the CTA has gone
        for (int j = max(0, ctl.issued - a.stages); j < ctl.issued; ++j)
            tc::mbar_drain(&ctl.full[j % a.stages], (j / a.stages) & 1);
    float *out = reinterpret_cast<float *>(ring);    // [nt][128]
    if (ok && warp >= 2) {
        float *to = out + 32 * (warp & 3) + lane;
        if (a.nt == 16) {
            float v[16];
            tc::tmem_ld8x2(tc::tmem_addr(tmem, warp, 0), tc::tmem_addr(tmem, warp, 8), v, v + 8);
#pragma unroll
            for (int j = 0; j < 16; ++j) to[j * kFeat] = v[j];
        } else {
            for (int c = 0; c < a.nt; c += 32) {
                float v[32];
                tc::tmem_ld32(tc::tmem_addr(tmem, warp, c), v);
#pragma unroll
                for (int j = 0; j < 32; ++j) to[(c + j) * kFeat] = v[j];
            }
        }
    }
    tc::tc_fence_before();
    if (splits > 1) tc::cluster_sync();
    else __syncthreads();
    tc::tc_fence_after();
    if (ok) {
        const uint32_t base = tc::smem_u32(out);
        const int step = splits * (kThreads / 32), rows = min(a.nt, a.tokens - t0);
        for (int j = rank * (kThreads / 32) + warp; j < rows; j += step) {
            const int at = j * kFeat + 4 * lane;
            float4 v;
            if (splits == 1) {
                v = *reinterpret_cast<const float4 *>(out + at);
            } else {
                float4 p[kMaxSplits];
#pragma unroll
                for (int r = 0; r < kMaxSplits; ++r)
                    if (r < splits) p[r] = tc::ld_cluster4(tc::map_rank(base + 4u * (uint32_t)at, r));
                v = p[0];
#pragma unroll
                for (int r = 1; r < kMaxSplits; ++r)
                    if (r < splits) v.x += p[r].x, v.y += p[r].y, v.z += p[r].z, v.w += p[r].w;
            }
            store_c4(a, t0 + j, f0 + 4 * lane, v);
        }
    }
    if (splits > 1) tc::cluster_sync();              // the others have read this CTA's tile
    if (warp == 1) tc::tmem_dealloc(tmem, (uint32_t)a.tmem_cols);
}

// ------------------------------------------------------------------ large products
// CTA pairs (cta_group::2) on tiles of 256 tokens x 256 features, persistent over the
// tiles.  A pair reads each operand tile once for both of its CTAs, which halves what an
// SM takes from L2 per MMA; the accumulators of two tiles share 448 TMEM columns, the
// last 64 of the one being the first 64 of the other, so that the epilogue of a tile
// runs under the next one's MMAs once it has taken those 64.
//
// 8192 x 12288 x 4096: 135 us in 4 bits (6.1 PFLOP/s, 3.2 times the measured bf16 rate), 243
// us in 8 (3.4); with the tokens' quantisation under the MMAs 143 and 265.  A stage's four MMAs take 512 cycles (247 ns); a stage takes 290 to 315 ns,
// bound by the hand-over between the loading warps, the MMA warp and its commits, and a tile
// 1.6 us more, in which its MMAs wait for the shared columns.  Tiles of 192 columns, which
// share none, took as long (138 and 253 us).
constexpr int kPairThreads = 224;                    // weights, MMA, four epilogue warps, tokens
constexpr int kPairQuantThreads = 256;               // more, where the tokens come unquantised
constexpr int kPairStages = 6;
constexpr int kPairAcc = 192;                        // column of the second accumulator
constexpr int kPairScales = 448;                     // columns of the scales: two sets of 24
constexpr int kPairOut = 4096;                       // a warp's staged 32 x 128-byte block of C

// The tokens' rows from `row0` on (whole tiles) that the product itself quantises, to where
// it reads them, in strips of up to kStrip spans of a row, or of 2^log_rows rows where those
// are short.  work[0] counts strips that warps have taken, work[1 + row / 128] those that
// are done; both begin at 0.
struct Unquantised {
    const void *x;                                   // null: all rows are there
    int fp32, row0, strips, log_rows;                // strips of a row
    uint8_t *data, *scales;
    uint32_t *work;
};
constexpr int kStrip = 16;

struct PairArgs {
    int M, N, K, kblocks, ktiles;
    int m_tiles, n_tiles;
    int rows_first;                                  // the order of tiles: rows of tiles are done one after the other
    int early_w;                                     // as in GemmArgs
    void *direct;                                    // C, where its rows start on no 16 bytes; null: TMA stores it
    Unquantised rest;
    int *status;
    long long spin_limit;
};

// Tile `i`: its row and column of tiles.
__device__ __forceinline__ int2 pair_tile(const PairArgs &a, int i) {
    const int inner = a.rows_first ? a.n_tiles : a.m_tiles, o = i / inner, n = i - o * inner;
    return a.rows_first ? make_int2(o, n) : make_int2(n, o);
}

struct PairControl {
    uint64_t full[kPairStages], empty[kPairStages], acc_full, acc_free, done;
    uint32_t tmem;
    int issued;
};

template <bool FP4>
constexpr int pair_stage_bytes() { return 32768 + (FP4 ? 3072 : 2048); }

template <bool FP4, typename TO>
__global__ void __launch_bounds__(kPairThreads + kPairQuantThreads) gemm_pair_kernel(const __grid_constant__ CUtensorMap map_x,
                                                             const __grid_constant__ CUtensorMap map_w,
                                                             const __grid_constant__ CUtensorMap map_sx,
                                                             const __grid_constant__ CUtensorMap map_sw,
                                                             const __grid_constant__ CUtensorMap map_c,
                                                             const PairArgs a) {
    constexpr int kStep = FP4 ? 64 : 32, kBlock = 4 * kStep, kScaleTiles = kBlock / 128;
    constexpr int kStage = pair_stage_bytes<FP4>();
    constexpr uint32_t kBytes = 32768u + 3u * 512u * kScaleTiles;    // of one CTA
    constexpr int kCols = 128 / (int)sizeof(TO);     // columns of a staged block
    extern __shared__ __align__(1024) uint8_t ring[];
    uint8_t *stage_out = ring + kPairStages * kStage;
    PairControl &ctl = *reinterpret_cast<PairControl *>(stage_out + 4 * kPairOut);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = a.m_tiles * a.n_tiles;

    if (tc::smem_u32(ring) & 1023u) {                // the swizzle's unit; every CTA alike
        if (threadIdx.x == 0) set_status(a.status, GDN_ERR_CUDA);
        return;
    }
    if (threadIdx.x == 32) {
        tc::prefetch_map(&map_x);
        tc::prefetch_map(&map_w);
        tc::prefetch_map(&map_sx);
        tc::prefetch_map(&map_sw);
        if (!a.direct) tc::prefetch_map(&map_c);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            tc::mbar_init(&ctl.full[s], 1);
            tc::mbar_init(&ctl.empty[s], 1);
        }
        tc::mbar_init(&ctl.acc_full, 1);
        tc::mbar_init(&ctl.acc_free, 8);             // the epilogue warps of both CTAs
        tc::mbar_init(&ctl.done, 1);
        ctl.issued = 0;
        tc::fence_barrier_init();
    }
    if (warp == 1) {
        if (!a.early_w) asm volatile("griddepcontrol.wait;" ::: "memory");   // as in gemm_kernel
        tc::tmem_alloc_pair(&ctl.tmem, 512);
    }
    tc::tc_fence_before();
    tc::cluster_sync();                              // both CTAs' barriers and TMEM are there
    tc::tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const uint32_t ring0 = tc::smem_u32(ring), full0 = tc::smem_u32(ctl.full), empty0 = tc::smem_u32(ctl.empty);
    if (warp == 0 || warp == 6) {
        // two warps, as one alone is late with a stage's four loads
        const bool weights = warp == 0;
        const uint32_t bar0 = tc::map_rank(full0, 0);
        auto load = [&](int kb, int row, int feat, int s) {
            const uint32_t st = ring0 + s * kStage;
            if (weights) {                           // and arms the pair's barrier for all that both CTAs get
                tc::expect_bytes(full0 + 8 * s, 2u * kBytes, rank == 0);
                tc::load_operand_pair(st + 16384, &map_w, kb * 128, (feat + rank) * 128,
                                      st + 32768 + 512 * kScaleTiles, &map_sw, kb * kScaleTiles, feat, bar0 + 8 * s);
            } else {
                tc::load_operand_pair(st, &map_x, kb * 128, row * 128, st + 32768, &map_sx, kb * kScaleTiles, row,
                                      bar0 + 8 * s);
            }
        };
        // the first tile's weights may come before the kernel ahead has written the tokens
        const int ahead = weights && a.early_w && pair < tiles ? min(kPairStages, a.kblocks) : 0;
        for (int i = 0; i < ahead; ++i) load(i, 0, pair_tile(a, pair).y * 2, i);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        int i = 0, s = 0;                            // stages asked for
        uint32_t parity = 1;                         // of the stage's last release; the first round has none
        bool ok = true;
        int ready = a.rest.x ? a.rest.row0 / 128 : a.m_tiles * 2;    // rows quantised, in 128s
        for (int tile = pair; tile < tiles && ok; tile += pairs) {
            const int2 at = pair_tile(a, tile);
            const int row = at.x * 2 + rank, feat = at.y * 2;    // in 128s
            // a wait that gives up is reported and the last one; every stage is filled all the
            // same, as the other loading warp has counted on it
            if (!weights && row >= ready && row * 128 < a.M)
                ready = tc::word_spin(a.rest.work + 1 + row, (128u >> a.rest.log_rows) * a.rest.strips, a.spin_limit,
                                      a.status) ? row + 1 : 2 * a.m_tiles;
            for (int kb = 0; kb < a.kblocks; ++kb, ++i) {
                if (i >= kPairStages) {
                    ok = tc::mbar_spin(empty0 + 8 * s, parity, a.spin_limit, a.status);
                    if (!ok) break;
                }
                if (i >= ahead) load(kb, row, feat, s);
                if (++s == kPairStages) s = 0, parity ^= 1;
            }
        }
        if (weights && lane == 0) ctl.issued = i;
    } else if (warp == 1) {
        asm volatile("griddepcontrol.wait;" ::: "memory");           // waits with a limit begin when work does
        if (rank == 0) {
            int i = 0, t = 0, s = 0;
            uint32_t parity = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs, ++t) {
                if (t > 0) {
                    ok = tc::mbar_spin(tc::smem_u32(&ctl.acc_free), (t - 1) & 1, a.spin_limit, a.status);
                    if (!ok) break;
                }
                tc::tc_fence_after();
                const uint32_t acc = tmem + (t & 1 ? kPairAcc : 0);
                for (int kb = 0; kb < a.kblocks; ++kb, ++i) {
                    const int at = s;
                    ok = tc::mbar_spin(full0 + 8 * at, parity, a.spin_limit, a.status);
                    if (!ok) break;
                    if (++s == kPairStages) s = 0, parity ^= 1;
                    const uint32_t st = ring0 + at * kStage;
                    const uint32_t tsx = tmem + kPairScales + (i & 1) * 24, tsw = tsx + 4 * kScaleTiles;
                    const uint64_t dx = tc::desc_sw128(st, 0, 1024), dw = tc::desc_sw128(st + 16384, 0, 1024);
                    if ((kb + 1) * kBlock <= a.K) {
                        tc::mma_mx_stage_pair<FP4>(acc, dx, dw, tc::desc_scales(st + 32768), tsx, tsw, kb > 0,
                                                   &ctl.empty[at]);
                        continue;
                    }
                    // the last block of a K that is not whole stages
                    const int st_tiles = min(kScaleTiles, a.ktiles - kb * kScaleTiles);
                    for (int k = 0; k < st_tiles; ++k) {
                        tc::copy_scales_pair(tsx + 4 * k, tc::desc_scales(st + 32768 + 512 * k));
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            tc::copy_scales_pair(tsw + 8 * k + 4 * b,
                                                 tc::desc_scales(st + 32768 + 512 * (kScaleTiles * (1 + b) + k)));
                    }
                    const int steps = (a.K - kb * kBlock + kStep - 1) / kStep;
                    for (int j = 0; j < steps; ++j) {
                        const int id = FP4 ? 2 * (j & 1) : j;
                        tc::mma_mx_pair<FP4>(acc, dx + 2 * j, dw + 2 * j, tc::idesc_mx(FP4, 256, 256, id),
                                             tsx + (FP4 ? 4 * (j >> 1) : 0), tsw + (FP4 ? 8 * (j >> 1) : 0),
                                             kb > 0 || j > 0);
                    }
                    tc::mma_commit_pair(&ctl.empty[at]);
                }
                if (ok) tc::mma_commit_pair(&ctl.acc_full);
            }
            tc::mma_commit_pair(&ctl.done);
        }
    } else if (warp >= kPairThreads / 32) {
        // Quantises strips in the tiles' order.  A strip belongs to the warp that took it and
        // no strip waits for anything, so that the loads' waits end whichever CTAs run.
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const Unquantised &r = a.rest;
        const int spans = (a.ktiles + 1) / 2;
        const unsigned total = (unsigned)(((a.M + 127) / 128 * 128 - r.row0) >> r.log_rows) * r.strips;
        unsigned next = lane == 0 ? atomicAdd(r.work, 1u) : 0u;
        for (;;) {
            const unsigned item = __shfl_sync(0xffffffffu, next, 0);
            if (item >= total) break;
            if (lane == 0) next = atomicAdd(r.work, 1u);
            const int row = r.row0 + (int)(item / r.strips << r.log_rows), first = (int)(item % r.strips) * kStrip;
            const int end = min(first + kStrip, spans);
            for (int i = 0; i < 1 << r.log_rows; ++i)
                if (r.fp32)
                    quantize_strip<float, FP4, false>((const float *)r.x, r.data, r.scales, row + i, first, end, a.M,
                                                      a.K, a.ktiles);
                else
                    quantize_strip<__nv_bfloat16, FP4, false>((const __nv_bfloat16 *)r.x, r.data, r.scales, row + i,
                                                              first, end, a.M, a.K, a.ktiles);
            tc::add_release(r.work + 1 + row / 128);
        }
    } else {
        // epilogue: each warp takes its 32 rows, 64 (bf16) or 32 (fp32) columns at a time,
        // through a swizzled block of its own to a TMA store, or, where C's rows start on no
        // 16 bytes, to plain stores along them (2048 x 50257 x 2048 4 bits 126 us, single
        // CTAs 196)
        asm volatile("griddepcontrol.wait;" ::: "memory");   // C may be written
        const int quarter = warp & 3;
        uint8_t *buf = stage_out + quarter * kPairOut;
        const uint32_t acc_free0 = tc::map_rank(tc::smem_u32(&ctl.acc_free), 0);
        int t = 0;
        for (int tile = pair; tile < tiles; tile += pairs, ++t) {
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&ctl.acc_full, t & 1, a.spin_limit, a.status))) break;
            tc::tc_fence_after();
            const int2 at = pair_tile(a, tile);
            const int row = (at.x * 2 + rank) * 128 + 32 * quarter, feat = at.y * 256;
            const uint32_t acc = tmem + (t & 1 ? kPairAcc : 0);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                // the 64 columns that the next tile's accumulator shares go first
                const int col = (t & 1 ? c : (c + 3) & 3) * 64;
                float v[64];
                tc::tmem_ld32x2(tc::tmem_addr(acc, quarter, col), tc::tmem_addr(acc, quarter, col + 32), v, v + 32);
                if (c == 0) {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_cluster(acc_free0);
                }
#pragma unroll
                for (int b = 0; b < 64 / kCols; ++b) {
                    if (lane == 0) tc::bulk_wait_read();     // the store before has left the block
                    __syncwarp();
                    if constexpr (sizeof(TO) == 2) {
                        tc::st_row64(buf, lane, v);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<float4 *>(buf + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                                make_float4(v[32 * b + 4 * k], v[32 * b + 4 * k + 1], v[32 * b + 4 * k + 2], v[32 * b + 4 * k + 3]);
                    }
                    if (a.direct) {
                        __syncwarp();
                        const int c0 = feat + col + b * kCols, rows = min(32, a.M - row);
                        TO *out = reinterpret_cast<TO *>(a.direct) + (long long)row * a.N + c0;
                        for (int r = 0; r < rows; ++r, out += a.N)
#pragma unroll
                            for (int e = lane; e < kCols; e += 32) {
                                const int at = e * (int)sizeof(TO), chunk = (at >> 4) ^ (r & 7);
                                if (c0 + e < a.N)
                                    out[e] = *reinterpret_cast<const TO *>(buf + r * 128 + (chunk << 4) + (at & 15));
                            }
                        __syncwarp();
                        continue;
                    }
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0 && row < a.M && feat + col + b * kCols < a.N) {
                        tc::tma_store_2d(&map_c, buf, feat + col + b * kCols, row);
                        tc::bulk_commit();
                    }
                }
            }
        }
        if (lane == 0) tc::bulk_wait_read();
        __syncwarp();
    }
    // every MMA done and every copy landed before TMEM is given back and a CTA goes
    if (warp < kPairThreads / 32) tc::mbar_drain(&ctl.done, 0);
    tc::tc_fence_before();
    tc::cluster_sync();
    if (threadIdx.x == 0 && rank == 0)
        for (int i = max(0, ctl.issued - kPairStages); i < ctl.issued; ++i)
            tc::mbar_drain(&ctl.full[i % kPairStages], (i / kPairStages) & 1);
    tc::cluster_sync();
    tc::tc_fence_after();
    if (warp == 1) tc::tmem_dealloc_pair(tmem, 512);
}

// Tiles are walked along the shorter side, whose operand then stays in L2 while the other
// passes once; along rows of tiles too where the weight takes half of L2 at most, so that
// the product can quantise rows under its MMAs.  MXFP8, K = 4096, rows first | columns
// first: 32768 x 4096 312 us | 370, 1024 x 65536 209 | 169, 8192 x 12288 242 | 238.
bool rows_first(const gdn_mx_matmul_args *a) {
    const long long bytes = (long long)a->N * (a->format == GDN_MXFP4 ? a->K / 2 : a->K);
    return a->N <= a->M || bytes <= 64ll << 20;
}

template <bool FP4, typename TO>
gdn_status run_pair(const gdn_mx_matmul_args *a, const LayerDevice &dev, bool early_w, const Unquantised &rest,
                    cudaStream_t q) {
    PairArgs g{};
    g.M = a->M, g.N = a->N, g.K = a->K;
    g.kblocks = (a->K + (FP4 ? 255 : 127)) / (FP4 ? 256 : 128);
    g.ktiles = (a->K + 127) / 128;
    g.m_tiles = (a->M + 255) / 256;
    g.n_tiles = (a->N + 255) / 256;
    g.rows_first = rows_first(a);
    g.early_w = early_w;
    g.rest = rest;
    g.status = dev.status;
    g.spin_limit = dev.spin_limit;
    const long long bytes = FP4 ? a->K / 2 : a->K;
    const int st = FP4 ? 2 : 1;
    g.direct = (long long)a->N * (int)sizeof(TO) % 16 ? a->c : nullptr;
    CUtensorMap mx, mw, msx, msw, mc = {};
    cudaError_t e;
    if ((e = tc::make_map_bytes(&mx, a->a, a->M, bytes, 128)) != cudaSuccess ||
        (e = tc::make_map_bytes(&mw, a->b, a->N, bytes, 128)) != cudaSuccess ||
        (e = tc::make_map_scales(&msx, a->a_scales, (a->M + 127) / 128, g.ktiles, st, 1)) != cudaSuccess ||
        (e = tc::make_map_scales(&msw, a->b_scales, (a->N + 127) / 128, g.ktiles, st, 2)) != cudaSuccess ||
        (!g.direct &&
         (e = tc::make_map_rows(&mc, a->c, a->M, a->N, sizeof(TO), 128 / (int)sizeof(TO), 32, true)) != cudaSuccess))
        return cuda_fail(e, "tensor map of a product");
    const size_t smem = kPairStages * pair_stage_bytes<FP4>() + 4 * kPairOut + sizeof(PairControl);
    auto k = gemm_pair_kernel<FP4, TO>;
    if ((e = allow_smem((const void *)k, smem)) != cudaSuccess)
        return cuda_fail(e, "shared memory of the product");
    const int pairs = (int)std::min<long long>((long long)g.m_tiles * g.n_tiles, dev.sms / 2);
    prof_before("mx_gemm_pair", q);
    e = launch_pdl_cluster(k, dim3(2 * pairs), dim3(kPairThreads + (rest.x ? kPairQuantThreads : 0)), smem, 2, q, mx, mw, msx, msw, mc, g);
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "mx product launch");
}

// Shared memory that a CTA of a cluster takes at least, for its TMEM columns.  Such a CTA holds
// its columns until the whole cluster has its own; if clusters, of this launch or of another
// stream's, each held on one SM what another needed there, none would ever end.  So the CTAs that
// fit an SM by their shared memory (228 KB, 1 KB of each CTA the system's) must fit its 512
// columns: more than 228 KB / (512 + 32) for each, as columns come by 32.  The pairs take 220 KB
// for 512.  CTAs of no cluster, here and in the delta rule, end whoever else waits.
constexpr size_t cluster_smem(int tmem_cols) { return (size_t)tmem_cols * 432 - 1024; }
static_assert(432 * (512 + 32) > 228 * 1024, "");
static_assert(kPairStages * pair_stage_bytes<false>() + 4 * kPairOut >= cluster_smem(512), "");

// Tokens of a tile: 16, or as many as there are up to 128.
int token_tile(int tokens) {
    int nt = 16;
    while (nt < 128 && nt < tokens) nt *= 2;
    return nt;
}

// Pairs take over from single CTAs where those are more than one wave, unless few tokens leave
// most of a pair's tile idle.  Us of single CTAs | pairs at K = 4096 in 4 bits: 384 x 4096 10.7 |
// 11.8, 128 x 16384 10.8 | 12.1, 512 x 12288 21.8 | 18.0; in 8 bits 384 x 4096 15.4 | 16.0, 128 x
// 16384 15.7 | 17.4, 512 x 12288 31.8 | 27.3; rows of C that start on no 16 bytes, 4 bits: 300 x
// 4097 10.6 | 13.8, 1000 x 4099 14.5 | 14.4, 512 x 12289 23.2 | 20.6; few tokens, 7 x 12288 6.7 | 16.2.
bool pair_fits(const gdn_mx_matmul_args *a, int sms) {
    const int nt = token_tile(a->M);
    const long long singles = (long long)((a->N + kFeat - 1) / kFeat) * ((a->M + nt - 1) / nt);
    const long long tiles = (long long)((a->M + 255) / 256) * ((a->N + 255) / 256);
    return nt > 32 && singles > sms && tiles < (1ll << 30);
}

// Rows to quantise ahead of the product: those of the pairs' first tiles (in 4 bits, whose
// MMAs take half as long, of the first two), the product itself taking the rest under its
// MMAs; or all of them where K, N or M is too short for the MMAs to cover that.  Us all ahead |
// the rest under the MMAs: 8192 x 12288 x 4096 in 4 bits 156 | 143, 8 bits 275 | 265; 8192 x
// 4096 x 4096 76 | 70, 105 | 98; 2048 x 12288 x 4096 49 | 47, 77 | 75; but 4096 x 16384 x 512
// 46 | 53, 50 | 55; 65536 x 1024 x 1024 84 | 103, 95 | 109.
int rows_ahead(const gdn_mx_matmul_args *a, int sms) {
    const int n_tiles = (a->N + 255) / 256, waves = a->format == GDN_MXFP4 ? 2 : 1;
    const int first = (sms / 2 + n_tiles - 1) / n_tiles * 256 * waves;
    return pair_fits(a, sms) && rows_first(a) && a->K >= 2048 && n_tiles >= 16 && a->M >= 2 * first ? first : a->M;
}

gdn_status run(const gdn_mx_matmul_args *a, const LayerDevice &dev, bool early_w, const Unquantised &rest,
               cudaStream_t q) {
    const bool fp4 = a->format == GDN_MXFP4;
    cudaError_t e = tc::encoder();
    if (e != cudaSuccess) return cuda_fail(e, "cuTensorMapEncodeTiled lookup");
    if (pair_fits(a, dev.sms)) {
        if (a->out_dtype == GDN_FP32) return fp4 ? run_pair<true, float>(a, dev, early_w, rest, q)
                                                    : run_pair<false, float>(a, dev, early_w, rest, q);
        return fp4 ? run_pair<true, __nv_bfloat16>(a, dev, early_w, rest, q)
                   : run_pair<false, __nv_bfloat16>(a, dev, early_w, rest, q);
    }
    GemmArgs g{};
    g.sx = a->a_scales;
    g.sw = a->b_scales;
    g.c = a->c;
    g.tokens = a->M, g.feats = a->N, g.K = a->K;
    g.nt = token_tile(a->M);
    g.token_tiles = (a->M + g.nt - 1) / g.nt;
    g.kblocks = (a->K + (fp4 ? 255 : 127)) / (fp4 ? 256 : 128);
    g.ktiles = (a->K + 127) / 128;
    g.stage_bytes = (kFeat + g.nt) * 128 + (fp4 ? 2048 : 1024);
    // The CTAs of a cluster share K, by powers of two (clusters of 3 took longer than no
    // cluster), while slots of the GPU are empty: two CTAs to an SM and up to 8 to a cluster
    // for few tokens; one and up to 4 for many, whose tiles take long to add up (4096 x
    // 4096, 128 tokens, 4 bits: 7.4 us with 4, 9.7 with 2, 13.5 with 8 at two to an SM).
    // Clusters of c leave about c SMs without one (37 of 4 fit, 36 of 8 at two to an SM), and
    // one cluster too many takes a second wave: 191 x 2432 x 4096 8 bits 14.7 us with 4, 11.7
    // with 2; 20 x 4864 x 4096 in 38 of 4 10.1 us at one to an SM, 6.3 at two.
    const long long tiles = (long long)((a->N + kFeat - 1) / kFeat) * g.token_tiles;
    const bool few = g.nt <= 32;
    int splits = 1;
    while (splits < (few ? kMaxSplits : 4) && 2 * splits <= g.kblocks &&
           2 * splits * tiles <= (few ? 2 : 1) * (dev.sms - 2 * splits))
        splits *= 2;
    const int per = (g.kblocks + splits - 1) / splits;
    g.stages = std::max(1, std::min({kMaxStages, per, (tiles * splits <= dev.sms - splits ? 200 : 100) * 1024 / g.stage_bytes}));
    g.early_w = early_w;
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
    size_t smem = std::max(g.stages * g.stage_bytes, g.nt * kFeat * 4) + 1024;
    if (splits > 1) smem = std::max(smem, cluster_smem(g.tmem_cols));
    auto k = fp4 ? gemm_kernel<true> : gemm_kernel<false>;
    if ((e = allow_smem((const void *)k, smem)) != cudaSuccess)
        return cuda_fail(e, "shared memory of the product");
    const long long ctas = tiles * splits;
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

static gdn_status check(const gdn_mx_matmul_args *a) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    if (a->M < 0 || a->N < 0 || a->K < 0)
        return fail(GDN_ERR_INVALID_ARG, "bad sizes M=%d N=%d K=%d", a->M, a->N, a->K);
    if (std::max({a->M, a->N, a->K}) > kMaxExtent)
        return fail(GDN_ERR_INVALID_ARG, "problem too large: M=%d N=%d K=%d", a->M, a->N, a->K);
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
    return GDN_OK;
}

// A product whose arguments check() has passed.  early_w: the kernel ahead in the stream is the
// quantisation, which began only when all before it, the writers of b among them, had ended, and
// takes no TMEM.
static gdn_status matmul(const gdn_mx_matmul_args *a, const LayerDevice &dev, bool early_w,
                         const mx::Unquantised &rest, void *stream) {
    if (a->M == 0 || a->N == 0) return GDN_OK;
    if (a->K == 0) {
        const cudaError_t e = cudaMemsetAsync(a->c, 0, (size_t)a->M * a->N * (a->out_dtype == GDN_FP32 ? 4 : 2),
                                              (cudaStream_t)stream);
        return e == cudaSuccess ? GDN_OK : cuda_fail(e, "clearing c");
    }
    return mx::run(a, dev, early_w, rest, (cudaStream_t)stream);
}

extern "C" gdn_status gdn_mx_matmul(const gdn_mx_matmul_args *a, void *stream) {
    gdn_status st = check(a);
    if (st != GDN_OK || a->M == 0 || a->N == 0) return st;
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    return matmul(a, dev, false, mx::Unquantised{}, stream);
}

// Bytes of X's elements in the workspace; its scales follow, then the counters of the
// product's own quantisation.
static size_t linear_data_bytes(const gdn_mx_linear_args *a) {
    const size_t n = (size_t)a->M * a->K;
    return ((a->format == GDN_MXFP4 ? n / 2 : n) + 255) / 256 * 256;
}

// The counters: one, and one for each 128 rows.
static int linear_words(const gdn_mx_linear_args *a) { return 1 + (int)((a->M + 127ll) / 128); }

extern "C" size_t gdn_mx_linear_workspace_size(const gdn_mx_linear_args *a) {
    if (!a || a->M < 0 || a->K < 0) {
        fail(GDN_ERR_INVALID_ARG, "null args or bad sizes");
        return 0;
    }
    if (std::max(a->M, a->K) > kMaxExtent) {
        fail(GDN_ERR_INVALID_ARG, "problem too large: M=%d K=%d", a->M, a->K);
        return 0;
    }
    return std::max<size_t>(256, linear_data_bytes(a) + gdn_mx_scale_bytes(a->M, a->K) + 4 * (size_t)linear_words(a));
}

extern "C" gdn_status gdn_mx_linear(const gdn_mx_linear_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    const size_t need = gdn_mx_linear_workspace_size(a);
    if (need == 0) return GDN_ERR_INVALID_ARG;
    if (!ws || misaligned(ws) || ws_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    uint8_t *data = (uint8_t *)ws, *scales = data + linear_data_bytes(a);
    const gdn_mx_matmul_args m{data, scales, a->w, a->w_scales, a->M, a->N, a->K, a->format, a->out_dtype, a->c};
    gdn_mx_quantize_args q{a->x, a->M, a->K, a->dtype, a->format, data, scales};
    // everything is checked before the quantisation is launched
    gdn_status st = check(&m);
    if (st == GDN_OK) st = check_quantize(&q);
    if (st != GDN_OK || a->M == 0 || a->N == 0) return st;
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    mx::Unquantised rest{};
    if (a->M >= 512) {                                         // at least two tiles of rows
        q.rows = mx::rows_ahead(&m, dev.sms);
        if (q.rows < a->M) {
            uint32_t *work = (uint32_t *)(scales + gdn_mx_scale_bytes(a->M, a->K));
            const int spans = (a->K + 255) / 256;
            int log_rows = 0;
            while (spans << (log_rows + 1) <= mx::kStrip) ++log_rows;
            rest = {a->x, a->dtype == GDN_FP32, q.rows, (spans + mx::kStrip - 1) / mx::kStrip, log_rows, data, scales, work};
        }
    }
    if ((st = mx_quantize(&q, rest.work, rest.x ? linear_words(a) : 0, stream)) != GDN_OK) return st;
    return matmul(&m, dev, a->K > 0, rest, stream);
}
