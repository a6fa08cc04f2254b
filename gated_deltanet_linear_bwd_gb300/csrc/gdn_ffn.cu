// gdn_ffn.cu -- gated feed-forward block y = (act(x Wg^T) * (x Wu^T)) Wd^T and its backward pass, bf16
// products on tcgen05 with their elementwise work in the epilogues:
//
//     forward    g = x Wg^T, u = x Wu^T, h = act(g) u          one product of 2 F features
//                y = h Wd^T
//     backward   dh = dy Wd;  dg = dh u act'(g), du = dh act(g), h = act(g) u
//                dx = dg Wg + du Wu                             one contraction over 2 F
//                dWg = dg^T x, dWu = du^T x, dWd = dy^T h       one launch
//
// Sums are fp32 in TMEM.  h, dg and du pass to the next product as bf16, the tensor cores' operand
// type: each is rounded once, by 2^-8 of itself at most.  Such roundings are of either sign, so that a
// sum of products with them is off by about as much as its own rounding to bf16 is.  Of few tokens,
// where there are few to average over, they pass whole.
#include <algorithm>

#include "gdn_layer_internal.h"
#include "gdn_ffn.cuh"
#include "tc_bf16_ptx.cuh"

namespace gdn {
namespace ffn {
namespace {

// ------------------------------------------------------------------ CTA pairs
// Tiles of 256 x 256 by two CTAs (cta_group::2), persistent over the tiles of up to three products;
// each CTA holds 128 rows of A and half the columns' rows of B.  Two accumulators of 256 columns fill
// TMEM, so that a tile's epilogue runs under the next tile's MMAs.  A stage's MMAs take 512 cycles at the
// least, and its 32 KB into either SM as long.  8192 x 4096 x 12288: into the block 843 us (1.96 PFLOP/s, 104% of
// the measured burst rate), out of it 432, backward dh 534, dx 874, the weights' gradients 1300.
enum Mode {
    kGated,      // A x, B gate's rows in the one CTA and up's in the other: a tile is 256 tokens x 128 features
    kDown,       // A h, B w_down
    kSlopes,     // A dy, B w_down across its rows: dh, from which dg, du and h
    kInput,      // A dg, then du, B w_gate, then w_up, across their rows: dx
    kWeights,    // three products of A and B across their rows: dWg, dWu, dWd
};
constexpr bool a_mn(int mode) { return mode == kWeights; }
constexpr bool b_mn(int mode) { return mode >= kSlopes; }

constexpr int kPairThreads = 224;                    // B, MMA, four epilogue warps, A
constexpr int kBlock = 4096;                         // a warp's staged 32 rows x 128 bytes
constexpr int kMaxStages = 8;
constexpr int stages(int mode, int tn) { return mode == kSlopes ? 5 : tn == 128 ? 8 : 6; }
constexpr int stage_bytes(int tn) { return 16384 + tn / 2 * 128; }
constexpr int blocks(int mode) { return mode == kSlopes ? 3 : 2; }    // of a warp
constexpr int kProducts = 3;

struct Maps {
    CUtensorMap a[kProducts], b[kProducts], c[kProducts];    // kSlopes: a[1] gate, a[2] up
};
struct PairArgs {
    int m_tiles[kProducts], n_tiles[kProducts], first[kProducts + 1];   // tiles of the products
    int cols[kProducts];                             // of C (kGated: features)
    int kblocks, parts;                              // blocks of 64 of a part of the contraction; kInput has two
    int c_rows[kProducts];
    int save;                                        // kGated: gate and up are stored too
    int gelu;
    int *status;
    long long spin_limit;
};
struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_free[2], done;
    uint64_t in[4];                                  // kSlopes: a warp's blocks of gate and up are there
    uint32_t tmem;
    int issued;
};

// A tile's product and its row and column of tiles: eight rows of tiles at a time, column after
// column, so that what the pairs work on together is near a square.
constexpr int kBand = 8;
__device__ __forceinline__ int3 tile_at(const PairArgs &a, int i) {
    int p = 0;
    while (p + 1 < kProducts && i >= a.first[p + 1]) ++p;
    i -= a.first[p];
    const int band = i / (kBand * a.n_tiles[p]), in = i - band * kBand * a.n_tiles[p];
    const int high = min(kBand, a.m_tiles[p] - band * kBand);
    return make_int3(p, band * kBand + in % high, in / high);
}

// A warp's 32 x 64 block of bf16 from registers to C, by TMA; two blocks are used in turn.
struct Stager {
    uint8_t *base;
    int used;
    __device__ __forceinline__ uint8_t *next(int lane) {
        if (used >= 2) {
            if (lane == 0) tc::bulk_wait_read_but_newest();
            __syncwarp();
        }
        return base + (used & 1) * kBlock;
    }
    __device__ __forceinline__ void send(const CUtensorMap *map, uint8_t *block, int col, int row, bool in, int lane) {
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            if (in) tc::tma_store_2d(map, block, col, row);
            tc::bulk_commit();                       // an empty group, where the block lies outside
        }
        ++used;
    }
};

template <int MODE, int TN>
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const __grid_constant__ Maps maps,
                                                            const __grid_constant__ PairArgs a) {
    constexpr bool A_MN = a_mn(MODE), B_MN = b_mn(MODE);
    constexpr int kStages = stages(MODE, TN), kStage = stage_bytes(TN);
    extern __shared__ __align__(1024) uint8_t ring[];
    uint8_t *stage_out = ring + kStages * kStage;
    Control &ctl = *reinterpret_cast<Control *>(stage_out + 4 * blocks(MODE) * kBlock);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = a.first[kProducts];
    const int kblocks = a.kblocks * a.parts;

    if (tc::smem_u32(ring) & 1023u) {                // the swizzle's unit; every CTA alike
        if (threadIdx.x == 0) set_status(a.status, GDN_ERR_CUDA);
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&ctl.full[s], 1);
            tc::mbar_init(&ctl.empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&ctl.acc_full[i], 1);
            tc::mbar_init(&ctl.acc_free[i], 8);      // the epilogue warps of both CTAs
        }
        for (int i = 0; i < 4; ++i) tc::mbar_init(&ctl.in[i], 1);
        tc::mbar_init(&ctl.done, 1);
        ctl.issued = 0;
        tc::fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("griddepcontrol.wait;" ::: "memory");           // the kernel ahead may hold TMEM
        tc::tmem_alloc_pair(&ctl.tmem, 512);
    }
    tc::tc_fence_before();
    tc::cluster_sync();                              // both CTAs' barriers and TMEM are there
    tc::tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const uint32_t ring0 = tc::smem_u32(ring), full0 = tc::smem_u32(ctl.full), empty0 = tc::smem_u32(ctl.empty);
    if (warp == 0 || warp == 6) {
        const bool is_b = warp == 0;
        const uint32_t bar0 = tc::map_rank(full0, 0);
        int i = 0, s = 0;                            // stages asked for
        uint32_t parity = 1;                         // of the stage's last release; the first round has none
        bool ok = true;
        for (int tile = pair; tile < tiles && ok; tile += pairs) {
            const int3 at = tile_at(a, tile);
            const int row = at.y * 256 + rank * 128;
            const int col = MODE == kGated ? at.z * 128 : at.z * TN + rank * (TN / 2);
            for (int kb = 0; kb < kblocks; ++kb, ++i) {
                if (i >= kStages) {
                    ok = tc::mbar_spin(empty0 + 8 * s, parity, a.spin_limit, a.status);
                    if (!ok) break;
                }
                const int part = MODE == kInput && kb >= a.kblocks ? 1 : 0, k = (kb - part * a.kblocks) * 64;
                const uint32_t st = ring0 + s * kStage, bar = bar0 + 8 * s;
                if (is_b) {                          // and arms the pair's barrier for all that both CTAs get
                    tc::expect_bytes(full0 + 8 * s, 2u * kStage, rank == 0);
                    const int b = MODE == kGated ? rank : MODE == kInput ? part : at.x;
                    tc::load_tile<B_MN, true, TN / 2>(st + 16384, &maps.b[b], col, k, bar);
                } else {
                    tc::load_tile<A_MN, true, 128>(st, &maps.a[MODE == kInput ? part : at.x], row, k, bar);
                }
                if (++s == kStages) s = 0, parity ^= 1;
            }
        }
        if (is_b && lane == 0) ctl.issued = i;
    } else if (warp == 1) {
        if (rank == 0) {
            int t = 0, s = 0;
            uint32_t parity = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs, ++t) {
                if (t >= 2) {
                    ok = tc::mbar_spin(tc::smem_u32(&ctl.acc_free[t & 1]), ((t >> 1) - 1) & 1, a.spin_limit, a.status);
                    if (!ok) break;
                }
                tc::tc_fence_after();
                const uint32_t acc = tmem + (t & 1) * 256;
                for (int kb = 0; kb < kblocks; ++kb) {
                    ok = tc::mbar_spin(full0 + 8 * s, parity, a.spin_limit, a.status);
                    if (!ok) break;
                    const uint32_t st = ring0 + s * kStage;
                    tc::mma_bf16_stage<A_MN, B_MN, true>(acc, tc::desc_tile<A_MN>(st), tc::desc_tile<B_MN>(st + 16384),
                                                         tc::idesc_bf16(256, TN, A_MN, B_MN), kb > 0, &ctl.empty[s]);
                    if (++s == kStages) s = 0, parity ^= 1;
                }
                if (ok) tc::mma_commit_pair(&ctl.acc_full[t & 1]);
            }
            tc::mma_commit_pair(&ctl.done);
        }
    } else {
        // epilogue: each warp takes its 32 rows, 64 columns at a time
        const int quarter = warp & 3;
        Stager out{stage_out + quarter * blocks(MODE) * kBlock, 0};
        const uint32_t free0 = tc::map_rank(tc::smem_u32(&ctl.acc_free[0]), 0);
        // kSlopes: the next block's gate and up, by TMA, under the products and the stores before it;
        // dg and du take their places, h a third block
        uint8_t *const gate = out.base, *const up = gate + kBlock, *const hidden = up + kBlock;
        int asked = 0, had = 0;
        const auto ask = [&](int tile, int c) {
            const int3 at = tile_at(a, tile);
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&ctl.in[quarter], 2 * kBlock);
                const int row = at.y * 256 + rank * 128 + 32 * quarter, col = at.z * 256 + c;
                tc::tma_load_2d(gate, &maps.a[1], &ctl.in[quarter], col, row);
                tc::tma_load_2d(up, &maps.a[2], &ctl.in[quarter], col, row);
            }
            ++asked;
        };
        if (MODE == kSlopes && pair < tiles) ask(pair, 0);
        int t = 0;
        for (int tile = pair; tile < tiles; tile += pairs, ++t) {
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&ctl.acc_full[t & 1], (t >> 1) & 1, a.spin_limit, a.status))) break;
            tc::tc_fence_after();
            const int3 at = tile_at(a, tile);
            const int row = at.y * 256 + rank * 128 + 32 * quarter, rows = a.c_rows[at.x], cols = a.cols[at.x];
            const uint32_t acc = tmem + (t & 1) * 256;
            if constexpr (MODE == kGated) {
#pragma unroll 1
                for (int c = 0; c < 128; c += 64) {
                    const int col = at.z * 128 + c;
                    const bool in = row < rows && col < cols;
                    float g[64], u[64];
                    tc::tmem_ld32x2(tc::tmem_addr(acc, quarter, c), tc::tmem_addr(acc, quarter, c + 32), g, g + 32);
                    tc::tmem_ld32x2(tc::tmem_addr(acc, quarter, 128 + c), tc::tmem_addr(acc, quarter, 160 + c), u, u + 32);
                    if (a.save) {
                        uint8_t *block = out.next(lane);
                        tc::st_row64(block, lane, g);
                        out.send(&maps.c[1], block, col, row, in, lane);
                        block = out.next(lane);
                        tc::st_row64(block, lane, u);
                        out.send(&maps.c[2], block, col, row, in, lane);
                    }
                    if (a.gelu) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) u[i] *= activation<true>(g[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 64; ++i) u[i] *= activation<false>(g[i]);
                    }
                    uint8_t *block = out.next(lane);
                    tc::st_row64(block, lane, u);
                    out.send(&maps.c[0], block, col, row, in, lane);
                }
            } else if constexpr (MODE == kSlopes) {
                bool there = true;
#pragma unroll 1
                for (int c = 0; c < 256; c += 64) {
                    const int col = at.z * 256 + c;
                    const bool in = row < rows && col < cols;
                    there = __all_sync(0xffffffffu, tc::mbar_wait(&ctl.in[quarter], had & 1, a.spin_limit, a.status));
                    if (!there) break;
                    ++had;
                    const auto slopes = [&](auto gelu) {
#pragma unroll
                        for (int b = 0; b < 64; b += 32) {
                            float v[32];
                            tc::tmem_ld32(tc::tmem_addr(acc, quarter, c + b), v);
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                const uint32_t off = tc::sw128_off(lane, b + i);
                                uint4 *pg = reinterpret_cast<uint4 *>(gate + off), *pu = reinterpret_cast<uint4 *>(up + off);
                                const uint4 gr = *pg, ur = *pu;
                                const __nv_bfloat16 *gs = reinterpret_cast<const __nv_bfloat16 *>(&gr);
                                const __nv_bfloat16 *us = reinterpret_cast<const __nv_bfloat16 *>(&ur);
                                float dg[8], du[8], h[8];
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const float g = to_f(gs[j]), u = to_f(us[j]);
                                    float slope;
                                    const float f = activation<decltype(gelu)::value>(g, slope);
                                    dg[j] = v[i + j] * u * slope;
                                    du[j] = v[i + j] * f;
                                    h[j] = f * u;
                                }
                                Vec<__nv_bfloat16, 8>::store(reinterpret_cast<__nv_bfloat16 *>(pg), dg);
                                Vec<__nv_bfloat16, 8>::store(reinterpret_cast<__nv_bfloat16 *>(pu), du);
                                Vec<__nv_bfloat16, 8>::store(reinterpret_cast<__nv_bfloat16 *>(hidden + off), h);
                            }
                        }
                    };
                    if (a.gelu) slopes(std::true_type());
                    else slopes(std::false_type());
                    if (c == 192) {                  // the accumulator is free
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive_cluster(free0 + 8 * (t & 1));
                    }
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        if (in) {
                            tc::tma_store_2d(&maps.c[0], gate, col, row);
                            tc::tma_store_2d(&maps.c[1], up, col, row);
                            tc::tma_store_2d(&maps.c[2], hidden, col, row);
                        }
                        tc::bulk_commit();
                        tc::bulk_wait_read();
                    }
                    __syncwarp();
                    if (c < 192) ask(tile, c + 64);
                    else if (tile + pairs < tiles) ask(tile + pairs, 0);
                }
                if (!there) break;
                continue;
            } else {
#pragma unroll 1
                for (int c = 0; c < TN; c += 64) {
                    const int col = at.z * TN + c;
                    float v[64];
                    tc::tmem_ld32x2(tc::tmem_addr(acc, quarter, c), tc::tmem_addr(acc, quarter, c + 32), v, v + 32);
                    uint8_t *block = out.next(lane);
                    tc::st_row64(block, lane, v);
                    out.send(&maps.c[at.x], block, col, row, row < rows && col < cols, lane);
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(free0 + 8 * (t & 1));
        }
        if (lane == 0) tc::bulk_wait_read();
        if (had < asked) tc::mbar_drain(&ctl.in[quarter], had & 1);
        __syncwarp();
    }
    // every MMA done and every copy landed before TMEM is given back and a CTA goes
    tc::mbar_drain(&ctl.done, 0);
    tc::tc_fence_before();
    tc::cluster_sync();
    if (threadIdx.x == 0 && rank == 0)
        for (int i = max(0, ctl.issued - kStages); i < ctl.issued; ++i)
            tc::mbar_drain(&ctl.full[i % kStages], (i / kStages) & 1);
    tc::cluster_sync();
    tc::tc_fence_after();
    if (warp == 1) tc::tmem_dealloc_pair(tmem, 512);
}

// As much shared memory for its TMEM columns as clusters take (the MX products' rule), and no more than
// there is.
constexpr size_t pair_smem(int mode, int tn) {
    return std::max<size_t>(stages(mode, tn) * stage_bytes(tn) + 4 * blocks(mode) * kBlock + sizeof(Control), 512 * 432 - 1024);
}
static_assert(pair_smem(kGated, 256) <= 227 * 1024 && pair_smem(kSlopes, 256) <= 227 * 1024 && pair_smem(kDown, 128) <= 227 * 1024, "");

// A matrix [rows, cols] as an operand (64-element boxes: `box` rows of it, or 64 of the contraction) or
// as a result (32 rows).
cudaError_t operand(CUtensorMap *m, const void *base, long long rows, long long cols, bool mn, int box) {
    return tc::make_map_rows(m, base, rows, cols, 2, 64, mn ? 64 : box, true);
}
cudaError_t result(CUtensorMap *m, const void *base, long long rows, long long cols) {
    return tc::make_map_rows(m, base, rows, cols, 2, 64, 32, true);
}

// One launch of up to three products.
struct Product {
    const void *a, *b, *b2;      // b2: kGated w_up; kInput: a2 and b2 are the second part; kSlopes: gate and up
    const void *a2;
    void *c[kProducts];          // kGated and kSlopes have three results, the others one
    long long m, n, k;           // C [m, n], contraction k
};
template <int MODE, int TN = 256>
gdn_status run_pair(const char *name, const Product *p, int count, PairArgs g, const LayerDevice &dev, cudaStream_t q) {
    Maps maps = {};
    cudaError_t e = tc::encoder();
    g.kblocks = (int)((p->k + 63) / 64);
    g.parts = MODE == kInput ? 2 : 1;
    long long tiles = 0;
    for (int i = 0; i < kProducts; ++i) {
        g.first[i] = (int)tiles;
        if (i >= count) continue;
        const bool amn = a_mn(MODE), bmn = b_mn(MODE);
        const auto op_a = [&](CUtensorMap *m, const void *base) {
            if (e == cudaSuccess) e = operand(m, base, amn ? p[i].k : p[i].m, amn ? p[i].m : p[i].k, amn, 128);
        };
        const auto op_b = [&](CUtensorMap *m, const void *base) {
            if (e == cudaSuccess) e = operand(m, base, bmn ? p[i].k : p[i].n, bmn ? p[i].n : p[i].k, bmn, TN / 2);
        };
        op_a(&maps.a[i], p[i].a);
        op_b(&maps.b[i], p[i].b);
        if (MODE == kInput) op_a(&maps.a[1], p[i].a2);
        if (MODE == kSlopes && e == cudaSuccess) e = result(&maps.a[1], p[i].a2, p[i].m, p[i].n);
        if (MODE == kSlopes && e == cudaSuccess) e = result(&maps.a[2], p[i].b2, p[i].m, p[i].n);
        if (MODE == kInput || MODE == kGated) op_b(&maps.b[1], p[i].b2);
        for (int j = 0; j < (MODE == kGated || MODE == kSlopes ? kProducts : 1); ++j)
            if (p[i].c[j] && e == cudaSuccess) e = result(&maps.c[i + j], p[i].c[j], p[i].m, p[i].n);
        g.m_tiles[i] = (int)((p[i].m + 255) / 256);
        g.n_tiles[i] = (int)((p[i].n + (MODE == kGated ? 127 : TN - 1)) / (MODE == kGated ? 128 : TN));
        g.c_rows[i] = (int)p[i].m;
        g.cols[i] = (int)p[i].n;
        tiles += (long long)g.m_tiles[i] * g.n_tiles[i];
        if (tiles >= (1ll << 30)) return fail(GDN_ERR_INVALID_ARG, "problem too large");
    }
    if (e != cudaSuccess) return cuda_fail(e, "tensor map of a product");
    g.first[kProducts] = (int)tiles;
    for (int i = count; i < kProducts; ++i) g.first[i] = (int)tiles;
    g.status = dev.status;
    g.spin_limit = dev.spin_limit;
    auto k = pair_kernel<MODE, TN>;
    if ((e = allow_smem((const void *)k, pair_smem(MODE, TN))) != cudaSuccess) return cuda_fail(e, "shared memory of the product");
    const int pairs = (int)std::min<long long>(tiles, dev.sms / 2);
    prof_before(name, q);
    e = launch_pdl_cluster(k, dim3(2 * pairs), dim3(kPairThreads), pair_smem(MODE, TN), 2, q, maps, g);
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "feed-forward product launch");
}

// Tiles of 256 x 128 where those of 256 x 256 would leave half of the pairs without one: 1000 x 5464 x
// 2048 41 us in 32 wide tiles, 33 in 64 narrow ones (not half, as a stage of either is bound by what
// comes into an SM).
bool narrow_fits(const Product &p, int sms) { return (p.m + 255) / 256 * ((p.n + 255) / 256) * 2 <= sms / 2; }

template <int MODE>
gdn_status run_pair_any(const char *name, const Product &p, const PairArgs &g, const LayerDevice &dev, cudaStream_t q) {
    return narrow_fits(p, dev.sms) ? run_pair<MODE, 128>(name, &p, 1, g, dev, q) : run_pair<MODE>(name, &p, 1, g, dev, q);
}

// ------------------------------------------------------------------ few tokens
// One CTA makes 128 rows of a weight (or 64 rows of w_gate and 64 of w_up) x `nt` tokens: the weight is
// the MMA's 128-row operand, so that few tokens cost a narrow MMA and not idle rows.  Where tiles are
// too few for the GPU the CTAs of a cluster share the contraction: each leaves its fp32 tile in its
// shared memory, and each adds up its share of the tokens, in rank order.  Bound by the weights' bytes.
constexpr int kFewThreads = 192;                     // loads, MMA, four epilogue warps
constexpr int kFewStages = 10, kMaxSplits = 8;
constexpr int kTmemBarrier = 1;                      // named: TMEM is there, and waits with a limit may begin

struct FewArgs {
    __nv_bfloat16 *c, *gate, *up;                    // gate, up: kGated, null = not stored
    int tokens, cols;                                // of C (kGated: features)
    int nt, token_tiles, kblocks, stages, stage_bytes, tmem_cols;
    int early_w;                                     // the kernel ahead began when all before it had ended, the weight's
                                                     // writers among them
    int gelu;
    int low;                                         // rows of C between its high parts and its low ones; not GATED: rows of
                                                     // tokens between those; 0 = no low parts
    int *status;
    long long spin_limit;
};
struct FewControl {
    uint64_t full[kFewStages], empty[kFewStages], done;
    uint32_t tmem;
    int failed, issued;
};
struct FewMaps {
    CUtensorMap x, w[2];
};

template <bool GATED>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
    extern __shared__ uint8_t raw[];
    __shared__ FewControl ctl;
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    constexpr int kRows = GATED ? 64 : 128;          // columns of C of a tile

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_rank(), splits = (int)tc::cluster_size();
    const int tile = blockIdx.x / splits;
    const int f0 = tile / a.token_tiles * kRows, t0 = tile % a.token_tiles * a.nt;
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
    __syncthreads();

    if (warp == 0) {
        const int n = kb1 - kb0;
        const uint32_t ring0 = tc::smem_u32(ring), full0 = tc::smem_u32(ctl.full), empty0 = tc::smem_u32(ctl.empty);
        auto load_w = [&](int kb, uint32_t st, uint32_t bar) {       // arms the stage for all it gets
            tc::expect_bytes(bar, (uint32_t)a.stage_bytes, true);
            if (GATED) {
                tc::load_box<false>(st, &maps.w[0], kb * 64, f0, bar);
                tc::load_box<false>(st + 8192, &maps.w[1], kb * 64, f0, bar);
            } else {
                tc::load_box<false>(st, &maps.w[0], kb * 64, f0, bar);
            }
        };
        // a ring's worth of weights may come before the kernel ahead has written the tokens
        const int ahead = a.early_w ? min(n, a.stages) : 0;
        for (int i = 0; i < ahead; ++i) load_w(kb0 + i, ring0 + i * a.stage_bytes, full0 + 8 * i);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");    // all before this kernel has ended
        int i = 0, s = 0;
        uint32_t parity = 1;                         // of the stage's last release; the first round has none
        auto fill = [&] {
            const uint32_t st = ring0 + s * a.stage_bytes, bar = full0 + 8 * s;
            if (i >= ahead) load_w(kb0 + i, st, bar);
            tc::load_box<false>(st + 16384, &maps.x, (kb0 + i) * 64, t0, bar);
            if (++s == a.stages) s = 0, parity ^= 1;
        };
        for (; i < min(n, a.stages); ++i) fill();
        tc::named_sync(kTmemBarrier, kFewThreads);
        for (; i < n; ++i) {
            if (!tc::mbar_spin(empty0 + 8 * s, parity, a.spin_limit, a.status)) {
                ctl.failed = 1;
                break;
            }
            fill();
        }
        if (lane == 0) ctl.issued = i;
    } else if (warp == 1) {
        asm volatile("griddepcontrol.wait;" ::: "memory");           // the kernel ahead may hold TMEM
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        tc::tmem_alloc(&ctl.tmem, (uint32_t)a.tmem_cols);
        tc::tmem_relinquish();
        tc::tc_fence_before();
        tc::named_sync(kTmemBarrier, kFewThreads);
        tc::tc_fence_after();
        const uint32_t tmem = ctl.tmem, idesc = tc::idesc_bf16(128, a.nt, false, false);
        int s = 0;
        uint32_t parity = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!tc::mbar_spin(tc::smem_u32(&ctl.full[s]), parity, a.spin_limit, a.status)) {
                ctl.failed = 1;
                break;
            }
            const uint32_t st = tc::smem_u32(ring + s * a.stage_bytes);
            tc::mma_bf16_stage<false, false, false>(tmem, tc::desc_tile<false>(st), tc::desc_tile<false>(st + 16384), idesc,
                                                    kb > kb0, &ctl.empty[s]);
            if (++s == a.stages) s = 0, parity ^= 1;
        }
        tc::mma_commit(&ctl.done);
    }
    if (warp > 1) {
        asm volatile("griddepcontrol.wait;" ::: "memory");              // C may be written
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        tc::named_sync(kTmemBarrier, kFewThreads);
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
        for (int c = 0; c < a.nt; c += 16) {
            float v[16];
            tc::tmem_ld8x2(tc::tmem_addr(tmem, warp, c), tc::tmem_addr(tmem, warp, c + 8), v, v + 8);
#pragma unroll
            for (int j = 0; j < 16; ++j) to[(c + j) * 128] = v[j];
        }
    }
    tc::tc_fence_before();
    if (splits > 1) tc::cluster_sync();
    else __syncthreads();
    tc::tc_fence_after();
    if (ok) {
        const uint32_t base = tc::smem_u32(out);
        const int step = splits * (kFewThreads / 32), rows = min(a.nt, GATED || !a.low ? a.tokens - t0 : a.low);
        for (int j = rank * (kFewThreads / 32) + warp; j < rows; j += step) {
            const int at = j * 128 + 4 * lane;
            float4 v;
            if (!GATED && a.low) {                   // of one tile of tokens: high and low parts
                v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int r = 0; r < 2 * splits; ++r) {
                    const uint32_t from = base + 4u * (uint32_t)(at + (r & 1) * a.low * 128);
                    const float4 p = tc::ld_cluster4(tc::map_rank(from, r / 2));
                    v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
                }
            } else if (splits == 1) {
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
            float x[4] = {v.x, v.y, v.z, v.w};
            const long long row = (long long)(t0 + j) * a.cols;
            if (!GATED) {
                if (f0 + 4 * lane < a.cols) tc::st4(a.c + row + f0 + 4 * lane, x);
                continue;
            }
            // lanes 0 - 15 have the gate of 64 features, 16 - 31 their up
            const int f = f0 + 4 * (lane & 15);
            const bool in = f < a.cols;
            __nv_bfloat16 *kept = lane < 16 ? a.gate : a.up;
            if (kept && in) tc::st4(kept + row + f, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = __shfl_down_sync(0xffffffffu, x[i], 16);
                x[i] = u * (a.gelu ? activation<true>(x[i]) : activation<false>(x[i]));
            }
            if (lane < 16 && in) {
                tc::st4(a.c + row + f, x);
                if (a.low) {                         // nothing of a value that bf16 rounds to infinity
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float high = __bfloat162float(__float2bfloat16_rn(x[i]));
                        x[i] = isinf(high) ? 0.f : x[i] - high;
                    }
                    tc::st4(a.c + row + (long long)a.low * a.cols + f, x);
                }
            }
        }
    }
    if (splits > 1) tc::cluster_sync();              // the others have read this CTA's tile
    if (warp == 1) tc::tmem_dealloc(tmem, (uint32_t)a.tmem_cols);
}

// Tokens of a tile: 16, or as many as there are up to 128.
int token_tile(int tokens) {
    int nt = 16;
    while (nt < 128 && nt < tokens) nt *= 2;
    return nt;
}

// Single CTAs for up to 128 tokens; of the product out of the block also while their tiles are three
// fifths of a wave at most.  Above, a stage of theirs takes 0.5 us, as long as its 32 KB to every SM, and
// CTA pairs, which take half as much for a product, are ahead.  Us of single CTAs | pairs, into the
// block: 128 x 4096 x 12288 47 | 55, 192 x 2048 x 5464 25 | 22, 256 x 4096 x 12288 68 | 56; out of it 256
// x 12288 x 4096 35 | 49, 512 x 5464 x 2048 27 | 33, 768 x 5464 x 2048 40 | 33, 1000 x 5464 x 2048 40 | 33.
bool few_fits(const Product &p, bool gated, int sms) {
    if (p.m <= 128) return true;
    return !gated && (p.n + 127) / 128 * ((p.m + 127) / 128) * 5 <= sms * 3;
}

template <bool GATED>
gdn_status run_few(const char *name, const Product &p, int gelu, int low, bool early_w, const LayerDevice &dev, cudaStream_t q) {
    FewMaps maps = {};
    FewArgs g{};
    g.c = (__nv_bfloat16 *)p.c[0];
    if (GATED) g.gate = (__nv_bfloat16 *)p.c[1], g.up = (__nv_bfloat16 *)p.c[2];
    g.tokens = (int)p.m;
    g.cols = (int)p.n;
    g.nt = token_tile((int)std::min<long long>(p.m, 128));
    g.token_tiles = (int)((p.m + g.nt - 1) / g.nt);
    g.kblocks = (int)((p.k + 63) / 64);
    g.stage_bytes = 16384 + g.nt * 128;
    g.early_w = early_w;
    g.gelu = gelu;
    g.low = low;
    g.status = dev.status;
    g.spin_limit = dev.spin_limit;
    // The CTAs of a cluster share the contraction, by powers of two, while slots of the GPU are empty:
    // two CTAs to an SM and up to 8 to a cluster for few tokens; one and up to 4 for many, whose tiles
    // take long to add up.  Clusters of c leave about c SMs without one.
    const int rows = GATED ? 64 : 128;
    const long long tiles = (p.n + rows - 1) / rows * g.token_tiles;
    const bool few = g.nt <= 32;
    int splits = 1;
    while (splits < (few ? kMaxSplits : 4) && 2 * splits <= g.kblocks &&
           2 * splits * tiles <= (few ? 2 : 1) * (dev.sms - 2 * splits))
        splits *= 2;
    const int per = (g.kblocks + splits - 1) / splits;
    g.stages = std::max(1, std::min({kFewStages, per, (tiles * splits <= dev.sms - splits ? 200 : 100) * 1024 / g.stage_bytes}));
    g.tmem_cols = 32;
    while (g.tmem_cols < g.nt) g.tmem_cols *= 2;
    cudaError_t e = tc::encoder();
    const auto map = [&](CUtensorMap *m, const void *base, long long r, int box) {
        if (e == cudaSuccess) e = tc::make_map_rows(m, base, r, p.k, 2, 64, box, true);
    };
    map(&maps.x, p.a, p.m, g.nt);
    map(&maps.w[0], p.b, p.n, rows);
    if (GATED) map(&maps.w[1], p.b2, p.n, rows);
    if (e != cudaSuccess) return cuda_fail(e, "tensor map of a product");
    size_t smem = std::max(g.stages * g.stage_bytes, g.nt * 128 * 4) + 1024;
    // a cluster's CTAs hold their TMEM until all have theirs: shared memory in proportion, as the MX products
    if (splits > 1) smem = std::max(smem, (size_t)g.tmem_cols * 432 - 1024);
    auto k = few_kernel<GATED>;
    if ((e = allow_smem((const void *)k, smem)) != cudaSuccess) return cuda_fail(e, "shared memory of the product");
    const long long ctas = tiles * splits;
    if (ctas >= (1ll << 31)) return fail(GDN_ERR_INVALID_ARG, "problem too large");
    prof_before(name, q);
    e = launch_pdl_cluster(k, dim3((unsigned)ctas), dim3(kFewThreads), smem, splits, q, maps, g);
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "feed-forward product launch");
}

gdn_status check(int M, int K, int F, int dtype, int activation) {
    if (M < 0 || K < 1 || F < 1) return fail(GDN_ERR_INVALID_ARG, "bad sizes M=%d K=%d F=%d", M, K, F);
    if (std::max({M, K, F}) > kMaxExtent) return fail(GDN_ERR_INVALID_ARG, "problem too large: M=%d K=%d F=%d", M, K, F);
    if (K % 8 != 0 || F % 8 != 0)
        return fail(GDN_ERR_UNSUPPORTED, "K = %d, F = %d: rows start on 16 bytes, multiples of 8", K, F);
    if (dtype != GDN_BF16) return fail(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_BF16", dtype);
    if (activation != GDN_ACT_SILU && activation != GDN_ACT_GELU)
        return fail(GDN_ERR_UNSUPPORTED, "activation %d is not GDN_ACT_SILU or GDN_ACT_GELU", activation);
    return GDN_OK;
}
// Bytes of an [M, F] tensor, to the next one's 256-byte boundary.
size_t hidden_bytes(int M, int F) { return ((size_t)M * F * 2 + 255) / 256 * 256; }

}  // namespace
}  // namespace ffn
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_ffn_fwd_workspace_size(const gdn_ffn_fwd_args *a) {
    if (!a) {
        fail(GDN_ERR_INVALID_ARG, "null args");
        return 0;
    }
    if (ffn::check(a->M, a->K, a->F, a->dtype, a->activation) != GDN_OK) return 0;
    return a->M == 0 ? 256 : std::max<size_t>(512, ffn::hidden_bytes(a->M <= ffn::kLowTokens ? 2 * a->M : a->M, a->F));
}

gdn_status gdn_ffn_fwd(const gdn_ffn_fwd_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = ffn::check(a->M, a->K, a->F, a->dtype, a->activation);
    if (st != GDN_OK || a->M == 0) return st;
    if (!a->x || !a->w_gate || !a->w_up || !a->w_down || !a->y || !a->gate != !a->up)
        return fail(GDN_ERR_INVALID_ARG, "x, w_gate, w_up, w_down and y are required, gate and up together or not at all");
    if (misaligned(a->x) || misaligned(a->w_gate) || misaligned(a->w_up) || misaligned(a->w_down) ||
        misaligned(a->y) || misaligned(a->gate) || misaligned(a->up))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    const size_t need = gdn_ffn_fwd_workspace_size(a);
    if (!ws || misaligned(ws) || ws_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    cudaStream_t q = (cudaStream_t)stream;
    ffn::PairArgs g{};
    g.save = a->gate != nullptr;
    g.gelu = a->activation == GDN_ACT_GELU;
    const ffn::Product up{a->x, a->w_gate, a->w_up, nullptr, {ws, a->gate, a->up}, a->M, a->F, a->K};
    // of few tokens h is two rows, what bf16 holds of it and of the rest: tokens to the second product
    const int low = a->M <= ffn::kLowTokens ? a->M : 0;
    const ffn::Product down{ws, a->w_down, nullptr, nullptr, {a->y}, a->M + low, a->K, a->F};
    const bool few = ffn::few_fits(up, true, dev.sms);
    st = few ? ffn::run_few<true>("ffn_gated_few", up, g.gelu, low, false, dev, q)
             : ffn::run_pair<ffn::kGated>("ffn_gated", &up, 1, g, dev, q);
    if (st != GDN_OK) return st;
    return ffn::few_fits(down, false, dev.sms) ? ffn::run_few<false>("ffn_down_few", down, 0, low, few, dev, q)
                                        : ffn::run_pair_any<ffn::kDown>("ffn_down", down, g, dev, q);
}

size_t gdn_ffn_bwd_workspace_size(const gdn_ffn_bwd_args *a) {
    if (!a) {
        fail(GDN_ERR_INVALID_ARG, "null args");
        return 0;
    }
    if (ffn::check(a->M, a->K, a->F, a->dtype, a->activation) != GDN_OK) return 0;
    if (a->M == 0) return 256;
    return std::max<size_t>(512, ffn::few_bwd_fits(a->M, a->K, a->F) ? ffn::few_bwd_bytes(a->M, a->K, a->F)
                                                                     : 3 * ffn::hidden_bytes(a->M, a->F));
}

gdn_status gdn_ffn_bwd(const gdn_ffn_bwd_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = ffn::check(a->M, a->K, a->F, a->dtype, a->activation);
    if (st != GDN_OK) return st;
    if (!a->dw_gate || !a->dw_up || !a->dw_down ||
        (a->M > 0 && (!a->d_y || !a->x || !a->w_gate || !a->w_up || !a->w_down || !a->gate || !a->up || !a->dx)))
        return fail(GDN_ERR_INVALID_ARG, "d_y, x, the weights, gate, up, dx and the weights' gradients are required");
    if (misaligned(a->d_y) || misaligned(a->x) || misaligned(a->w_gate) || misaligned(a->w_up) ||
        misaligned(a->w_down) || misaligned(a->gate) || misaligned(a->up) || misaligned(a->dx) ||
        misaligned(a->dw_gate) || misaligned(a->dw_up) || misaligned(a->dw_down))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    const size_t need = gdn_ffn_bwd_workspace_size(a);
    if (need > 256 && (!ws || misaligned(ws) || ws_bytes < need))
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    cudaStream_t q = (cudaStream_t)stream;
    if (a->M == 0) {                                 // gradients of no tokens
        const size_t bytes = (size_t)a->F * a->K * 2;
        cudaError_t e = cudaMemsetAsync(a->dw_gate, 0, bytes, q);
        if (e == cudaSuccess) e = cudaMemsetAsync(a->dw_up, 0, bytes, q);
        if (e == cudaSuccess) e = cudaMemsetAsync(a->dw_down, 0, bytes, q);
        return e == cudaSuccess ? GDN_OK : cuda_fail(e, "clearing the weights' gradients");
    }
    if (ffn::few_bwd_fits(a->M, a->K, a->F)) {
        const cudaError_t e = ffn::few_bwd(a, (float *)ws, q);
        return e == cudaSuccess ? GDN_OK : cuda_fail(e, "feed-forward backward launch");
    }
    uint8_t *dg = (uint8_t *)ws, *du = dg + ffn::hidden_bytes(a->M, a->F), *h = du + ffn::hidden_bytes(a->M, a->F);
    ffn::PairArgs g{};
    g.gelu = a->activation == GDN_ACT_GELU;
    const ffn::Product dh{a->d_y, a->w_down, a->up, a->gate, {dg, du, h}, a->M, a->F, a->K};
    const ffn::Product dx{dg, a->w_gate, a->w_up, du, {a->dx}, a->M, a->K, a->F};
    const ffn::Product dw[3] = {{dg, a->x, nullptr, nullptr, {a->dw_gate}, a->F, a->K, a->M},
                                {du, a->x, nullptr, nullptr, {a->dw_up}, a->F, a->K, a->M},
                                {a->d_y, h, nullptr, nullptr, {a->dw_down}, a->K, a->F, a->M}};
    st = ffn::run_pair<ffn::kSlopes>("ffn_slopes", &dh, 1, g, dev, q);
    if (st == GDN_OK) st = ffn::run_pair_any<ffn::kInput>("ffn_input", dx, g, dev, q);
    if (st == GDN_OK) st = ffn::run_pair<ffn::kWeights>("ffn_weights", dw, 3, g, dev, q);
    return st;
}

}  // extern "C"
