// gdn_linrec.cu -- per-channel gated linear recurrence h_t = a_t h_{t-1} + x_t,
// its backward pass and its one-token step.
//
// A token's map h -> a h + x composes as (A, B) then (A', B') = (A A', A' B + B'),
// so a run of tokens is one pair per channel.  A CTA takes 64 channels of one sequence
// and walks it in tiles of W x R tokens that TMA keeps coming.  Each warp reduces its R
// tokens to a pair, the pairs meet in shared memory, and every warp, knowing the value
// before its first token, forms its R results from the decays it still holds in
// registers: one pass over memory.
//
// Where channels and sequences are too few for the GPU, a cluster of S CTAs shares
// a sequence: its CTAs take neighbouring tiles, each sends its tile's pair into
// every other's shared memory, and each folds the pairs of the tiles before its own.
// No CTA ever waits on global memory, and the order of every sum is fixed.  A cluster
// has 8 CTAs at most; long sequences of few channels are instead cut into parts that are
// walked twice, first for their pairs alone, then, the pairs joined, for the results.
//
// Bound by memory and, gated, nearly as much by the gate's arithmetic: 16 x (512 .. 8192) tokens
// x 4096 gated bf16 forward 262 us, 96% of the measured copy rate; 4 x 4096 x 4096 backward 118
// us, 84%; 65536 x 2048 in clusters of 8 159 us, 75% (the rounds' length: each waits for the
// slowest of 8 CTAs).
#include <algorithm>
#include <type_traits>

#include "gdn_layer_internal.h"
#include "tc_mx_ptx.cuh"

namespace gdn {
namespace linrec {
namespace {

constexpr int kChannels = 64;      // of a CTA: two to a lane
constexpr int kMaxCluster = 8;

// The two channels a lane carries, as two elements of T side by side.
__device__ __forceinline__ float2 get2(uint32_t r) {
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}
__device__ __forceinline__ float2 get2(float2 r) { return r; }
__device__ __forceinline__ uint32_t put2(float2 v, const __nv_bfloat16 *) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ float2 put2(float2 v, const float *) { return v; }
template <typename T>
struct Raw2;
template <>
struct Raw2<__nv_bfloat16> {
    using type = uint32_t;
};
template <>
struct Raw2<float> {
    using type = float2;
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float bounded(float x) { return fminf(x, 3e38f); }

// A token's gate: the decay a = exp(l) with l = g, or -s softplus(g); and for the
// backward pass softplus(g) in units of kUnit and its derivative, the logistic function.
//
// fp32 tensors take the accurate functions.  For bf16 ones the two exponentials and the
// logarithm are the hardware's: with the accurate ones the pass is bound by arithmetic (106
// instructions for a token of two channels, 46% of the memory rate; 44 in this form).
// What a slow channel needs of them is small relative errors of the log decay, however small
// that is:
// - It multiplies a thousand decays near 1 together, and the hardware exponential's errors
//   there lean one way (2e-8 on average, 2e-5 in the fp32 state of such a channel).  So for
//   |y| < 1/32 2^y is 1 + y q(y), q the polynomial through (2^y - 1) / y at the three Chebyshev
//   points of -1/32 .. 1/32: off by 1.1e-7 of y, and by a rounding that points either way.
// - softplus(g) ~ e^g of a steady logit of -15 decides what is left after 65536 tokens, and
//   d(gate_scale) is a sum of such terms.  The logarithm of the rounded 1 + e^g loses it (1% at
//   -12, all of it at -17).  So for e < 1/8 log2(1 + e) is e p(e), p the polynomial through
//   log2(1 + e) / e at the four Chebyshev points of 0 .. 1/8: off by 3.1e-7 of itself, where the
//   logarithm of a larger e is off by 2^-22 of at least 0.17.  e^g itself is off by 2^-23 |g| of
//   itself, the rounding of its exponent.  (One polynomial of eight terms for all e needs no
//   logarithm and took longer, the FMA pipe being the fuller one: 65536 x 2048 forward 163 us
//   against 159, backward 273 against 263.)
template <typename T, bool GATED>
struct Gate {
    static constexpr float kUnit = 1.f;      // of softplus
    static __device__ __forceinline__ float decay(float g, float s, float &sp) {
        sp = 0.f;
        if (GATED) sp = fmaxf(g, 0.f) + log1pf(expf(-fabsf(g)));
        return expf(GATED ? -s * sp : g);
    }
    static __device__ __forceinline__ float2 decay(float2 g, float2 s, float2 &sp) {
        return make_float2(decay(g.x, s.x, sp.x), decay(g.y, s.y, sp.y));
    }
    static __device__ __forceinline__ float slope(float g) {
        const float e = expf(-fabsf(g));
        return (g >= 0.f ? 1.f : e) / (1.f + e);
    }
    static __device__ __forceinline__ float2 slope(float2 g, float2) {
        return make_float2(slope(g.x), slope(g.y));
    }
};
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
template <bool GATED>
struct Gate<__nv_bfloat16, GATED> {
    static constexpr float kUnit = kLn2;
    static __device__ __forceinline__ float2 decay(float2 g, float2 s, float2 &sp) {
        float2 y = mul2(g, both(kLog2e));
        if (GATED) {
            const float2 e = make_float2(ex2(-fabsf(y.x)), ex2(-fabsf(y.y)));
            const float2 u = add2(e, both(1.f));
            float2 q = fma2(e, both(-2.9770274392e-1f), both(4.7618794121e-1f));
            q = fma2(q, e, both(-7.2123178461e-1f));
            q = mul2(fma2(q, e, both(1.4426945903f)), e);
            sp = add2(make_float2(fmaxf(y.x, 0.f), fmaxf(y.y, 0.f)),
                      make_float2(e.x < 0.125f ? q.x : lg2(u.x), e.y < 0.125f ? q.y : lg2(u.y)));
            y = mul2(sp, make_float2(-s.x, -s.y));
        }
        float2 p = fma2(y, both(5.5505085252e-2f), both(2.4023355157e-1f));
        p = fma2(p, y, both(kLn2));
        p = fma2(p, y, both(1.f));
        return make_float2(fabsf(y.x) < 0.03125f ? p.x : ex2(y.x), fabsf(y.y) < 0.03125f ? p.y : ex2(y.y));
    }
    // the logistic function is e^g / (1 + e^g) = 2^(g log2 e - softplus(g)); an infinite g
    // as the largest number, whose softplus it is too
    static __device__ __forceinline__ float2 slope(float2 g, float2 sp) {
        const float2 y = mul2(g, both(kLog2e));
        return make_float2(ex2(bounded(y.x) - bounded(sp.x)), ex2(bounded(y.y) - bounded(sp.y)));
    }
};

struct Shape {
    const int32_t *cu;
    long long T;               // tokens per row, or of the packed batch
    int N, D, groups;          // sequences, channels, channel groups
    int lanes_n;               // clusters that share a channel group's sequences
    int cluster;               // CTAs of a cluster
    int parts;                 // parts a sequence is cut into (then cluster is 1)
    float2 *pair;              // parts > 1: [N][parts][D] a part's pair, written by the first walk
    float *start;              // parts > 1: [N][parts][D] the value before a part, for the second
    int reduce;                // the first walk
    int longest_first;         // a CTA takes one sequence, and the first CTAs the longest
    int *status;
    long long spin_limit;
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

// The sequence of the `j`-th CTAs of a packed batch whose CTAs come in several waves: the
// j-th longest, so that no long one is left for the end.  16 x (512 .. 8192) tokens x 4096
// gated bf16 forward, backward, the longest last: 303, 535 us in order, 262, 447 so.
constexpr int kMaxOrdered = 128;
__device__ __forceinline__ int sequence_of(const Shape &s, int j, void *scratch) {
    if (!s.longest_first) return j;
    int *len = reinterpret_cast<int *>(scratch), *found = len + kMaxOrdered, t = threadIdx.x;
    if (t < s.N) len[t] = s.cu[t + 1] - s.cu[t];
    __syncthreads();
    if (t < s.N) {
        const int mine = len[t];
        int rank = 0;
        for (int u = 0; u < s.N; ++u) rank += len[u] > mine || (len[u] == mine && u < t);
        if (rank == j) *found = t;
    }
    __syncthreads();
    const int n = *found;
    __syncthreads();
    return n;
}

// Part `part` of a sequence, from its first token on (from its last, BACK); true if
// tokens of the sequence lie before it.
template <bool BACK>
__device__ __forceinline__ bool cut(const Shape &s, int part, long long &bos, long long &len) {
    const long long per = ((len + s.parts - 1) / s.parts + 127) / 128 * 128, off = min(part * per, len);
    const long long mine = min(per, len - off), before = BACK ? len - off - mine : off;
    bos += before;
    len = mine;
    return before > 0;
}

// Pairs (A and B of two channels) of a tile's warps, and of a round's tiles in the
// cluster.  Two of each: a tile's are written while the one before it may still be read.
template <int W>
struct Pairs {
    float4 warp[2][W][32];
    float4 tile[2][kMaxCluster][32];
    uint64_t got[2];           // one phase a round: the pairs of every CTA have come
};

// 16 bytes into another CTA's shared memory, counted by that CTA's barrier.
__device__ __forceinline__ void send(uint32_t addr, uint32_t bar, float4 v) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(addr),
        "r"(bar), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
        : "memory");
}

// The pair of a warp's tokens joins the others' in two halves, so that other work fits
// between them.  offer() leaves it where the tile's, or the cluster's, warps find it;
// take() turns the value before the round's first tile (carry) into the value before
// this warp's first token, and carry into the value after the round.
//
// The pairs of a cluster travel by st.async, each counted by the receiver's barrier,
// and no CTA waits for more than them.  (The cluster's own barrier, whose release
// also waits for the results stored to global memory before it, made a round of
// 65536 x 2048 tokens by 8 CTAs 3.5 us long instead of 2.5.)  A CTA can be two rounds
// ahead of none: its pair of the next round is what lets the others go on.
template <int W>
struct Join {
    Pairs<W> &p;
    int warp, lane, rank, size;
    const Shape &s;
    float2 A, B;               // of the tile's warps before this one (clusters only)
    bool alive;                // no wait for pairs gave up
    float2 product;            // of every decay so far (single CTAs only)

    // Past its barrier every warp of the CTA is done with the tile before.
    __device__ __forceinline__ void offer(int round, float2 a, float2 b) {
        const int buf = round & 1;
        p.warp[buf][warp][lane] = make_float4(a.x, a.y, b.x, b.y);
        __syncthreads();
        if (size == 1) return;
        if (!alive) return;
        if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(&p.got[buf], (uint32_t)size * 512u);
        float2 allA = both(1.f), allB = both(0.f);
        A = allA, B = allB;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == warp) A = allA, B = allB;
            const float4 q = p.warp[buf][w][lane];
            allA = mul2(allA, make_float2(q.x, q.y));
            allB = fma2(make_float2(q.x, q.y), allB, make_float2(q.z, q.w));
        }
        for (int to = warp; to < size; to += W)      // the warps share the receivers out
            send(tc::map_rank(tc::smem_u32(&p.tile[buf][rank][lane]), to),
                 tc::map_rank(tc::smem_u32(&p.got[buf]), to), make_float4(allA.x, allA.y, allB.x, allB.y));
    }
    __device__ __forceinline__ float2 take(int round, float2 &carry) {
        const int buf = round & 1;
        float2 before = carry;
        if (size == 1) {
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w == warp) before = carry;
                const float4 q = p.warp[buf][w][lane];
                carry = fma2(make_float2(q.x, q.y), carry, make_float2(q.z, q.w));
                product = mul2(product, make_float2(q.x, q.y));
            }
            return before;
        }
        // a limit of its own: the pairs come whether or not a wait for tiles gave up.  If
        // they do not, nothing more is counted or sent, and the others stop a round later.
        if (alive) alive = tc::mbar_wait(&p.got[buf], (round >> 1) & 1, 1ll << 22, s.status);
        for (int k = 0; k < size; ++k) {
            if (k == rank) before = carry;
            const float4 q = p.tile[buf][k][lane];
            carry = fma2(make_float2(q.x, q.y), carry, make_float2(q.z, q.w));
        }
        return fma2(A, before, B);
    }
};

// Where a lane's channels are, and which of the two exist.
struct Place {
    int warp, lane, rank, size, cluster, ch;
    int from;                  // ch, or of a lane that has none the last channel there is
    bool in0, in1;
};
__device__ __forceinline__ Place place(const Shape &s) {
    Place p;
    p.warp = threadIdx.x >> 5, p.lane = threadIdx.x & 31;
    p.rank = (int)tc::cluster_rank(), p.size = (int)tc::cluster_size();
    p.cluster = blockIdx.x / p.size;
    p.ch = p.cluster % s.groups * kChannels + 2 * p.lane;
    p.in0 = p.ch < s.D, p.in1 = p.ch + 1 < s.D;
    p.from = min(p.ch, s.D - 1);
    return p;
}
__device__ __forceinline__ float2 load_state(const float *base, long long at, const Place &p) {
    return make_float2(base && p.in0 ? base[at] : 0.f, base && p.in1 ? base[at + 1] : 0.f);
}
__device__ __forceinline__ void store_state(float *base, long long at, const Place &p, float2 v) {
    if (p.in0) base[at] = v.x;
    if (p.in1) base[at + 1] = v.y;
}

__device__ __forceinline__ void store_pair(float2 *base, long long at, const Place &p, float2 A, float2 B) {
    if (p.in0) base[at] = make_float2(A.x, B.x);
    if (p.in1) base[at + 1] = make_float2(A.y, B.y);
}

// Two elements at p, which may be on no 4- or 8-byte boundary (PAIRS false) and of
// which the second may not exist.
template <typename T, bool PAIRS>
__device__ __forceinline__ float2 load2(const T *p, const Place &at) {
    if (PAIRS) return get2(*reinterpret_cast<const typename Raw2<T>::type *>(p));
    return make_float2(to_f(p[0]), at.in1 ? to_f(p[1]) : 0.f);
}
template <typename T, bool PAIRS>
__device__ __forceinline__ void store2(T *p, const Place &at, float2 v) {
    if (PAIRS) {
        *reinterpret_cast<typename Raw2<T>::type *>(p) = put2(v, (const T *)nullptr);
    } else {
        from_f(p, v.x);
        if (at.in1) from_f(p + 1, v.y);
    }
}

// A ring of stages, each a tile of every input: rows of kChannels elements.  TMA
// fills stage i % S with tile i; the barrier in Join::offer() is what frees a stage, so one
// thread keeps the ring S - 1 tiles ahead without further waiting.
template <typename T, int W, int R, int INPUTS, int STAGES>
struct Ring {
    static constexpr int kTile = W * R;
    T tile[STAGES][INPUTS][kTile][kChannels];
    Pairs<W> pairs;
    uint64_t full[STAGES];
};

struct FwdArgs {
    const void *x, *g;
    const float *scale, *h0;
    void *h;
    float *ht;
};

// Forward over TMA tiles (TMA true), or with plain loads for widths whose rows do not
// start on 16 bytes.
template <typename T, bool GATED, int W, int R, int STAGES, bool TMA>
__global__ void __launch_bounds__(32 * W, TMA ? 1 : 3) fwd_kernel(const __grid_constant__ CUtensorMap map_x,
                                                       const __grid_constant__ CUtensorMap map_g,
                                                       const FwdArgs a, const Shape s) {
    using Ring = linrec::Ring<T, W, R, 2, STAGES>;
    constexpr int kTile = Ring::kTile;
    constexpr uint32_t kBytes = 2u * kTile * kChannels * sizeof(T);
    extern __shared__ __align__(128) uint8_t raw[];
    Ring &ring = *reinterpret_cast<Ring *>(raw);
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(&ring.full[i], 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(&ring.pairs.got[i], 1);
        tc::fence_barrier_init();
    }
    __syncthreads();
    pdl_enter();

    const Place at = place(s);
    const int ch0 = at.ch - 2 * at.lane;
    const float2 sc = GATED ? load_state(a.scale, at.ch, at) : both(0.f);
    if (at.size > 1) tc::cluster_sync();     // the others' barriers are ready

    Join<W> join{ring.pairs, at.warp, at.lane, at.rank, at.size, s, both(1.f), both(0.f), true, both(1.f)};
    bool ok = true;                // no wait gave up
    int tiles = 0, issued = 0;     // tiles walked and asked for, over all sequences
    for (int unit = sequence_of(s, at.cluster / s.groups, &ring.pairs); unit < s.N * s.parts; unit += s.lanes_n) {
        const int n = unit / s.parts;
        long long bos, len;
        range(s, n, bos, len);
        if (s.parts > 1) cut<false>(s, unit - n * s.parts, bos, len);
        const long long step = (long long)at.size * kTile, state = (long long)n * s.D + at.ch;
        const long long part = (long long)unit * s.D + at.ch;
        float2 carry = both(0.f);
        if (!s.reduce) carry = s.parts > 1 ? load_state(s.start, part, at) : load_state(a.h0, state, at);
        join.product = both(1.f);
        const int base = tiles;
        const int rounds = (int)((len + step - 1) / step);
        auto ask = [&](int round) {          // thread 0: tile `round` of this sequence
            const int st = (base + round) % STAGES;
            const int row = (int)(bos + round * step + at.rank * kTile);
            tc::mbar_arrive_expect_tx(&ring.full[st], kBytes);
            tc::tma_load_2d(&ring.tile[st][0], &map_x, &ring.full[st], ch0, row);
            tc::tma_load_2d(&ring.tile[st][1], &map_g, &ring.full[st], ch0, row);
            ++issued;
        };
        if (TMA && threadIdx.x == 0)
            for (int i = 0; i < STAGES - 1 && i < rounds && ok; ++i) ask(i);
        auto token = [&](int i) { return i * step + at.rank * kTile + at.warp * R; };
        // tokens this warp has of tile i, the same for lanes past the last channel, which walk
        // TMA's zeros or the last channel: in two branches a warp would take twice as long
        auto rows_of = [&](int i) { return ok ? (int)max(0ll, min((long long)R, len - token(i))) : 0; };
        auto cell = [&](int i, int input, int r) {
            return get2(*reinterpret_cast<const typename Raw2<T>::type *>(
                &ring.tile[(base + i) % STAGES][input][at.warp * R + r][2 * at.lane]));
        };
        // tile i: its decays and its pair
        auto scan = [&](int i, float2 (&al)[R], float2 (&xv)[TMA ? 1 : R], float2 &A, float2 &B) {
            if (TMA && ok)
                ok = tc::mbar_wait(&ring.full[(base + i) % STAGES], ((base + i) / STAGES) & 1, s.spin_limit, s.status);
            const int rows = rows_of(i);
            auto go = [&](auto whole) {
                if constexpr (!TMA) {
                    const long long row0 = (bos + token(i)) * s.D + at.from;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const bool in = whole.value || r < rows;
                        xv[r] = in ? load2<T, false>(reinterpret_cast<const T *>(a.x) + row0 + (long long)r * s.D, at) : both(0.f);
                        al[r] = in ? load2<T, false>(reinterpret_cast<const T *>(a.g) + row0 + (long long)r * s.D, at) : both(0.f);
                    }
                }
                A = both(1.f), B = both(0.f);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 g = TMA ? cell(i, 1, r) : al[r];
                    float2 x = TMA ? cell(i, 0, r) : xv[TMA ? 0 : r];
                    float2 sp;
                    al[r] = Gate<T, GATED>::decay(g, sc, sp);
                    if (!whole.value && r >= rows) al[r] = both(1.f), x = both(0.f);
                    A = mul2(A, al[r]);
                    B = fma2(al[r], B, x);
                }
            };
            if (rows == R) go(std::true_type());
            else go(std::false_type());
        };
        // tile i's results from the value before this warp's first token
        auto emit = [&](int i, const float2 (&al)[R], const float2 (&xv)[TMA ? 1 : R], float2 h) {
            const int rows = at.in0 ? rows_of(i) : 0;
            auto go = [&](auto whole) {
                T *out = reinterpret_cast<T *>(a.h) + (bos + token(i)) * s.D + at.ch;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    h = fma2(al[r], h, TMA ? cell(i, 0, r) : xv[TMA ? 0 : r]);
                    if (whole.value || r < rows) store2<T, TMA>(out, at, h);
                    out += s.D;
                }
            };
            if (rows == R) go(std::true_type());
            else if (rows > 0) go(std::false_type());
        };
        auto refill = [&](int i) {           // after offer(i): the stage of tile i - 1 is free
            if (TMA && threadIdx.x == 0 && ok && i + STAGES - 1 < rounds) ask(i + STAGES - 1);
        };
        for (int i = 0; i < rounds; ++i) {
            float2 al[R], xv[TMA ? 1 : R], A, B;
            scan(i, al, xv, A, B);
            join.offer(base + i, A, B);
            refill(i);
            const float2 before = join.take(base + i, carry);
            if (!s.reduce) emit(i, al, xv, before);
        }
        tiles += rounds;
        // the next sequence's first tiles go into stages that this one's last are read from
        __syncthreads();
        if (at.rank == 0 && at.warp == 0) {
            if (s.reduce) store_pair(s.pair, part, at, join.product, carry);
            else if (a.ht && s.parts == 1) store_state(a.ht, state, at, carry);
        }
    }
    if (at.size > 1) tc::cluster_sync();     // nor does a CTA go before the others are done
    if (TMA && threadIdx.x == 0 && !ok)      // nothing may land after the CTA has gone
        for (int i = max(0, issued - STAGES); i < issued; ++i)
            tc::mbar_drain(&ring.full[i % STAGES], (i / STAGES) & 1);
}

struct BwdArgs {
    const void *dh, *g, *h;
    const float *scale, *h0, *dht;
    void *dx, *dg;
    float *dh0, *partial;      // partial: [lanes_n * cluster][D], or null
};

// The same walk from the last token to the first: with e_t = dh_t + c_t, a token's
// map on the carried gradient is c -> a (dh + c), the pair (a, a dh).  Row u of the
// walk is token len - 1 - u, so a tile's rows lie in shared memory from its last to
// its first; the tile of h is one token earlier than the others.
template <typename T, bool GATED, int W, int R, int STAGES, bool TMA>
__global__ void __launch_bounds__(32 * W, TMA ? 1 : 2) bwd_kernel(const __grid_constant__ CUtensorMap map_dh,
                                                       const __grid_constant__ CUtensorMap map_g,
                                                       const __grid_constant__ CUtensorMap map_h,
                                                       const BwdArgs a, const Shape s) {
    using Ring = linrec::Ring<T, W, R, 3, STAGES>;
    constexpr int kTile = Ring::kTile;
    constexpr uint32_t kBytes = 3u * kTile * kChannels * sizeof(T);
    extern __shared__ __align__(128) uint8_t raw[];
    Ring &ring = *reinterpret_cast<Ring *>(raw);
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(&ring.full[i], 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(&ring.pairs.got[i], 1);
        tc::fence_barrier_init();
    }
    __syncthreads();
    pdl_enter();

    const Place at = place(s);
    const int ch0 = at.ch - 2 * at.lane;
    const float2 sc = GATED ? load_state(a.scale, at.ch, at) : both(0.f);
    const float2 minus = make_float2(-sc.x, -sc.y);
    float2 dscale = both(0.f);
    if (at.size > 1) tc::cluster_sync();     // the others' barriers are ready

    Join<W> join{ring.pairs, at.warp, at.lane, at.rank, at.size, s, both(1.f), both(0.f), true, both(1.f)};
    bool ok = true;
    int tiles = 0, issued = 0;
    const uint32_t bytes = s.reduce ? kBytes / 3 * 2 : kBytes;       // a pair needs no h
    for (int unit = sequence_of(s, at.cluster / s.groups, &ring.pairs); unit < s.N * s.parts; unit += s.lanes_n) {
        const int n = unit / s.parts;
        long long bos, len;
        range(s, n, bos, len);
        const bool lead = s.parts > 1 && cut<true>(s, unit - n * s.parts, bos, len);
        const long long step = (long long)at.size * kTile, state = (long long)n * s.D + at.ch;
        const long long part = (long long)unit * s.D + at.ch;
        float2 carry = both(0.f);
        if (!s.reduce) carry = s.parts > 1 ? load_state(s.start, part, at) : load_state(a.dht, state, at);
        join.product = both(1.f);
        const float2 h0 = load_state(a.h0, state, at);
        const int base = tiles;
        const int rounds = (int)((len + step - 1) / step);
        auto ask = [&](int round) {
            const int st = (base + round) % STAGES;
            const int row = (int)(bos + len - kTile - (round * step + at.rank * kTile));
            tc::mbar_arrive_expect_tx(&ring.full[st], bytes);
            tc::tma_load_2d(&ring.tile[st][0], &map_dh, &ring.full[st], ch0, row);
            tc::tma_load_2d(&ring.tile[st][1], &map_g, &ring.full[st], ch0, row);
            if (!s.reduce) tc::tma_load_2d(&ring.tile[st][2], &map_h, &ring.full[st], ch0, row - 1);
            ++issued;
        };
        if (TMA && threadIdx.x == 0)
            for (int i = 0; i < STAGES - 1 && i < rounds && ok; ++i) ask(i);
        for (int i = 0; i < rounds; ++i, ++tiles) {
            const int st = tiles % STAGES;
            const long long u = i * step + at.rank * kTile + at.warp * R, top = len - 1 - u;
            int rows = (int)max(0ll, min((long long)R, len - u));
            if (TMA) {
                if (ok) ok = tc::mbar_wait(&ring.full[st], (tiles / STAGES) & 1, s.spin_limit, s.status);
                if (!ok) rows = 0;
            }
            // row r of the walk: r rows back from the tile's row kTile - 1 - warp * R
            auto cell = [&](int input, int r) {
                return get2(*reinterpret_cast<const typename Raw2<T>::type *>(
                    &ring.tile[st][input][kTile - 1 - at.warp * R - r][2 * at.lane]));
            };
            const long long row0 = (bos + top) * s.D + at.ch;
            const long long from = row0 - at.ch + at.from;
            const T *gd = reinterpret_cast<const T *>(a.dh) + from, *gg = reinterpret_cast<const T *>(a.g) + from;
            const T *gh = reinterpret_cast<const T *>(a.h) + from;
            float2 al[R], sp[GATED ? R : 1], dv[TMA ? 1 : R], gv[TMA ? 1 : R], hv[TMA ? 1 : R];
            float2 A = both(1.f), B = both(0.f);
            auto first = [&](auto whole) {
                if constexpr (!TMA) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const bool in = whole.value || r < rows;
                        const long long off = (long long)r * s.D;
                        dv[r] = in ? load2<T, false>(gd - off, at) : both(0.f);
                        gv[r] = in ? load2<T, false>(gg - off, at) : both(0.f);
                        hv[r] = in && !s.reduce && (lead || r < top) ? load2<T, false>(gh - off - s.D, at) : both(0.f);
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float2 d = TMA ? cell(0, r) : dv[TMA ? 0 : r];
                    al[r] = Gate<T, GATED>::decay(TMA ? cell(1, r) : gv[TMA ? 0 : r], sc, sp[GATED ? r : 0]);
                    if (!whole.value && r >= rows) al[r] = both(1.f), d = both(0.f);
                    A = mul2(A, al[r]);
                    B = mul2(al[r], add2(B, d));
                }
            };
            if (rows == R) first(std::true_type());
            else first(std::false_type());
            join.offer(tiles, A, B);
            if (TMA && threadIdx.x == 0 && ok && i + STAGES - 1 < rounds) ask(i + STAGES - 1);
            float2 c = join.take(tiles, carry);
            auto second = [&](auto whole) {
                T *dx = reinterpret_cast<T *>(a.dx) + row0, *dg = reinterpret_cast<T *>(a.dg) + row0;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float2 hp = TMA ? cell(2, r) : hv[TMA ? 0 : r];
                    if (!whole.value && !lead && r == top) hp = h0;     // before the first token is h0
                    const float2 e = add2(TMA ? cell(0, r) : dv[TMA ? 0 : r], c);
                    c = mul2(al[r], e);
                    float2 dl = mul2(c, hp);
                    if (whole.value || r < rows) {
                        if (GATED) {
                            // softplus finite even for an infinite gate, whose decay of 0 is in dl
                            const float2 q = sp[GATED ? r : 0];
                            dscale = fma2(dl, make_float2(bounded(q.x), bounded(q.y)), dscale);
                            dl = mul2(mul2(dl, minus), Gate<T, GATED>::slope(TMA ? cell(1, r) : gv[TMA ? 0 : r], q));
                        }
                        store2<T, TMA>(dx, at, e);
                        store2<T, TMA>(dg, at, dl);
                    }
                    dx -= s.D, dg -= s.D;
                }
            };
            if (s.reduce) continue;
            const int mine = at.in0 ? rows : 0;
            if (mine == R && (lead || top >= R)) second(std::true_type());
            else if (mine > 0) second(std::false_type());
        }
        __syncthreads();
        if (at.rank == 0 && at.warp == 0) {
            if (s.reduce) store_pair(s.pair, part, at, join.product, carry);
            else if (a.dh0 && s.parts == 1) store_state(a.dh0, state, at, carry);
        }
    }
    if (at.size > 1) tc::cluster_sync();
    if (TMA && threadIdx.x == 0 && !ok)
        for (int i = max(0, issued - STAGES); i < issued; ++i)
            tc::mbar_drain(&ring.full[i % STAGES], (i / STAGES) & 1);
    if (GATED && a.partial && !s.reduce) {   // the CTA's sum, its warps in order
        float2 *sum = reinterpret_cast<float2 *>(ring.pairs.warp);
        sum[at.warp * 32 + at.lane] = mul2(dscale, both(-Gate<T, GATED>::kUnit));
        __syncthreads();
        if (at.warp == 0) {
            float2 t = both(0.f);
            for (int w = 0; w < W; ++w) t = add2(t, sum[w * 32 + at.lane]);
            store_state(a.partial, ((long long)(at.cluster / s.groups) * at.size + at.rank) * s.D + at.ch, at, t);
        }
    }
}

// The parts' pairs joined: the value before each part, and after the last one.  A channel's
// parts are shared out over the 32 warps of a block, which first meet with the pairs of
// theirs: one thread for all of a channel's parts took 0.14 us for each.
__global__ void __launch_bounds__(1024) parts_kernel(const float2 *pair, float *start, const float *init,
                                                     float *final, int N, int parts, int D) {
    __shared__ float2 all[32][33];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long i = blockIdx.x * 32ll + lane;
    const bool in = i < (long long)N * D;
    const long long n = i / D, ch = i - n * D, at = n * parts * D + ch;
    const int per = (parts + 31) / 32, first = warp * per, end = in ? min(first + per, parts) : 0;
    float2 q = make_float2(1.f, 0.f);
#pragma unroll 8
    for (int k = first; k < end; ++k) {
        const float2 r = pair[at + (long long)k * D];
        q = make_float2(r.x * q.x, r.x * q.y + r.y);
    }
    all[warp][lane] = q;
    __syncthreads();
    float v = in && init ? init[i] : 0.f;
    for (int w = 0; w < warp; ++w) v = all[w][lane].x * v + all[w][lane].y;
#pragma unroll 8
    for (int k = first; k < end; ++k) {
        const float2 r = pair[at + (long long)k * D];
        start[at + (long long)k * D] = v;
        v = r.x * v + r.y;
    }
    if (in && final && warp == 31) final[i] = v;
}

// One token: VEC neighbouring channels to a thread, which takes the same ones of every
// gridDim.y-th group of blockDim.y sequences.
template <typename T, int VEC>
struct Few;
template <>
struct Few<__nv_bfloat16, 4> {
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float *v) {
        const uint2 r = *reinterpret_cast<const uint2 *>(p);
        const float2 a = get2(r.x), b = get2(r.y);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(put2(make_float2(v[0], v[1]), p), put2(make_float2(v[2], v[3]), p));
    }
};
template <>
struct Few<float, 4> {
    static __device__ __forceinline__ void load(const float *p, float *v) {
        const float4 r = *reinterpret_cast<const float4 *>(p);
        v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
    }
    static __device__ __forceinline__ void store(float *p, const float *v) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <typename T>
struct Few<T, 1> {
    static __device__ __forceinline__ void load(const T *p, float *v) { v[0] = to_f(*p); }
    static __device__ __forceinline__ void store(T *p, const float *v) { from_f(p, v[0]); }
};

template <typename T, bool GATED, int VEC>
__global__ void __launch_bounds__(256) step_kernel(const T *x, const T *g, const float *scale,
                                                   const float *state, T *h, float *out, int N, int D) {
    pdl_enter();
    const int ch = (blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (ch >= D) return;
    float s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[j] = 0.f;
    if (GATED) Few<float, VEC>::load(scale + ch, s);
    for (int n = blockIdx.y * blockDim.y + threadIdx.y; n < N; n += gridDim.y * blockDim.y) {
        const long long at = (long long)n * D + ch;
        float xv[VEC], gv[VEC], v[VEC];
        Few<T, VEC>::load(x + at, xv);
        Few<T, VEC>::load(g + at, gv);
        Few<float, VEC>::load(state + at, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float sp;
            v[j] = Gate<float, GATED>::decay(gv[j], s[j], sp) * v[j] + xv[j];
        }
        Few<float, VEC>::store(out + at, v);
        Few<T, VEC>::store(h + at, v);
    }
}

template <typename T, bool GATED>
cudaError_t run_step(const gdn_linrec_step_args *a, int sms, cudaStream_t q) {
    // rows that start on 16 bytes are read by fours
    const int vec = a->D % 4 == 0 ? 4 : 1, chunks = a->D / vec;
    int wide = 1;
    while (wide < 256 && wide < chunks) wide *= 2;
    const dim3 block(wide, 256 / wide);
    const int across = (chunks + wide - 1) / wide;
    const int down = (int)std::min<long long>((a->N + block.y - 1) / block.y, std::max(1, 16 * sms / across));
    return launch_pdl(vec == 4 ? step_kernel<T, GATED, 4> : step_kernel<T, GATED, 1>, dim3(across, down), block, 0, q,
                      (const T *)a->x, (const T *)a->g, a->gate_scale, a->state, (T *)a->h, a->out_state, a->N, a->D);
}

// Clusters that share a channel group's sequences: one each, but no more than fill
// the GPU several times over, so that the per-CTA partial sums of d(gate_scale)
// stay small beside the data.
int group_lanes(int N, int groups) {
    const int most = std::max(1, 4096 / groups);
    return std::min(N, std::max(most, 64));
}

// Warps, tokens to a warp and stages: about 100 KB of tiles to a CTA, two CTAs to an SM.
// Every warp reads every warp's pair, so that few warps with many tokens each do best:
// forward, 65536 x 2048 gated bf16, 8 warps of 16 tokens 198 us, 4 of 32 160 us, 16 of 8
// 437 us; backward, 4 x 4096 x 4096, 8 of 8 130 us, 4 of 16 119 us, 6 of 10 132 us.
template <typename T>
struct Tiles {
    static constexpr bool kHalf = sizeof(T) == 2;
    static constexpr int kFwdWarps = 4, kFwdRows = kHalf ? 32 : 16, kFwdStages = 3;
    static constexpr int kBwdWarps = 4, kBwdRows = kHalf ? 16 : 8, kBwdStages = 4;
};

// CTAs that share a sequence: doubled while the grid leaves slots of the GPU (two
// CTAs per SM) empty and the sequences have a tile for each; of a packed batch, whose
// longest sequence may be the last to end, up to twice that (us of 16 x (512 .. 8192) tokens
// x 1000 gated bf16 forward, backward: 124, 202 in single CTAs, 81, 129 in pairs, 89, 139 in
// fours; 16 x 4096 tokens each 77, 121 in single CTAs, 86, 136 in pairs).  Clusters of c leave about c SMs without
// one (74 of 4 fit, 36 of 8), and one cluster too many takes a second wave: 2 x 8192 x 2432
// fp32 146 us in 76 clusters of 4, 130 in as many of 2.
int cluster_of(long long clusters, long long mean_len, bool packed) {
    int c = 1;
    while (c < kMaxCluster && clusters * c <= (packed ? 2 : 1) * (kSms - 2 * c) && mean_len > (long long)c * 128) c *= 2;
    return c;
}

// What the choice between clusters and parts goes by.
struct Kind {
    bool fp32, gated, back, tma;
};

// Parts of a sequence, or 1: as many as fill the GPU with a CTA each, of 128 tokens at
// least, where two walks of them and the two more launches (5 us) take less than the
// cluster's rounds, each of which is 1.6 times a tile of 128 tokens long.  The walks read twice, at
// 7 TB/s in all.  Us in clusters | parts: 4096 x 64 gated bf16
// forward 9.9 | 9.5, backward 16.3 | 12.4; 16384 x 64 31 | 12, 51 | 15, in fp32 67 | 17, 141 |
// 24; 65536 x 1024 157 | 119, 260 | 173; but fp32 and not gated 186 | 204, 312 | 293.
int parts_of(long long clusters, int cluster, long long mean_len, const Kind &k, double bytes) {
    if (cluster < 4) return 1;
    const long long parts = std::min(2 * kSms / clusters, mean_len / 128);
    if (parts < 2) return 1;
    const double tile = (k.fp32 ? (k.gated ? 3.3 : 1.8) : k.tma ? 1.2 : 2.2) * (k.back ? 1.6 : 1.0);
    const long long rounds = (mean_len + 128 * cluster - 1) / (128 * cluster);
    const long long tiles = 2 * ((mean_len + 128 * parts - 1) / (128 * parts));
    const double walks = std::max((double)tiles * tile, bytes * (k.back ? 7 : 5) / 7e6);
    return walks + 5 < (double)rounds * 1.6 * tile ? (int)parts : 1;
}

gdn_status check(int B, int T, int D, int N, int dtype, bool packed) {
    if (B < 1 || T < 0 || D < 1) return fail(GDN_ERR_INVALID_ARG, "bad sizes B=%d T=%d D=%d", B, T, D);
    if (dtype != GDN_FP32 && dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_FP32 or GDN_BF16", dtype);
    if (packed && (B != 1 || N < 1))
        return fail(GDN_ERR_INVALID_ARG, "cu_seqlens needs B == 1 and N >= 1 (B=%d N=%d)", B, N);
    if ((long long)B * T >= (1ll << 31) - (1 << 16) || D > (1 << 24) || (long long)(packed ? N : B) * D >= (1ll << 40))
        return fail(GDN_ERR_INVALID_ARG, "problem too large");
    return GDN_OK;
}

// Rows that start on 16 bytes, as TMA wants them.
bool tma_rows(int dtype, int D) { return D % (dtype == GDN_BF16 ? 8 : 4) == 0; }

Shape shape_of(const int32_t *cu, int B, int T, int D, int N, const Kind &kind) {
    Shape s = {};
    s.cu = cu;
    s.T = T;
    s.N = cu ? N : B;
    s.D = D;
    s.groups = (D + kChannels - 1) / kChannels;
    const long long mean = cu ? T / s.N : T;
    s.lanes_n = group_lanes(s.N, s.groups);
    s.cluster = cluster_of((long long)s.groups * s.lanes_n, mean, cu != nullptr);
    s.parts = parts_of((long long)s.groups * s.lanes_n, s.cluster, mean, kind,
                       (double)(cu ? T : (long long)T * s.N) * D * (kind.fp32 ? 4 : 2));
    if (s.parts > 1) {
        s.cluster = 1;
        s.lanes_n = group_lanes(s.N * s.parts, s.groups);
    }
    s.longest_first = cu && s.parts == 1 && s.lanes_n == s.N && s.N <= kMaxOrdered &&
                      (long long)s.groups * s.N * s.cluster > 2 * kSms;
    return s;
}

// Workspace of the parts' pairs and starting values.
size_t parts_bytes(const Shape &s) { return s.parts > 1 ? (size_t)s.N * s.parts * s.D * 12 : 0; }
void place_parts(Shape &s, void *ws) {
    s.pair = (float2 *)ws;
    s.start = (float *)(s.pair + (size_t)s.N * s.parts * s.D);
}

template <typename... KArgs, typename... Args>
cudaError_t launch(const char *name, void (*kernel)(KArgs...), int warps, size_t smem, const Shape &s, cudaStream_t st,
                   const Args &...args) {
    cudaError_t e = allow_smem((const void *)kernel, smem);
    if (e != cudaSuccess) return e;
    prof_before(name, st);
    e = launch_pdl_cluster(kernel, dim3((unsigned)((long long)s.groups * s.lanes_n * s.cluster)), dim3(32 * warps),
                           smem, s.cluster, st, args..., s);
    prof_after(st);
    return e;
}

// [tokens, D] of T, boxes of kChannels channels x `rows` tokens (an empty tensor's map
// is never used).
template <typename T>
cudaError_t map_of(CUtensorMap *m, const void *base, const Shape &s, int rows) {
    const long long tokens = s.cu ? s.T : s.T * s.N;
    return tokens == 0 ? cudaSuccess : tc::make_map_rows(m, base, tokens, s.D, sizeof(T), kChannels, rows);
}

// A walk, or with parts the walk for their pairs, their joining and the walk for the results.
template <typename Walk>
cudaError_t in_parts(Shape s, const float *init, float *final, cudaStream_t q, Walk walk) {
    if (s.parts == 1) return walk(s);
    s.reduce = 1;
    cudaError_t e = walk(s);
    if (e != cudaSuccess) return e;
    prof_before("linrec_parts", q);
    e = launch_pdl(parts_kernel, dim3((unsigned)(((long long)s.N * s.D + 31) / 32)), dim3(1024), 0, q,
                   (const float2 *)s.pair, s.start, init, final, s.N, s.parts, s.D);
    prof_after(q);
    if (e != cudaSuccess) return e;
    s.reduce = 0;
    return walk(s);
}

template <typename T, bool GATED>
cudaError_t run_fwd(const FwdArgs &f, const Shape &s, bool tma, cudaStream_t q) {
    constexpr int W = Tiles<T>::kFwdWarps, R = Tiles<T>::kFwdRows, S = Tiles<T>::kFwdStages;
    CUtensorMap mx = {}, mg = {};
    if (!tma)
        return in_parts(s, f.h0, f.ht, q, [&](const Shape &w) {
            return launch("linrec_fwd_plain", fwd_kernel<T, GATED, 8, 8, 1, false>, 8, sizeof(Ring<T, 8, 8, 2, 1>),
                          w, q, mx, mg, f);
        });
    cudaError_t e = tc::encoder();
    if (e == cudaSuccess) e = map_of<T>(&mx, f.x, s, W * R);
    if (e == cudaSuccess) e = map_of<T>(&mg, f.g, s, W * R);
    if (e != cudaSuccess) return e;
    return in_parts(s, f.h0, f.ht, q, [&](const Shape &w) {
        return launch("linrec_fwd", fwd_kernel<T, GATED, W, R, S, true>, W, sizeof(Ring<T, W, R, 2, S>), w, q, mx, mg, f);
    });
}

template <typename T, bool GATED>
cudaError_t run_bwd(const BwdArgs &b, const Shape &s, bool tma, cudaStream_t q) {
    constexpr int W = Tiles<T>::kBwdWarps, R = Tiles<T>::kBwdRows, S = Tiles<T>::kBwdStages;
    CUtensorMap md = {}, mg = {}, mh = {};
    if (!tma)
        return in_parts(s, b.dht, b.dh0, q, [&](const Shape &w) {
            return launch("linrec_bwd_plain", bwd_kernel<T, GATED, 8, 8, 1, false>, 8, sizeof(Ring<T, 8, 8, 3, 1>),
                          w, q, md, mg, mh, b);
        });
    cudaError_t e = tc::encoder();
    if (e == cudaSuccess) e = map_of<T>(&md, b.dh, s, W * R);
    if (e == cudaSuccess) e = map_of<T>(&mg, b.g, s, W * R);
    if (e == cudaSuccess) e = map_of<T>(&mh, b.h, s, W * R);
    if (e != cudaSuccess) return e;
    return in_parts(s, b.dht, b.dh0, q, [&](const Shape &w) {
        return launch("linrec_bwd", bwd_kernel<T, GATED, W, R, S, true>, W, sizeof(Ring<T, W, R, 3, S>), w, q,
                      md, mg, mh, b);
    });
}

// The answer to a workspace query: 256 stands for none.
size_t asked_for(size_t need) { return need == 0 ? 256 : std::max<size_t>(512, need); }

Shape shape_of(const gdn_linrec_fwd_args *a) {
    return shape_of(a->cu_seqlens, a->B, a->T, a->D, a->N,
                    {a->dtype == GDN_FP32, a->gate_scale != nullptr, false, tma_rows(a->dtype, a->D)});
}
Shape shape_of(const gdn_linrec_bwd_args *a) {
    return shape_of(a->cu_seqlens, a->B, a->T, a->D, a->N,
                    {a->dtype == GDN_FP32, a->gate_scale != nullptr, true, tma_rows(a->dtype, a->D)});
}

// Workspace: parts, then a row of d(gate_scale) for each CTA of a channel group.
size_t fwd_workspace(const gdn_linrec_fwd_args *a) {
    return parts_bytes(shape_of(a));
}
size_t bwd_workspace(const gdn_linrec_bwd_args *a) {
    const Shape s = shape_of(a);
    const bool sums = a->gate_scale && a->d_gate_scale;
    return parts_bytes(s) + (sums ? (size_t)s.lanes_n * s.cluster * s.D * sizeof(float) : 0);
}

}  // namespace
}  // namespace linrec
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_linrec_fwd_workspace_size(const gdn_linrec_fwd_args *a) {
    if (!a) {
        fail(GDN_ERR_INVALID_ARG, "null args");
        return 0;
    }
    if (linrec::check(a->B, a->T, a->D, a->N, a->dtype, a->cu_seqlens != nullptr) != GDN_OK) return 0;
    return linrec::asked_for(linrec::fwd_workspace(a));
}

gdn_status gdn_linrec_fwd(const gdn_linrec_fwd_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = linrec::check(a->B, a->T, a->D, a->N, a->dtype, a->cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (a->T > 0 && (!a->x || !a->g || !a->h))
        return fail(GDN_ERR_INVALID_ARG, "x, g and h are required");
    if (misaligned(a->x) || misaligned(a->g) || misaligned(a->h) || misaligned(a->gate_scale) ||
        misaligned(a->initial_state) || misaligned(a->cu_seqlens) || misaligned(a->final_state))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    const size_t need = linrec::fwd_workspace(a);
    if (need > 0 && (!ws || misaligned(ws) || ws_bytes < need))
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    linrec::Shape s = linrec::shape_of(a);
    s.status = dev.status;
    s.spin_limit = dev.spin_limit;
    linrec::place_parts(s, ws);
    const bool tma = linrec::tma_rows(a->dtype, a->D), bf = a->dtype == GDN_BF16;
    const bool gated = a->gate_scale != nullptr;
    const linrec::FwdArgs f{a->x, a->g, a->gate_scale, a->initial_state, a->h, a->final_state};
    cudaStream_t q = (cudaStream_t)stream;
    const cudaError_t e = bf ? (gated ? linrec::run_fwd<__nv_bfloat16, true>(f, s, tma, q)
                                      : linrec::run_fwd<__nv_bfloat16, false>(f, s, tma, q))
                             : (gated ? linrec::run_fwd<float, true>(f, s, tma, q)
                                      : linrec::run_fwd<float, false>(f, s, tma, q));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "linear recurrence launch");
}

size_t gdn_linrec_bwd_workspace_size(const gdn_linrec_bwd_args *a) {
    if (!a) {
        fail(GDN_ERR_INVALID_ARG, "null args");
        return 0;
    }
    if (linrec::check(a->B, a->T, a->D, a->N, a->dtype, a->cu_seqlens != nullptr) != GDN_OK) return 0;
    return linrec::asked_for(linrec::bwd_workspace(a));
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
    const size_t need = linrec::bwd_workspace(a);
    if (need > 0 && (!ws || misaligned(ws) || ws_bytes < need))
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    linrec::Shape s = linrec::shape_of(a);
    s.status = dev.status;
    s.spin_limit = dev.spin_limit;
    linrec::place_parts(s, ws);
    float *partial = sums ? (float *)((char *)ws + linrec::parts_bytes(s)) : nullptr;
    const bool tma = linrec::tma_rows(a->dtype, a->D), bf = a->dtype == GDN_BF16;
    const linrec::BwdArgs b{a->d_h, a->g, a->h, a->gate_scale, a->initial_state, a->d_final_state,
                            a->dx, a->dg, a->d_initial_state, partial};
    cudaStream_t q = (cudaStream_t)stream;
    cudaError_t e = bf ? (gated ? linrec::run_bwd<__nv_bfloat16, true>(b, s, tma, q)
                                : linrec::run_bwd<__nv_bfloat16, false>(b, s, tma, q))
                       : (gated ? linrec::run_bwd<float, true>(b, s, tma, q)
                                : linrec::run_bwd<float, false>(b, s, tma, q));
    if (e == cudaSuccess && sums) e = column_sum(partial, s.lanes_n * s.cluster, a->D, a->d_gate_scale, q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "linear recurrence backward launch");
}

gdn_status gdn_linrec_step(const gdn_linrec_step_args *a, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    if (a->N < 0 || a->D < 1) return fail(GDN_ERR_INVALID_ARG, "bad sizes N=%d D=%d", a->N, a->D);
    if (a->D > (1 << 24) || a->N > (1 << 30)) return fail(GDN_ERR_INVALID_ARG, "problem too large");
    if (a->dtype != GDN_FP32 && a->dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_FP32 or GDN_BF16", a->dtype);
    if (a->N == 0) return GDN_OK;
    if (!a->x || !a->g || !a->state || !a->h || !a->out_state)
        return fail(GDN_ERR_INVALID_ARG, "x, g, state, h and out_state are required");
    if (misaligned(a->x) || misaligned(a->g) || misaligned(a->gate_scale) || misaligned(a->state) ||
        misaligned(a->h) || misaligned(a->out_state))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    if (shifted(a->state, a->out_state, (size_t)a->N * a->D * 4))
        return fail(GDN_ERR_INVALID_ARG, "out_state overlaps state without being it");
    LayerDevice dev;
    const gdn_status st = layer_device(&dev);
    if (st != GDN_OK) return st;
    cudaStream_t q = (cudaStream_t)stream;
    prof_before("linrec_step", q);
    const bool gated = a->gate_scale != nullptr;
    const cudaError_t e = a->dtype == GDN_BF16
                              ? (gated ? linrec::run_step<__nv_bfloat16, true>(a, dev.sms, q)
                                       : linrec::run_step<__nv_bfloat16, false>(a, dev.sms, q))
                              : (gated ? linrec::run_step<float, true>(a, dev.sms, q)
                                       : linrec::run_step<float, false>(a, dev.sms, q));
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "linear recurrence step launch");
}

}  // extern "C"
