// gdn_ssm.cu -- selective state space scan, its backward pass and its one-token step.
//
// Per channel d and state s of S, with the step delta = softplus(dt + dt_bias) (or dt):
//
//     h_t = exp(delta_t a) h_{t-1} + delta_t x_t b_t,   y_t = (<c_t, h_t> + skip x_t) silu(z_t)
//
// A channel's states are shared out to LP lanes, eight to each (four in the backward pass), which stay
// in registers while the lanes walk the tokens; x, dt, z, b and c come through shared memory a tile at a
// time, the step's softplus and the gate taken once for all lanes.  <c, h> of a few tokens is added up
// over the lanes together.
//
// Where sequences and channels are too few for the GPU, sequences are cut into parts that are
// walked twice: first for a part's end state from zero and the sum of its steps (whose exponential
// is the part's decay), then, these joined, for the outputs.  The backward pass always cuts into
// segments of 32 tokens, whose start states and end gradients one joined walk gives.
//
// A token and channel of 16 states is 16 exponentials and 64 multiply-adds (1.7 ps of the GPU's
// either), and 122 instructions in all (3.2 ps): bound by instruction issue, 63% of whose slots the 16
// warps of an SM fill.  Packed 16 x (256 .. 4096) tokens x 4096 gated bf16 600 us (4.2 ps), 32768 x 2048
// in parts 538; 4 x 4096 x 2048 backward 1035, of which the segments' gradients (466 instructions) are
// 744; the memory's floors are 172, 81 and 70.  Whether sequences are cut goes by their mean length: of
// a packed batch of one of 32768 tokens and fifteen of 100, x 2048, all are walked whole (5.2 ms).
#include <algorithm>
#include <type_traits>

#include "gdn_layer_internal.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace ssm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 256;
constexpr int kMaxStates = 64;
constexpr int kSegment = 32;                       // tokens of the backward pass's segments
constexpr int kSub = 4;                            // tokens whose decays it holds in registers

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The decays 2^y.  What matters is a small error that leans neither way, as a slow state multiplies
// thousands of decays near 1 together.  The hardware's exponential leans down by 0.5e-8 .. 3.3e-8 of
// itself there, 1.8e-8 on average over steps spread by their logarithm: a constant added to y, free in
// the product's instruction, takes 1.2e-8 of that away (a step of 0 still gives exactly 1).  fp32 tensors
// take for |y| < 1/32 the polynomial 1 + y q(y), q through (2^y - 1) / y at the three Chebyshev points of
// -1/32 .. 1/32 (1.1e-7 of y).
template <typename T>
__device__ __forceinline__ float2 decay(float2 step, float2 a2) {
    if (sizeof(T) == 2) {
        const float2 y = __ffma2_rn(step, a2, both(1.73e-8f));
        return make_float2(ex2(y.x), ex2(y.y));
    }
    const float2 y = __fmul2_rn(step, a2);
    float2 p = __ffma2_rn(y, both(5.5505085252e-2f), both(2.4023355157e-1f));
    p = __ffma2_rn(p, y, both(0.6931471805599453f));
    p = __ffma2_rn(p, y, both(1.f));
    return make_float2(fabsf(y.x) < 0.03125f ? p.x : ex2(y.x), fabsf(y.y) < 0.03125f ? p.y : ex2(y.y));
}

// Sequences cut into parts of `part` tokens.  A part's slot is cu[n] / part + n + its number in the
// sequence, which no two share, so that a packed batch needs no table: sequence n + 1's first slot is
// at least sequence n's number of parts (one at least) behind sequence n's.
struct Cut {
    Seqs s;
    int part, per;                                 // per: parts of a row
    int slots;
    int *status;
};
struct Part {
    int n;
    long long first;                               // its first token
    int len;                                       // tokens, 0 only for an empty sequence
    bool ends;                                     // the sequence
};
// False where no part has the slot.
__device__ __forceinline__ bool part_of(const Cut &c, int slot, Part &p) {
    long long bos, len, off;
    if (!c.s.cu) {
        p.n = slot / c.per;
        bos = (long long)p.n * c.s.T;
        len = c.s.T;
        off = (long long)(slot - p.n * c.per) * c.part;
    } else {
        int lo = 0, hi = c.s.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((long long)c.s.cu[mid] / c.part + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
        p.n = lo;
        if (!seq_tokens(c.s, lo, bos, len)) return false;
        off = (slot - bos / c.part - lo) * c.part;
    }
    if (off < 0 || (off > 0 && off >= len)) return false;
    p.first = bos + off;
    p.len = (int)min((long long)c.part, len - off);
    p.ends = off + p.len == len;
    return true;
}
// The first slot and the number of parts of sequence n.
__device__ __forceinline__ int parts_of(const Cut &c, int n, int &count) {
    long long bos, len;
    if (!seq_tokens(c.s, n, bos, len)) {
        count = 0;
        return 0;
    }
    count = (int)max(1ll, (len + c.part - 1) / c.part);
    return c.s.cu ? (int)(bos / c.part) + n : n * c.per;
}

// The lanes of a channel have SP places for its S states.  Those past the last state hold copies of
// real ones, whose c is shared out among a state's copies (by halves, which is exact): <c, h> stays the
// same sum, and no place multiplies a zero by what may be infinite (an input, a step).  Fours of places
// are fours of states where S is a multiple of four.
struct Place {
    int state;
    float share;
};
template <int SP>
__device__ __forceinline__ Place place_of(int i, int S) {
    const int P = S > 1 ? 1 << (32 - __clz(S - 1)) : 1;      // the power of two from S on
    const int s = i & (P - 1);
    const bool copy = s >= S, copied = s < P / 2 && s + P / 2 >= S;
    return {copy ? s - P / 2 : s, (copy || copied ? 0.5f : 1.f) * (float)P / SP};
}

// A lane's 2 P neighbouring states, from s0 on, of a row of a [.., D, S] tensor; past the last one copies
// (COPIES), or zeros.
template <int SP, bool COPIES, int P>
__device__ __forceinline__ void load_states(const float *base, long long row, int S, int s0, bool in, float2 (&v)[P]) {
    const float *p = base + row * S;
    const bool there = base && in;
    const auto at = [&](int i) { return COPIES ? place_of<SP>(s0 + i, S).state : s0 + i; };
    const auto one = [&](int i) { return there && (COPIES || s0 + i < S) ? p[at(i)] : 0.f; };
#pragma unroll
    for (int i = 0; i < P; i += 2) {
        if ((S & 3) == 0) {
            const float4 f = there && (COPIES || s0 + 2 * i < S) ? *reinterpret_cast<const float4 *>(p + at(2 * i))
                                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            v[i] = make_float2(f.x, f.y);
            v[i + 1] = make_float2(f.z, f.w);
        } else {
#pragma unroll
            for (int j = i; j < i + 2; ++j) v[j] = make_float2(one(2 * j), one(2 * j + 1));
        }
    }
}
template <int P>
__device__ __forceinline__ void store_states(float *base, long long row, int S, int s0, bool in, const float2 (&v)[P]) {
    if (!in) return;
    float *p = base + row * S + s0;
#pragma unroll
    for (int i = 0; i < P; i += 2) {
        if ((S & 3) == 0) {
            if (s0 + 2 * i < S) *reinterpret_cast<float4 *>(p + 2 * i) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
        } else {
#pragma unroll
            for (int j = i; j < i + 2; ++j) {
                if (s0 + 2 * j < S) p[2 * j] = v[j].x;
                if (s0 + 2 * j + 1 < S) p[2 * j + 1] = v[j].y;
            }
        }
    }
}

// Adds up NV values over NL lanes that are STRIDE apart, `lane` being this one's place among them.
// While values are left to share, each round leaves half of them to either half of the lanes;
// then v[0 .. max(1, NV / NL)) are the sums of the values from the returned index on, and lanes that
// share one all have it.
template <int NV, int NL, int STRIDE>
__device__ __forceinline__ int share_sum(float *v, int lane) {
    int from = 0;
    int n = NV;
#pragma unroll
    for (int o = NL / 2; o > 0; o /= 2) {
        if (n > 1) {
            const int half = n / 2;
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int k = 0; k < NV / 2; ++k)
                if (k < half) {
                    const float give = up ? v[k] : v[k + half], keep = up ? v[k + half] : v[k];
                    v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o * STRIDE);
                }
            if (up) from += half;
            n = half;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o * STRIDE);
        }
    }
    return from;
}

// ------------------------------------------------------------------ forward, and parts' pairs
struct Inputs {
    const void *x, *dt, *b, *c, *z, *dy;
    const float *a, *skip, *dt_bias;
    int D, S, groups;                              // groups of channels
};
struct FwdArgs {
    Inputs in;
    const float *h0;
    void *y;
    float *ht;
    const float *start;                            // [slots][D][S] states before the parts; null: h0
    float *end, *back, *steps;                     // pairs: [slots][D][S], [slots][D][S], [slots][D]
    Cut cut;
    int longest_first;
};
// The outputs; a part's end state from zero and the sum of its steps; and with those the gradient
// that its tokens leave to the state before it.
enum Mode { kOutputs, kPairs, kBothPairs };

// A lane has eight states of two channels, LP lanes share a pair of channels.  What bounds the walk
// beside its arithmetic is what the lanes read of shared memory: b and c, which every channel needs.
// Two channels to a lane, and states by pairs through the arithmetic on two numbers at once, take 80
// bytes for 16 states; four states of one channel 40 bytes for four, and pairs of channels, with b and
// c there twice, 144 for 16 (4.9 ps a token and channel of 16 states, the rate of shared memory).
//
// The lanes take U tokens at a time, each lane U / LP of them as its own: it loads their x, dt and z
// kAhead groups ahead, by cp.async to shared memory (of loads to registers a warp can only await all
// that are in flight), makes their steps and gates, leaves the steps to the others in shared memory,
// and stores their y when the lanes have added up <c, h>.  So a warp waits for the CTA's others only
// for b and c, of TB tokens at a time (whole pairs of groups).
constexpr int kFwdThreads = 128;
constexpr int kStates = 8;                         // of a lane and channel
constexpr int kAhead = 4;
template <typename T, int LP>
struct Lanes {
    static constexpr int CH = 2 * kFwdThreads / LP, SP = kStates * LP;
    static constexpr int U = LP <= 4 ? 4 : LP, OWN = U / LP, TB = LP <= 4 ? 64 / LP : 2 * U;
    struct Two {
        T e[2];
    };
    struct Shared {
        float4 b[2][TB * SP / 4], c[2][TB * SP / 4];
        float4 du[2][U][kFwdThreads / LP];         // steps and steps x, two groups in turn
        float2 ds[2][U][kFwdThreads / LP];         // and gradients before the gate
        alignas(16) Two raw[kAhead + 1][OWN][4][kFwdThreads];    // a lane's x, dt, z, dy
    };
};

// The j-th longest of up to kMaxOrdered sequences: long ones are not left for the end.
constexpr int kMaxOrdered = kFwdThreads;
__device__ __forceinline__ int longest(const Seqs &s, int j, int *scratch) {
    const int t = threadIdx.x;
    if (t < s.N) scratch[t] = s.cu[t + 1] - s.cu[t];
    __syncthreads();
    if (t < s.N) {
        const int mine = scratch[t];
        int rank = 0;
        for (int u = 0; u < s.N; ++u) rank += scratch[u] > mine || (scratch[u] == mine && u < t);
        if (rank == j) scratch[kMaxOrdered] = t;
    }
    __syncthreads();
    const int n = scratch[kMaxOrdered];
    __syncthreads();
    return n;
}

// b or c of a tile, [tokens][S] as [tokens][SP], a few of a place to a thread.
template <typename T, int TT, int SP, int THREADS>
struct Coefficients {
    static constexpr int N = (TT * SP + THREADS - 1) / THREADS;
    static_assert(THREADS % SP == 0, "a thread's are of one place");
    T v[N];                                        // converted only when they are put down: that waits for them
    // Tokens from `token` on, `live` of them (FULL: all of the tile's).
    template <bool FULL>
    __device__ __forceinline__ void fetch(const void *from, long long token, int live, int S) {
        const T *p = (const T *)from + token * S + place_of<SP>(threadIdx.x % SP, S).state;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = (threadIdx.x + i * THREADS) / SP;
            v[i] = (FULL ? N * THREADS == TT * SP || t < TT : t < live) ? p[t * S] : T(0.f);
        }
    }
    __device__ __forceinline__ void put(float4 *to, float share) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (N * THREADS == TT * SP || threadIdx.x + i * THREADS < TT * SP)
                reinterpret_cast<float *>(to)[threadIdx.x + i * THREADS] = to_f(v[i]) * share;
    }
};

// Two neighbouring elements of T, of which the second may not exist; PAIRS: rows of even width, which
// cp.async can copy them from.
template <typename T, bool PAIRS>
__device__ __forceinline__ void copy2(T *to, const T *from, bool both_in) {
    if (PAIRS) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                     "n"(2 * (int)sizeof(T))
                     : "memory");
    } else {
        to[0] = from[0];
        if (both_in) to[1] = from[1];
    }
}
template <typename T, bool PAIRS>
__device__ __forceinline__ void load2(T *to, const T *from, bool both_in) {
    if (PAIRS) {
        *reinterpret_cast<typename Vec<T, 2>::Raw *>(to) = Vec<T, 2>::raw(from);
    } else {
        to[0] = from[0];
        if (both_in) to[1] = from[1];
    }
}
template <typename T>
__device__ __forceinline__ float2 get2(const T *e) {
    float f[2];
    Vec<T, 2>::load(e, f);
    return make_float2(f[0], f[1]);
}
template <typename T, bool PAIRS>
__device__ __forceinline__ void store2(T *p, bool both_in, float2 v) {
    if (PAIRS) {
        const float f[2] = {v.x, v.y};
        Vec<T, 2>::store(p, f);
    } else {
        from_f(p, v.x);
        if (both_in) from_f(p + 1, v.y);
    }
}

// A lane's states of two channels, [channel][pairs of states]: of each channel 4 (i LP + s) to + 3, i = 0
// and 1, so that the lanes' b and c lie side by side.
using LaneStates = float2[2][kStates / 2];
template <int LP>
__device__ __forceinline__ void load_lane(const float *base, long long row, int S, int s, bool in0, bool in1, LaneStates &v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 p[2];
        load_states<kStates * LP, true>(base, row + (i & 1), S, 4 * (i / 2 * LP + s), i & 1 ? in1 : in0, p);
        v[i & 1][i / 2 * 2] = p[0];
        v[i & 1][i / 2 * 2 + 1] = p[1];
    }
}
template <int LP>
__device__ __forceinline__ void store_lane(float *base, long long row, int S, int s, bool in0, bool in1, const LaneStates &v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p[2] = {v[i & 1][i / 2 * 2], v[i & 1][i / 2 * 2 + 1]};
        store_states(base, row + (i & 1), S, 4 * (i / 2 * LP + s), i & 1 ? in1 : in0, p);
    }
}

// Reports impossible ranges, of which some may have no slot.  Not inlined: the walk behind it came out
// with other registers, a tenth slower.
__device__ __noinline__ void report_ranges(const int32_t *cu, long long T, int N, int *status) {
    if (!cu) return;
    for (int n = threadIdx.x; n < N; n += kFwdThreads) {
        long long bos, len;
        if (!seq_tokens({cu, T, N}, n, bos, len)) set_status(status, GDN_ERR_BAD_SEQLENS);
    }
}

template <typename T, int LP, bool PAIRS, int MODE>
__global__ void __launch_bounds__(kFwdThreads, 4) fwd_kernel(FwdArgs a) {
    using L = Lanes<T, LP>;
    constexpr int U = L::U, OWN = L::OWN;
    extern __shared__ __align__(16) uint8_t shared[];
    typename L::Shared &m = *reinterpret_cast<typename L::Shared *>(shared);
    pdl_wait();
    if (blockIdx.x == 0) report_ranges(a.cut.s.cu, a.cut.s.T, a.cut.s.N, a.cut.status);

    const int group = blockIdx.x % a.in.groups;
    int slot = blockIdx.x / a.in.groups;
    if (a.longest_first) slot = longest(a.cut.s, slot, reinterpret_cast<int *>(shared));
    Part part;
    if (!part_of(a.cut, slot, part)) return;
    const int D = a.in.D, S = a.in.S, len = part.len, blocks = (len + L::TB - 1) / L::TB;
    const int pair = threadIdx.x / LP, s = threadIdx.x % LP;
    const int ch = group * L::CH + 2 * pair;
    const bool in0 = ch < D, in1 = ch + 1 < D;

    Coefficients<T, L::TB, L::SP, kFwdThreads> nb, nc;
    const auto fetch = [&](int k) {
        const long long token = part.first + k * L::TB;
        const int left = len - k * L::TB;
        if (left >= L::TB) {
            nb.template fetch<true>(a.in.b, token, left, S);
            if (MODE != kPairs) nc.template fetch<true>(a.in.c, token, left, S);
        } else if (left > 0) {
            nb.template fetch<false>(a.in.b, token, left, S);
            if (MODE != kPairs) nc.template fetch<false>(a.in.c, token, left, S);
        }
    };
    const auto put = [&](int k) {
        nb.put(m.b[k & 1], 1.f);
        if (MODE != kPairs) nc.put(m.c[k & 1], MODE == kOutputs ? place_of<L::SP>(threadIdx.x % L::SP, S).share : 1.f);
    };
    // this lane's tokens of a group, OWN from t on; what lies past the end keeps what was there.
    // Pointers that move a group at a time: 631 -> 600 us against addresses from the token's number.
    const long long mine0 = (part.first + s * OWN) * D + ch, group_step = (long long)U * D;
    const T *px = (const T *)a.in.x + mine0, *pdt = (const T *)a.in.dt + mine0, *pz = (const T *)a.in.z + mine0,
            *pdy = (const T *)a.in.dy + mine0;
    T *py = (T *)a.y + mine0;
    int asked = 0, taken = 0;
    const auto ask = [&](int t) {
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            if (t + j >= len || !in0) continue;
            const auto copy = [&](int what, const T *from) {
                copy2<T, PAIRS>(m.raw[asked][j][what][threadIdx.x].e, from + (long long)j * D, in1);
            };
            copy(0, px);
            copy(1, pdt);
            if (MODE != kPairs && a.in.z) copy(2, pz);
            if (MODE == kBothPairs) copy(3, pdy);
        }
        px += group_step, pdt += group_step, pz += group_step, pdy += group_step;
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++asked == kAhead + 1) asked = 0;
    };
    const auto param = [&](const float *p) { return make_float2(p && in0 ? p[ch] : 0.f, p && in1 ? p[ch + 1] : 0.f); };
    const float2 bias = param(a.in.dt_bias), skip = param(a.in.skip);

#pragma unroll
    for (int g = 0; g < kAhead; ++g) ask(g * U + s * OWN);
    fetch(0);
    LaneStates a2, h, prod, acc;
    float2 steps = both(0.f);
    load_lane<LP>(a.in.a, ch, S, s, in0, in1, a2);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < kStates / 2; ++i) {
            a2[c][i] = __fmul2_rn(a2[c][i], both(kLog2e));
            h[c][i] = acc[c][i] = both(0.f);
            prod[c][i] = both(1.f);
        }
    if (MODE == kOutputs)
        load_lane<LP>(a.start ? a.start : a.h0, (long long)(a.start ? slot : part.n) * D + ch, S, s, in0, in1, h);
    put(0);
    fetch(1);
    __syncthreads();

    // Of the group from token t on: this lane's tokens' steps, and what their outputs will take.
    struct Gates {
        float2 sx[OWN], gate[OWN];
    };
    const auto own_tokens = [&](int which, int t, Gates &g) {
        const int own = t + s * OWN;
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const auto mine = [&](int j, int what) { return get2(m.raw[taken][j][what][threadIdx.x].e); };
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const float2 xi = mine(j, 0);
            float2 st = mine(j, 1);
            if (a.in.dt_bias) st = softplus2<T>(__fadd2_rn(st, bias));
            const bool live = own + j < len;
            float2 u = __fmul2_rn(st, xi);
            if (!live) st = u = both(0.f);
            m.du[which][s * OWN + j][pair] = make_float4(st.x, st.y, u.x, u.y);
            if (MODE == kPairs) continue;
            g.gate[j] = both(1.f);
            if (a.in.z) {
                g.gate[j] = mine(j, 2);
                g.gate[j] = __fmul2_rn(g.gate[j], logistic2<T>(g.gate[j]));
            }
            // without skip no product with x, which may be infinite
            if (MODE == kOutputs) g.sx[j] = a.in.skip ? __fmul2_rn(skip, xi) : both(0.f);
            else m.ds[which][s * OWN + j][pair] = live ? __fmul2_rn(g.gate[j], mine(j, 3)) : both(0.f);
        }
        if (++taken == kAhead + 1) taken = 0;
        ask(own + kAhead * U);
    };
    const auto walk = [&](int which, int t, const Gates &g, const float4 *bt, const float4 *ct) {
        float v[2 * U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const float4 du = m.du[which][j][pair];
            const float2 ds = MODE == kBothPairs ? m.ds[which][j][pair] : both(0.f);
            float2 dot[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {          // four states
                const float4 b4 = bt[(j * 2 + q) * LP], c4 = MODE != kPairs ? ct[(j * 2 + q) * LP] : b4;
#pragma unroll
                for (int o = 0; o < 2; ++o) {      // two of them
                    const int i = 2 * q + o;
                    const float2 b = o ? make_float2(b4.z, b4.w) : make_float2(b4.x, b4.y);
                    const float2 cc = o ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float2 e = decay<T>(both(c ? du.y : du.x), a2[c][i]);
                        h[c][i] = __ffma2_rn(e, h[c][i], __fmul2_rn(both(c ? du.w : du.z), b));
                        if (MODE == kOutputs) dot[c] = i ? __ffma2_rn(cc, h[c][i], dot[c]) : __fmul2_rn(cc, h[c][i]);
                        if (MODE == kBothPairs) {
                            prod[c][i] = __fmul2_rn(prod[c][i], e);
                            acc[c][i] = __ffma2_rn(prod[c][i], __fmul2_rn(both(c ? ds.y : ds.x), cc), acc[c][i]);
                        }
                    }
                }
            }
            if (MODE == kOutputs) {
                v[2 * j] = dot[0].x + dot[0].y;
                v[2 * j + 1] = dot[1].x + dot[1].y;
            } else {
                steps = __fadd2_rn(steps, make_float2(du.x, du.y));
            }
        }
        if (MODE != kOutputs) return;
        share_sum<2 * U, LP, 1>(v, s);             // those of this lane's tokens
        const int own = t + s * OWN;
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            if (own + j >= len || !in0) continue;
            const float2 y = __fmul2_rn(__fadd2_rn(make_float2(v[2 * j], v[2 * j + 1]), g.sx[j]), g.gate[j]);
            store2<T, PAIRS>(py + (long long)j * D, in1, y);
        }
        py += group_step;
    };
    // a group's steps are read behind a __syncwarp, and the next group's are put elsewhere
    Gates g;
    for (int k = 0; k < blocks; ++k) {
        const float4 *bt = m.b[k & 1] + s, *ct = m.c[k & 1] + s;
        const int t0 = k * L::TB, t1 = min(t0 + L::TB, len);
#pragma unroll 1
        for (int t = t0; t < t1; t += 2 * U, bt += U * L::SP / 2, ct += U * L::SP / 2) {
            own_tokens(0, t, g);
            __syncwarp();
            walk(0, t, g, bt, ct);
            own_tokens(1, t + U, g);
            __syncwarp();
            walk(1, t + U, g, bt + U * L::SP / 4, ct + U * L::SP / 4);
        }
        if (k + 1 < blocks) {
            put(k + 1);
            fetch(k + 2);
        }
        __syncthreads();
    }
    if (MODE == kOutputs) {
        if (part.ends && a.ht) store_lane<LP>(a.ht, (long long)part.n * D + ch, S, s, in0, in1, h);
    } else {
        const long long row = (long long)slot * D + ch;
        store_lane<LP>(a.end, row, S, s, in0, in1, h);
        if (MODE == kBothPairs) store_lane<LP>(a.back, row, S, s, in0, in1, acc);
        if (s == 0 && in0) a.steps[row] = steps.x;
        if (s == 0 && in1) a.steps[row + 1] = steps.y;
    }
}

// Parts joined: end[slot] becomes the state before the part, back[slot] (if given) the gradient that
// reaches its last state from behind.  A thread takes one state of a channel of a sequence.
struct JoinArgs {
    const float *a, *steps, *h0, *dht;
    float *end, *back, *dh0;
    int D, S;
    Cut cut;
};
__global__ void __launch_bounds__(256) join_kernel(JoinArgs a) {
    pdl_wait();
    const long long states = (long long)a.D * a.S, i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int n = blockIdx.y;
    if (i >= states) return;
    const int d = (int)(i / a.S);
    int count;
    const int first = parts_of(a.cut, n, count);
    const float a2 = a.a[i] * kLog2e;
    constexpr int kAhead = 16;                     // parts whose loads are in flight
    // one direction to a thread: parts in order for the states, from the last for the gradients
    const bool back = blockIdx.z == 1;
    float *const pairs = back ? a.back : a.end;
    const float *const from = back ? a.dht : a.h0;
    const auto at = [&](int j) { return (long long)(first + (back ? count - 1 - j : j)); };
    float v = from ? from[n * states + i] : 0.f;
    for (int j = 0; j < count; j += kAhead) {
        float e[kAhead], st[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (j + k < count) {
                e[k] = pairs[at(j + k) * states + i];
                st[k] = a.steps[at(j + k) * a.D + d];
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (j + k < count) {
                pairs[at(j + k) * states + i] = v;
                // a part's decay may underflow where no token's does: an infinite state stays one
                const float decay = ex2(st[k] * a2);
                v = decay == 0.f && isinf(v) ? v + e[k] : fmaf(decay, v, e[k]);
            }
    }
    if (back && a.dh0 && count > 0) a.dh0[n * states + i] = v;
}

// ------------------------------------------------------------------ backward
struct BwdArgs {
    Inputs in;
    float *start;                                  // [slots][D][S] states before the segments; then da's parts
    const float *behind;                           // [slots][D][S] gradients from behind them
    void *dx, *ddt, *dz;
    float *dskip, *dbias;                          // [slots][D] each segment's part
    float *dbc;                                    // [lanes][tokens][2 S]: of groups of channels
    void *db, *dc;                                 // written here where one lane has all channels
    long long tokens;
    int lanes;                                     // CTAs that share a segment's channels
    Cut cut;
};

// A lane has four states of two channels here, LP lanes a pair of channels: the decays and decayed
// states of a sub-segment's tokens are 64 registers.  4 x 4096 x 2048 x 16 gated bf16, this kernel alone:
// segments of 64 tokens in sub-segments of 8 (128 registers, 8 warps to an SM) 846 us, so (12 warps) 744.
template <int LP>
struct Segment {
    static constexpr int CP = LP <= 4 ? 32 : 128 / LP, CH = 2 * CP, NT = CP * LP, WARPS = NT / 32;
    static constexpr int SP = 4 * LP, V = 2 * SP;  // states, and gradients of b and c of a token
    float4 du[kSegment][CP];                       // steps, steps x; then <e, b>, <e a, p>
    float2 ds[kSegment][CP];                       // gradients before the gate; then <c, h>
    float4 b[kSegment * LP], c[kSegment * LP];
    float4 saved[kSegment / kSub - 1][2][NT];      // states before the sub-segments; then sums of dskip, dbias
    float red[2][WARPS][kSub][V];
    float acc[kSegment * V];
};
constexpr int kBwdThreads = 384;                   // on an SM at once
using SubStates = float2[2][2];                    // [channel][pair of states]

template <typename T, int LP, bool PAIRS>
__global__ void __launch_bounds__(Segment<LP>::NT, kBwdThreads / Segment<LP>::NT) bwd_kernel(BwdArgs a) {
    using G = Segment<LP>;
    extern __shared__ __align__(16) uint8_t shared[];
    G &m = *reinterpret_cast<G *>(shared);
    pdl_wait();

    const int slot = blockIdx.x / a.lanes, lane_no = blockIdx.x - slot * a.lanes;
    const int D = a.in.D, S = a.in.S, tid = threadIdx.x;
    const int g0 = (int)((long long)a.in.groups * lane_no / a.lanes), g1 = (int)((long long)a.in.groups * (lane_no + 1) / a.lanes);
    const int s = tid % LP, pair = tid / LP, warp = tid / 32;
    Part part;
    const bool there = part_of(a.cut, slot, part) && part.len > 0;
    if (!there) {                                  // its parts of the sums
        for (int g = g0; g < g1; ++g)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int ch = g * G::CH + 2 * pair + c;
                const float2 none[2] = {both(0.f), both(0.f)};
                store_states(a.start, (long long)slot * D + ch, S, 4 * s, ch < D, none);
                if (ch < D && s == 0) {
                    if (a.dskip) a.dskip[(long long)slot * D + ch] = 0.f;
                    if (a.dbias) a.dbias[(long long)slot * D + ch] = 0.f;
                }
            }
        return;
    }
    const int len = part.len, subs = (len + kSub - 1) / kSub;
    {
        Coefficients<T, kSegment, G::SP, G::NT> co;
        co.template fetch<false>(a.in.b, part.first, len, S);
        co.put(m.b, 1.f);
        co.template fetch<false>(a.in.c, part.first, len, S);
        co.put(m.c, tid % G::SP < S ? 1.f : 0.f);  // copies take no part in the gradients
    }
    for (int k = tid; k < kSegment * G::V; k += G::NT) m.acc[k] = 0.f;

    // as one that loads and stores: a pair of channels, every LP-th token
    const int mp = tid % G::CP, mt = tid / G::CP;
    struct alignas(16) Raw {
        T x[2], dt[2], z[2], dy[2];
    };
    for (int g = g0; g < g1; ++g) {
        const int mch = g * G::CH + 2 * mp;
        const bool m0 = mch < D, m1 = mch + 1 < D;
        const auto param = [&](const float *p) { return make_float2(p && m0 ? p[mch] : 0.f, p && m1 ? p[mch + 1] : 0.f); };
        const float2 bias = param(a.in.dt_bias), skip = param(a.in.skip);
        const long long base = part.first * D + mch;
        const auto fetch = [&](int t, Raw &r) {
            r = {};
            if (t >= len || !m0) return;
            const long long at = base + (long long)t * D;
            load2<T, PAIRS>(r.x, (const T *)a.in.x + at, m1);
            load2<T, PAIRS>(r.dt, (const T *)a.in.dt + at, m1);
            if (a.in.z) load2<T, PAIRS>(r.z, (const T *)a.in.z + at, m1);
            load2<T, PAIRS>(r.dy, (const T *)a.in.dy + at, m1);
        };
        constexpr int kBatch = 8 < kSegment / LP ? 8 : kSegment / LP;    // tokens whose loads are in flight
        for (int t0 = mt; t0 < kSegment; t0 += kBatch * LP) {
            Raw r[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) fetch(t0 + j * LP, r[j]);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int t = t0 + j * LP;
                float2 step = get2(r[j].dt), ds = get2(r[j].dy);
                if (a.in.dt_bias) step = softplus2<T>(__fadd2_rn(step, bias));
                if (t >= len) step = both(0.f);
                if (a.in.z) {
                    const float2 z = get2(r[j].z);
                    ds = __fmul2_rn(ds, __fmul2_rn(z, logistic2<T>(z)));
                }
                const float2 u = __fmul2_rn(step, get2(r[j].x));
                m.du[t][mp] = make_float4(step.x, step.y, u.x, u.y);
                m.ds[t][mp] = ds;
            }
        }
        SubStates an, a2, hs, carry, da;
        const int ch = g * G::CH + 2 * pair;
        const long long row = (long long)slot * D + ch;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            load_states<G::SP, true>(a.in.a, ch + c, S, 4 * s, ch + c < D, an[c]);
            load_states<G::SP, false>(a.start, row + c, S, 4 * s, ch + c < D, hs[c]);
            load_states<G::SP, false>(a.behind, row + c, S, 4 * s, ch + c < D, carry[c]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a2[c][i] = __fmul2_rn(an[c][i], both(kLog2e));
                da[c][i] = both(0.f);
            }
        }
        __syncthreads();

        // the states before every sub-segment
        {
            SubStates h = {{hs[0][0], hs[0][1]}, {hs[1][0], hs[1][1]}};
            for (int q = 0; q + 1 < subs; ++q) {
#pragma unroll
                for (int k = 0; k < kSub; ++k) {
                    const int t = q * kSub + k;
                    const float4 du = m.du[t][pair], b = m.b[t * LP + s];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            h[c][i] = __ffma2_rn(decay<T>(both(c ? du.y : du.x), a2[c][i]), h[c][i],
                                                 __fmul2_rn(both(c ? du.w : du.z), i ? make_float2(b.z, b.w) : make_float2(b.x, b.y)));
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) m.saved[q][c][tid] = make_float4(h[c][0].x, h[c][0].y, h[c][1].x, h[c][1].y);
            }
        }
        // TAIL: the sequence ends inside the sub-segment
        const auto gradients = [&](int q, auto tail) {
            constexpr bool TAIL = decltype(tail)::value;
            SubStates h = {{hs[0][0], hs[0][1]}, {hs[1][0], hs[1][1]}}, e[kSub], p[kSub];
            if (q > 0)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float4 v = m.saved[q - 1][c][tid];
                    h[c][0] = make_float2(v.x, v.y);
                    h[c][1] = make_float2(v.z, v.w);
                }
#pragma unroll
            for (int k = 0; k < kSub; ++k) {
                const int t = q * kSub + k;
                const float4 du = m.du[t][pair], b = m.b[t * LP + s];
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        e[k][c][i] = decay<T>(both(c ? du.y : du.x), a2[c][i]);
                        p[k][c][i] = __fmul2_rn(e[k][c][i], h[c][i]);
                        h[c][i] = __ffma2_rn(both(c ? du.w : du.z), i ? make_float2(b.z, b.w) : make_float2(b.x, b.y), p[k][c][i]);
                    }
            }
            // past the last token nothing: an infinite state times the step there, 0, would be NaN in da
            if (TAIL)
#pragma unroll
                for (int k = 1; k < kSub; ++k)
                    if (q * kSub + k >= len)
#pragma unroll
                        for (int c = 0; c < 2; ++c) p[k][c][0] = p[k][c][1] = both(0.f);
            // <c, h>, <e, b> and <e a, p> of this lane's states, [token][channel]
            float hc[2 * kSub], eb[2 * kSub], ep[2 * kSub];
            float *red = &m.red[q & 1][warp][0][0];
#pragma unroll
            for (int k = kSub - 1; k >= 0; --k) {
                const int t = q * kSub + k;
                const float4 du = m.du[t][pair], b4 = m.b[t * LP + s], c4 = m.c[t * LP + s];
                const float2 ds2 = m.ds[t][pair];
                float2 gb[2], gc[2];               // gradients of b and c, of both channels
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float2 step = both(c ? du.y : du.x), u = both(c ? du.w : du.z), ds = both(c ? ds2.y : ds2.x);
                    float2 vh, vb, vp;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 b = i ? make_float2(b4.z, b4.w) : make_float2(b4.x, b4.y);
                        const float2 cc = i ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
                        const float2 hh = __ffma2_rn(u, b, p[k][c][i]);
                        const float2 grad = __ffma2_rn(cc, ds, carry[c][i]);
                        const float2 lost = __fmul2_rn(grad, p[k][c][i]);
                        gc[i] = c ? __ffma2_rn(ds, hh, gc[i]) : __fmul2_rn(ds, hh);
                        gb[i] = c ? __ffma2_rn(grad, u, gb[i]) : __fmul2_rn(grad, u);
                        vh = i ? __ffma2_rn(cc, hh, vh) : __fmul2_rn(cc, hh);
                        vb = i ? __ffma2_rn(grad, b, vb) : __fmul2_rn(grad, b);
                        vp = i ? __ffma2_rn(lost, an[c][i], vp) : __fmul2_rn(lost, an[c][i]);
                        da[c][i] = __ffma2_rn(lost, step, da[c][i]);
                        carry[c][i] = __fmul2_rn(e[k][c][i], grad);
                    }
                    hc[2 * k + c] = vh.x + vh.y;
                    eb[2 * k + c] = vb.x + vb.y;
                    ep[2 * k + c] = vp.x + vp.y;
                }
                float v[8] = {gb[0].x, gb[0].y, gb[1].x, gb[1].y, gc[0].x, gc[0].y, gc[1].x, gc[1].y};
                constexpr int NL = 32 / LP, LEFT = NL >= 8 ? 1 : 8 / NL;
                const int lane = (tid & 31) / LP, from = share_sum<8, NL, LP>(v, lane);
                if (NL <= 8 || (lane & (NL / 8 - 1)) == 0) {
#pragma unroll
                    for (int i = 0; i < LEFT; ++i) {
                        const int w = from + i;    // 0 - 3: b's, 4 - 7: c's
                        red[k * G::V + (w >> 2) * G::SP + 4 * s + (w & 3)] = v[i];
                    }
                }
            }
            // over the channels' lanes; every lane has read its tokens' steps and gradients
            {
                constexpr int LEFT = LP < 2 * kSub ? 2 * kSub / LP : 1;
                const int from = share_sum<2 * kSub, LP, 1>(hc, s);
                share_sum<2 * kSub, LP, 1>(eb, s);
                share_sum<2 * kSub, LP, 1>(ep, s);
                __syncwarp();
                const int t = q * kSub + from / 2;
                if constexpr (LEFT >= 2) {
#pragma unroll
                    for (int i = 0; i < LEFT; i += 2) {
                        m.du[t + i / 2][pair] = make_float4(eb[i], eb[i + 1], ep[i], ep[i + 1]);
                        m.ds[t + i / 2][pair] = make_float2(hc[i], hc[i + 1]);
                    }
                } else if (LP <= 2 * kSub || (s & (LP / (2 * kSub) - 1)) == 0) {    // one channel's
                    const int c = from & 1;
                    float *sums = reinterpret_cast<float *>(&m.du[t][pair]);
                    sums[c] = eb[0];
                    sums[2 + c] = ep[0];
                    reinterpret_cast<float *>(&m.ds[t][pair])[c] = hc[0];
                }
            }
            __syncthreads();
            for (int k = tid; k < kSub * G::V; k += G::NT) {
                float v = m.acc[q * kSub * G::V + k];
#pragma unroll
                for (int w = 0; w < G::WARPS; ++w) v += (&m.red[q & 1][w][0][0])[k];
                m.acc[q * kSub * G::V + k] = v;
            }
        };
        int q = subs - 1;
        if (len % kSub != 0) gradients(q--, std::true_type());
        for (; q >= 0; --q) gradients(q, std::false_type());
#pragma unroll
        for (int c = 0; c < 2; ++c) store_states(a.start, row + c, S, 4 * s, ch + c < D, da[c]);
        __syncthreads();                           // every channel's sums are there

        float2 gs = both(0.f), gbias = both(0.f);
        for (int t0 = mt; t0 < len; t0 += kBatch * LP) {
            Raw r[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) fetch(t0 + j * LP, r[j]);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int t = t0 + j * LP;
                if (t >= len || !m0) continue;
                const float4 sums = m.du[t][mp];
                const float2 x = get2(r[j].x), dy = get2(r[j].dy), hc = m.ds[t][mp];
                float2 step = get2(r[j].dt), slope = both(1.f), ds = dy;
                if (a.in.dt_bias) {
                    const float2 raw = __fadd2_rn(step, bias);
                    step = softplus2<T>(raw);
                    slope = logistic2<T>(raw);
                }
                const long long at = base + (long long)t * D;
                if (a.in.z) {
                    const float2 z = get2(r[j].z), sg = logistic2<T>(z), y = a.in.skip ? __ffma2_rn(skip, x, hc) : hc;
                    store2<T, PAIRS>((T *)a.dz + at, m1,
                                     __fmul2_rn(__fmul2_rn(dy, y), make_float2(silu_slope(z.x, sg.x), silu_slope(z.y, sg.y))));
                    ds = __fmul2_rn(dy, __fmul2_rn(z, sg));
                }
                const float2 eb = make_float2(sums.x, sums.y);
                const float2 ddt = __fmul2_rn(slope, __ffma2_rn(x, eb, make_float2(sums.z, sums.w)));
                float2 dx = __fmul2_rn(step, eb);
                if (a.in.skip) dx = __ffma2_rn(skip, ds, dx);
                store2<T, PAIRS>((T *)a.dx + at, m1, dx);
                store2<T, PAIRS>((T *)a.ddt + at, m1, ddt);
                gs = __ffma2_rn(ds, x, gs);
                gbias = __fadd2_rn(gbias, ddt);
            }
        }
        // over the threads that took the same channels
        float4 *sums = &m.saved[0][0][0];
        sums[mt * G::CP + mp] = make_float4(gs.x, gs.y, gbias.x, gbias.y);
        __syncthreads();
        if (tid < G::CP) {
            float4 v = sums[tid];
#pragma unroll
            for (int r = 1; r < LP; ++r) {
                const float4 w = sums[r * G::CP + tid];
                v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
            }
            const long long at = (long long)slot * D + mch;
            if (a.dskip && m0) a.dskip[at] = v.x;
            if (a.dskip && m1) a.dskip[at + 1] = v.y;
            if (a.dbias && m0) a.dbias[at] = v.z;
            if (a.dbias && m1) a.dbias[at + 1] = v.w;
        }
        __syncthreads();                           // before the next channels' tile
    }
    for (int k = tid; k < len * 2 * S; k += G::NT) {
        const int t = k / (2 * S), w = k % (2 * S);
        const float v = m.acc[t * G::V + (w >= S ? G::SP + w - S : w)];
        if (a.lanes == 1) from_f((T *)(w >= S ? a.dc : a.db) + (part.first + t) * S + (w >= S ? w - S : w), v);
        else a.dbc[((long long)lane_no * a.tokens + part.first + t) * 2 * S + w] = v;
    }
}

// db and dc from the lanes' parts; tokens that no sequence has are left alone.
template <typename T>
__global__ void __launch_bounds__(256) dbc_kernel(const float *parts, int lanes, long long tokens, int S, Seqs s,
                                                  T *db, T *dc) {
    pdl_enter();
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < tokens * 2 * S;
         i += (long long)gridDim.x * blockDim.x) {
        const long long t = i / (2 * S);
        const int w = (int)(i - t * 2 * S);
        if (s.cu) {
            long long bos, len;
            if (!seq_tokens(s, seq_of(s, t), bos, len)) continue;
        }
        float v = 0.f;
        for (int l = 0; l < lanes; ++l) v += parts[(long long)l * tokens * 2 * S + i];
        from_f((w >= S ? dc : db) + t * S + (w >= S ? w - S : w), v);
    }
}

// ------------------------------------------------------------------ one token
struct StepArgs {
    Inputs in;
    const float *state;
    void *y;
    float *out;
    int N;
};
// A thread takes four states of a channel, of every gridDim.y-th sequence.
template <typename T, int LP>
__global__ void __launch_bounds__(kThreads) step_kernel(StepArgs a) {
    pdl_enter();
    const int D = a.in.D, S = a.in.S, s = threadIdx.x % LP, ch = blockIdx.x * (kThreads / LP) + threadIdx.x / LP;
    const bool in = ch < D;
    constexpr int SP = 4 * LP;
    float2 a2[2];
    load_states<SP, false>(a.in.a, ch, S, 4 * s, in, a2);
    a2[0] = __fmul2_rn(a2[0], both(kLog2e));
    a2[1] = __fmul2_rn(a2[1], both(kLog2e));
    const float bias = a.in.dt_bias && in ? a.in.dt_bias[ch] : 0.f, skip = a.in.skip && in ? a.in.skip[ch] : 0.f;
    const auto coefficients = [&](const void *base, long long n, float (&v)[4]) {
        const T *p = (const T *)base + n * S + 4 * s;
        if ((S & 3) == 0 && 4 * s < S) {
            Vec<T, 4>::load(p, v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = 4 * s + i < S ? to_f(p[i]) : 0.f;
        }
    };
    for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
        const long long row = (long long)n * D + ch;
        float2 h[2];
        load_states<SP, false>(a.state, row, S, 4 * s, in, h);
        float b[4], cc[4], step = 0.f, x = 0.f, z = 0.f;
        coefficients(a.in.b, n, b);
        coefficients(a.in.c, n, cc);
        if (in) {
            x = to_f(((const T *)a.in.x)[row]);
            step = to_f(((const T *)a.in.dt)[row]);
            if (a.in.z) z = to_f(((const T *)a.in.z)[row]);
        }
        if (a.in.dt_bias) step = softplus<T>(step + bias);
        float2 dot = both(0.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            h[i] = __ffma2_rn(decay<T>(both(step), a2[i]), h[i],
                              __fmul2_rn(both(step * x), make_float2(b[2 * i], b[2 * i + 1])));
            // of states that there are not nothing counts, whatever the step and x
            dot = __ffma2_rn(make_float2(cc[2 * i], cc[2 * i + 1]),
                             make_float2(4 * s + 2 * i < S ? h[i].x : 0.f, 4 * s + 2 * i + 1 < S ? h[i].y : 0.f), dot);
        }
        store_states(a.out, row, S, 4 * s, in, h);
        float y = dot.x + dot.y;
#pragma unroll
        for (int o = LP / 2; o > 0; o /= 2) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (!in || s != 0) continue;
        if (a.in.skip) y = fmaf(skip, x, y);
        if (a.in.z) y *= z * logistic<T>(z);
        from_f((T *)a.y + row, y);
    }
}

// ------------------------------------------------------------------ host
// Lanes of a channel, with so many states to each.
int lanes_of(int S, int states) {
    int lp = 1;
    while (states * lp < S) lp *= 2;
    return lp;
}
// Of the forward pass two at least: alone with eight states or fewer a lane has so much to do for its own
// tokens that they hold the walk up (8 x 2048 x 4096 x 8 bf16 533 us, with two 453).
int fwd_lanes(int S) { return std::max(2, lanes_of(S, kStates)); }
template <int MOST, typename F>
auto by_lanes(int lp, F f) {
    if constexpr (MOST > 8)
        if (lp == 1) return f(std::integral_constant<int, 1>());
    if (lp == 2) return f(std::integral_constant<int, 2>());
    if (lp == 4) return f(std::integral_constant<int, 4>());
    if (lp == 8 || MOST == 8) return f(std::integral_constant<int, 8>());
    return f(std::integral_constant<int, MOST>());
}
template <typename F>
auto by_type(int dtype, F f) {
    return dtype == GDN_BF16 ? f((__nv_bfloat16 *)nullptr) : f((float *)nullptr);
}
template <typename F>
auto by_alignment(bool whole, F f) {
    return whole ? f(std::true_type()) : f(std::false_type());
}

gdn_status check(int B, int T, int D, int S, int N, int dtype, bool packed) {
    if (B < 1 || T < 0 || D < 1 || S < 1)
        return fail(GDN_ERR_INVALID_ARG, "bad sizes B=%d T=%d D=%d S=%d", B, T, D, S);
    if (S > kMaxStates) return fail(GDN_ERR_UNSUPPORTED, "S = %d (at most %d)", S, kMaxStates);
    if (dtype != GDN_FP32 && dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_FP32 or GDN_BF16", dtype);
    if (packed && (B != 1 || N < 1))
        return fail(GDN_ERR_INVALID_ARG, "cu_seqlens needs B == 1 and N >= 1 (B=%d N=%d)", B, N);
    // a CTA for 16 channels and 32 tokens or a sequence at least, numbered by an int; sequences by a
    // grid's second dimension
    const long long n = packed ? N : B, tokens = (long long)B * T;
    if (tokens >= (1ll << 31) - (1 << 16) || D > (1 << 23) || n > 65535 ||
        (tokens / kSegment + 2 * n) * ((D + 15) / 16) >= (1ll << 31))
        return fail(GDN_ERR_INVALID_ARG, "problem too large");
    return GDN_OK;
}

Cut cut_of(const int32_t *cu, int B, int T, int N, int part) {
    Cut c{};
    c.s = {cu, T, cu ? N : B};
    c.part = part;
    c.per = std::max(1, (int)(((long long)T + part - 1) / part));
    c.slots = cu ? (int)((long long)T / part) + N : B * c.per;
    return c;
}

// Tokens of a part of the forward pass, T + 1 for sequences left whole.  Parts, of 32 tokens at least,
// pay, with their second walk and two launches, from sequences of 192 tokens on where whole ones are no
// more than a CTA to an SM, which waits for its own arithmetic.  Us whole | in parts, 16 states gated bf16:
// 8 x 2048 x 2048 360 | 321, 2 x 400 x 4096 72 | 41, 2 x 200 x 4096 37 | 31, 2 x 1000 x 1024 175 | 31.
int fwd_part(int B, int T, int D, int S, int N, bool packed) {
    const int lp = fwd_lanes(S), ch = 2 * kFwdThreads / lp;
    const long long n = packed ? N : B, ctas = n * ((D + ch - 1) / ch), mean = packed ? T / n : T;
    const long long fill = 4 * kSms / std::max(1ll, ctas), parts = std::min(fill, mean / 32);
    if (fill < 4 || mean < 192) return T + 1;
    return (int)((mean + parts - 1) / parts + 7) / 8 * 8;
}

struct FwdPlan {
    Cut cut;
    bool parts;
    size_t states, steps;          // floats of each
};
FwdPlan plan_of(const gdn_ssm_fwd_args *a) {
    FwdPlan p{};
    const int part = fwd_part(a->B, a->T, a->D, a->S, a->N, a->cu_seqlens != nullptr);
    p.parts = part <= a->T;
    p.cut = cut_of(a->cu_seqlens, a->B, a->T, a->N, part);
    if (p.parts) {
        p.states = (size_t)p.cut.slots * a->D * a->S;
        p.steps = (size_t)p.cut.slots * a->D;
    }
    return p;
}

struct BwdPlan {
    Cut cut;
    int lanes;
    size_t states, rows, dbc;      // floats: of states (twice), of a row (three times), of db and dc
};
BwdPlan plan_of(const gdn_ssm_bwd_args *a) {
    BwdPlan p{};
    p.cut = cut_of(a->cu_seqlens, a->B, a->T, a->N, kSegment);
    const int lp = lanes_of(a->S, 4), ch = lp <= 4 ? 64 : 256 / lp, groups = (a->D + ch - 1) / ch;
    // CTAs for about four waves, so that the last one is short
    const long long want = (8ll * kSms + p.cut.slots - 1) / p.cut.slots;
    p.lanes = (int)std::max(1ll, std::min<long long>(groups, want));
    p.states = (size_t)p.cut.slots * a->D * a->S;
    p.rows = (size_t)p.cut.slots * a->D;
    p.dbc = p.lanes > 1 ? (size_t)p.lanes * a->B * a->T * 2 * a->S : 0;
    return p;
}
size_t padded(size_t floats) { return (floats + 3) / 4 * 4; }
size_t fwd_bytes(const FwdPlan &p) { return 4 * (padded(p.states) + padded(p.steps)); }
size_t bwd_bytes(const BwdPlan &p) { return 4 * (2 * padded(p.states) + 3 * padded(p.rows) + padded(p.dbc)); }
size_t asked_for(size_t need) { return need == 0 ? 256 : std::max<size_t>(512, need); }

template <int MODE>
cudaError_t launch_fwd(const char *name, FwdArgs f, int dtype, cudaStream_t q) {
    return by_type(dtype, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return by_lanes<8>(fwd_lanes(f.in.S), [&](auto lp) {
            return by_alignment(f.in.D % 2 == 0, [&](auto vect) {
                constexpr int LP = decltype(lp)::value;
                auto k = fwd_kernel<T, LP, decltype(vect)::value, MODE>;
                cudaError_t e = allow_smem((const void *)k, sizeof(typename Lanes<T, LP>::Shared));
                if (e != cudaSuccess) return e;
                f.in.groups = (f.in.D + Lanes<T, LP>::CH - 1) / Lanes<T, LP>::CH;
                prof_before(name, q);
                e = launch_pdl(k, dim3((unsigned)((long long)f.in.groups * f.cut.slots)),
                               dim3(kFwdThreads), sizeof(typename Lanes<T, LP>::Shared), q, f);
                prof_after(q);
                return e;
            });
        });
    });
}

cudaError_t launch_join(const JoinArgs &j, cudaStream_t q) {
    const long long states = (long long)j.D * j.S;
    prof_before("ssm_join", q);
    const cudaError_t e = launch_pdl(join_kernel, dim3((unsigned)((states + 255) / 256), j.cut.s.N, j.back ? 2 : 1),
                                     dim3(256), 0, q, j);
    prof_after(q);
    return e;
}

template <typename T>
cudaError_t launch_bwd(BwdArgs b, cudaStream_t q) {
    cudaError_t e = by_lanes<16>(lanes_of(b.in.S, 4), [&](auto lp) {
        return by_alignment(b.in.D % 2 == 0, [&](auto vect) {
            constexpr int LP = decltype(lp)::value;
            using G = Segment<LP>;
            auto k = bwd_kernel<T, LP, decltype(vect)::value>;
            cudaError_t r = allow_smem((const void *)k, sizeof(G));
            if (r != cudaSuccess) return r;
            b.in.groups = (b.in.D + G::CH - 1) / G::CH;
            prof_before("ssm_bwd", q);
            r = launch_pdl(k, dim3((unsigned)((long long)b.lanes * b.cut.slots)), dim3(G::NT), sizeof(G), q, b);
            prof_after(q);
            return r;
        });
    });
    if (e != cudaSuccess || b.lanes == 1 || b.tokens == 0) return e;
    const long long n = b.tokens * 2 * b.in.S;
    prof_before("ssm_dbc", q);
    e = launch_pdl(dbc_kernel<T>, dim3((unsigned)std::min<long long>((n + 255) / 256, 1 << 16)), dim3(256), 0, q,
                   (const float *)b.dbc, b.lanes, b.tokens, b.in.S, b.cut.s, (T *)b.db, (T *)b.dc);
    prof_after(q);
    return e;
}

}  // namespace
}  // namespace ssm
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_ssm_fwd_workspace_size(const gdn_ssm_fwd_args *a) {
    if (!a) {
        fail(GDN_ERR_INVALID_ARG, "null args");
        return 0;
    }
    if (ssm::check(a->B, a->T, a->D, a->S, a->N, a->dtype, a->cu_seqlens != nullptr) != GDN_OK) return 0;
    return ssm::asked_for(ssm::fwd_bytes(ssm::plan_of(a)));
}

gdn_status gdn_ssm_fwd(const gdn_ssm_fwd_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = ssm::check(a->B, a->T, a->D, a->S, a->N, a->dtype, a->cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (!a->a || (a->T > 0 && (!a->x || !a->dt || !a->b || !a->c || !a->y)))
        return fail(GDN_ERR_INVALID_ARG, "x, dt, a, b, c and y are required");
    if (misaligned(a->x) || misaligned(a->dt) || misaligned(a->a) || misaligned(a->b) || misaligned(a->c) ||
        misaligned(a->skip) || misaligned(a->z) || misaligned(a->dt_bias) || misaligned(a->initial_state) ||
        misaligned(a->cu_seqlens) || misaligned(a->y) || misaligned(a->final_state))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    ssm::FwdPlan p = ssm::plan_of(a);
    const size_t need = ssm::fwd_bytes(p);
    if (need > 0 && (!ws || misaligned(ws) || ws_bytes < need))
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    p.cut.status = dev.status;
    cudaStream_t q = (cudaStream_t)stream;
    ssm::FwdArgs f{};
    f.in = {a->x, a->dt, a->b, a->c, a->z, nullptr, a->a, a->skip, a->dt_bias, a->D, a->S, 0};
    f.h0 = a->initial_state;
    f.y = a->y;
    f.ht = a->final_state;
    f.cut = p.cut;
    f.longest_first = a->cu_seqlens && !p.parts && a->N <= ssm::kMaxOrdered;
    cudaError_t e = cudaSuccess;
    if (p.parts) {
        f.end = (float *)ws;
        f.steps = f.end + ssm::padded(p.states);
        e = ssm::launch_fwd<ssm::kPairs>("ssm_pairs", f, a->dtype, q);
        if (e == cudaSuccess)
            e = ssm::launch_join({a->a, f.steps, a->initial_state, nullptr, f.end, nullptr, nullptr, a->D, a->S, p.cut}, q);
        f.start = f.end;
    }
    if (e == cudaSuccess) e = ssm::launch_fwd<ssm::kOutputs>("ssm_fwd", f, a->dtype, q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "state space scan launch");
}

size_t gdn_ssm_bwd_workspace_size(const gdn_ssm_bwd_args *a) {
    if (!a) {
        fail(GDN_ERR_INVALID_ARG, "null args");
        return 0;
    }
    if (ssm::check(a->B, a->T, a->D, a->S, a->N, a->dtype, a->cu_seqlens != nullptr) != GDN_OK) return 0;
    return ssm::asked_for(ssm::bwd_bytes(ssm::plan_of(a)));
}

gdn_status gdn_ssm_bwd(const gdn_ssm_bwd_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = ssm::check(a->B, a->T, a->D, a->S, a->N, a->dtype, a->cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (!a->a || !a->da ||
        (a->T > 0 && (!a->d_y || !a->x || !a->dt || !a->b || !a->c || !a->dx || !a->ddt || !a->db || !a->dc ||
                      (a->z && !a->dz))))
        return fail(GDN_ERR_INVALID_ARG, "d_y, x, dt, a, b, c, dx, ddt, da, db, dc and (with z) dz are required");
    if (misaligned(a->d_y) || misaligned(a->x) || misaligned(a->dt) || misaligned(a->a) || misaligned(a->b) ||
        misaligned(a->c) || misaligned(a->skip) || misaligned(a->z) || misaligned(a->dt_bias) ||
        misaligned(a->initial_state) || misaligned(a->cu_seqlens) || misaligned(a->d_final_state) ||
        misaligned(a->dx) || misaligned(a->ddt) || misaligned(a->da) || misaligned(a->db) || misaligned(a->dc) ||
        misaligned(a->dskip) || misaligned(a->dz) || misaligned(a->ddt_bias) || misaligned(a->d_initial_state))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    ssm::BwdPlan p = ssm::plan_of(a);
    const size_t need = ssm::bwd_bytes(p);
    if (!ws || misaligned(ws) || ws_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    p.cut.status = dev.status;
    cudaStream_t q = (cudaStream_t)stream;
    ssm::FwdArgs f{};
    f.in = {a->x, a->dt, a->b, a->c, a->z, a->d_y, a->a, a->skip, a->dt_bias, a->D, a->S, 0};
    f.cut = p.cut;
    f.end = (float *)ws;
    f.back = f.end + ssm::padded(p.states);
    f.steps = f.back + ssm::padded(p.states);
    cudaError_t e = ssm::launch_fwd<ssm::kBothPairs>("ssm_bwd_pairs", f, a->dtype, q);
    if (e == cudaSuccess)
        e = ssm::launch_join({a->a, f.steps, a->initial_state, a->d_final_state, f.end, f.back, a->d_initial_state,
                              a->D, a->S, p.cut}, q);
    ssm::BwdArgs b{};
    b.in = f.in;
    b.start = f.end;
    b.behind = f.back;
    b.dx = a->dx, b.ddt = a->ddt, b.dz = a->dz, b.db = a->db, b.dc = a->dc;
    float *rows = f.steps + ssm::padded(p.rows);
    const bool skip = a->skip && a->dskip, bias = a->dt_bias && a->ddt_bias;
    b.dskip = skip ? rows : nullptr;
    b.dbias = bias ? rows + ssm::padded(p.rows) : nullptr;
    b.dbc = rows + 2 * ssm::padded(p.rows);
    b.tokens = (long long)a->B * a->T;
    b.lanes = p.lanes;
    b.cut = p.cut;
    if (e == cudaSuccess)
        e = a->dtype == GDN_BF16 ? ssm::launch_bwd<__nv_bfloat16>(b, q) : ssm::launch_bwd<float>(b, q);
    if (e == cudaSuccess) e = column_sum(b.start, p.cut.slots, a->D * a->S, a->da, q);
    if (e == cudaSuccess && skip) e = column_sum(b.dskip, p.cut.slots, a->D, a->dskip, q);
    if (e == cudaSuccess && bias) e = column_sum(b.dbias, p.cut.slots, a->D, a->ddt_bias, q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "state space scan backward launch");
}

gdn_status gdn_ssm_step(const gdn_ssm_step_args *a, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    if (a->N < 0) return fail(GDN_ERR_INVALID_ARG, "bad sizes N=%d D=%d S=%d", a->N, a->D, a->S);
    gdn_status st = ssm::check(1, 1, a->D, a->S, 1, a->dtype, false);
    if (st != GDN_OK) return st;
    if (a->N > (1 << 30)) return fail(GDN_ERR_INVALID_ARG, "problem too large");
    if (a->N == 0) return GDN_OK;
    if (!a->x || !a->dt || !a->a || !a->b || !a->c || !a->state || !a->y || !a->out_state)
        return fail(GDN_ERR_INVALID_ARG, "x, dt, a, b, c, state, y and out_state are required");
    if (misaligned(a->x) || misaligned(a->dt) || misaligned(a->a) || misaligned(a->b) || misaligned(a->c) ||
        misaligned(a->skip) || misaligned(a->z) || misaligned(a->dt_bias) || misaligned(a->state) ||
        misaligned(a->y) || misaligned(a->out_state))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    if (shifted(a->state, a->out_state, (size_t)a->N * a->D * a->S * 4))
        return fail(GDN_ERR_INVALID_ARG, "out_state overlaps state without being it");
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    cudaStream_t q = (cudaStream_t)stream;
    ssm::StepArgs s{{a->x, a->dt, a->b, a->c, a->z, nullptr, a->a, a->skip, a->dt_bias, a->D, a->S, 0},
                    a->state, a->y, a->out_state, a->N};
    prof_before("ssm_step", q);
    const cudaError_t e = ssm::by_type(a->dtype, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return ssm::by_lanes<16>(ssm::lanes_of(a->S, 4), [&](auto lp) {
            constexpr int LP = decltype(lp)::value, rows = ssm::kThreads / LP;
            const int across = (a->D + rows - 1) / rows, down = std::min(a->N, std::max(1, 16 * dev.sms / across));
            return launch_pdl(ssm::step_kernel<T, LP>, dim3(across, down), dim3(ssm::kThreads), 0, q, s);
        });
    });
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "state space step launch");
}

}  // extern "C"
