// gdn_conv.cu -- short causal convolution along the tokens, per channel, with its
// activation; its backward pass and its one-token step.
//
//     pre_t = bias + sum_k w_k xp_{t + k},  y = act(pre);  xp = the W - 1 inputs before, then x
//
// A thread carries VEC neighbouring channels down a run of tokens with the last W - 1 inputs in
// registers, so that each input is read once (and W - 1 more for each run).  The tokens are taken
// as one long row: where a sequence begins, the registers are filled from its initial state.
// Bound by memory: 16 x (512 .. 8192) tokens x 4096 bf16 forward 176 us, 97% of the measured copy
// rate; 4 x 4096 x 4096 backward 94 us, 64%, with 16 warps to an SM that fill 55% of the issue slots.  Of
// few channels the backward pass is held up by the sums over its many runs (2^20 x 16 94 us, 15 of bytes).
#include <algorithm>
#include <type_traits>

#include "gdn_layer_internal.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace conv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTaps = 4;

// VEC neighbouring channels as pairs, for arithmetic on two numbers at once (of a single channel the
// second of the pair is not there).
template <int VEC>
constexpr int kPairs = VEC > 1 ? VEC / 2 : 1;
template <typename T, int VEC>
__device__ __forceinline__ void get(const typename Vec<T, VEC>::Raw &r, float2 (&v)[kPairs<VEC>]) {
    float f[VEC];
    Vec<T, VEC>::get(r, f);
#pragma unroll
    for (int i = 0; i < kPairs<VEC>; ++i) v[i] = make_float2(f[2 * i], VEC > 1 ? f[2 * i + (VEC > 1)] : 0.f);
}
template <typename T, int VEC>
__device__ __forceinline__ void load(const T *p, float2 (&v)[kPairs<VEC>]) {
    get<T, VEC>(Vec<T, VEC>::raw(p), v);
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T *p, const float2 (&v)[kPairs<VEC>]) {
    float f[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = i & 1 ? v[i / 2].y : v[i / 2].x;
    Vec<T, VEC>::store(p, f);
}
template <int P>
__device__ __forceinline__ void clear(float2 (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = make_float2(0.f, 0.f);
}
// A thread's own loads, GROUPS groups of kAhead tokens of N tensors in flight, by cp.async to shared
// memory: in registers there is no room for enough of them (16 x (512 .. 8192) x 4096 bf16 forward 200
// us from registers, 176 so; backward of 4 x 4096 x 4096 110, 97).  Only the thread that asked reads
// them, so that no barrier is needed.
constexpr int kAhead = 4;
template <typename T, int VEC, int N, int GROUPS>
struct Ahead {
    using Raw = typename Vec<T, VEC>::Raw;
    static constexpr int kSlots = GROUPS + 1;          // one is being read
    Raw (*slot)[kAhead][N][kThreads];
    int asked, taken;
    static constexpr size_t kBytes = sizeof(Raw) * kSlots * kAhead * N * kThreads;

    __device__ __forceinline__ explicit Ahead(uint8_t *shared)
        : slot(reinterpret_cast<Raw(*)[kAhead][N][kThreads]>(shared)), asked(0), taken(0) {}
    // A group: tokens from `t` on that are below `end`, of each tensor from p[i] on.
    __device__ __forceinline__ void ask(const T *const (&&p)[N], int t, int end, long long D) {
        const int me = threadIdx.y * blockDim.x + threadIdx.x;
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (t + j < end)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    Raw *to = &slot[asked][j][i][me];
                    if constexpr (sizeof(Raw) >= 4)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                                         (uint32_t)__cvta_generic_to_shared(to)),
                                     "l"(p[i] + j * D), "n"((int)sizeof(Raw))
                                     : "memory");
                    else *to = Vec<T, VEC>::raw(p[i] + j * D);
                }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++asked == kSlots) asked = 0;
    }
    // The oldest group.
    __device__ __forceinline__ void take(Raw (&r)[kAhead][N]) {
        const int me = threadIdx.y * blockDim.x + threadIdx.x;
        asm volatile("cp.async.wait_group %0;" ::"n"(GROUPS - 1) : "memory");
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) r[j][i] = slot[taken][j][i][me];
        if (++taken == kSlots) taken = 0;
    }
};
template <typename T, int VEC>
using FwdAhead = Ahead<T, VEC, 1, 4>;
template <typename T, int VEC>
using BwdAhead = Ahead<T, VEC, 2, 5>;

struct FwdArgs {
    const void *x, *w, *bias, *h0;
    void *y, *ht;
    Seqs s;
    int tokens, D, run, runs;      // tokens of a run, runs; the items ahead of them write final states
    int *status;
};

// A thread's channels down a run of tokens: the sequence they are in, and its last W - 1 inputs.
template <typename T, int VEC, int W>
struct Walk {
    static constexpr int P = kPairs<VEC>;
    const T *x, *h0;
    const Seqs &s;
    int D, ch;
    int n, bos, end;               // the sequence and its tokens
    bool good;
    float2 hist[W - 1][P];         // the oldest first

    // Inputs of the W - 1 places ahead of token t.  Nothing outside x and h0 is read whatever cu holds.
    __device__ __forceinline__ void enter(int t) {
        n = seq_of(s, t);
        long long b, len;
        good = seq_tokens(s, n, b, len);
        bos = (int)b;
        end = (int)(b + len);
        fill(t);
    }
    __device__ __forceinline__ void fill(int t) {
        const int local = t - bos;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int back = W - 1 - k;               // tokens before t
            if (local >= back && t >= back) load<T, VEC>(x + (long long)(t - back) * D + ch, hist[k]);
            else if (h0 && local >= 0 && local < back)
                load<T, VEC>(h0 + ((long long)n * (W - 1) + (k + local)) * D + ch, hist[k]);
            else clear(hist[k]);
        }
    }
    // Before token t: into its sequence, if it is not this one's (behind the last one there is none).
    __device__ __forceinline__ void reach(int t) {
        if (t >= end && n + 1 < s.N) enter(t);
    }
    __device__ __forceinline__ void push(const float2 (&v)[P]) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k) hist[k][i] = hist[k + 1][i];
            hist[W - 2][i] = v[i];
        }
    }
};

// Weights and bias of VEC channels: VEC W neighbouring elements, in loads of up to 16 bytes.
template <typename T, int VEC, int W>
struct Taps {
    static constexpr int P = kPairs<VEC>, kBytes = VEC * W * (int)sizeof(T);
    static constexpr int kLoad = (kBytes & -kBytes) < 16 ? (kBytes & -kBytes) : 16;
    float2 w[W][P], b[P];
    __device__ __forceinline__ Taps(const void *weight, const void *bias, int ch) {
        using Raw = typename RawBytes<kLoad>::type;
        Raw raw[kBytes / kLoad];
#pragma unroll
        for (int i = 0; i < kBytes / kLoad; ++i) raw[i] = reinterpret_cast<const Raw *>((const T *)weight + (long long)ch * W)[i];
        const T *e = reinterpret_cast<const T *>(raw);
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int k = 0; k < W; ++k)
                w[k][i] = make_float2(to_f(e[2 * i * W + k]), VEC > 1 ? to_f(e[(2 * i + (VEC > 1)) * W + k]) : 0.f);
        if (bias) load<T, VEC>((const T *)bias + ch, b);
        else clear(b);
    }
    // Before the activation; v is the token's own input.
    __device__ __forceinline__ float2 pre(const float2 (&hist)[W - 1][P], const float2 (&v)[P], int i) const {
        float2 p = b[i];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) p = __ffma2_rn(w[k][i], hist[k][i], p);
        return __ffma2_rn(w[W - 1][i], v[i], p);
    }
};

template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, 3) fwd_kernel(FwdArgs a) {
    pdl_enter();
    constexpr int P = kPairs<VEC>;
    using Raw = typename Vec<T, VEC>::Raw;
    extern __shared__ __align__(16) uint8_t shared[];
    const int ch = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    if (ch >= a.D) return;
    int item = blockIdx.x * blockDim.y + threadIdx.y;
    Walk<T, VEC, W> walk{(const T *)a.x, (const T *)a.h0, a.s, a.D, ch};
    if (item < a.s.N) {
        // the last W - 1 inputs of a sequence's state and tokens, and the check of its range
        const int n = item;
        long long bos, len;
        const bool good = seq_tokens(a.s, n, bos, len);
        if (!good && ch == 0) set_status(a.status, GDN_ERR_BAD_SEQLENS);
        if (!a.ht) return;
        walk.n = n, walk.bos = (int)bos;
        walk.fill((int)(bos + len));
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store<T, VEC>((T *)a.ht + ((long long)n * (W - 1) + j) * a.D + ch, walk.hist[j]);
        return;
    }
    item -= a.s.N;
    if (item >= a.runs) return;
    const int t0 = item * a.run, t1 = min(t0 + a.run, a.tokens);
    const T *x = (const T *)a.x + (long long)t0 * a.D + ch;
    T *y = (T *)a.y + (long long)t0 * a.D + ch;
    FwdAhead<T, VEC> ahead(shared);
    const long long D = a.D;
    int asked = t0;
    const auto ask = [&] {
        ahead.ask({x}, asked, t1, D);
        asked += kAhead;
        x += kAhead * D;
    };
#pragma unroll
    for (int g = 0; g < 4; ++g) ask();
    const Taps<T, VEC, W> taps(a.w, a.bias, ch);
    walk.enter(t0);
    for (int t = t0; t < t1; t += kAhead) {
        Raw raw[kAhead][1];
        ahead.take(raw);
        ask();
        const auto token = [&](int j) {
            float2 v[P], out[P];
            get<T, VEC>(raw[j][0], v);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 p = taps.pre(walk.hist, v, i);
                out[i] = SILU ? __fmul2_rn(p, logistic2<T>(p)) : p;
            }
            walk.push(v);
            if (walk.good) store<T, VEC>(y, out);
            y += a.D;
        };
        if (t + kAhead <= min(t1, walk.end)) {         // all of this sequence
#pragma unroll
            for (int j = 0; j < kAhead; ++j) token(j);
        } else {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (t + j >= t1) break;
                walk.reach(t + j);
                token(j);
            }
        }
    }
}

struct BwdArgs {
    const void *dy, *x, *w, *bias, *h0, *dht;
    void *dx, *dh0;
    float *partial;                // [runs][D][W + 1]: each run's dweight and dbias
    Seqs s;
    int tokens, D, run, runs;
    int *status;
};

// The gradient before the activation, from the inputs under the taps.
template <typename T, bool SILU>
__device__ __forceinline__ float2 before_activation(float2 pre, float2 g) {
    if (!SILU) return g;
    const float2 s = logistic2<T>(pre);
    // s (1 + pre (1 - s))
    const float2 one = make_float2(1.f, 1.f), r = __ffma2_rn(s, make_float2(-1.f, -1.f), one);
    return __fmul2_rn(g, __fmul2_rn(s, __ffma2_rn(pre, r, one)));
}

// Token t is tap W - 1 - j of token t + j: its gradient gathers, in acc[j], what the tokens up to
// now have given, and leaves when the W - 1 tokens behind it (fewer at a sequence's end) are done.
template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, 2) bwd_kernel(BwdArgs a) {
    pdl_enter();
    constexpr int P = kPairs<VEC>;
    using Raw = typename Vec<T, VEC>::Raw;
    extern __shared__ __align__(16) uint8_t shared[];
    const int ch = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    if (ch >= a.D) return;
    int item = blockIdx.x * blockDim.y + threadIdx.y;
    const T *dht = (const T *)a.dht;
    Walk<T, VEC, W> walk{(const T *)a.x, (const T *)a.h0, a.s, a.D, ch};
    if (item < a.s.N) {
        const int n = item;
        long long bos, len;
        const bool good = seq_tokens(a.s, n, bos, len);
        if (!good && ch == 0) set_status(a.status, GDN_ERR_BAD_SEQLENS);
        if (!a.dh0) return;
        // row j of the state is tap k of token j - k
        const Taps<T, VEC, W> taps(a.w, a.bias, ch);
        float2 d[W - 1][P];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            clear(d[j]);
            if (dht && j >= len) load<T, VEC>(dht + ((long long)n * (W - 1) + (j - len)) * a.D + ch, d[j]);
        }
        walk.n = n, walk.bos = (int)bos;
        walk.fill((int)bos);
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {
            if (t >= len) break;
            float2 v[P], g[P];
            load<T, VEC>((const T *)a.x + (bos + t) * a.D + ch, v);
            load<T, VEC>((const T *)a.dy + (bos + t) * a.D + ch, g);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                g[i] = before_activation<T, SILU>(taps.pre(walk.hist, v, i), g[i]);
#pragma unroll
                for (int j = t; j < W - 1; ++j) d[j][i] = __ffma2_rn(taps.w[j - t][i], g[i], d[j][i]);
            }
            walk.push(v);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store<T, VEC>((T *)a.dh0 + ((long long)n * (W - 1) + j) * a.D + ch, d[j]);
        return;
    }
    item -= a.s.N;
    if (item >= a.runs) return;
    const int t0 = item * a.run, t1 = min(t0 + a.run, a.tokens);
    const int t2 = min(t1 + W - 1, a.tokens);          // the tokens behind the run give to it too
    const T *x = (const T *)a.x + (long long)t0 * a.D + ch, *dy = (const T *)a.dy + (long long)t0 * a.D + ch;
    T *dx = (T *)a.dx + ((long long)t0 - (W - 1)) * a.D + ch;
    BwdAhead<T, VEC> ahead(shared);
    const long long D = a.D;
    int asked = t0;
    const auto ask = [&] {
        ahead.ask({x, dy}, asked, t2, D);
        asked += kAhead;
        x += kAhead * D;
        dy += kAhead * D;
    };
#pragma unroll
    for (int g = 0; g < 5; ++g) ask();
    const Taps<T, VEC, W> taps(a.w, a.bias, ch);
    float2 acc[W][P], dw[W][P], db[P];
    clear(db);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        clear(acc[k]);
        clear(dw[k]);
    }
    unsigned fine = 0;                                 // bit j: token t - j is one of an intact range
    walk.enter(t0);
    for (int t = t0; t < t1 + W - 1; t += kAhead) {
        Raw raw[kAhead][2];
        ahead.take(raw);
        ask();
        // INSIDE: of an intact sequence, W - 1 tokens and more from either end of it, and of this run
        const auto token = [&](int j, auto inside) {
            constexpr bool INSIDE = decltype(inside)::value;
            const int now = t + j;
            if (INSIDE || now < t2) {
                if (!INSIDE) walk.reach(now);
                const int local = now - walk.bos, tail = now + (W - 1) - walk.end;
                float2 v[P], g[P];
                get<T, VEC>(raw[j][0], v);
                get<T, VEC>(raw[j][1], g);
                if (!INSIDE && dht && walk.good && tail >= 0 && tail < W - 1)
                    load<T, VEC>(dht + ((long long)walk.n * (W - 1) + tail) * a.D + ch, acc[0]);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    g[i] = before_activation<T, SILU>(taps.pre(walk.hist, v, i), g[i]);
                    if (!INSIDE && !walk.good) g[i] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < W; ++k)        // token t - k may be of the sequence before
                        if (INSIDE || k <= local) acc[k][i] = __ffma2_rn(taps.w[W - 1 - k][i], g[i], acc[k][i]);
                    if (INSIDE || now < t1) {
                        db[i] = __fadd2_rn(db[i], g[i]);
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) dw[k][i] = __ffma2_rn(g[i], walk.hist[k][i], dw[k][i]);
                        dw[W - 1][i] = __ffma2_rn(g[i], v[i], dw[W - 1][i]);
                    }
                }
                walk.push(v);
            }
            if (!INSIDE) fine = fine << 1 | (walk.good ? 1u : 0u);
            if (INSIDE || (now - (W - 1) >= t0 && (fine >> (W - 1) & 1))) store<T, VEC>(dx, acc[W - 1]);
            dx += a.D;
#pragma unroll
            for (int k = W - 1; k > 0; --k)
#pragma unroll
                for (int i = 0; i < P; ++i) acc[k][i] = acc[k - 1][i];
            clear(acc[0]);
        };
        if (walk.good && t >= max(t0, walk.bos) + W - 1 && t + kAhead <= min(t1, walk.end - (W - 1))) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) token(j, std::true_type());
            fine = ~0u;
        } else {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (t + j >= t1 + W - 1) break;
                token(j, std::false_type());
            }
        }
    }
    float *p = a.partial + ((long long)item * a.D + ch) * (W + 1);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) p[i * (W + 1) + k] = i & 1 ? dw[k][i / 2].y : dw[k][i / 2].x;
        p[i * (W + 1) + W] = i & 1 ? db[i / 2].y : db[i / 2].x;
    }
}

// dweight and dbias from the runs' sums, [runs][D][W + 1], in a fixed order.
__global__ void __launch_bounds__(256) sums_kernel(const float *partial, int runs, int D, int W, float *dweight, float *dbias) {
    __shared__ float strip[8][32];
    pdl_enter();
    const int lane = threadIdx.x & 31, strip_no = threadIdx.x >> 5, columns = D * (W + 1);
    const int i = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (i < columns)
        for (int r = strip_no; r < runs; r += 8) t += partial[(long long)r * columns + i];
    strip[strip_no][lane] = t;
    __syncthreads();
    if (strip_no > 0 || i >= columns) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) t += strip[k][lane];
    const int d = i / (W + 1), k = i - d * (W + 1);
    if (k < W) dweight[d * W + k] = t;
    else if (dbias) dbias[d] = t;
}

template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) step_kernel(const T *x, const T *w, const T *bias, const T *state, T *y,
                                                        T *out, int N, int D) {
    pdl_enter();
    const int ch = (blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (ch >= D) return;
    constexpr int P = kPairs<VEC>;
    const Taps<T, VEC, W> taps(w, bias, ch);
    for (long long n = (long long)blockIdx.y * blockDim.y + threadIdx.y; n < N; n += gridDim.y * blockDim.y) {
        float2 hist[W - 1][P], v[P], r[P];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) load<T, VEC>(state + (n * (W - 1) + k) * D + ch, hist[k]);
        load<T, VEC>(x + n * D + ch, v);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 p = taps.pre(hist, v, i);
            r[i] = SILU ? __fmul2_rn(p, logistic2<T>(p)) : p;
        }
        store<T, VEC>(y + n * D + ch, r);
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) store<T, VEC>(out + (n * (W - 1) + k) * D + ch, hist[k + 1]);
        store<T, VEC>(out + (n * (W - 1) + W - 2) * D + ch, v);
    }
}

// CTAs of 256 threads: channels across, as many runs (or sequences) as fit beside them.
struct Block {
    dim3 threads;
    int across;                    // CTAs along the channels
};
Block block_of(int D, int vec) {
    const int chunks = (D + vec - 1) / vec;
    int wide = 1;
    while (wide < kThreads && wide < chunks) wide *= 2;
    return {dim3(wide, kThreads / wide), (chunks + wide - 1) / wide};
}

// Channels to a thread: as many as the rows' alignment allows, `most` at most (a power of two).
int vec_of(int D, int most) {
    int v = most;
    while (D % v != 0) v /= 2;
    return v;
}

// Tokens of a run: as few as keep the GPU's threads (`threads` to an SM) in one wave, but enough that
// the W - 1 inputs read before a run, and its weights, are little beside it.
int run_of(long long tokens, int D, int vec, int threads, int least) {
    const Block b = block_of(D, vec);
    const long long runs = std::max<long long>(1, (long long)kSms * (threads / kThreads) * b.threads.y / b.across);
    return (int)std::max<long long>(least, (tokens + runs - 1) / runs);
}

gdn_status check(int B, int T, int D, int N, int W, int dtype, int activation, bool packed) {
    if (B < 1 || T < 0 || D < 1) return fail(GDN_ERR_INVALID_ARG, "bad sizes B=%d T=%d D=%d", B, T, D);
    if (W < 2 || W > kMaxTaps) return fail(GDN_ERR_UNSUPPORTED, "W = %d (2 to %d)", W, kMaxTaps);
    if (dtype != GDN_FP32 && dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d is not GDN_FP32 or GDN_BF16", dtype);
    if (activation != GDN_ACT_NONE && activation != GDN_ACT_SILU)
        return fail(GDN_ERR_UNSUPPORTED, "activation %d is not GDN_ACT_NONE or GDN_ACT_SILU", activation);
    if (packed && (B != 1 || N < 1))
        return fail(GDN_ERR_INVALID_ARG, "cu_seqlens needs B == 1 and N >= 1 (B=%d N=%d)", B, N);
    if ((long long)B * T >= (1ll << 31) - (1 << 16) || D > (1 << 23) || (packed ? N : B) > (1 << 30))
        return fail(GDN_ERR_INVALID_ARG, "problem too large");
    return GDN_OK;
}

// f(W, SILU) with both as constants.
template <typename F>
cudaError_t pick(int W, int activation, F f) {
    const auto with = [&](auto w) {
        return activation == GDN_ACT_SILU ? f(w, std::true_type()) : f(w, std::false_type());
    };
    switch (W) {
        case 2: return with(std::integral_constant<int, 2>());
        case 3: return with(std::integral_constant<int, 3>());
        default: return with(std::integral_constant<int, 4>());
    }
}

template <typename T, int VEC>
cudaError_t run_fwd(FwdArgs f, int W, int activation, cudaStream_t q) {
    const Block b = block_of(f.D, VEC);
    f.run = run_of(f.tokens, f.D, VEC, 768, 32);
    f.runs = (f.tokens + f.run - 1) / f.run;
    const long long items = (long long)f.runs + f.s.N;
    return pick(W, activation, [&](auto w, auto silu) {
        auto k = fwd_kernel<T, VEC, decltype(w)::value, decltype(silu)::value>;
        constexpr size_t smem = FwdAhead<T, VEC>::kBytes;
        cudaError_t e = allow_smem((const void *)k, smem);
        if (e != cudaSuccess) return e;
        prof_before("conv_fwd", q);
        e = launch_pdl(k, dim3((unsigned)((items + b.threads.y - 1) / b.threads.y), b.across), b.threads, smem, q, f);
        prof_after(q);
        return e;
    });
}

template <typename T, int VEC>
cudaError_t run_bwd(BwdArgs g, int W, int activation, float *dweight, float *dbias, cudaStream_t q) {
    const Block b = block_of(g.D, VEC);
    const long long items = (long long)g.runs + g.s.N;
    cudaError_t e = pick(W, activation, [&](auto w, auto silu) {
        auto k = bwd_kernel<T, VEC, decltype(w)::value, decltype(silu)::value>;
        constexpr size_t smem = BwdAhead<T, VEC>::kBytes;
        cudaError_t r = allow_smem((const void *)k, smem);
        if (r != cudaSuccess) return r;
        prof_before("conv_bwd", q);
        r = launch_pdl(k, dim3((unsigned)((items + b.threads.y - 1) / b.threads.y), b.across), b.threads, smem, q, g);
        prof_after(q);
        return r;
    });
    if (e != cudaSuccess) return e;
    prof_before("conv_sums", q);
    e = launch_pdl(sums_kernel, dim3((unsigned)(((long long)g.D * (W + 1) + 31) / 32)), dim3(256), 0, q, (const float *)g.partial,
                   g.runs, g.D, W, dweight, dbias);
    prof_after(q);
    return e;
}

template <typename T, int VEC>
cudaError_t run_step(const gdn_conv_step_args *a, int sms, cudaStream_t q) {
    const Block b = block_of(a->D, VEC);
    const int down = (int)std::min<long long>((a->N + b.threads.y - 1) / b.threads.y, std::max(1, 16 * sms / b.across));
    return pick(a->W, a->activation, [&](auto w, auto silu) {
        return launch_pdl(step_kernel<T, VEC, decltype(w)::value, decltype(silu)::value>, dim3(b.across, down),
                          b.threads, 0, q, (const T *)a->x, (const T *)a->weight, (const T *)a->bias,
                          (const T *)a->state, (T *)a->y, (T *)a->out_state, a->N, a->D);
    });
}

// Channels to a thread: 8 bytes in the forward pass and of single tokens, 4 (fp32 8) in the backward pass,
// which holds some 20 numbers for each.
int fwd_vec(int dtype, int D) { return vec_of(D, dtype == GDN_BF16 ? 4 : 2); }
int bwd_vec(int D) { return vec_of(D, 2); }

int tokens_of(int B, int T) { return B * T; }

// Runs of the backward pass, each of which leaves a row of partial sums.
int bwd_run(int tokens, int D) { return run_of(tokens, D, bwd_vec(D), 512, 16); }
int bwd_runs(const gdn_conv_bwd_args *a) {
    const int tokens = tokens_of(a->B, a->T), run = bwd_run(tokens, a->D);
    return (int)(((long long)tokens + run - 1) / run);
}

// f(type, VEC) with both as types.
template <typename F>
cudaError_t by_type(int dtype, int vec, F f) {
    using bf16 = __nv_bfloat16;
    if (dtype == GDN_BF16) switch (vec) {
            case 4: return f((bf16 *)nullptr, std::integral_constant<int, 4>());
            case 2: return f((bf16 *)nullptr, std::integral_constant<int, 2>());
            default: return f((bf16 *)nullptr, std::integral_constant<int, 1>());
        }
    switch (vec) {
        case 2: return f((float *)nullptr, std::integral_constant<int, 2>());
        default: return f((float *)nullptr, std::integral_constant<int, 1>());
    }
}

}  // namespace
}  // namespace conv
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_conv_fwd(const gdn_conv_fwd_args *a, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = conv::check(a->B, a->T, a->D, a->N, a->W, a->dtype, a->activation, a->cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (!a->weight || (a->T > 0 && (!a->x || !a->y))) return fail(GDN_ERR_INVALID_ARG, "x, weight and y are required");
    if (misaligned(a->x) || misaligned(a->weight) || misaligned(a->bias) || misaligned(a->initial_state) ||
        misaligned(a->cu_seqlens) || misaligned(a->y) || misaligned(a->final_state))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    const conv::FwdArgs f{a->x, a->weight, a->bias, a->initial_state, a->y, a->final_state,
                          {a->cu_seqlens, a->T, a->cu_seqlens ? a->N : a->B}, conv::tokens_of(a->B, a->T), a->D, 0, 0,
                          dev.status};
    const cudaError_t e = conv::by_type(a->dtype, conv::fwd_vec(a->dtype, a->D), [&](auto *t, auto vec) {
        return conv::run_fwd<std::remove_pointer_t<decltype(t)>, decltype(vec)::value>(f, a->W, a->activation,
                                                                                       (cudaStream_t)stream);
    });
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "convolution launch");
}

size_t gdn_conv_bwd_workspace_size(const gdn_conv_bwd_args *a) {
    if (!a) {
        fail(GDN_ERR_INVALID_ARG, "null args");
        return 0;
    }
    if (conv::check(a->B, a->T, a->D, a->N, a->W, a->dtype, a->activation, a->cu_seqlens != nullptr) != GDN_OK)
        return 0;
    const size_t need = (size_t)conv::bwd_runs(a) * a->D * (a->W + 1) * sizeof(float);
    return need == 0 ? 256 : std::max<size_t>(512, need);
}

gdn_status gdn_conv_bwd(const gdn_conv_bwd_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    gdn_status st = conv::check(a->B, a->T, a->D, a->N, a->W, a->dtype, a->activation, a->cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (!a->weight || !a->dweight || (a->T > 0 && (!a->d_y || !a->x || !a->dx)))
        return fail(GDN_ERR_INVALID_ARG, "d_y, x, weight, dx and dweight are required");
    if (misaligned(a->d_y) || misaligned(a->x) || misaligned(a->weight) || misaligned(a->bias) ||
        misaligned(a->initial_state) || misaligned(a->cu_seqlens) || misaligned(a->d_final_state) ||
        misaligned(a->dx) || misaligned(a->dweight) || misaligned(a->dbias) || misaligned(a->d_initial_state))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    const size_t need = gdn_conv_bwd_workspace_size(a);
    if (need > 256 && (!ws || misaligned(ws) || ws_bytes < need))
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    const int tokens = conv::tokens_of(a->B, a->T), vec = conv::bwd_vec(a->D);
    const conv::BwdArgs b{a->d_y, a->x, a->weight, a->bias, a->initial_state, a->d_final_state, a->dx,
                          a->d_initial_state, (float *)ws, {a->cu_seqlens, a->T, a->cu_seqlens ? a->N : a->B}, tokens,
                          a->D, conv::bwd_run(tokens, a->D), conv::bwd_runs(a), dev.status};
    const cudaError_t e = conv::by_type(a->dtype, vec, [&](auto *t, auto v) {
        return conv::run_bwd<std::remove_pointer_t<decltype(t)>, std::min(2, decltype(v)::value)>(
            b, a->W, a->activation, a->dweight, a->dbias, (cudaStream_t)stream);
    });
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "convolution backward launch");
}

gdn_status gdn_conv_step(const gdn_conv_step_args *a, void *stream) {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "null args");
    if (a->N < 0) return fail(GDN_ERR_INVALID_ARG, "bad sizes N=%d D=%d", a->N, a->D);
    gdn_status st = conv::check(1, 1, a->D, a->N, a->W, a->dtype, a->activation, false);
    if (st != GDN_OK) return st;
    if (a->N == 0) return GDN_OK;
    if (!a->x || !a->weight || !a->state || !a->y || !a->out_state)
        return fail(GDN_ERR_INVALID_ARG, "x, weight, state, y and out_state are required");
    if (misaligned(a->x) || misaligned(a->weight) || misaligned(a->bias) || misaligned(a->state) ||
        misaligned(a->y) || misaligned(a->out_state))
        return fail(GDN_ERR_INVALID_ARG, "every tensor must be 16-byte aligned");
    if (shifted(a->state, a->out_state, (size_t)a->N * (a->W - 1) * a->D * (a->dtype == GDN_BF16 ? 2 : 4)))
        return fail(GDN_ERR_INVALID_ARG, "out_state overlaps state without being it");
    LayerDevice dev;
    if ((st = layer_device(&dev)) != GDN_OK) return st;
    cudaStream_t q = (cudaStream_t)stream;
    prof_before("conv_step", q);
    const cudaError_t e = conv::by_type(a->dtype, conv::fwd_vec(a->dtype, a->D), [&](auto *t, auto v) {
        return conv::run_step<std::remove_pointer_t<decltype(t)>, decltype(v)::value>(a, dev.sms, q);
    });
    prof_after(q);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "convolution step launch");
}

}  // extern "C"
