// gdn_conv.cu -- short causal convolution along the tokens, per channel, with its
// activation; its backward pass and its one-token step.
//
//     pre_t = bias + sum_k w_k xp_{t + k},  y = act(pre);  xp = the W - 1 inputs before, then x
//
// A thread carries VEC neighbouring channels down a run of tokens with the last W - 1 inputs in
// registers, so that each input is read once (and W - 1 more for each run).  The tokens are taken
// as one long row: where a sequence begins, the registers are filled from its initial state.
#include <algorithm>
#include <type_traits>

#include "gdn_layer_internal.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace conv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTaps = 4;

struct FwdArgs {
    const void *x, *w, *bias, *h0;
    void *y, *ht;
    Seqs s;
    long long tokens;
    int D, run, runs;              // tokens of a run, runs; the CTAs behind them write final states
    int *status;
};

// Inputs xp of the W - 1 places ahead of token t, which is the local-th of sequence n: hist[0] is
// the oldest.  Nothing outside x and h0 is read whatever cu holds.
template <typename T, int VEC, int W>
__device__ __forceinline__ void history(const T *x, const T *h0, long long t, long long local, int n, int D, int ch,
                                        float (&hist)[W - 1][VEC]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const long long back = W - 1 - k;             // tokens before t
        if (local >= back && t >= back) {
            Vec<T, VEC>::load(x + (t - back) * D + ch, hist[k]);
        } else if (h0 && local >= 0 && local < back) {
            Vec<T, VEC>::load(h0 + ((long long)n * (W - 1) + (k + local)) * D + ch, hist[k]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) hist[k][i] = 0.f;
        }
    }
}

// Weights and bias of VEC channels.
template <typename T, int VEC, int W>
__device__ __forceinline__ void weights(const T *w, const T *bias, int ch, float (&wt)[W][VEC], float (&b)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) wt[k][i] = to_f(w[(long long)(ch + i) * W + k]);
        b[i] = bias ? to_f(bias[ch + i]) : 0.f;
    }
}

template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) fwd_kernel(FwdArgs a) {
    pdl_enter();
    constexpr int kAhead = VEC >= 8 ? 4 : 8;          // tokens whose loads are in flight
    const T *x = (const T *)a.x, *h0 = (const T *)a.h0;
    T *y = (T *)a.y, *ht = (T *)a.ht;
    const int ch = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    if (ch >= a.D) return;
    const long long item = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (item >= a.runs) {
        // the last W - 1 inputs of a sequence's state and tokens, and the check of its range
        const long long seq = item - a.runs;
        if (seq >= a.s.N) return;
        const int n = (int)seq;
        long long bos, len;
        const bool good = seq_tokens(a.s, n, bos, len);
        if (!good && ch == 0) set_status(a.status, GDN_ERR_BAD_SEQLENS);
        if (!ht) return;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const long long at = len + j;             // in the W - 1 + len inputs
            float v[VEC];
            if (at >= W - 1) {
                Vec<T, VEC>::load(x + (bos + at - (W - 1)) * a.D + ch, v);
            } else if (h0) {
                Vec<T, VEC>::load(h0 + ((long long)n * (W - 1) + at) * a.D + ch, v);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[i] = 0.f;
            }
            Vec<T, VEC>::store(ht + ((long long)n * (W - 1) + j) * a.D + ch, v);
        }
        return;
    }
    const long long t0 = item * a.run, t1 = min(t0 + a.run, a.tokens);
    float wt[W][VEC], b[VEC], hist[W - 1][VEC];
    weights<T, VEC, W>((const T *)a.w, (const T *)a.bias, ch, wt, b);
    int n = seq_of(a.s, t0);
    long long bos, len;
    bool good = seq_tokens(a.s, n, bos, len);
    history<T, VEC, W>(x, h0, t0, t0 - bos, n, a.D, ch, hist);
    for (long long t = t0; t < t1; t += kAhead) {
        typename Vec<T, VEC>::Raw raw[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (t + j < t1) raw[j] = Vec<T, VEC>::raw(x + (t + j) * a.D + ch);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (t + j >= t1) break;
            if (t + j >= bos + len && n + 1 < a.s.N) {
                // past the sequence: the one that holds the token, its inputs from the state
                n = seq_of(a.s, t + j);
                good = seq_tokens(a.s, n, bos, len);
                history<T, VEC, W>(x, h0, t + j, t + j - bos, n, a.D, ch, hist);
            }
            float v[VEC], pre[VEC];
            Vec<T, VEC>::get(raw[j], v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float p = b[i];
#pragma unroll
                for (int k = 0; k < W - 1; ++k) p += wt[k][i] * hist[k][i];
                p += wt[W - 1][i] * v[i];
#pragma unroll
                for (int k = 0; k + 1 < W - 1; ++k) hist[k][i] = hist[k + 1][i];
                hist[W - 2][i] = v[i];
                pre[i] = SILU ? p * logistic<T>(p) : p;
            }
            if (good) Vec<T, VEC>::store(y + (t + j) * a.D + ch, pre);
        }
    }
}

struct BwdArgs {
    const void *dy, *x, *w, *bias, *h0, *dht;
    void *dx, *dh0;
    float *partial;                // [runs][D][W], then [runs][D]: each run's dweight and dbias
    Seqs s;
    long long tokens;
    int D, run, runs;
    int *status;
};

// The gradient before the activation, from the inputs under the taps.
template <typename T, int VEC, int W, bool SILU>
__device__ __forceinline__ void before_activation(const float (&wt)[W][VEC], const float (&b)[VEC],
                                                  const float (&hist)[W - 1][VEC], const float (&x)[VEC],
                                                  float (&g)[VEC]) {
    if (!SILU) return;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float p = b[i];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) p += wt[k][i] * hist[k][i];
        p += wt[W - 1][i] * x[i];
        g[i] *= silu_slope(p, logistic<T>(p));
    }
}

// Token t is tap W - 1 - j of token t + j: its gradient gathers, in acc[j], what the tokens up to
// now have given, and leaves when the W - 1 tokens behind it (fewer at a sequence's end) are done.
template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) bwd_kernel(BwdArgs a) {
    pdl_enter();
    constexpr int kAhead = 4;
    const T *x = (const T *)a.x, *h0 = (const T *)a.h0, *dy = (const T *)a.dy, *dht = (const T *)a.dht;
    T *dx = (T *)a.dx, *dh0 = (T *)a.dh0;
    const int ch = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    if (ch >= a.D) return;
    const long long item = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    float wt[W][VEC], b[VEC], hist[W - 1][VEC];
    if (item >= a.runs) {
        const long long seq = item - a.runs;
        if (seq >= a.s.N) return;
        const int n = (int)seq;
        long long bos, len;
        const bool good = seq_tokens(a.s, n, bos, len);
        if (!good && ch == 0) set_status(a.status, GDN_ERR_BAD_SEQLENS);
        if (!dh0) return;
        // row j of the state is tap k of token j - k
        weights<T, VEC, W>((const T *)a.w, (const T *)a.bias, ch, wt, b);
        float d[W - 1][VEC];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) d[j][i] = 0.f;
            if (dht && j >= len) Vec<T, VEC>::load(dht + ((long long)n * (W - 1) + (j - len)) * a.D + ch, d[j]);
        }
        history<T, VEC, W>(x, h0, bos, 0, n, a.D, ch, hist);
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {
            if (t >= len) break;
            float v[VEC], g[VEC];
            Vec<T, VEC>::load(x + (bos + t) * a.D + ch, v);
            Vec<T, VEC>::load(dy + (bos + t) * a.D + ch, g);
            before_activation<T, VEC, W, SILU>(wt, b, hist, v, g);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
#pragma unroll
                for (int j = t; j < W - 1; ++j) d[j][i] += wt[j - t][i] * g[i];
#pragma unroll
                for (int k = 0; k + 1 < W - 1; ++k) hist[k][i] = hist[k + 1][i];
                hist[W - 2][i] = v[i];
            }
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) Vec<T, VEC>::store(dh0 + ((long long)n * (W - 1) + j) * a.D + ch, d[j]);
        return;
    }
    const long long t0 = item * a.run, t1 = min(t0 + a.run, a.tokens);
    const long long t2 = min(t1 + W - 1, a.tokens);    // the tokens behind the run give to it too
    weights<T, VEC, W>((const T *)a.w, (const T *)a.bias, ch, wt, b);
    float acc[W][VEC], dw[W][VEC], db[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) acc[k][i] = dw[k][i] = 0.f;
    }
    int n = seq_of(a.s, t0);
    long long bos, len;
    bool good = seq_tokens(a.s, n, bos, len);
    unsigned fine = 0;                                 // bit j: token t - j is one of an intact range
    history<T, VEC, W>(x, h0, t0, t0 - bos, n, a.D, ch, hist);
    for (long long t = t0; t < t1 + W - 1; t += kAhead) {
        typename Vec<T, VEC>::Raw rx[kAhead], rg[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (t + j < t2) {
                rx[j] = Vec<T, VEC>::raw(x + (t + j) * a.D + ch);
                rg[j] = Vec<T, VEC>::raw(dy + (t + j) * a.D + ch);
            }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const long long now = t + j;
            if (now >= t1 + W - 1) break;
            if (now < t2) {
                if (now >= bos + len && n + 1 < a.s.N) {
                    n = seq_of(a.s, now);
                    good = seq_tokens(a.s, n, bos, len);
                    history<T, VEC, W>(x, h0, now, now - bos, n, a.D, ch, hist);
                }
                const long long local = now - bos, tail = local + (W - 1) - len;
                float v[VEC], g[VEC];
                Vec<T, VEC>::get(rx[j], v);
                Vec<T, VEC>::get(rg[j], g);
                before_activation<T, VEC, W, SILU>(wt, b, hist, v, g);
                if (dht && good && tail >= 0 && tail < W - 1)
                    Vec<T, VEC>::load(dht + ((long long)n * (W - 1) + tail) * a.D + ch, acc[0]);
                if (good) {
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        if (local < k) break;          // token t - k is of the sequence before
#pragma unroll
                        for (int i = 0; i < VEC; ++i) acc[k][i] += wt[W - 1 - k][i] * g[i];
                    }
                    if (now < t1) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            db[i] += g[i];
#pragma unroll
                            for (int k = 0; k < W - 1; ++k) dw[k][i] += g[i] * hist[k][i];
                            dw[W - 1][i] += g[i] * v[i];
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
#pragma unroll
                    for (int k = 0; k + 1 < W - 1; ++k) hist[k][i] = hist[k + 1][i];
                    hist[W - 2][i] = v[i];
                }
            }
            fine = fine << 1 | (good ? 1u : 0u);
            const long long done = now - (W - 1);
            if (done >= t0 && (fine >> (W - 1) & 1)) Vec<T, VEC>::store(dx + done * a.D + ch, acc[W - 1]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
#pragma unroll
                for (int k = W - 1; k > 0; --k) acc[k][i] = acc[k - 1][i];
                acc[0][i] = 0.f;
            }
        }
    }
    float *pw = a.partial + (item * a.D + ch) * W, *pb = a.partial + (long long)a.runs * a.D * W + item * a.D + ch;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) pw[i * W + k] = dw[k][i];
        pb[i] = db[i];
    }
}

template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) step_kernel(const T *x, const T *w, const T *bias, const T *state, T *y,
                                                        T *out, int N, int D) {
    pdl_enter();
    const int ch = (blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (ch >= D) return;
    float wt[W][VEC], b[VEC];
    weights<T, VEC, W>(w, bias, ch, wt, b);
    for (long long n = (long long)blockIdx.y * blockDim.y + threadIdx.y; n < N; n += gridDim.y * blockDim.y) {
        float v[W][VEC], r[VEC];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) Vec<T, VEC>::load(state + (n * (W - 1) + k) * D + ch, v[k]);
        Vec<T, VEC>::load(x + n * D + ch, v[W - 1]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float p = b[i];
#pragma unroll
            for (int k = 0; k < W; ++k) p += wt[k][i] * v[k][i];
            r[i] = SILU ? p * logistic<T>(p) : p;
        }
        Vec<T, VEC>::store(y + n * D + ch, r);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) Vec<T, VEC>::store(out + (n * (W - 1) + k) * D + ch, v[k + 1]);
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

constexpr int kFwdRun = 32;
// Runs of the backward pass, each of which leaves a row of partial sums: as many as fill the GPU
// (its SM count enters the workspace's size, which is asked for without a device, so that of the
// largest part is taken), of 16 tokens at least.
constexpr int kSms = 160;
int bwd_run(long long tokens, int D, int vec) {
    const Block b = block_of(D, vec);
    const long long runs = std::max<long long>(1, (long long)kSms * 4 * b.threads.y / b.across);
    return (int)std::max<long long>(16, (tokens + runs - 1) / runs);
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
    f.run = kFwdRun;
    f.runs = (int)((f.tokens + f.run - 1) / f.run);
    // the final states' items follow the runs; without tokens only they are there
    const long long items = (long long)f.runs + f.s.N;
    return pick(W, activation, [&](auto w, auto silu) {
        prof_before("conv_fwd", q);
        const cudaError_t e = launch_pdl(fwd_kernel<T, VEC, decltype(w)::value, decltype(silu)::value>,
                                         dim3((unsigned)((items + b.threads.y - 1) / b.threads.y), b.across), b.threads,
                                         0, q, f);
        prof_after(q);
        return e;
    });
}

template <typename T, int VEC>
cudaError_t run_bwd(BwdArgs g, int W, int activation, float *dweight, float *dbias, cudaStream_t q) {
    const Block b = block_of(g.D, VEC);
    const long long items = (long long)g.runs + g.s.N;
    cudaError_t e = pick(W, activation, [&](auto w, auto silu) {
        prof_before("conv_bwd", q);
        const cudaError_t r = launch_pdl(bwd_kernel<T, VEC, decltype(w)::value, decltype(silu)::value>,
                                         dim3((unsigned)((items + b.threads.y - 1) / b.threads.y), b.across), b.threads,
                                         0, q, g);
        prof_after(q);
        return r;
    });
    if (e == cudaSuccess) e = column_sum(g.partial, g.runs, g.D * W, dweight, q);
    if (e == cudaSuccess && dbias)
        e = column_sum(g.partial + (long long)g.runs * g.D * W, g.runs, g.D, dbias, q);
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

// Channels to a thread of the three passes: 16 bytes, and four in the backward pass, which holds
// some 20 numbers for each.
int fwd_vec(int dtype, int D) { return vec_of(D, dtype == GDN_BF16 ? 8 : 4); }
int bwd_vec(int D) { return vec_of(D, 4); }

long long tokens_of(int B, int T) { return (long long)B * T; }

int bwd_runs(const gdn_conv_bwd_args *a) {
    const long long tokens = tokens_of(a->B, a->T), run = bwd_run(tokens, a->D, bwd_vec(a->D));
    return (int)((tokens + run - 1) / run);
}

// f.template operator()<T, VEC>() for the type and the channels to a thread.
template <typename F>
cudaError_t by_type(int dtype, int vec, F f) {
    using bf16 = __nv_bfloat16;
    if (dtype == GDN_BF16) switch (vec) {
            case 8: return f((bf16 *)nullptr, std::integral_constant<int, 8>());
            case 4: return f((bf16 *)nullptr, std::integral_constant<int, 4>());
            case 2: return f((bf16 *)nullptr, std::integral_constant<int, 2>());
            default: return f((bf16 *)nullptr, std::integral_constant<int, 1>());
        }
    switch (vec) {
        case 4: return f((float *)nullptr, std::integral_constant<int, 4>());
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
    const long long tokens = conv::tokens_of(a->B, a->T);
    const int vec = conv::bwd_vec(a->D);
    const conv::BwdArgs b{a->d_y, a->x, a->weight, a->bias, a->initial_state, a->d_final_state, a->dx,
                          a->d_initial_state, (float *)ws, {a->cu_seqlens, a->T, a->cu_seqlens ? a->N : a->B}, tokens,
                          a->D, conv::bwd_run(tokens, a->D, vec), conv::bwd_runs(a), dev.status};
    const cudaError_t e = conv::by_type(a->dtype, vec, [&](auto *t, auto v) {
        return conv::run_bwd<std::remove_pointer_t<decltype(t)>, std::min(4, decltype(v)::value)>(
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
