// The block's short causal convolution ("xLSTM: Extended Long Short-Term Memory"
// section 2.4, Figure 10: a depthwise convolution of width 4 in front of the
// cell, with the Swish activation), for prompts, single tokens and training.
//
//   pre_t[c] = bias[c] + sum_k w[c][k] x_{t-K+1+k}[c],   y_t = act(pre_t)
//
// with the K-1 inputs before the sequence taken from a carried state.  Backward,
// with d_t = dy_t act'(pre_t) (pre is formed again from x, nothing is saved):
//   dx_t = sum_j w[K-1-j] d_{t+j},  dw[k] = sum_t d_t x_{t-K+1+k},  dbias = sum_t d_t
//
// Channels are last and independent, so a thread owns a few of them and walks along
// a run of tokens with its last inputs in registers: x is read once (plus K-1 tokens
// at each run's start), and the floor is HBM's.  What keeps the kernels from it is
// issue: two special functions and about 60 instructions per four channels and token
// forward, 60 per two backward.  Measured on one B200 (bf16, K 4, Swish; floor at
// 6.53 TB/s): 16384 x 2048 forward 30 us (21), 4 x 2048 x 2048 backward 34 us (15),
// one token of 256 x 4096 5.8 us (2.6), 4.5 with its 17 MB in L2, as a decode step that
// comes back to them within 126 MB finds them.
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "profile.h"
#include "vec.cuh"

namespace xlstm {
namespace {

constexpr int kThreads = 256;

// Two channels' activation and its slope.  Where e^-v overflows (v < -88) the
// logistic is 0, as the formula's limit.
template <bool SILU> __device__ __forceinline__ float2 activate(float2 v) {
    return SILU ? mul2(v, make_float2(logistic(v.x), logistic(v.y))) : v;
}
template <bool SILU> __device__ __forceinline__ float2 slope(float2 v) {
    if (!SILU) return both(1.f);
    const float2 s = make_float2(logistic(v.x), logistic(v.y));
    return mul2(s, fma2(v, make_float2(1.f - s.x, 1.f - s.y), both(1.f)));
}

// The weights of 2 * P channels from c on ([C, K]: 2 * P * K consecutive floats), as
// pairs of channels; and their biases.
template <int K, int P> __device__ __forceinline__ void load_weights(const float *w, int c, float2 (*f)[P]) {
    float t[2 * P * K];
#pragma unroll
    for (int i = 0; i < 2 * P * K; i += 2) {
        const float2 v = __ldg(reinterpret_cast<const float2 *>(w + (size_t)c * K + i));
        t[i] = v.x;
        t[i + 1] = v.y;
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e) f[k][e] = make_float2(t[2 * e * K + k], t[(2 * e + 1) * K + k]);
}
template <int P> __device__ __forceinline__ void load_bias(const float *bias, int c, float2 *f) {
#pragma unroll
    for (int e = 0; e < P; ++e) f[e] = bias ? __ldg(reinterpret_cast<const float2 *>(bias + c) + e) : both(0.f);
}

// Index i of a grid's threads as (column, row) of rows of n; 32-bit where it can be.
__device__ __forceinline__ void split_index(long long i, long long total, int n, int &col, int &row) {
    if (total < (1LL << 31)) {
        row = (int)((unsigned)i / (unsigned)n);
        col = (int)((unsigned)i - (unsigned)row * (unsigned)n);
    } else {
        row = (int)(i / n);
        col = (int)(i - (long long)row * n);
    }
}

struct ConvArgs {
    const void *x;
    const float *w, *bias;
    const void *state0;
    const int *lengths;
    void *y, *state_out;
    int B, S, C;
    int run, runs;              // tokens per thread, runs per sequence
};

__device__ __forceinline__ int length_of(const int *lengths, int b, int S) {
    if (!lengths) return S;
    const int n = lengths[b];
    return n < 0 ? 0 : n > S ? S : n;
}

// W neighbouring channels (4 or 2) as they lie in memory.
template <typename T, int W> struct Raw;
template <> struct Raw<float, 4> { using type = float4; };
template <> struct Raw<float, 2> { using type = float2; };
template <> struct Raw<__nv_bfloat16, 4> { using type = uint2; };
template <> struct Raw<__nv_bfloat16, 2> { using type = uint32_t; };
__device__ __forceinline__ void spread(float4 v, float2 *f) { f[0] = make_float2(v.x, v.y); f[1] = make_float2(v.z, v.w); }
__device__ __forceinline__ void spread(float2 v, float2 *f) { f[0] = v; }
__device__ __forceinline__ void spread(uint32_t v, float2 *f) {
    f[0] = make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ void spread(uint2 v, float2 *f) { spread(v.x, f); spread(v.y, f + 1); }
__device__ __forceinline__ uint32_t round2(float2 f) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void gather(const float2 *f, float4 &v) { v = make_float4(f[0].x, f[0].y, f[1].x, f[1].y); }
__device__ __forceinline__ void gather(const float2 *f, float2 &v) { v = f[0]; }
__device__ __forceinline__ void gather(const float2 *f, uint2 &v) { v = make_uint2(round2(f[0]), round2(f[1])); }
__device__ __forceinline__ void gather(const float2 *f, uint32_t &v) { v = round2(f[0]); }
template <typename R> __device__ __forceinline__ R zeros() { return R{}; }

// The inputs of one thread's W channels in one batch row, by time: the carried
// state before 0, zeros before that and from S on.
template <typename T, int K, int W> struct Channel {
    using R = typename Raw<T, W>::type;
    const T *x, *state0;
    int S;
    size_t C;
    __device__ __forceinline__ Channel(const void *x_, const void *s_, int b, int c, int S_, int C_)
        : x((const T *)x_ + (size_t)b * S_ * C_ + c),
          state0(s_ ? (const T *)s_ + (size_t)b * (K - 1) * C_ + c : nullptr), S(S_), C(C_) {}
    __device__ __forceinline__ R at(int t) const {
        if (t >= 0) return t < S ? __ldg(reinterpret_cast<const R *>(x + t * C)) : zeros<R>();
        if (state0 && t >= -(K - 1)) return __ldg(reinterpret_cast<const R *>(state0 + (K - 1 + t) * C));
        return zeros<R>();
    }
};

// Four channels a thread in either type: at eight, the weights and the window took
// 127 registers and left too few threads to cover HBM's latency (46 us against 21
// for 16384 x 2048 bf16).
template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a) {
    constexpr int W = 4, P = W / 2, U = 8;           // channels, their pairs, tokens' loads in flight
    using R = typename Raw<T, W>::type;
    const int nvec = a.C / W, parts = a.runs + (a.state_out ? 1 : 0);
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x, total = (long long)a.B * parts * nvec;
    if (i >= total) return;
    int col, br;
    split_index(i, total, nvec, col, br);
    const int c = col * W, b = br / parts, r = br - b * parts;
    const int len = length_of(a.lengths, b, a.S);
    const Channel<T, K, W> in(a.x, a.state0, b, c, a.S, a.C);
    if (r == a.runs) {                               // the last K-1 inputs
        T *out = (T *)a.state_out + (size_t)b * (K - 1) * a.C + c;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) *reinterpret_cast<R *>(out + (size_t)j * a.C) = in.at(len - (K - 1) + j);
        return;
    }
    const int t0 = r * a.run, t1 = min(t0 + a.run, len);
    if (t0 >= len) return;
    float2 w[K][P], bias[P], win[4][P];              // the last inputs, by time modulo 4 (U is a multiple)
    R next[U];
    const T *x = in.x + (size_t)t0 * a.C;
#pragma unroll
    for (int u = 0; u < U; ++u) next[u] = t0 + u < t1 ? __ldg(reinterpret_cast<const R *>(x + (size_t)u * a.C)) : zeros<R>();
#pragma unroll
    for (int j = 1; j < K; ++j) spread(in.at(t0 - j), win[(4 - j) % 4]);
    load_weights<K, P>(a.w, c, w);
    load_bias<P>(a.bias, c, bias);
    T *y = (T *)a.y + ((size_t)b * a.S + t0) * a.C + c;
    for (int t = t0; t < t1; t += U, x += (size_t)U * a.C, y += (size_t)U * a.C) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1) break;
            spread(next[u], win[u % 4]);
            if (t + U + u < t1) next[u] = __ldg(reinterpret_cast<const R *>(x + (size_t)(U + u) * a.C));
            float2 out[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                float2 p = bias[e];
#pragma unroll
                for (int k = 0; k < K; ++k) p = fma2(w[k][e], win[(u + 4 - (K - 1) + k) % 4][e], p);
                out[e] = activate<SILU>(p);
            }
            R v;
            gather(out, v);
            __stcs(reinterpret_cast<R *>(y + (size_t)u * a.C), v);
        }
    }
}

struct ConvStepArgs {
    const void *x;
    const float *w, *bias;
    void *state, *y;
    int B, C;
};

// Four channels of ROWS batch rows a thread: the weights, more bytes than a row's data,
// are read once for the rows.  256 x 4096 bf16, in L2: 4.6 us with four rows, 8.6 with one; one
// where four would not give every SM a CTA.
template <typename T, int K, bool SILU, int ROWS>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvStepArgs a) {
    constexpr int W = 4, P = W / 2;
    using R = typename Raw<T, W>::type;
    const int nvec = a.C / W;
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x, total = (long long)((a.B + ROWS - 1) / ROWS) * nvec;
    if (i >= total) return;
    int col, group;
    split_index(i, total, nvec, col, group);
    const int c = col * W, b0 = group * ROWS;
    R raw[ROWS][K];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (b0 + r >= a.B) continue;
        const T *st = (const T *)a.state + (size_t)(b0 + r) * (K - 1) * a.C + c;
#pragma unroll
        for (int k = 0; k < K - 1; ++k) raw[r][k] = *reinterpret_cast<const R *>(st + (size_t)k * a.C);
        raw[r][K - 1] = __ldcs(reinterpret_cast<const R *>((const T *)a.x + (size_t)(b0 + r) * a.C + c));
    }
    float2 w[K][P], bias[P];
    load_weights<K, P>(a.w, c, w);
    load_bias<P>(a.bias, c, bias);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (b0 + r >= a.B) continue;
        T *st = (T *)a.state + (size_t)(b0 + r) * (K - 1) * a.C + c;
        float2 out[P];
#pragma unroll
        for (int e = 0; e < P; ++e) out[e] = bias[e];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float2 v[P];
            spread(raw[r][k], v);
#pragma unroll
            for (int e = 0; e < P; ++e) out[e] = fma2(w[k][e], v[e], out[e]);
            if (k > 0) *reinterpret_cast<R *>(st + (size_t)(k - 1) * a.C) = raw[r][k];
        }
#pragma unroll
        for (int e = 0; e < P; ++e) out[e] = activate<SILU>(out[e]);
        R v;
        gather(out, v);
        __stcs(reinterpret_cast<R *>((T *)a.y + (size_t)(b0 + r) * a.C + c), v);
    }
}

// ---------------------------------------------------------------- backward
struct ConvBwdArgs {
    const void *x;
    const float *w, *bias;
    const void *state0, *dy, *dstate;
    void *dx, *dstate0;
    float *partial;             // [B * runs, C * (K + 1)]: dw as [C, K], then dbias [C]
    int B, S, C;
    int run, runs;              // input times per thread; the K-1 carried ones are times -(K-1)..-1
};

// One thread's walk along a run of input times [tau0, tau1), U tokens at a time.  Blocks
// of tokens at the ends of the sequence or of the run look at every token's place (times
// outside the sequence, the carried state, the final state's cotangent, tokens whose
// share of dw is the next run's); the blocks between, nearly all, need none of that.
template <typename T, int K, bool SILU>
__device__ __forceinline__ void conv_bwd_walk(const ConvBwdArgs &a, int c, int b, int tau0, int tau1, const float2 *w, float2 bias,
                                              float2 *dw, float2 &db) {
    constexpr int W = 2, U = sizeof(T) == 2 ? 8 : 4; // channels, tokens' loads in flight
    using R = typename Raw<T, W>::type;
    const int S = a.S;
    const size_t C = a.C;
    const Channel<T, K, W> in(a.x, a.state0, b, c, S, a.C);
    const T *dy = (const T *)a.dy + (size_t)b * S * C + c;
    const T *dstate = a.dstate ? (const T *)a.dstate + (size_t)b * (K - 1) * C + c : nullptr;
    T *dx = (T *)a.dx + (size_t)b * S * C + c;
    T *dstate0 = a.dstate0 ? (T *)a.dstate0 + (size_t)b * (K - 1) * C + c : nullptr;
    float2 win[4], d[4];                             // the last inputs and d's, by time modulo 4 (U is a multiple)
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = both(0.f);
#pragma unroll
    for (int j = 1; j < K; ++j) spread(in.at(tau0 - j), &win[(4 - j) % 4]);
    // outputs' times t; the input time t - (K-1) is complete once d_t is known
    const int t_end = tau1 + K - 1;
    R xn[U], yn[U];
    auto load = [&](int t, int u) {
        xn[u] = in.at(t);
        yn[u] = t >= 0 && t < S ? __ldg(reinterpret_cast<const R *>(dy + t * C)) : zeros<R>();
    };
    auto token = [&](int u, bool inside, bool own) {
        float2 dyv, p = bias;
        spread(yn[u], &dyv);
#pragma unroll
        for (int k = 0; k < K; ++k) p = fma2(w[k], win[(u + 4 - (K - 1) + k) % 4], p);
        d[u % 4] = inside ? mul2(dyv, slope<SILU>(p)) : both(0.f);
        if (own) {
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k] = fma2(d[u % 4], win[(u + 4 - (K - 1) + k) % 4], dw[k]);
            db = add2(db, d[u % 4]);
        }
        float2 g = both(0.f);
#pragma unroll
        for (int j = 0; j < K; ++j) g = fma2(w[K - 1 - j], d[(u + 4 - (K - 1) + j) % 4], g);
        return g;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) load(tau0 + u, u);
    for (int t = tau0; t < t_end; t += U) {
        if (t >= K - 1 && t > tau0 && t + U <= tau1 && t + 2 * U <= S) {
            const T *xp = in.x + (t + U) * C, *yp = dy + (t + U) * C;
            T *out = dx + (t - (K - 1)) * C;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                spread(xn[u], &win[u % 4]);
                const float2 g = token(u, true, true);
                xn[u] = __ldg(reinterpret_cast<const R *>(xp + u * C));
                yn[u] = __ldg(reinterpret_cast<const R *>(yp + u * C));
                R v;
                gather(&g, v);
                __stcs(reinterpret_cast<R *>(out + u * C), v);
            }
            continue;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int tt = t + u, tau = tt - (K - 1);
            if (tt >= t_end) break;
            spread(xn[u], &win[u % 4]);
            const bool inside = tt >= 0 && tt < S;                       // outside the sequence there is no output
            float2 g = token(u, inside, inside && tt < tau1);
            load(tt + U, u);
            if (tau < tau0) continue;                                    // the run before completes it
            const int place = tt - S;                                    // in the final state
            if (dstate && place >= 0) {
                float2 ds;
                spread(__ldg(reinterpret_cast<const R *>(dstate + place * C)), &ds);
                g = add2(g, ds);
            }
            R v;
            gather(&g, v);
            if (tau >= 0) __stcs(reinterpret_cast<R *>(dx + tau * C), v);
            else if (dstate0) *reinterpret_cast<R *>(dstate0 + (K - 1 + tau) * C) = v;
        }
    }
}

// Two channels a thread, one packed pair: four took 154 registers and 140 us for
// 4 x 2048 x 2048 bf16.
template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(kThreads, 2) conv_bwd_kernel(ConvBwdArgs a) {
    const int nvec = a.C / 2;
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x, total = (long long)a.B * a.runs * nvec;
    if (i >= total) return;
    int col, br;
    split_index(i, total, nvec, col, br);
    const int c = col * 2, b = br / a.runs, r = br - b * a.runs;
    const int tau0 = r * a.run - (K - 1), tau1 = min(tau0 + a.run, a.S);
    float2 w[K][1], bias, dw[K], db = both(0.f);
    load_weights<K, 1>(a.w, c, w);
    load_bias<1>(a.bias, c, &bias);
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k] = both(0.f);
    conv_bwd_walk<T, K, SILU>(a, c, b, tau0, tau1, &w[0][0], bias, dw, db);
    pdl_launch_dependents();
    float *part = a.partial + (size_t)br * a.C * (K + 1);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        part[(size_t)c * K + k] = dw[k].x;
        part[(size_t)(c + 1) * K + k] = dw[k].y;
    }
    *reinterpret_cast<float2 *>(part + (size_t)a.C * K + c) = db;
}

// Tokens per thread, a multiple of 8.  A large problem is cut so that its CTAs are one
// wave (`per_sm` are resident: a second, nearly empty wave would double the time);
// beyond `most` tokens the waves are many and even out.  A small problem gets short
// runs, so that it has threads enough.
int run_length(int B, int times, int columns, int per_sm, int least, int most) {
    const long long room = (long long)per_sm * num_sms_current_device();
    int run = least;
    while (run < most) {
        const long long runs = (times + run - 1) / run;
        if (((long long)B * runs * columns + kThreads - 1) / kThreads <= room) break;
        run += 8;
    }
    return run;
}

unsigned blocks_for(long long n) { return (unsigned)((n + kThreads - 1) / kThreads); }

#define XLSTM_CONV_WIDTHS(T)                                                         \
    if (K == 2) { if (silu) { XLSTM_LAUNCH(T, 2, true) } else { XLSTM_LAUNCH(T, 2, false) } } \
    if (K == 3) { if (silu) { XLSTM_LAUNCH(T, 3, true) } else { XLSTM_LAUNCH(T, 3, false) } } \
    if (K == 4) { if (silu) { XLSTM_LAUNCH(T, 4, true) } else { XLSTM_LAUNCH(T, 4, false) } }
#define XLSTM_CONV_DISPATCH                                                          \
    if (bf16) { XLSTM_CONV_WIDTHS(__nv_bfloat16) } else { XLSTM_CONV_WIDTHS(float) } \
    return cudaErrorInvalidValue;

cudaError_t launch_conv_fwd(const ConvArgs &a, int K, bool silu, bool bf16, cudaStream_t st) {
    const unsigned grid = blocks_for((long long)a.B * (a.runs + (a.state_out ? 1 : 0)) * (a.C / 4));
    if (grid == 0) return cudaSuccess;
    KernelTimer timer("conv_fwd", st);
#define XLSTM_LAUNCH(T, KK, A) conv_fwd_kernel<T, KK, A><<<grid, kThreads, 0, st>>>(a); return cudaGetLastError();
    XLSTM_CONV_DISPATCH
#undef XLSTM_LAUNCH
}
cudaError_t launch_conv_step(const ConvStepArgs &a, int K, bool silu, bool bf16, cudaStream_t st) {
    const long long columns = a.C / 4;
    const bool rows = (a.B / 4) * columns >= (long long)kThreads * num_sms_current_device();
    const unsigned grid = blocks_for((rows ? (a.B + 3) / 4 : a.B) * columns);
    KernelTimer timer("conv_step", st);
#define XLSTM_LAUNCH(T, KK, A)                                                    \
    if (rows) conv_step_kernel<T, KK, A, 4><<<grid, kThreads, 0, st>>>(a);        \
    else conv_step_kernel<T, KK, A, 1><<<grid, kThreads, 0, st>>>(a);             \
    return cudaGetLastError();
    XLSTM_CONV_DISPATCH
#undef XLSTM_LAUNCH
}
cudaError_t launch_conv_bwd(const ConvBwdArgs &a, int K, bool silu, bool bf16, cudaStream_t st) {
    const unsigned grid = blocks_for((long long)a.B * a.runs * (a.C / 2));
    KernelTimer timer("conv_bwd", st);
#define XLSTM_LAUNCH(T, KK, A) conv_bwd_kernel<T, KK, A><<<grid, kThreads, 0, st>>>(a); return cudaGetLastError();
    XLSTM_CONV_DISPATCH
#undef XLSTM_LAUNCH
}

xlstm_status check_conv(int B, int S, int C, int K, xlstm_dtype dt, xlstm_conv_act act) {
    if (dt != XLSTM_F32 && dt != XLSTM_BF16) return XLSTM_ERR_DTYPE;
    if (act != XLSTM_CONV_NONE && act != XLSTM_CONV_SILU) return XLSTM_ERR_DTYPE;
    if (B < 0 || S < 0 || C < 8 || C > 65536 || C % 8 != 0) return XLSTM_ERR_SHAPE;
    if (K < 2 || K > 4) return XLSTM_ERR_SHAPE;
    if (S > (1 << 30) || (long long)B * (S + K) >= (1LL << 31)) return XLSTM_ERR_SHAPE;   // rows of tokens are ints
    return XLSTM_OK;
}

void plan_conv_bwd(int B, int S, int C, int K, int *run, int *runs) {
    *run = run_length(B, S + K - 1, C / 2, 2, 16, 256);
    *runs = (S + K - 1 + *run - 1) / *run;
}

}  // namespace
}  // namespace xlstm

extern "C" xlstm_status xlstm_causal_conv_fwd(const void *x, const float *w, const float *bias,
                                              const void *state0, const int *lengths, void *y,
                                              void *state_out, int B, int S, int C, int K,
                                              xlstm_dtype dt, xlstm_conv_act act, void *cuda_stream) {
    using namespace xlstm;
    CallRange range("xlstm_causal_conv_fwd");
    const xlstm_status bad = check_conv(B, S, C, K, dt, act);
    if (bad != XLSTM_OK) return bad;
    if (B == 0) return XLSTM_OK;
    if (!w || (S > 0 && (!x || !y))) return XLSTM_ERR_NULL;
    const void *ptrs[] = {x, w, bias, state0, y, state_out};
    for (const void *p : ptrs)
        if (misaligned16(p)) return XLSTM_ERR_ALIGN;
    if (misaligned4(lengths)) return XLSTM_ERR_ALIGN;          // read one by one
    const void *in[] = {x, w, bias, state0, lengths}, *out[] = {y, state_out};
    for (const void *o : out)
        for (const void *i : in)
            if (o && o == i) return XLSTM_ERR_UNSUPPORTED;
    if (y && y == state_out) return XLSTM_ERR_UNSUPPORTED;
    const bool bf16 = dt == XLSTM_BF16;
    ConvArgs a = {x, w, bias, state0, lengths, y, state_out, B, S, C, 0, 0};
    a.run = run_length(B, S, C / 4, bf16 ? 3 : 2, 8, 128);
    a.runs = (S + a.run - 1) / a.run;
    return launch_conv_fwd(a, K, act == XLSTM_CONV_SILU, bf16, (cudaStream_t)cuda_stream) == cudaSuccess
               ? XLSTM_OK : XLSTM_ERR_CUDA;
}

extern "C" xlstm_status xlstm_causal_conv_step(const void *x, const float *w, const float *bias,
                                               void *state, void *y, int B, int C, int K,
                                               xlstm_dtype dt, xlstm_conv_act act, void *cuda_stream) {
    using namespace xlstm;
    CallRange range("xlstm_causal_conv_step");
    const xlstm_status bad = check_conv(B, 1, C, K, dt, act);
    if (bad != XLSTM_OK) return bad;
    if (B == 0) return XLSTM_OK;
    if (!x || !w || !state || !y) return XLSTM_ERR_NULL;
    const void *ptrs[] = {x, w, bias, state, y};
    for (const void *p : ptrs)
        if (misaligned16(p)) return XLSTM_ERR_ALIGN;
    if (state == x || state == y || y == x || y == (const void *)w || y == (const void *)bias ||
        state == (const void *)w || state == (const void *)bias)
        return XLSTM_ERR_UNSUPPORTED;
    ConvStepArgs a = {x, w, bias, state, y, B, C};
    return launch_conv_step(a, K, act == XLSTM_CONV_SILU, dt == XLSTM_BF16, (cudaStream_t)cuda_stream) == cudaSuccess
               ? XLSTM_OK : XLSTM_ERR_CUDA;
}

extern "C" xlstm_status xlstm_causal_conv_bwd_workspace_size(int B, int S, int C, int K, xlstm_dtype dt,
                                                             size_t *bytes) {
    using namespace xlstm;
    if (!bytes) return XLSTM_ERR_NULL;
    const xlstm_status bad = check_conv(B, S, C, K, dt, XLSTM_CONV_NONE);
    if (bad != XLSTM_OK) return bad;
    int run, runs;
    plan_conv_bwd(B, S, C, K, &run, &runs);
    *bytes = (size_t)B * runs * C * (K + 1) * sizeof(float);
    return XLSTM_OK;
}

extern "C" xlstm_status xlstm_causal_conv_bwd(const void *x, const float *w, const float *bias,
                                              const void *state0, const void *dy, const void *dstate,
                                              void *dx, float *dw, float *dbias, void *dstate0,
                                              int B, int S, int C, int K, xlstm_dtype dt,
                                              xlstm_conv_act act, void *workspace,
                                              size_t workspace_bytes, void *cuda_stream) {
    using namespace xlstm;
    CallRange range("xlstm_causal_conv_bwd");
    const xlstm_status bad = check_conv(B, S, C, K, dt, act);
    if (bad != XLSTM_OK) return bad;
    if (!w || !dw || (B > 0 && S > 0 && (!x || !dy || !dx))) return XLSTM_ERR_NULL;
    const void *ptrs[] = {x, w, bias, state0, dy, dstate, dx, dw, dbias, dstate0, workspace};
    for (const void *p : ptrs)
        if (misaligned16(p)) return XLSTM_ERR_ALIGN;
    const void *in[] = {x, w, bias, state0, dy, dstate}, *out[] = {dx, dw, dbias, dstate0};
    for (int i = 0; i < 4; ++i) {
        if (!out[i]) continue;
        for (const void *p : in)
            if (out[i] == p) return XLSTM_ERR_UNSUPPORTED;
        for (int j = 0; j < i; ++j)
            if (out[i] == out[j]) return XLSTM_ERR_UNSUPPORTED;
    }
    ConvBwdArgs a = {x, w, bias, state0, dy, dstate, dx, dstate0, (float *)workspace, B, S, C, 0, 0};
    plan_conv_bwd(B, S, C, K, &a.run, &a.runs);
    const size_t need = (size_t)B * a.runs * C * (K + 1) * sizeof(float);
    if (need > 0 && (!workspace || workspace_bytes < need)) return XLSTM_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    if (B > 0 && launch_conv_bwd(a, K, act == XLSTM_CONV_SILU, dt == XLSTM_BF16, st) != cudaSuccess)
        return XLSTM_ERR_CUDA;
    return launch_sum_rows((const float *)workspace, dw, dbias, C * K, B * a.runs, C * (K + 1), st) == cudaSuccess
               ? XLSTM_OK : XLSTM_ERR_CUDA;
}
