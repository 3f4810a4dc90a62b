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
// Channels are last and independent, so a thread owns one vector of channels
// and walks along the tokens with its K-1 last inputs in registers: x is read
// once (plus K-1 tokens at each run's start) and the op is bound by HBM.
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "profile.h"
#include "vec.cuh"

namespace xlstm {
namespace {

constexpr int kThreads = 256;

// 1 / (1 + e^-v) from CUDA's fast exponential and division: relative error about
// 1e-6, 0 at -inf (v = -inf only meets it as v * 0 below) and 1 at +inf.
__device__ __forceinline__ float fast_sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// Where e^-v overflows (v < -88) __fdividef returns 0, as the formula's limit.
template <bool SILU> __device__ __forceinline__ float activate(float v) { return SILU ? v * fast_sigmoid(v) : v; }
template <bool SILU> __device__ __forceinline__ float slope(float v) {
    if (!SILU) return 1.f;
    const float s = fast_sigmoid(v);
    return s * (1.f + v * (1.f - s));
}

// The weights of VN channels from c on ([C, K]: VN * K consecutive floats, a
// multiple of four) by 16-byte loads.
template <int K, int VN> __device__ __forceinline__ void load_weights(const float *w, int c, float (*f)[VN]) {
#pragma unroll
    for (int i = 0; i < K * VN; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(w + (size_t)c * K + i));
        f[i % K][i / K] = v.x;
        f[(i + 1) % K][(i + 1) / K] = v.y;
        f[(i + 2) % K][(i + 2) / K] = v.z;
        f[(i + 3) % K][(i + 3) / K] = v.w;
    }
}
template <int VN> __device__ __forceinline__ void load_bias(const float *bias, int c, float *f) {
#pragma unroll
    for (int e = 0; e < VN; e += 4) {
        const float4 v = bias ? __ldg(reinterpret_cast<const float4 *>(bias + c + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
        f[e] = v.x; f[e + 1] = v.y; f[e + 2] = v.z; f[e + 3] = v.w;
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

// The input at time t of batch row b (t < 0: the carried state), one vector.
template <typename T, int K>
__device__ __forceinline__ uint4 input_at(const T *x, const T *state0, int b, int t, int S, int nvec, int cv) {
    if (t >= 0) return __ldg(reinterpret_cast<const uint4 *>(x) + ((size_t)b * S + t) * nvec + cv);
    if (state0 && t >= -(K - 1))
        return __ldg(reinterpret_cast<const uint4 *>(state0) + ((size_t)b * (K - 1) + (K - 1 + t)) * nvec + cv);
    return make_uint4(0, 0, 0, 0);
}

template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a) {
    constexpr int VN = Vec<T>::N, U = 4;             // U tokens' loads in flight per thread
    const int nvec = a.C / VN;
    const int parts = a.runs + (a.state_out ? 1 : 0);
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)a.B * parts * nvec) return;
    const int cv = (int)(i % nvec);
    const long long br = i / nvec;
    const int b = (int)(br / parts), r = (int)(br - (long long)b * parts);
    const int len = length_of(a.lengths, b, a.S);
    const T *x = (const T *)a.x, *state0 = (const T *)a.state0;
    if (r == a.runs) {                               // the last K-1 inputs
        uint4 *out = reinterpret_cast<uint4 *>(a.state_out) + (size_t)b * (K - 1) * nvec + cv;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) out[(size_t)j * nvec] = input_at<T, K>(x, state0, b, len - (K - 1) + j, a.S, nvec, cv);
        return;
    }
    const int t0 = r * a.run;
    if (t0 >= len) return;
    const int t1 = min(t0 + a.run, len);
    float w[K][VN], bias[VN], win[K][VN];
    load_weights<K, VN>(a.w, cv * VN, w);
    load_bias<VN>(a.bias, cv * VN, bias);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) unpack<T>(input_at<T, K>(x, state0, b, t0 - (K - 1) + k, a.S, nvec, cv), win[k]);
    const uint4 *xv = reinterpret_cast<const uint4 *>(x) + (size_t)b * a.S * nvec + cv;
    uint4 *yv = reinterpret_cast<uint4 *>(a.y) + (size_t)b * a.S * nvec + cv;
    for (int t = t0; t < t1; t += U) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < t1) raw[u] = __ldg(xv + (size_t)(t + u) * nvec);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1) break;
            unpack<T>(raw[u], win[K - 1]);
            float out[VN];
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                float p = bias[e];
#pragma unroll
                for (int k = 0; k < K; ++k) p += w[k][e] * win[k][e];
                out[e] = activate<SILU>(p);
#pragma unroll
                for (int k = 0; k < K - 1; ++k) win[k][e] = win[k + 1][e];
            }
            __stcs(yv + (size_t)(t + u) * nvec, pack<T>(out));
        }
    }
}

struct ConvStepArgs {
    const void *x;
    const float *w, *bias;
    void *state, *y;
    int B, C;
};

template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvStepArgs a) {
    constexpr int VN = Vec<T>::N;
    const int nvec = a.C / VN;
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)a.B * nvec) return;
    const int cv = (int)(i % nvec);
    const long long b = i / nvec;
    uint4 *st = reinterpret_cast<uint4 *>(a.state) + (size_t)b * (K - 1) * nvec + cv;
    uint4 raw[K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) raw[k] = st[(size_t)k * nvec];
    raw[K - 1] = __ldcs(reinterpret_cast<const uint4 *>(a.x) + i);
    float out[VN], w[K][VN];
    load_weights<K, VN>(a.w, cv * VN, w);
    load_bias<VN>(a.bias, cv * VN, out);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float v[VN];
        unpack<T>(raw[k], v);
#pragma unroll
        for (int e = 0; e < VN; ++e) out[e] += w[k][e] * v[e];
        if (k > 0) st[(size_t)(k - 1) * nvec] = raw[k];
    }
#pragma unroll
    for (int e = 0; e < VN; ++e) out[e] = activate<SILU>(out[e]);
    __stcs(reinterpret_cast<uint4 *>(a.y) + i, pack<T>(out));
}

// ---------------------------------------------------------------- backward
// Four channels per thread in either type, so that the weights, their gradient
// and both windows fit in registers.
template <typename T> __device__ __forceinline__ void load4(const T *p, float *f);
template <> __device__ __forceinline__ void load4<float>(const float *p, float *f) {
    const float4 v = __ldg(reinterpret_cast<const float4 *>(p));
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
template <> __device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16 *p, float *f) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
}
template <typename T> __device__ __forceinline__ void store4(T *p, const float *f);
template <> __device__ __forceinline__ void store4<float>(float *p, const float *f) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, const float *f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    __stcs(reinterpret_cast<uint2 *>(p), make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                                    *reinterpret_cast<const uint32_t *>(&b)));
}

struct ConvBwdArgs {
    const void *x;
    const float *w, *bias;
    const void *state0, *dy, *dstate;
    void *dx, *dstate0;
    float *partial;             // [B * runs, C * (K + 1)]: dw as [C, K], then dbias [C]
    int B, S, C;
    int run, runs;              // input times per thread; the K-1 carried ones are times -(K-1)..-1
};

template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvBwdArgs a) {
    constexpr int VN = 4, U = 4;
    const int nvec = a.C / VN;
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)a.B * a.runs * nvec) return;
    const int c = (int)(i % nvec) * VN;
    const long long br = i / nvec;
    const int b = (int)(br / a.runs), r = (int)(br - (long long)b * a.runs);
    const int S = a.S, C = a.C;
    const int tau0 = r * a.run - (K - 1), tau1 = min(tau0 + a.run, S);
    const T *x = (const T *)a.x + (size_t)b * S * C + c;
    const T *dy = (const T *)a.dy + (size_t)b * S * C + c;
    const T *state0 = a.state0 ? (const T *)a.state0 + (size_t)b * (K - 1) * C + c : nullptr;
    const T *dstate = a.dstate ? (const T *)a.dstate + (size_t)b * (K - 1) * C + c : nullptr;
    T *dx = (T *)a.dx + (size_t)b * S * C + c;
    T *dstate0 = a.dstate0 ? (T *)a.dstate0 + (size_t)b * (K - 1) * C + c : nullptr;

    float w[K][VN], bias[VN], win[K][VN], d[K][VN], dw[K][VN], db[VN];
    load_weights<K, VN>(a.w, c, w);
    load_bias<VN>(a.bias, c, bias);
#pragma unroll
    for (int e = 0; e < VN; ++e) {
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][e] = d[k][e] = 0.f;
        db[e] = 0.f;
    }
    auto input = [&](int t, float *f) {
        if (t >= 0 && t < S) load4<T>(x + (size_t)t * C, f);
        else if (t < 0 && state0 && t >= -(K - 1)) load4<T>(state0 + (size_t)(K - 1 + t) * C, f);
        else f[0] = f[1] = f[2] = f[3] = 0.f;
    };
#pragma unroll
    for (int k = 0; k < K - 1; ++k) input(tau0 - (K - 1) + k, win[k]);
    // outputs' times t; the input time t - (K-1) is complete once d_t is known
    const int t_end = tau1 + K - 1;
    for (int t = tau0; t < t_end; t += U) {
        float xin[U][VN], dyin[U][VN];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            input(t + u, xin[u]);
            if (t + u >= 0 && t + u < S) load4<T>(dy + (size_t)(t + u) * C, dyin[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int tt = t + u;
            if (tt >= t_end) break;
            const bool out_time = tt >= 0 && tt < S;
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                win[K - 1][e] = xin[u][e];
                float p = bias[e];
#pragma unroll
                for (int k = 0; k < K; ++k) p += w[k][e] * win[k][e];
                d[K - 1][e] = out_time ? dyin[u][e] * slope<SILU>(p) : 0.f;
                if (tt < tau1) {                       // a later time's share is the next run's
#pragma unroll
                    for (int k = 0; k < K; ++k) dw[k][e] += d[K - 1][e] * win[k][e];
                    db[e] += d[K - 1][e];
                }
            }
            const int tau = tt - (K - 1);
            if (tau >= tau0) {
                float g[VN];
#pragma unroll
                for (int e = 0; e < VN; ++e) {
                    g[e] = 0.f;
#pragma unroll
                    for (int j = 0; j < K; ++j) g[e] += w[K - 1 - j][e] * d[j][e];
                }
                const int slot = tau - (S - (K - 1));  // its place in the final state
                if (dstate && slot >= 0) {
                    float ds[VN];
                    load4<T>(dstate + (size_t)slot * C, ds);
#pragma unroll
                    for (int e = 0; e < VN; ++e) g[e] += ds[e];
                }
                if (tau >= 0) store4<T>(dx + (size_t)tau * C, g);
                else if (dstate0) store4<T>(dstate0 + (size_t)(K - 1 + tau) * C, g);
            }
#pragma unroll
            for (int e = 0; e < VN; ++e) {
#pragma unroll
                for (int k = 0; k < K - 1; ++k) {
                    win[k][e] = win[k + 1][e];
                    d[k][e] = d[k + 1][e];
                }
            }
        }
    }
    float *part = a.partial + (size_t)br * C * (K + 1);
#pragma unroll
    for (int e = 0; e < VN; ++e) {
#pragma unroll
        for (int k = 0; k < K; ++k) part[(size_t)(c + e) * K + k] = dw[k][e];
        part[(size_t)C * K + c + e] = db[e];
    }
}

// Tokens per thread: long runs read fewer tokens twice, short ones give a small
// problem more threads.
int fwd_run(long long tokens_times_vectors, int num_sms) {
    return tokens_times_vectors / 16 >= 512LL * num_sms ? 16 : 4;
}
int bwd_run(long long tokens_times_vectors, int num_sms) {
    return tokens_times_vectors / 64 >= 256LL * num_sms ? 64 : 16;
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
    const int vn = bf16 ? 8 : 4;
    const unsigned grid = blocks_for((long long)a.B * (a.runs + (a.state_out ? 1 : 0)) * (a.C / vn));
    if (grid == 0) return cudaSuccess;
    KernelTimer timer("conv_fwd", st);
#define XLSTM_LAUNCH(T, KK, A) conv_fwd_kernel<T, KK, A><<<grid, kThreads, 0, st>>>(a); return cudaGetLastError();
    XLSTM_CONV_DISPATCH
#undef XLSTM_LAUNCH
}
cudaError_t launch_conv_step(const ConvStepArgs &a, int K, bool silu, bool bf16, cudaStream_t st) {
    const unsigned grid = blocks_for((long long)a.B * (a.C / (bf16 ? 8 : 4)));
    KernelTimer timer("conv_step", st);
#define XLSTM_LAUNCH(T, KK, A) conv_step_kernel<T, KK, A><<<grid, kThreads, 0, st>>>(a); return cudaGetLastError();
    XLSTM_CONV_DISPATCH
#undef XLSTM_LAUNCH
}
cudaError_t launch_conv_bwd(const ConvBwdArgs &a, int K, bool silu, bool bf16, cudaStream_t st) {
    const unsigned grid = blocks_for((long long)a.B * a.runs * (a.C / 4));
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
    if (S > (1 << 30) || (long long)B * (S + K) > (1LL << 40) / C) return XLSTM_ERR_SHAPE;
    return XLSTM_OK;
}

void plan_conv_bwd(int B, int S, int C, int K, int *run, int *runs) {
    *run = bwd_run((long long)B * S * (C / 4), num_sms_current_device());
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
    const void *ptrs[] = {x, w, bias, state0, lengths, y, state_out};
    for (const void *p : ptrs)
        if (misaligned16(p)) return XLSTM_ERR_ALIGN;
    const void *in[] = {x, w, bias, state0, lengths}, *out[] = {y, state_out};
    for (const void *o : out)
        for (const void *i : in)
            if (o && o == i) return XLSTM_ERR_UNSUPPORTED;
    if (y && y == state_out) return XLSTM_ERR_UNSUPPORTED;
    const bool bf16 = dt == XLSTM_BF16;
    ConvArgs a = {x, w, bias, state0, lengths, y, state_out, B, S, C, 0, 0};
    a.run = fwd_run((long long)B * S * (C / (bf16 ? 8 : 4)), num_sms_current_device());
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
